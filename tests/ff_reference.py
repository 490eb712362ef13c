"""The feed-forward operators from their formulas in 64 bits (torch on the
CPU), with the error bounds their tests hold the kernels to.

Bounds.  A product summed in FP32 is within TOL * sum |a||b| of the exact one
(the library's bar for FP32 accuracy, whatever the order of the sum), a
result rounded to BF16 within 2^-8 of itself (8 significant bits: in [1, 2)
they are 2^-7 apart, so at most 2^-8 off), to FP32 within 2^-24.  act and act' are computed in FP32 from a
handful of operations: within ACT * (1 + |g|), ACT = 1e-6 with the accurate
exponential (FP32) and 4e-6 with the fast one (BF16); |act'| <= 1.13 for
every activation, which carries an error of g over to act(g)."""
import math

import torch

TOL = 1e-5
SLOPE = 1.13
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
ACT = {torch.float32: 1e-6, torch.bfloat16: 4e-6}


def act_both(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        p = 0.5 * torch.erfc(-g * math.sqrt(0.5))
        return g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g ** 3))
        return (0.5 * g * (1 + t),
                0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g))
    return torch.clamp(g, min=0), (g > 0).double()


def forward(X, Wg, Wu, act):
    """{name: (value, bound)} of H, G, U; bounds before rounding to dt are for dt's kernels."""
    dt = X.dtype
    X, Wg, Wu = (t.double().cpu() for t in (X, Wg, Wu))
    G, U = X @ Wg, X @ Wu
    eG, eU = TOL * (X.abs() @ Wg.abs()), TOL * (X.abs() @ Wu.abs())
    a, _ = act_both(G, act)
    ea = SLOPE * eG + ACT[dt] * (1 + G.abs())
    H, eH = a * U, ea * U.abs() + a.abs() * eU + ea * eU
    f32 = torch.float32  # G and U are kept in FP32
    return {k: (v, e + ROUND[t] * (v.abs() + e) + 1e-37)
            for k, v, e, t in (("H", H, eH, dt), ("G", G, eG, f32), ("U", U, eU, f32))}


def backward(dH, X, Wg, Wu, G, U, act):
    """{name: (value, bound)} of dX, dWg, dWu."""
    dt = X.dtype
    dH, X, Wg, Wu, G, U = (t.double().cpu() for t in (dH, X, Wg, Wu, G, U))
    a, d = act_both(G, act)
    dG, dU = dH * U * d, dH * a
    ea = ACT[dt] * (1 + G.abs())
    # three FP32 products, then rounded to dt
    eG = (dH * U).abs() * ea + (dG.abs() + (dH * U).abs() * ea) * (3 * 2.0 ** -24 + ROUND[dt])
    eU = dH.abs() * ea + (dU.abs() + dH.abs() * ea) * (2.0 ** -24 + ROUND[dt])
    out = {"dX": (dG @ Wg.t() + dU @ Wu.t(),
                  eG @ Wg.abs().t() + eU @ Wu.abs().t() +
                  TOL * ((dG.abs() + eG) @ Wg.abs().t() + (dU.abs() + eU) @ Wu.abs().t())),
           "dWg": (X.t() @ dG, X.abs().t() @ eG + TOL * (X.abs().t() @ (dG.abs() + eG))),
           "dWu": (X.t() @ dU, X.abs().t() @ eU + TOL * (X.abs().t() @ (dU.abs() + eU)))}
    return {k: (v, e + ROUND[dt] * (v.abs() + e) + 1e-37) for k, (v, e) in out.items()}


def codes(q, K):
    q = q.cpu()
    return torch.stack((q & 15, q >> 4), 2).reshape(q.shape[0], -1)[:, :K].double()


def q4(X, q, s, z, group):
    """(Y, bound before rounding): zero points and codes may be summed apart."""
    K = X.shape[1]
    X, s = X.double().cpu(), s.double().cpu()
    c = codes(q, K)
    at = torch.arange(K) // group
    zz = torch.full_like(s, 8.0) if z is None else z.double().cpu()
    W = s[:, at] * (c - zz[:, at])
    D = s[:, at].abs() * ((c - 8).abs() + (zz[:, at] - 8).abs())
    return X @ W.t(), TOL * (X.abs() @ D.t())


def q4_rounded(X, q, s, z, group):
    y, e = q4(X, q, s, z, group)
    return y, e + ROUND[X.dtype] * (y.abs() + e) + 1e-37


def q4_gated(X, g, u, group, act):
    dt = X.dtype
    G, eG = q4(X, *g, group)
    U, eU = q4(X, *u, group)
    a, _ = act_both(G, act)
    ea = SLOPE * eG + ACT[dt] * (1 + G.abs())
    H, e = a * U, ea * U.abs() + a.abs() * eU + ea * eU
    return H, e + ROUND[dt] * (H.abs() + e) + 1e-37


def worst(got, value_bound):
    """Largest error over its bound (<= 1 passes); inf where a value is not finite,
    unless the exact one is beyond the type's range and the value the Inf of its sign."""
    v, e = value_bound
    over = v.to(got.dtype).isinf()
    got = got.double().cpu()
    assert got.shape == v.shape, (got.shape, v.shape)
    if not torch.equal(got[over], v[over].sign() * math.inf):
        return math.inf
    got, v, e = got[~over], v[~over], e[~over]
    if v.numel() == 0:
        return 0.0
    r = ((got - v).abs() / e).max()
    return float(r) if torch.isfinite(r) else math.inf
