"""The feed-forward operators as a program calls them, over the range of their sizes.

Four operators of one layer's life: the gated feed-forward block
H = act(X Wg) * (X Wu) (one call in a forward pass), the same block trained
(forward, then the gradients of X, Wg and Wu from dH), its products with 4-bit
weights for a few tokens (one matrix, or the gated pair), and the clipping of
all gradients by their global norm.  ``run`` computes each in its plain form,
in elementary torch operations in 32 bits, or (``own``) through
``roofline_gb300.feedforward``.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("silu", "gelu", "gelu_tanh", "relu")
CLIP_EPS = 1e-6


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a prefill or evaluation batch of a large layer, weights stored out x in
        dict(name="ff bf16 4096x4096x14336", op="ff", M=4096, D=4096, F=14336, dtype="bf16",
             act="silu", order="oi", pad=0),
        # a decode step of a few dozen sequences at once
        dict(name="ff bf16 48x4096x14336", op="ff", M=48, D=4096, F=14336, dtype="bf16",
             act="silu", order="oi", pad=0),
        # one token with unquantised weights
        dict(name="ff bf16 1x4096x11008", op="ff", M=1, D=4096, F=11008, dtype="bf16",
             act="silu", order="oi", pad=0),
        # FP32 with every size odd (no 16-byte rows), weights stored in x out
        dict(name="ff f32 1023x777x1025", op="ff", M=1023, D=777, F=1025, dtype="f32",
             act="gelu_tanh", order="io", pad=0),
        # a training step of a large layer
        dict(name="train bf16 8192x4096x11008", op="train", M=8192, D=4096, F=11008,
             dtype="bf16", act="silu", order="oi", pad=0),
        # a training step of a small layer in FP32, weights stored in x out
        dict(name="train f32 2048x1024x2816", op="train", M=2048, D=1024, F=2816, dtype="f32",
             act="gelu", order="io", pad=0),
        # packed sequences of odd length, odd widths, rows that are slices of wider buffers
        dict(name="train bf16 1025x777x1341", op="train", M=1025, D=777, F=1341, dtype="bf16",
             act="gelu_tanh", order="oi", pad=3),
        # one token through one quantised projection: the smallest call, latency counts
        dict(name="q4 bf16 1x4096x4096", op="q4", M=1, N=4096, K=4096, group=128, dtype="bf16",
             zeros=False, gated=False, act="silu"),
        # one token through the quantised gated pair
        dict(name="q4 gated bf16 1x14336x4096", op="q4", M=1, N=14336, K=4096, group=128,
             dtype="bf16", zeros=False, gated=True, act="silu"),
        # a batch of 16 tokens, the longest rows, zero points and small groups
        dict(name="q4 bf16 16x8192x28672", op="q4", M=16, N=8192, K=28672, group=64,
             dtype="bf16", zeros=True, gated=False, act="silu"),
        # the gradients of a small model, FP32
        dict(name="clip f32 40 of 1.3M", op="clip", count=40, total=1_300_000, share_f32=1.0,
             align=1, clipped=True),
        # the gradients of a large model, most of them bf16, a few FP32
        dict(name="clip mixed 400 of 600M", op="clip", count=400, total=600_000_000,
             share_f32=0.1, align=8, clipped=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ff", "train", "q4", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    act = rng.choice(ACTS)
    if op == "ff":
        return dict(op=op, M=_log(rng, 1, 4096), D=_log(rng, 64, 4096), F=_log(rng, 64, 14336),
                    dtype=dtype, act=act, order=rng.choice(["oi", "io"]),
                    pad=rng.choice([0, 0, 8, 3]))
    if op == "train":
        return dict(op=op, M=_log(rng, 1, 8192), D=_log(rng, 64, 4096), F=_log(rng, 64, 11008),
                    dtype=dtype, act=act, order=rng.choice(["oi", "io"]),
                    pad=rng.choice([0, 0, 8, 3]))
    if op == "q4":
        return dict(op=op, M=_log(rng, 1, 16), N=_log(rng, 64, 16384), K=_log(rng, 64, 28672),
                    group=rng.choice([32, 64, 128]), dtype=dtype, zeros=rng.random() < 0.5,
                    gated=rng.random() < 0.5, act=act)
    count = _log(rng, 1, 400)
    return dict(op=op, count=count, total=max(count, _log(rng, 1000, 600_000_000)),
                share_f32=rng.choice([0.0, 0.1, 1.0]) if dtype == "bf16" else 1.0,
                align=rng.choice([1, 8, 64]), clipped=rng.random() < 0.8)


def _sizes(case):
    """The tensors' sizes: a few large matrices, many small vectors, as a model has them."""
    rng = random.Random(case["count"] * 1_000_003 + case["total"])
    w = [math.exp(rng.uniform(0.0, 9.0)) for _ in range(case["count"])]
    s = sum(w)
    return [max(1, int(case["total"] * x / s)) for x in w]


def _placed(case):
    """[(dtype, first element, size)] of each tensor, and each arena's length."""
    rng = random.Random(case["count"])
    ends, out = {"bf16": 0, "f32": 0}, []
    for n in _sizes(case):
        d = "f32" if rng.random() < case["share_f32"] else "bf16"
        at = -(-ends[d] // case["align"]) * case["align"]
        out.append((d, at, n))
        ends[d] = at + n
    return out, ends


def work(case):
    if case["op"] in ("ff", "train"):
        M, D, F, b = case["M"], case["D"], case["F"], 2 if case["dtype"] == "bf16" else 4
        if case["op"] == "ff":  # X, both weights in; H out
            return {"bytes": b * (M * D + 2 * D * F + M * F), "flops": 4.0 * M * D * F}
        # X, both weights, dH in; H, dX and both weight gradients out
        return {"bytes": b * (2 * M * D + 4 * D * F + 2 * M * F), "flops": 12.0 * M * D * F}
    if case["op"] == "q4":
        M, N, K, b = case["M"], case["N"], case["K"], 2 if case["dtype"] == "bf16" else 4
        side = 2 if case["gated"] else 1
        per_row = (K + 1) // 2 + -(-K // case["group"]) * b * (2 if case["zeros"] else 1)
        return {"bytes": side * N * per_row + b * M * (K + N), "flops": 2.0 * side * M * N * K}
    n = sum((2 if d == "bf16" else 4) * s for d, _, s in _placed(case)[0])
    return {"bytes": 2 * n, "flops": 3.0 * sum(s for _, _, s in _placed(case)[0])}


# ------------------------------------------------------------------ the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, rows, cols, scale, dtype, pad):
    """A rows x cols matrix whose rows are slices of a buffer `pad` columns wider."""
    t = torch.randn((rows, cols + pad), generator=g, device="cuda")
    return (t * scale).to(dtype)[:, :cols]


def _quantised(g, N, K, group, dtype, zeros):
    """4-bit codes (two a byte, the even column in the low half), scales and zero points
    of a normal weight matrix, each group over its own range."""
    groups = -(-K // group)
    w = torch.randn((N, groups * group), generator=g, device="cuda") * K ** -0.5
    w = w.view(N, groups, group)
    if zeros:
        lo, hi = w.amin(2), w.amax(2)
        s = ((hi - lo) / 15).to(dtype)
        z = torch.round(-lo / s.float()).clamp(0, 15).to(dtype)
        q = torch.round(w / s.float()[..., None]) + z.float()[..., None]
    else:
        s, z = (w.abs().amax(2) / 7).to(dtype), None
        q = torch.round(w / s.float()[..., None]) + 8
    q = q.clamp_(0, 15).to(torch.uint8).view(N, -1)
    q[:, K:] = 0
    q = q[:, :2 * ((K + 1) // 2)]
    return (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous(), s.contiguous(), z


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] in ("ff", "train"):
        M, D, F, dt, pad = case["M"], case["D"], case["F"], DTYPES[case["dtype"]], case["pad"]
        st = {"case": case, "X": _normal(g, M, D, 1.0, dt, pad)}
        for w in ("Wg", "Wu"):
            st[w] = (_normal(g, F, D, D ** -0.5, dt, pad).t() if case["order"] == "oi"
                     else _normal(g, D, F, D ** -0.5, dt, pad))
        if case["op"] == "train":
            st["dH"] = _normal(g, M, F, F ** -0.5, dt, pad)
        return st
    if case["op"] == "q4":
        dt = DTYPES[case["dtype"]]
        st = {"case": case, "X": torch.randn((case["M"], case["K"]), generator=g,
                                             device="cuda").to(dt)}
        for k in range(2 if case["gated"] else 1):
            st["W%d" % k] = _quantised(g, case["N"], case["K"], case["group"], dt, case["zeros"])
        return st
    placed, ends = _placed(case)
    st = {"case": case, "grads": [], "outs": []}
    for d, n in ends.items():
        flat = torch.randn(n, generator=g, device="cuda")
        flat = flat.mul_(1e-3 * (1.0 + 9.0 * torch.rand(1, generator=g, device="cuda")))
        st["flat_" + d] = flat.to(DTYPES[d])
        st["out_" + d] = torch.zeros(n, dtype=DTYPES[d], device="cuda")
    last = {"bf16": 0, "f32": 0}
    for d, at, n in placed:
        st["flat_" + d][last[d]:at] = 0  # the gap before an aligned tensor holds no gradient
        last[d] = at + n
        st["grads"].append(st["flat_" + d][at:at + n])
        st["outs"].append(st["out_" + d][at:at + n])
    # gradients of norm 1e-3 * (1 to 10) * sqrt(n): clipped to about a tenth, or left alone
    st["max_norm"] = (1e-4 if case["clipped"] else 1e-1) * math.sqrt(case["total"])
    return st


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"ff": _own_ff, "train": _own_train, "q4": _own_q4, "clip": _own_clip}[op](state)
    return {"ff": _ff, "train": _train, "q4": _q4, "clip": _clip}[op](state)


def _own_ff(st):
    from roofline_gb300 import feedforward as ff
    return ff.gated_ff(st["X"], st["Wg"], st["Wu"], act=st["case"]["act"])


def _own_train(st):
    from roofline_gb300 import feedforward as ff
    act = st["case"]["act"]
    H, G, U = ff.gated_ff(st["X"], st["Wg"], st["Wu"], act=act, save=True)
    dX, dWg, dWu = ff.gated_ff_backward(st["dH"], st["X"], st["Wg"], st["Wu"], G, U, act=act)
    return {"H": H, "dX": dX, "dWg": dWg, "dWu": dWu}


def _own_q4(st):
    from roofline_gb300 import feedforward as ff
    c = st["case"]
    q, s, z = st["W0"]
    if not c["gated"]:
        return ff.q4_matmul(st["X"], q, s, zeros=z, group=c["group"])
    q1, s1, z1 = st["W1"]
    return ff.q4_gated(st["X"], q, s, q1, s1, zeros_g=z, zeros_u=z1, group=c["group"],
                       act=c["act"])


def _own_clip(st):
    from roofline_gb300 import feedforward as ff
    norm = ff.clip_grad_norm(st["grads"], st["max_norm"], out=st["outs"])
    return {"norm": norm, "bf16": st["out_bf16"], "f32": st["out_f32"]}


def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        p = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return (0.5 * g * (1.0 + t),
                0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 0.134145 * g * g))
    on = (g > 0).to(g.dtype)
    return g * on, on


def _ff(st):
    X = st["X"].float()
    a, _ = _act(X @ st["Wg"].float(), st["case"]["act"])
    return (a * (X @ st["Wu"].float())).to(st["X"].dtype)


def _train(st):
    X, Wg, Wu, dH = (st[k].float() for k in ("X", "Wg", "Wu", "dH"))
    dt = st["X"].dtype
    U = X @ Wu
    a, da = _act(X @ Wg, st["case"]["act"])
    dG, dU = dH * U * da, dH * a
    return {"H": (a * U).to(dt), "dX": (dG @ Wg.t() + dU @ Wu.t()).to(dt),
            "dWg": (X.t() @ dG).to(dt), "dWu": (X.t() @ dU).to(dt)}


def _dequantised(w, K, group, dtype):
    q, s, z = w
    n = torch.stack((q & 15, q >> 4), 2).view(q.shape[0], -1)[:, :K].to(dtype)
    at = torch.arange(K, device=q.device) // group
    zero = 8.0 if z is None else z.to(dtype)[:, at]
    return (n - zero) * s.to(dtype)[:, at]


def _q4(st):
    c, X = st["case"], st["X"].float()
    y = X @ _dequantised(st["W0"], c["K"], c["group"], torch.float32).t()
    if c["gated"]:
        y = _act(y, c["act"])[0] * (X @ _dequantised(st["W1"], c["K"], c["group"],
                                                      torch.float32).t())
    return y.to(st["X"].dtype)


def _clip(st):
    b, f = st["flat_bf16"].float(), st["flat_f32"]
    norm = torch.sqrt((b * b).sum() + (f * f).sum())
    c = torch.clamp(st["max_norm"] / (norm + CLIP_EPS), max=1.0)
    return {"norm": norm, "bf16": (b * c).to(torch.bfloat16), "f32": f * c}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "clip":
        flat = {d: st["flat_" + d].double() for d in ("bf16", "f32")}
        norm = math.sqrt(sum(float(torch.dot(t, t)) for t in flat.values()))
        c = min(1.0, st["max_norm"] / (norm + CLIP_EPS))
        return {"norm": norm, "bf16": flat["bf16"].mul_(c), "f32": flat["f32"].mul_(c)}
    nn = torch.nn.functional
    act = {"silu": nn.silu, "gelu": nn.gelu, "relu": nn.relu,
           "gelu_tanh": lambda g: nn.gelu(g, approximate="tanh")}[case["act"]]
    X = st["X"].double()
    if case["op"] == "q4":
        K, y = case["K"], []
        for k in range(2 if case["gated"] else 1):
            q, s, z = st["W%d" % k]
            acc = torch.zeros((case["M"], case["N"]), dtype=torch.float64, device="cuda")
            for at in range(0, s.shape[1]):  # group by group
                lo, hi = at * case["group"], min(K, (at + 1) * case["group"])
                code = torch.empty((case["N"], hi - lo), dtype=torch.float64, device="cuda")
                code[:, 0::2] = (q[:, lo // 2:(hi + 1) // 2] % 16).double()
                code[:, 1::2] = (q[:, lo // 2:hi // 2] // 16).double()
                code -= 8.0 if z is None else z[:, at:at + 1].double()
                acc += (X[:, lo:hi] @ code.t()) * s[:, at].double()
            y.append(acc)
        return act(y[0]) * y[1] if case["gated"] else y[0]
    leaves = [t.requires_grad_(case["op"] == "train")
              for t in (X, st["Wg"].double(), st["Wu"].double())]
    H = act(leaves[0] @ leaves[1]) * (leaves[0] @ leaves[2])
    if case["op"] == "ff":
        return H
    dX, dWg, dWu = torch.autograd.grad(H, leaves, st["dH"].double())
    return {"H": H.detach(), "dX": dX, "dWg": dWg, "dWu": dWu}
