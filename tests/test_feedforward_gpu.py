"""The feed-forward operators on the GPU against their formulas in 64 bits,
at the sizes, strides and values where they can go wrong.  The tolerances are
the bounds of ff_reference."""
import math

import pytest
import torch

from tests import ff_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
ACTS = ["silu", "gelu", "gelu_tanh", "relu"]


@pytest.fixture(scope="module")
def ff():
    from roofline_gb300 import build, feedforward
    build.build()
    return feedforward


def _mat(g, rows, cols, dt, scale=1.0, pad=0, off=0):
    """rows x cols, cut out of a buffer `pad` columns wider from column `off` on."""
    t = torch.randn((rows, cols + pad), generator=g) * scale
    return t.to(dt).cuda()[:, off:off + cols]


def _weight(g, D, F, dt, order, pad=0, off=0):
    s = max(D, 1) ** -0.5
    return _mat(g, F, D, dt, s, pad, off).t() if order == "oi" else _mat(g, D, F, dt, s, pad, off)


def _case(seed, M, D, F, dt, order, pad=0, off=0):
    g = torch.Generator().manual_seed(seed)
    return (_mat(g, M, D, dt, 1.0, pad, off), _weight(g, D, F, dt, order, pad, off),
            _weight(g, D, F, dt, order, pad, off), _mat(g, M, F, dt, 1.0, pad, off))


def _check_forward(ff, X, Wg, Wu, act):
    want = ref.forward(X, Wg, Wu, act)
    H, G, U = ff.gated_ff(X, Wg, Wu, act=act, save=True)
    H2 = ff.gated_ff(X, Wg, Wu, act=act)
    torch.cuda.synchronize()
    for name, t in (("H", H), ("G", G), ("U", U), ("H", H2)):
        assert ref.worst(t, want[name]) <= 1.0, name
    return G, U


def _check_backward(ff, dH, X, Wg, Wu, G, U, act):
    got = ff.gated_ff_backward(dH, X, Wg, Wu, G, U, act=act)
    torch.cuda.synchronize()
    want = ref.backward(dH, X, Wg, Wu, G, U, act)
    for name, t in zip(("dX", "dWg", "dWu"), got):
        assert ref.worst(t, want[name]) <= 1.0, name


SIZES = [(1, 1, 1), (1, 64, 64), (2, 8, 16), (3, 5, 7), (17, 100, 33), (31, 129, 127),
         (64, 64, 64), (128, 256, 128), (129, 72, 200), (257, 136, 264), (300, 520, 130),
         (1, 1000, 515), (8, 515, 1000), (33, 2048, 96), (700, 40, 300), (1030, 260, 1032)]


@pytest.mark.parametrize("order", ["oi", "io"])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES)
def test_forward_and_backward(ff, size, dt, order):
    act = ACTS[sum(size) % 4]
    X, Wg, Wu, dH = _case(sum(size), *size, dt, order)
    G, U = _check_forward(ff, X, Wg, Wu, act)
    _check_backward(ff, dH, X, Wg, Wu, G, U, act)


@pytest.mark.parametrize("order", ["oi", "io"])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [(1100, 200, 2100), (2500, 2200, 264), (264, 2200, 2500)])
def test_products_that_fill_the_gpu(ff, size, dt, order):
    """Enough tiles for pairs of CTAs: the forward product, dX and dW in turn."""
    X, Wg, Wu, dH = _case(sum(size), *size, dt, order)
    G, U = _check_forward(ff, X, Wg, Wu, "silu")
    _check_backward(ff, dH, X, Wg, Wu, G, U, "silu")


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [(2300, 64, 2200), (2300, 200, 2200), (2200, 2300, 130),
                                  (2048, 256, 2304)])
def test_fewer_blocks_of_k_than_stages(ff, size, dt):
    """Sums so short that a worker's blocks of K do not fill the ring of stages (tiles of
    pairs, and of one CTA): call after call, where each finds the shared memory and the
    tensor memory as the one before it left them, gives the same bits."""
    from roofline_gb300 import gemm
    X, Wg, Wu, dH = _case(sum(size), *size, dt, "oi")
    G, U = _check_forward(ff, X, Wg, Wu, "silu")
    H = ff.gated_ff(X, Wg, Wu)
    grads = ff.gated_ff_backward(dH, X, Wg, Wu, G, U)
    for _ in range(20):
        assert torch.equal(ff.gated_ff(X, Wg, Wu), H)
        for a, b in zip(ff.gated_ff_backward(dH, X, Wg, Wu, G, U), grads):
            assert torch.equal(a, b)
    assert gemm.check_status() == gemm.OK


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_activations(ff, dt, act):
    """Every activation over gate values from deep in one tail to deep in the other."""
    g = torch.Generator().manual_seed(5)
    D, F, M = 16, 160, 70
    X = torch.zeros(M, D)
    X[:, 0] = torch.linspace(-30, 30, M)  # G(i, j) = x_i * w_j: from -90 to 90
    X[:, 1:] = torch.randn((M, D - 1), generator=g) * 0.1
    Wg = torch.randn((D, F), generator=g) * 0.1
    Wg[0] = torch.linspace(-3, 3, F)
    Wu = torch.randn((D, F), generator=g)
    X, Wg, Wu = (t.to(dt).cuda() for t in (X, Wg, Wu))
    dH = torch.randn((M, F), generator=g).to(dt).cuda()
    G, U = _check_forward(ff, X, Wg, Wu, act)
    _check_backward(ff, dH, X, Wg, Wu, G, U, act)


@pytest.mark.parametrize("order", ["oi", "io"])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("pad,off", [(8, 0), (8, 8), (3, 0), (5, 1), (16, 3)])
@pytest.mark.parametrize("size", [(5, 96, 72), (130, 200, 136)])
def test_strided_and_misaligned(ff, size, pad, off, dt, order):
    X, Wg, Wu, dH = _case(pad + off, *size, dt, order, pad, off)
    G, U = _check_forward(ff, X, Wg, Wu, "silu")
    _check_backward(ff, dH, X, Wg, Wu, G, U, "silu")


@pytest.mark.parametrize("order", ["oi", "io"])
@pytest.mark.parametrize("pad", [0, 4, 3])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 7, 8, 9, 13, 16, 17])
def test_few_tokens_f32(ff, M, pad, order):
    """Around each number of tokens where FP32's few-token kernels change, with rows and
    sums that end inside a block's share, aligned and not; the same bits again with a
    workspace of the stated size."""
    D, F = (1036, 330) if M % 2 else (270, 1100)
    X, Wg, Wu, dH = _case(M + pad, M, D, F, F32, order, pad, pad)
    G, U = _check_forward(ff, X, Wg, Wu, ACTS[M % 4])
    _check_backward(ff, dH, X, Wg, Wu, G, U, ACTS[M % 4])
    op = 1 if order == "oi" else 0
    ws = [torch.empty(max(ff.gated_ff_workspace(M, D, F, ff.DT_F32, op, b), 1),
                      dtype=torch.uint8, device="cuda") for b in (False, True)]
    assert torch.equal(ff.gated_ff(X, Wg, Wu, workspace=ws[0]), ff.gated_ff(X, Wg, Wu))
    for a, b in zip(ff.gated_ff_backward(dH, X, Wg, Wu, G, U, workspace=ws[1]),
                    ff.gated_ff_backward(dH, X, Wg, Wu, G, U)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M", [2, 200])
def test_output_rows_of_wider_buffers_are_left_alone(ff, M, dt):
    """H goes into columns of a wider buffer; what is around them stays."""
    D, F = 72, 131
    X, Wg, Wu, _ = _case(9, M, D, F, dt, "oi")
    wide = torch.full((M + 1, F + 9), 7.0, dtype=dt, device="cuda")
    ff.gated_ff(X, Wg, Wu, out=wide[:M, 4:4 + F])
    torch.cuda.synchronize()
    assert ref.worst(wide[:M, 4:4 + F], ref.forward(X, Wg, Wu, "silu")["H"]) <= 1.0
    wide[:M, 4:4 + F] = 7.0
    assert bool((wide == 7.0).all())


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_empty_extents(ff, dt):
    for M, D, F in ((0, 8, 8), (4, 8, 0), (4, 0, 8), (0, 0, 0)):
        X, Wg, Wu, dH = _case(1, M, D, F, dt, "io")
        H, G, U = ff.gated_ff(X, Wg, Wu, save=True)
        dX, dWg, dWu = ff.gated_ff_backward(dH, X, Wg, Wu, G, U)
        torch.cuda.synchronize()
        for t, shape in ((H, (M, F)), (dX, (M, D)), (dWg, (D, F)), (dWu, (D, F))):
            assert tuple(t.shape) == shape and not bool(t.float().abs().sum())


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_nan_and_inf(ff, dt):
    """A NaN in a token's row reaches that row only; an Inf in X gives no finite G in its
    row (Inf or NaN), and leaves the others alone."""
    X, Wg, Wu, dH = _case(2, 140, 80, 96, dt, "oi")
    X = X.clone()
    X[3, 5] = math.nan
    X[130, 0] = math.inf
    H, G, U = ff.gated_ff(X, Wg, Wu, save=True)
    torch.cuda.synchronize()
    rows = torch.ones(140, dtype=torch.bool)
    rows[3] = rows[130] = False
    clean = X.clone()
    clean[~rows.cuda()] = 0
    want = ref.forward(clean, Wg, Wu, "silu")
    for name, t in (("H", H), ("G", G), ("U", U)):
        assert ref.worst(t[rows.cuda()], tuple(x[rows] for x in want[name])) <= 1.0
    assert bool(G[3].isnan().all()) and bool(H[3].isnan().all())
    assert not bool(G[130].isfinite().any())


def test_large_and_small_values_f32(ff):
    """FP32 inputs near the ends of the range: what is representable comes out."""
    g = torch.Generator().manual_seed(8)
    X = torch.randn((40, 64), generator=g) * 1e18
    Wg = torch.randn((64, 48), generator=g) * 1e-18
    Wu = torch.randn((64, 48), generator=g) * 1e-15
    X[0, 0], Wg[0, 0], Wu[0, 0] = 3.4e38, 1e-25, 1e-28
    X, Wg, Wu = X.cuda(), Wg.cuda(), Wu.cuda()
    _check_forward(ff, X, Wg, Wu, "gelu")


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_some_gradients_only(ff, dt):
    X, Wg, Wu, dH = _case(4, 90, 64, 80, dt, "io")
    _, G, U = ff.gated_ff(X, Wg, Wu, save=True)
    full = ff.gated_ff_backward(dH, X, Wg, Wu, G, U)
    dX, none1, none2 = ff.gated_ff_backward(dH, X, Wg, Wu, G, U, need_dw=False)
    none3, dWg, dWu = ff.gated_ff_backward(dH, X, Wg, Wu, G, U, need_dx=False)
    torch.cuda.synchronize()
    assert none1 is None and none2 is None and none3 is None
    for a, b in zip(full, (dX, dWg, dWu)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("act", ACTS)
def test_gradient_against_differences(ff, act):
    """The kernel's gradients against central differences of the kernel's own
    forward pass in FP32.  The difference of the loss L = sum dH * H over 2h is
    off by the bounds of H at both points over 2h, and by what the difference
    of the 64-bit formula with the same h is off."""
    M, D, F, h = 24, 40, 48, 2.0 ** -5
    X, Wg, Wu, dH = _case(11, M, D, F, F32, "io")
    _, G, U = ff.gated_ff(X, Wg, Wu, act=act, save=True)
    grads = ff.gated_ff_backward(dH, X, Wg, Wu, G, U, act=act)
    g = torch.Generator().manual_seed(12)
    for k in range(3):
        v = torch.randn(grads[k].shape, generator=g).cuda()
        v /= v.norm()
        num = num64 = slack = 0.0
        for sign in (1.0, -1.0):
            at = [X, Wg, Wu]
            at[k] = at[k] + sign * h * v
            H = ff.gated_ff(*at, act=act).double()
            val, e = ref.forward(*at, act)["H"]
            num += sign * float((dH.double() * H).sum()) / (2 * h)
            num64 += sign * float((dH.double().cpu() * val).sum()) / (2 * h)
            slack += float((dH.double().cpu().abs() * e).sum()) / (2 * h)
        want = float((grads[k].double() * v.double()).sum())
        exact = ref.backward(dH, X, Wg, Wu, G, U, act)[("dX", "dWg", "dWu")[k]]
        true = float((exact[0] * v.double().cpu()).sum())
        own = float((exact[1] * v.double().cpu().abs()).sum())
        # v rounded into at[k] moves the point by 2^-24 of it: within slack's 1e-5
        assert abs(num - want) <= abs(num64 - true) + slack + own
        # and the check has teeth: that slack is well under the gradient itself
        assert abs(num64 - true) + slack + own <= 0.5 * float(grads[k].norm())


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_own_stream_and_workspace(ff, dt):
    """Inputs made on one stream, the call on another, its own workspace; too small a one
    is refused; repeated calls give the same bits."""
    from roofline_gb300 import gemm
    M, D, F = 150, 77, 90
    X, Wg, Wu, dH = _case(6, M, D, F, dt, "oi")
    code = ff.DT_F32 if dt == F32 else ff.DT_BF16
    _, G0, U0 = ff.gated_ff(X, Wg, Wu, save=True)
    first = ff.gated_ff_backward(dH, X, Wg, Wu, G0, U0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    need = [max(ff.gated_ff_workspace(M, D, F, code, gemm.OP_T, b), 256) for b in (False, True)]
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in need]
    H, G, U = ff.gated_ff(X, Wg, Wu, save=True, stream=side, workspace=ws[0])
    got = ff.gated_ff_backward(dH, X, Wg, Wu, G, U, stream=side, workspace=ws[1])
    torch.cuda.synchronize()
    assert torch.equal(G, G0) and torch.equal(U, U0)
    for a, b in zip(first, got):
        assert torch.equal(a, b)
    with pytest.raises(gemm.GemmError):
        ff.gated_ff_backward(dH, X, Wg, Wu, G, U, workspace=ws[1][:256])
    assert gemm.check_status() == gemm.OK


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_captured_in_a_graph(ff, dt):
    X, Wg, Wu, dH = _case(6, 200, 128, 144, dt, "oi")
    H, G, U = ff.gated_ff(X, Wg, Wu, save=True)
    want = ff.gated_ff_backward(dH, X, Wg, Wu, G, U)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        H2, G2, U2 = ff.gated_ff(X, Wg, Wu, save=True)
        got = ff.gated_ff_backward(dH, X, Wg, Wu, G2, U2)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(H, H2)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("size", [(256, 256, 128), (1100, 200, 2100)], ids=["one", "pairs"])
def test_stalled_pipeline_reports_timeout(ff, size, monkeypatch):
    """With a test hook the producer issues no copy: the waits run out (no copy or MMA is in
    flight), the status says so, and the next call is right.  Tiles of one CTA and of pairs."""
    from roofline_gb300 import gemm
    X, Wg, Wu, _ = _case(3, *size, BF16, "oi")
    assert gemm.check_status() == gemm.OK
    with monkeypatch.context() as m:
        m.setenv("GEMM_DEBUG_STALL_PRODUCER", "1")
        m.setenv("GEMM_DEBUG_WAIT_LIMIT_NS", "2000000")  # 2 ms
        ff.gated_ff(X, Wg, Wu)
        assert gemm.check_status() == gemm.ERR_DEVICE_TIMEOUT
    assert gemm.check_status() == gemm.OK
    _check_forward(ff, X, Wg, Wu, "silu")
    assert gemm.check_status() == gemm.OK


@pytest.mark.parametrize("order", ["oi", "io"])
@pytest.mark.parametrize("size", [(70, 70000, 200), (300, 33000, 1100), (1, 32800, 40),
                                  (40000, 72, 130), (70000, 40, 300), (130, 100, 20000),
                                  (300, 600, 16400)])
def test_long_sums_bf16(ff, size, order):
    """Sums longer than an accumulator keeps, of the block (one CTA a tile and pairs), of dX
    and of dW, and launches whose other product's sums are short: the bounds of short ones,
    and equal bits on repeat."""
    from roofline_gb300 import gemm
    X, Wg, Wu, dH = _case(sum(size), *size, BF16, order)
    G, U = _check_forward(ff, X, Wg, Wu, "silu")
    _check_backward(ff, dH, X, Wg, Wu, G, U, "silu")
    H = ff.gated_ff(X, Wg, Wu)
    grads = ff.gated_ff_backward(dH, X, Wg, Wu, G, U)
    for _ in range(5):
        assert torch.equal(ff.gated_ff(X, Wg, Wu), H)
        for a, b in zip(ff.gated_ff_backward(dH, X, Wg, Wu, G, U), grads):
            assert torch.equal(a, b)
    assert gemm.check_status() == gemm.OK


@pytest.mark.parametrize("K", [32768, 32769, 90000, 400000])
def test_long_sums_of_one_sign_bf16(ff, K):
    """Products of one sign, where every rounding towards zero has the same sign: however
    long, a sum is off by no more than a part of 32768 is.  An MMA adds 16 of K by at most two
    roundings of 2^-23 to a sum that grows evenly: 2^-12 over 2048 of them.  Parts are
    added in FP32, 2^-24 each."""
    g = torch.Generator().manual_seed(K)
    tol = 2.0 ** -12 + (K // 32768 + 1) * 2.0 ** -24
    X = (torch.rand((40, K), generator=g) + 0.5).to(BF16).cuda()
    Wg = (torch.rand((24, K), generator=g) + 0.5).to(BF16).cuda().t()
    _, G, U = ff.gated_ff(X, Wg, Wg, act="relu", save=True)
    want = X.double() @ Wg.double()
    assert bool(((G.double() - want).abs() <= tol * want).all()) and torch.equal(G, U)
    # dW over K tokens, dG = dU = dH exactly
    X, dH = X.t()[:, :16].contiguous(), X.t()[:, 16:32].contiguous()
    one = torch.ones((K, 16), device="cuda")
    W = torch.ones((16, 16), dtype=BF16, device="cuda")
    _, dWg, dWu = ff.gated_ff_backward(dH, X, W, W, one, one, act="relu", need_dx=False)
    want = X.double().t() @ dH.double()
    torch.cuda.synchronize()
    # rounding keeps the order: the result lies between the rounded ends of what the sum may be
    low, high = ((want * (1 + d)).float().to(BF16) for d in (-tol, tol))
    assert bool(((dWg >= low) & (dWg <= high)).all())
    assert torch.equal(dWg, dWu)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_wait_limit_grows_with_the_sum(ff, dt, monkeypatch):
    """A sum that takes longer than the limit of a short wait (here 0.1 ms, for 4096 blocks of
    K of 0.2 us each or more) is not taken for a stalled one."""
    from roofline_gb300 import gemm
    M, D, F = 40, 1 << 18, 64
    X, Wg, Wu, _ = _case(5, M, D, F, dt, "oi")
    want = ff.gated_ff(X, Wg, Wu)
    assert gemm.check_status() == gemm.OK
    with monkeypatch.context() as m:
        m.setenv("GEMM_DEBUG_WAIT_LIMIT_NS", "100000")
        got = ff.gated_ff(X, Wg, Wu)
        assert gemm.check_status() == gemm.OK
    assert torch.equal(got, want)


# ------------------------------------------------------------------ 4-bit products

def _quant(g, N, K, group, dt, zeros, pad=0):
    """Random codes (all 16 values), scales of both signs, zero points off the grid too."""
    q = torch.randint(0, 256, (N, (K + 1) // 2 + pad), generator=g, dtype=torch.uint8)
    groups = -(-K // group)
    s = (torch.randn((N, groups), generator=g) * max(K, 1) ** -0.5).to(dt).cuda()
    z = (torch.rand((N, groups), generator=g) * 15).to(dt).cuda() if zeros else None
    return q.cuda()[:, :(K + 1) // 2], s, z


Q4_SIZES = [(1, 1, 1), (1, 8, 32), (1, 16, 64), (2, 3, 5), (3, 17, 33), (1, 64, 127),
            (4, 100, 256), (5, 33, 300), (7, 130, 1025), (8, 256, 512), (9, 65, 640),
            (16, 48, 2048), (17, 96, 1000), (33, 40, 96), (1, 1031, 4096), (2, 40, 9001)]


@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("zeros", [False, True], ids=["z8", "zeros"])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", Q4_SIZES)
def test_q4(ff, size, dt, zeros, group):
    M, N, K = size
    g = torch.Generator().manual_seed(M + N + K + group)
    X = _mat(g, M, K, dt)
    w, u = _quant(g, N, K, group, dt, zeros), _quant(g, N, K, group, dt, zeros)
    Y = ff.q4_matmul(X, w[0], w[1], zeros=w[2], group=group)
    act = ACTS[(M + N) % 4]
    H = ff.q4_gated(X, w[0], w[1], u[0], u[1], zeros_g=w[2], zeros_u=u[2], group=group, act=act)
    torch.cuda.synchronize()
    assert ref.worst(Y, ref.q4_rounded(X, *w, group)) <= 1.0
    assert ref.worst(H, ref.q4_gated(X, w, u, group, act)) <= 1.0


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M", [64, 100, 257, 1000])
@pytest.mark.parametrize("N,K", [(70, 513), (300, 2048)])
def test_q4_many_tokens(ff, N, K, M, dt):
    """Prompts: many passes over the weights, the last one not full."""
    g = torch.Generator().manual_seed(N + M)
    X = _mat(g, M, K, dt)
    w, u = _quant(g, N, K, 128, dt, True), _quant(g, N, K, 128, dt, True)
    Y = ff.q4_matmul(X, w[0], w[1], zeros=w[2], group=128)
    H = ff.q4_gated(X, w[0], w[1], u[0], u[1], zeros_g=w[2], zeros_u=u[2], group=128, act="gelu")
    torch.cuda.synchronize()
    assert ref.worst(Y, ref.q4_rounded(X, *w, 128)) <= 1.0
    assert ref.worst(H, ref.q4_gated(X, w, u, 128, "gelu")) <= 1.0


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 3, 16, 19])
@pytest.mark.parametrize("N,K", [(5, 20000), (33, 12345), (200, 8192), (1000, 8200), (3000, 4104)])
def test_q4_few_rows_long_sums(ff, N, K, M, dt):
    """Blocks of rows whose sums several thread blocks share, each a part that need not
    be whole steps; equal calls give equal bits."""
    g = torch.Generator().manual_seed(N + M)
    X = _mat(g, M, K, dt)
    w, u = _quant(g, N, K, 64, dt, True), _quant(g, N, K, 64, dt, True)
    Y = ff.q4_matmul(X, w[0], w[1], zeros=w[2], group=64)
    H = ff.q4_gated(X, w[0], w[1], u[0], u[1], zeros_g=w[2], zeros_u=u[2], group=64, act="silu")
    again = ff.q4_matmul(X, w[0], w[1], zeros=w[2], group=64)
    torch.cuda.synchronize()
    assert torch.equal(Y, again)
    assert ref.worst(Y, ref.q4_rounded(X, *w, 64)) <= 1.0
    assert ref.worst(H, ref.q4_gated(X, w, u, 64, "silu")) <= 1.0


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("pad,off", [(0, 1), (1, 0), (3, 1), (16, 0), (15, 5)])
@pytest.mark.parametrize("K", [96, 513])
def test_q4_strides(ff, K, pad, off, dt):
    """Rows of codes any number of bytes apart, X and Y cut out of wider buffers."""
    M, N, group = 5, 70, 64
    g = torch.Generator().manual_seed(pad + off + K)
    X = _mat(g, M, K, dt, 1.0, pad + off, off)
    q, s, z = _quant(g, N, K, group, dt, True, pad)
    wide = torch.full((M, N + pad + 2), 7.0, dtype=dt, device="cuda")
    ff.q4_matmul(X, q, s, zeros=z, group=group, out=wide[:, 1:1 + N])
    torch.cuda.synchronize()
    assert ref.worst(wide[:, 1:1 + N], ref.q4_rounded(X, q, s, z, group)) <= 1.0
    wide[:, 1:1 + N] = 7.0
    assert bool((wide == 7.0).all())


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_q4_empty_and_nan(ff, dt):
    g = torch.Generator().manual_seed(1)
    q, s, z = _quant(g, 20, 100, 32, dt, True)
    assert ff.q4_matmul(_mat(g, 0, 100, dt), q, s, zeros=z, group=32).shape == (0, 20)
    # K = 0: zeros
    q0 = torch.zeros((20, 0), dtype=torch.uint8, device="cuda")
    s0 = torch.zeros((20, 0), dtype=dt, device="cuda")
    y = ff.q4_matmul(_mat(g, 3, 0, dt), q0, s0, group=32)
    torch.cuda.synchronize()
    assert y.shape == (3, 20) and not bool(y.any())
    # a NaN in one token reaches its row only; the last code of an odd K is not read as a weight
    X = _mat(g, 12, 99, dt).clone()
    X[4, 7] = math.nan
    q, s, z = _quant(g, 20, 99, 32, dt, False)
    Y = ff.q4_matmul(X, q, s, group=32)
    torch.cuda.synchronize()
    rows = [i for i in range(12) if i != 4]
    X[4] = 0
    val, e = ref.q4_rounded(X, q, s, None, 32)
    assert ref.worst(Y[rows], (val[rows], e[rows])) <= 1.0
    assert bool(Y[4].isnan().all())


def _by_ieee(got, want, bound):
    """NaN where the formula's value is NaN, Inf of its sign where it is Inf or beyond the
    type, and within the bound elsewhere."""
    got = got.cpu()
    assert torch.equal(got.isnan(), want.isnan())
    ok = ~want.isnan()
    assert ref.worst(got[ok], (want[ok], bound[ok])) <= 1.0


# few and many rows, sums that several thread blocks share, one token to three passes
Q4_RANGE_SIZES = [(1, 40, 256), (2, 200, 300), (5, 33, 8200), (19, 70, 999), (40, 24, 513)]


@pytest.mark.parametrize("group", [32, 128, 256])
@pytest.mark.parametrize("zeros", [False, True], ids=["z8", "zeros"])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", Q4_RANGE_SIZES)
def test_q4_inf_by_ieee_rules(ff, size, dt, zeros, group):
    """Inf and NaN in X end where the formula in 64 bits says: Inf of the sign of the weight
    that one Inf meets, NaN where it meets a weight of zero, an Inf of the other sign or a
    NaN; tokens without any are as they were."""
    M, N, K = size
    g = torch.Generator().manual_seed(sum(size) + group)
    X = _mat(g, M, K, dt).clone()
    w, u = _quant(g, N, K, group, dt, zeros), _quant(g, N, K, group, dt, zeros)
    if zeros:
        for t in (w[2], u[2]):
            t[::3] = 5.0  # zero points that codes meet
    X[0, K // 3] = math.inf
    if M > 1:
        X[M - 1, K - 1] = -math.inf
    if M > 4:
        X[2, 1], X[2, K - 2] = math.inf, -math.inf
        X[3, 4] = math.nan
    Y = ff.q4_matmul(X, w[0], w[1], zeros=w[2], group=group)
    H = ff.q4_gated(X, w[0], w[1], u[0], u[1], zeros_g=w[2], zeros_u=u[2], group=group, act="relu")
    again = ff.q4_matmul(X, w[0], w[1], zeros=w[2], group=group)
    torch.cuda.synchronize()
    clean = X.clone()
    clean[~X.isfinite()] = 0
    bound, bound_h = ref.q4_rounded(clean, *w, group)[1], ref.q4_gated(clean, w, u, group, "relu")[1]
    want, want_u = ref.q4(X, *w, group)[0], ref.q4(X, *u, group)[0]
    assert not bool(want[0].isfinite().any()) and bool(want[0].isinf().any())
    _by_ieee(Y, want, bound)
    _by_ieee(H, torch.clamp(want, min=0) * want_u, bound_h)
    assert torch.equal(Y.nan_to_num(), again.nan_to_num())


@pytest.mark.parametrize("group", [32, 128, 256])
@pytest.mark.parametrize("zeros", [False, True], ids=["z8", "zeros"])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", Q4_RANGE_SIZES)
def test_q4_large_values(ff, size, dt, zeros, group):
    """X near the end of the type's range, of one sign in some tokens, by scales that bring
    the exact sums back into it: what is representable comes out, within the bounds."""
    M, N, K = size
    g = torch.Generator().manual_seed(sum(size) + group + 1)
    X = torch.randn((M, K), generator=g).clamp(-4, 4)
    X[::2] = X[::2].abs()
    X = (X * 2.0 ** 125).to(dt).cuda()   # up to 2^127
    q, s, z = _quant(g, N, K, group, dt, zeros)
    s = (s.float() * 2.0 ** -16).to(dt)  # sums of K terms of about 2^(125 - 16 + 3) K^-1/2
    Y = ff.q4_matmul(X, q, s, zeros=z, group=group)
    torch.cuda.synchronize()
    want = ref.q4_rounded(X, q, s, z, group)
    assert float(want[0].abs().max()) < 3e38
    assert ref.worst(Y, want) <= 1.0


def test_q4_on_another_stream_and_in_a_graph(ff):
    g = torch.Generator().manual_seed(1)
    X = _mat(g, 1, 512, BF16)
    q, s, z = _quant(g, 300, 512, 128, BF16, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = ff.q4_matmul(X, q, s, zeros=z, stream=side)
    b = ff.q4_matmul(X, q, s, zeros=z)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = ff.q4_matmul(X, q, s, zeros=z)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, c)


# ------------------------------------------------------------------ norm and clipping

def _grads(g, specs, scale=0.1):
    """Tensors given as (size, dtype, offset of the first element in its buffer)."""
    out = []
    for n, dt, off in specs:
        t = (torch.randn(n + off, generator=g) * scale).to(dt).cuda()
        out.append(t[off:])
    return out


def _norm64(ts):
    return math.sqrt(sum(float((t.double() ** 2).sum()) for t in ts))


def _check_clip(ts, outs, norm, max_norm):
    """norm: squares and sums of a thread's few values in FP32 (2^-24 each, at most 64 of
    them, half of that after the root), the rest in 64 bits, one rounding: 2^-18.  Outputs:
    the norm's error, two roundings of the factor, one product, one rounding."""
    n64 = _norm64(ts)
    assert abs(float(norm) - n64) <= 2.0 ** -18 * n64
    c = min(1.0, max_norm / (n64 + 1e-6))
    for t, o in zip(ts, outs):
        want = t.double() * c
        tol = 2.0 ** -17 + ref.ROUND[t.dtype]
        # a result below the normal range is rounded to a multiple of 2^-149 (FP32)
        # or 2^-133 (BF16)
        tiny = 2.0 ** -149 if t.dtype == F32 else 2.0 ** -133
        assert bool(((o.double() - want).abs() <= tol * want.abs() + tiny).all())


SPECS = {
    "one": [(1, F32, 0)],
    "small": [(5, F32, 0), (0, F32, 0), (7, BF16, 1), (1, BF16, 0), (0, BF16, 0)],
    "odd offsets": [(1000 + 37 * i, F32 if i % 3 else BF16, i % 9) for i in range(30)],
    "large and small": [(3_000_001, BF16, 0), (3, F32, 1), (1_000_003, F32, 3), (1, BF16, 5)],
    "many": [(1 + (i * 7919) % 997, BF16 if i % 2 else F32, i % 4) for i in range(2500)],
}


@pytest.mark.parametrize("max_norm", [0.5, 1e6, 0.0])
@pytest.mark.parametrize("name", list(SPECS))
def test_clip(ff, name, max_norm):
    g = torch.Generator().manual_seed(len(name))
    ts = _grads(g, SPECS[name])
    before = [t.clone() for t in ts]
    outs = [torch.full_like(t, 9.0) for t in ts]
    norm = ff.clip_grad_norm(ts, max_norm, out=outs)
    only = ff.grad_norm(ts)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    assert float(norm) == float(only)
    _check_clip(before, outs, norm, max_norm)
    # in place: the same bits
    norm2 = ff.clip_grad_norm(ts, max_norm)
    torch.cuda.synchronize()
    assert float(norm2) == float(norm)
    assert all(torch.equal(a, b) for a, b in zip(ts, outs))


def test_clip_neighbours_are_left_alone(ff):
    """Tensors next to one another in one buffer, inputs and outputs aligned differently."""
    g = torch.Generator().manual_seed(3)
    for dt in (F32, BF16):
        flat = torch.randn(5000, generator=g).to(dt).cuda()
        dest = torch.full((5003,), 9.0, dtype=dt, device="cuda")
        cuts = [0, 1, 9, 10, 1033, 1040, 3001, 4999]
        ts = [flat[a:b] for a, b in zip(cuts, cuts[1:])]
        outs = [dest[a + 3:b + 3] for a, b in zip(cuts, cuts[1:])]
        norm = ff.clip_grad_norm(ts, 1.0, out=outs)
        torch.cuda.synchronize()
        _check_clip(ts, outs, norm, 1.0)
        assert bool((dest[:3] == 9.0).all()) and float(dest[5002]) == 9.0


def test_clip_no_tensors_and_empty_ones(ff):
    norm = ff.clip_grad_norm([], 1.0)
    empty = ff.clip_grad_norm([torch.zeros(0, device="cuda")], 1.0)
    zero = [torch.zeros(1000, device="cuda")]
    nz = ff.clip_grad_norm(zero, 1.0)
    torch.cuda.synchronize()
    assert float(norm) == 0.0 and float(empty) == 0.0 and float(nz) == 0.0
    assert not bool(zero[0].any())


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_clip_not_finite(ff, dt):
    """Inf: the norm is Inf, the factor 0 (Inf * 0 = NaN at the Inf); NaN: all NaN."""
    for bad in (math.inf, math.nan):
        t = torch.ones(2000, dtype=dt, device="cuda")
        t[1234] = bad
        norm = ff.clip_grad_norm([t], 1.0)
        torch.cuda.synchronize()
        if bad == math.inf:
            assert float(norm) == math.inf
            assert bool(t[1234].isnan()) and int(t.isnan().sum()) == 1 and float(t[0]) == 0.0
        else:
            assert math.isnan(float(norm)) and bool(t.isnan().all())


def test_clip_range(ff):
    """Squares beyond FP32's range: 1e25 squared overflows a float, 1e-30 squared underflows."""
    for v in (1e25, 1e-30):
        t = torch.full((3000,), v, device="cuda")
        norm = ff.grad_norm([t])
        torch.cuda.synchronize()
        want = float(t[0].double()) * math.sqrt(3000.0)
        assert abs(float(norm) - want) <= 2.0 ** -18 * want


def test_clip_stream_graph_and_workspace(ff):
    from roofline_gb300 import gemm
    g = torch.Generator().manual_seed(3)
    ts = _grads(g, SPECS["odd offsets"])
    outs = [torch.empty_like(t) for t in ts]
    norm = ff.clip_grad_norm(ts, 0.25, out=outs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(int(gemm.load().grad_norm_clip_workspace(len(ts))), dtype=torch.uint8,
                     device="cuda")
    outs2 = [torch.empty_like(t) for t in ts]
    norm2 = ff.clip_grad_norm(ts, 0.25, out=outs2, stream=side, workspace=ws)
    torch.cuda.synchronize()
    assert float(norm) == float(norm2) and all(torch.equal(a, b) for a, b in zip(outs, outs2))
    with pytest.raises(gemm.GemmError):
        ff.clip_grad_norm(ts, 0.25, out=outs2, workspace=ws[:64])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm3 = ff.clip_grad_norm(ts, 0.25, out=outs2)
    for o in outs2:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert float(norm) == float(norm3) and all(torch.equal(a, b) for a, b in zip(outs, outs2))


# ------------------------------------------------------------------ refusals of tensor calls

def test_integers_beyond_an_int_are_refused(ff):
    """A group or act that a C int does not hold is refused, not cut to its low 32 bits (a
    group so cut reads scales that its tensor does not have); nothing of the call runs."""
    from roofline_gb300 import gemm
    g = torch.Generator().manual_seed(2)
    X = _mat(g, 2, 256, BF16)
    q = torch.zeros((8, 128), dtype=torch.uint8, device="cuda")
    s = torch.ones((8, 1), dtype=BF16, device="cuda")  # one group, as 2^32 + 32 would have
    for group in (2 ** 32 + 32, 2 ** 32 + 128, 2 ** 63 - 1, 2 ** 63, -32, 0, 1.5, None):
        with pytest.raises(ValueError):
            ff.q4_matmul(X, q, s, group=group)
        with pytest.raises(ValueError):
            ff.q4_gated(X, q, s, q, s, group=group)
    with pytest.raises(gemm.GemmError):  # an int, but not a group that there is
        ff.q4_matmul(X, q, s, group=512)
    X, Wg, Wu, dH = _case(3, 4, 8, 6, F32, "io")
    _, G, U = ff.gated_ff(X, Wg, Wu, save=True)
    for act in (2 ** 32, -2 ** 32, 2 ** 64, 1.5):
        with pytest.raises(ValueError):
            ff.gated_ff(X, Wg, Wu, act=act)
        with pytest.raises(ValueError):
            ff.gated_ff_backward(dH, X, Wg, Wu, G, U, act=act)
    with pytest.raises(gemm.GemmError):
        ff.gated_ff(X, Wg, Wu, act=4)
    with pytest.raises(ValueError):
        ff.clip_grad_norm([X], "much")


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_expanded_matrices_are_refused(ff, dt):
    """One value expanded to a column (or to a row of a W.t()) has one element behind it,
    not one a row: refused, as input and as output.  One row expanded has no second row."""
    M, D, F = 40, 24, 16
    X, Wg, Wu, dH = _case(3, M, D, F, dt, "io")
    one = torch.ones((1, 1), dtype=dt, device="cuda")
    bad = []
    wg1, wu1 = Wg[:1], Wu[:1]                               # D = 1
    bad.append(lambda: ff.gated_ff(one.expand(M, 1), wg1, wu1))
    bad.append(lambda: ff.gated_ff(X, one.expand(D, 1), Wu[:, :1]))   # F = 1
    bad.append(lambda: ff.gated_ff(X, Wg[:, :1], one.expand(D, 1)))
    bad.append(lambda: ff.gated_ff(X[:, :1], one.expand(1, F), wu1))  # D = 1, by columns
    bad.append(lambda: ff.gated_ff(X, Wg[:, :1], Wu[:, :1], out=one.expand(M, 1)))
    bad.append(lambda: ff.gated_ff(X[:1].expand(M, D), Wg, Wu))
    _, G, U = ff.gated_ff(X, Wg[:, :1], Wu[:, :1], save=True)
    f1 = torch.ones((1, 1), device="cuda").expand(M, 1)
    d1 = dH[:, :1].contiguous()
    for args in ((one.expand(M, 1), X, G, U), (d1, X, f1, U), (d1, X, G, f1)):
        bad.append(lambda a=args: ff.gated_ff_backward(a[0], a[1], Wg[:, :1], Wu[:, :1], a[2], a[3]))
    q = torch.zeros((1, 1), dtype=torch.uint8, device="cuda")
    s = torch.ones((F, 1), dtype=dt, device="cuda")
    bad.append(lambda: ff.q4_matmul(X[:, :2], q.expand(F, 1), s, group=32))
    bad.append(lambda: ff.q4_matmul(one.expand(M, 1), torch.zeros((F, 1), dtype=torch.uint8,
                                                                  device="cuda"), s, group=32))
    bad.append(lambda: ff.q4_matmul(X[:, :2], torch.zeros((1, 1), dtype=torch.uint8, device="cuda"),
                                    s[:1], group=32, out=one.expand(M, 1)))
    for call in bad:
        with pytest.raises(ValueError):
            call()
    # what is expanded along one row or column only, or empty, is what it says
    row = torch.randn((1, D), generator=torch.Generator().manual_seed(4)).to(dt).cuda()
    h = ff.gated_ff(row.expand(1, D), Wg, Wu)
    torch.cuda.synchronize()
    assert ref.worst(h, ref.forward(row, Wg, Wu, "silu")["H"]) <= 1.0
    assert ff.gated_ff(one.expand(0, 1), wg1, wu1).shape == (0, F)
    assert ff.gated_ff(one[:, :0].expand(M, 0), Wg[:0], Wu[:0]).shape == (M, F)


# ------------------------------------------------------------------ streams and memory

def _calls(ff):
    """{name: f(stream) -> its new tensors} of every operator, on inputs that stay."""
    g = torch.Generator().manual_seed(5)
    M, D, F = 70, 96, 264
    X, Wg, Wu, dH = _case(5, M, D, F, BF16, "oi")
    _, G, U = ff.gated_ff(X, Wg, Wu, save=True)
    w = _quant(g, F, D, 32, BF16, True)
    grads = [X, dH, G]
    outs = [torch.empty_like(t) for t in grads]
    return {
        "forward": lambda s: ff.gated_ff(X, Wg, Wu, save=True, stream=s),
        "backward": lambda s: ff.gated_ff_backward(dH, X, Wg, Wu, G, U, stream=s),
        "q4": lambda s: (ff.q4_matmul(X, w[0], w[1], zeros=w[2], group=32, stream=s),),
        "q4 gated": lambda s: (ff.q4_gated(X, w[0], w[1], w[0], w[1], zeros_g=w[2], zeros_u=w[2],
                                           group=32, stream=s),),
        "norm": lambda s: (ff.grad_norm(grads, stream=s),),
        "clip": lambda s: (ff.clip_grad_norm(grads, 0.5, out=outs, stream=s),),
    }


def _write_later(tensors):
    """Frees blocks of these tensors' sizes on the current stream, with writes to them
    enqueued there that run some 25 ms from now."""
    blocks = [torch.empty(t.untyped_storage().nbytes(), dtype=torch.uint8, device="cuda")
              for t in tensors]
    torch.cuda._sleep(50_000_000)
    for b in blocks:
        b.fill_(7)


@pytest.mark.parametrize("name", ["forward", "backward", "q4", "q4 gated", "norm", "clip"])
def test_new_outputs_on_another_stream(ff, name):
    """Memory that the current stream is still to write is not given to a call on another
    stream that does not wait for it; what the current stream enqueues on an output after
    waiting for the call is done before the output's memory is used again there."""
    call = _calls(ff)[name]
    want = call(None)
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        _write_later(want)
        got = call(side)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    # used on the current stream behind 25 ms of work, freed, and allocated again on `side`
    copies = [torch.empty_like(t) for t in got]
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    for c, t in zip(copies, got):
        c.copy_(t)
    del got, t, a, b
    more = call(side)
    with torch.cuda.stream(side):
        for m in more:
            m.fill_(7)
    torch.cuda.synchronize()
    for c, b in zip(copies, want):
        assert torch.equal(c, b)


def test_calls_on_two_streams_at_once(ff):
    """Calls without a workspace share none: on two streams at once, with other inputs, each
    gives the bits that it gives alone."""
    from roofline_gb300 import gemm
    cases = [_case(20 + i, 300, 203, 1111, dt, "oi", 3) for i, dt in enumerate((F32, BF16))]
    grads = [[torch.randn(50_000 + 999 * i + j).cuda() for j in range(20)] for i in range(2)]

    def step(i, stream):
        X, Wg, Wu, dH = cases[i]
        H, G, U = ff.gated_ff(X, Wg, Wu, save=True, stream=stream)
        return [H, G, U, *ff.gated_ff_backward(dH, X, Wg, Wu, G, U, stream=stream),
                ff.grad_norm(grads[i], stream=stream)]
    want = [step(i, None) for i in range(2)]
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s in sides:
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)  # both queues fill before either runs
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            got[i].append(step(i, sides[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for call in got[i]:
            for a, b in zip(call, want[i]):
                assert torch.equal(a, b)
    assert gemm.check_status() == gemm.OK


def test_graph_keeps_its_workspace(ff):
    """A captured call's scratch stays its own when a later call needs more."""
    X, Wg, Wu, dH = _case(30, 100, 72, 136, F32, "io")
    ts = [torch.randn(5000).cuda() for _ in range(10)]
    H, G, U = ff.gated_ff(X, Wg, Wu, save=True)
    want = [H, *ff.gated_ff_backward(dH, X, Wg, Wu, G, U), ff.grad_norm(ts)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        H2, G2, U2 = ff.gated_ff(X, Wg, Wu, save=True)
        got = [H2, *ff.gated_ff_backward(dH, X, Wg, Wu, G2, U2), ff.grad_norm(ts)]
    large = _case(31, 2000, 1024, 2816, F32, "io")
    for _ in range(2):
        _, G3, U3 = ff.gated_ff(*large[:3], save=True)
        ff.gated_ff_backward(large[3], *large[:3], G3, U3)
        ff.grad_norm([t for t in ts for _ in range(300)])
        torch.cuda.synchronize()
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_workspaces_that_are_none_are_refused(ff):
    from roofline_gb300 import gemm
    X, Wg, Wu, dH = _case(6, 40, 64, 72, F32, "io")
    _, G, U = ff.gated_ff(X, Wg, Wu, save=True)
    need = ff.gated_ff_workspace(40, 64, 72, ff.DT_F32, backward=True)
    host = torch.empty(need, dtype=torch.uint8)
    one = torch.empty(1, dtype=torch.uint8, device="cuda").expand(need)
    apart = torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2]
    for ws in (host, one, apart, 4096):
        for call in (lambda: ff.gated_ff(X, Wg, Wu, workspace=ws),
                     lambda: ff.gated_ff_backward(dH, X, Wg, Wu, G, U, workspace=ws),
                     lambda: ff.grad_norm([X], workspace=ws),
                     lambda: ff.clip_grad_norm([X], 1.0, workspace=ws)):
            with pytest.raises(ValueError):
                call()
    ts = [X, G]
    ws = torch.empty(ff.grad_norm_workspace(2), dtype=torch.uint8, device="cuda")
    a, b = ff.grad_norm(ts, workspace=ws), ff.grad_norm(ts)
    torch.cuda.synchronize()
    assert float(a) == float(b)
    with pytest.raises(gemm.GemmError):
        ff.grad_norm(ts, workspace=ws[:8])


@pytest.mark.parametrize("order", ["oi", "io"])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_clip_what_the_backward_pass_returns(ff, dt, order):
    """The gradients of weights in either order of storage are clipped as they come: in
    place, and into outputs of the same order; with a few other dense orders."""
    X, Wg, Wu, dH = _case(8, 60, 50, 33, dt, order)
    _, G, U = ff.gated_ff(X, Wg, Wu, save=True)
    ts = list(ff.gated_ff_backward(dH, X, Wg, Wu, G, U))
    cube = torch.randn(3, 5, 7).to(dt).cuda()
    ts += [cube.permute(2, 0, 1), cube.clone().transpose(0, 2), cube[:, :1].contiguous().expand(3, 1, 7)]
    torch.cuda.synchronize()
    before = [t.clone() for t in ts]
    outs = [torch.full_like(t, 9.0) for t in ts]
    norm = ff.clip_grad_norm(ts, 0.5, out=outs)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    _check_clip(before, outs, norm, 0.5)
    norm2 = ff.clip_grad_norm(ts, 0.5)
    torch.cuda.synchronize()
    assert float(norm2) == float(norm) == float(ff.grad_norm(before))
    assert all(torch.equal(a, b) for a, b in zip(ts, outs))


def test_clip_refuses_what_is_not_dense(ff):
    t = torch.randn(8, 6).cuda()
    for bad in (t[:, :3], t[::2], t[:1].expand(8, 6), t[:, :1].expand(8, 6)):
        with pytest.raises(ValueError):
            ff.grad_norm([bad])
        with pytest.raises(ValueError):
            ff.clip_grad_norm([torch.zeros_like(t)[:, :bad.shape[1]].contiguous()], 1.0, out=[bad])
    a, b = t.t(), torch.empty(6, 8, device="cuda")  # one size, two orders
    with pytest.raises(ValueError):
        ff.clip_grad_norm([a], 1.0, out=[b])
    with pytest.raises(ValueError):
        ff.clip_grad_norm([b], 1.0, out=[a])
    with pytest.raises(ValueError):
        ff.clip_grad_norm([a], 1.0, out=[t])
    with pytest.raises(ValueError):
        ff.clip_grad_norm([t], 1.0, out=[t.bfloat16()])


# ------------------------------------------------------------------ the activations' tails

def _act64(g, act):
    """act and act' in 64 bits with the accuracy of their tails, and how far FP32 rounding of
    the exponent's argument moves each, relative (2^-23 of the argument)."""
    g = g.double()
    if act == "silu":
        s, c, arg = torch.sigmoid(g), torch.sigmoid(-g), torch.zeros_like(g)
        return g * s, s + g * s * c, (s + (g * s * c).abs()), arg
    if act == "gelu":
        p = 0.5 * torch.erfc(-g * math.sqrt(0.5))
        f = torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
        return g * p, p + g * f, p + (g * f).abs(), g * g
    k = math.sqrt(2 / math.pi)
    u = 2 * k * (g + 0.044715 * g ** 3)
    s, c = torch.sigmoid(u), torch.sigmoid(-u)
    t = 2 * g * s * c * k * (1 + 0.134145 * g * g)
    return g * s, s + t, s + t.abs(), u.abs()


def _tail_points(act, limit):
    """Gate values of both signs from 1e-3 on to where act's negative tail passes `limit`."""
    top = {"silu": math.log(limit) * -1.06, "gelu": math.sqrt(-2 * math.log(limit)),
           "gelu_tanh": (-math.log(limit) / 0.0713) ** (1 / 3)}[act]
    g = torch.logspace(-3, math.log10(top), 150)
    g = torch.cat((g, -g))
    return g[_act64(g, act)[0].abs() >= limit]


@pytest.mark.parametrize("M", [4, 64])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_activation_tails(ff, dt, act, M):
    """H = act(G) for G as given (a width of 2, U = 1), relative to act(G) itself down to where
    it leaves the normal numbers.  FP32: erfcf and expf within 4 units of 2^-23, a quotient,
    sums and two products within 4 more, and the argument's rounding, which the
    exponential multiplies: 3 of 2^-23.  BF16: the fast exponential, 2 + 1.2 |x| of 2^-23, and
    the rounding of the result; erf's 2^-23 is of 1, not of its tail."""
    points = _tail_points(act, 2.0 ** -125).to(dt)
    n = -(-points.numel() // M) * M
    g = torch.cat((points, points[:1].expand(n - points.numel()))).view(M, -1)
    F = g.shape[1]
    for j in range(F):  # one column of gates a call: G(m, j) = X(m, 0)
        X = torch.ones((M, 2), dtype=dt)
        X[:, 0] = g[:, j]
        Wg, Wu = torch.zeros((2, 1), dtype=dt), torch.zeros((2, 1), dtype=dt)
        Wg[0], Wu[1] = 1.0, 1.0
        X, Wg, Wu = X.cuda(), Wg.cuda(), Wu.cuda()
        H, G, U = ff.gated_ff(X, Wg, Wu, act=act, save=True)
        torch.cuda.synchronize()
        assert torch.equal(G, X[:, :1].float()) and bool((U == 1).all())
        want, _, _, arg = _act64(g[:, j], act)
        if dt == F32:
            tol = (8 + 3 * arg) * 2.0 ** -23 * want.abs()
        else:
            e = arg if act == "gelu_tanh" else g[:, j].double().abs()
            tol = want.abs() * (2.0 ** -8 + (8 + 6 * e) * 2.0 ** -23)
            if act == "gelu":
                tol = tol + g[:, j].double().abs() * 2.0 ** -23
        assert bool(((H[:, 0].double().cpu() - want).abs() <= tol + 2.0 ** -133).all())


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activation_gradient_tails_f32(ff, act):
    """dX of a width of 2 with Wg = (1, 0), Wu = (0, 1), dH = U = 1 is (act'(G), act(G)): the
    bound of act for each term of act', relative to the terms."""
    points = _tail_points(act, 2.0 ** -110)
    n = -(-points.numel() // 16) * 16
    g = torch.cat((points, points[:1].expand(n - points.numel()))).view(16, -1)
    Wg, Wu = torch.zeros((2, 1)).cuda(), torch.zeros((2, 1)).cuda()
    Wg[0], Wu[1] = 1.0, 1.0
    one = torch.ones((16, 1)).cuda()
    for j in range(g.shape[1]):
        dX, _, _ = ff.gated_ff_backward(one, torch.ones((16, 2)).cuda(), Wg, Wu,
                                        g[:, j:j + 1].cuda(), one, act=act, need_dw=False)
        torch.cuda.synchronize()
        a, d, terms, arg = _act64(g[:, j], act)
        tol = (12 + 3 * arg) * 2.0 ** -23
        got = dX.double().cpu()
        assert bool(((got[:, 0] - d).abs() <= tol * terms + 2.0 ** -140).all())
        assert bool(((got[:, 1] - a).abs() <= tol * a.abs() + 2.0 ** -140).all())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_activations_of_huge_gates(ff, dt, act):
    """Gates whose square or cube leaves FP32's range, up to its end: act is g or 0, act' 1 or
    0, exactly (the exponential is 0, erf 1)."""
    g = torch.tensor([1e6, 1e13, 3e19, 1e25, 3e38])
    g = torch.cat((g, -g))[:, None].cuda()
    n = g.shape[0]
    Wg, Wu = torch.zeros((2, 1), dtype=dt).cuda(), torch.zeros((2, 1), dtype=dt).cuda()
    Wg[0], Wu[1] = 1.0, 1.0
    X = torch.ones((n, 2), dtype=dt, device="cuda")
    dX, _, _ = ff.gated_ff_backward(X[:, :1].contiguous(), X, Wg, Wu, g, torch.ones_like(g),
                                    act=act, need_dw=False)
    torch.cuda.synchronize()
    assert torch.equal(dX[:, 0], (g[:, 0] > 0).to(dt))
    assert torch.equal(dX[:, 1], torch.clamp(g[:, 0], min=0).to(dt))


def test_tensors_written_in_place_count_as_modified(ff):
    """Autograd refuses to use a saved tensor that a call has written since; the version of
    what a call only reads stays."""
    X, Wg, Wu, _ = _case(7, 20, 16, 24, F32, "io")
    q, s, _ = _quant(torch.Generator().manual_seed(1), 24, 16, 32, F32, False)
    outs = [torch.zeros((20, 24), device="cuda") for _ in range(3)]
    for out, call in zip(outs, (
            lambda o: ff.gated_ff(X, Wg, Wu, out=o), lambda o: ff.q4_matmul(X, q, s, group=32, out=o),
            lambda o: ff.q4_gated(X, q, s, q, s, group=32, out=o))):
        x = torch.ones((20, 24), device="cuda", requires_grad=True)
        y = (x * out).sum()  # keeps `out` for the gradient of x
        before = out._version
        assert call(out) is out and out._version > before
        with pytest.raises(RuntimeError, match="modified"):
            y.backward()
    grads = [torch.ones(100, device="cuda"), torch.ones(7, device="cuda")]
    dest = [torch.ones(100, device="cuda"), torch.ones(7, device="cuda")]
    versions = [t._version for t in (X, Wg, q, s, *grads)]
    ff.grad_norm(grads)
    ff.clip_grad_norm(grads, 1.0, out=dest)
    assert versions == [t._version for t in (X, Wg, q, s, *grads)]
    assert all(t._version > 0 for t in dest)
    ff.clip_grad_norm(grads, 1.0)
    assert all(t._version > v for t, v in zip(grads, versions[-2:]))
    with torch.inference_mode():
        t = torch.ones(100, device="cuda")
        ff.clip_grad_norm([t], 1.0)
        assert abs(float(t.norm()) - 1.0) < 1e-5
    torch.cuda.synchronize()
