"""Host side of the feed-forward operators, without a GPU: refusals before any
device work, workspace sizes, and the 64-bit gradients of the tests' reference
against central differences."""
import ctypes

import pytest
import torch

from tests import ff_reference as ref
from roofline_gb300 import build, feedforward as ff, gemm

P = 256  # a well-aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gemm.load()


def _ff(lib, dtype=0, act=0, op=0, M=4, D=8, F=6, X=P, ldx=8, Wg=P, ldg=8, Wu=P, ldu=8, H=P,
        ldh=8, G=None, ldG=8, U=None, ldU=8, ws=None, wsb=0):
    return lib.gated_ff(dtype, act, op, M, D, F, X, ldx, Wg, ldg, Wu, ldu, H, ldh, G, ldG, U,
                        ldU, ws, wsb, None)


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(dtype=-1), dict(act=4), dict(act=-1), dict(op=2), dict(M=-1), dict(D=-1),
    dict(F=-1), dict(X=None), dict(Wg=None), dict(Wu=None), dict(H=None), dict(ldx=7),
    dict(ldg=5), dict(op=1, ldu=7), dict(ldh=5), dict(G=P), dict(U=P), dict(G=P, U=P, ldG=5),
    dict(X=P + 2), dict(dtype=1, X=P + 1), dict(H=P + 1), dict(ws=P + 16, wsb=1 << 20),
    dict(ldx=1 << 40)])
def test_gated_ff_refuses(lib, bad):
    assert _ff(lib, **bad) == gemm.ERR_INVALID_ARG


def test_gated_ff_sizes(lib):
    assert _ff(lib, M=0, X=None, H=None) == gemm.OK       # no tokens
    assert _ff(lib, F=0, Wg=None, Wu=None, H=None) == gemm.OK
    assert _ff(lib, M=1 << 31, ldx=8) == gemm.ERR_UNSUPPORTED
    if not torch.cuda.is_available():
        assert _ff(lib) == gemm.ERR_NO_DEVICE


def _bw(lib, dtype=0, act=0, op=0, M=4, D=8, F=6, dX=P, dWg=P, dWu=P, ldw=8, G=P, X=P, Wg=P,
        dH=P, ws=None, lddx=8):
    return lib.gated_ff_backward(dtype, act, op, M, D, F, dH, 8, X, 8, Wg, 8, P, 8, G, 8, P, 8,
                                 dX, lddx, dWg, ldw, dWu, ldw, ws, 0, None)


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(act=9), dict(op=5), dict(M=-2), dict(dH=None), dict(G=None), dict(X=None),
    dict(Wg=None), dict(dWg=None), dict(dWu=None), dict(dX=None, dWg=None, dWu=None),
    dict(ldw=5), dict(op=1, ldw=7), dict(lddx=7), dict(dX=P + 2), dict(ws=P + 1)])
def test_gated_ff_backward_refuses(lib, bad):
    assert _bw(lib, **bad) == gemm.ERR_INVALID_ARG


def test_gated_ff_backward_sizes(lib):
    assert _bw(lib, D=0) == gemm.OK
    assert _bw(lib, M=0, F=0) == gemm.OK
    if not torch.cuda.is_available():
        assert _bw(lib) == gemm.ERR_NO_DEVICE
        assert _bw(lib, dX=None) == gemm.ERR_NO_DEVICE
        assert _bw(lib, dWg=None, dWu=None, X=None) == gemm.ERR_NO_DEVICE


def test_workspace_sizes(lib):
    out = ctypes.c_uint64(7)
    assert lib.gated_ff_workspace(0, 0, 0, 4, 8, 6, 0, None) == gemm.ERR_INVALID_ARG
    assert lib.gated_ff_workspace(0, 5, 0, 4, 8, 6, 0, out) == gemm.ERR_INVALID_ARG
    assert lib.gated_ff_workspace(0, 0, 0, -4, 8, 6, 0, out) == gemm.ERR_INVALID_ARG
    for backward in (False, True):
        for dt in (ff.DT_F32, ff.DT_BF16):
            for op in (gemm.OP_N, gemm.OP_T):
                # any strides need at least what aligned ones do
                need = ff.gated_ff_workspace(100, 200, 300, dt, op, backward)
                assert need >= ff.gated_ff_workspace(100, 200, 300, dt, op, backward, True)
    # the backward pass keeps dG and dU
    assert ff.gated_ff_workspace(100, 200, 300, ff.DT_BF16, backward=True, aligned=True) >= \
        2 * 100 * 300 * 2


def _q4(lib, dtype=0, M=2, N=3, K=9, X=P, ldx=9, Q=P, ldq=5, S=P, Z=None, group=32, Y=P, ldy=3):
    return lib.q4_matmul(dtype, M, N, K, X, ldx, Q, ldq, S, Z, group, Y, ldy, None)


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(M=-1), dict(N=-1), dict(K=-1), dict(group=0), dict(group=48),
    dict(group=-32), dict(group=512), dict(X=None), dict(Q=None), dict(S=None), dict(Y=None),
    dict(ldx=8), dict(ldq=4), dict(ldy=2), dict(X=P + 2), dict(S=P + 1), dict(Z=P + 1),
    dict(Y=P + 2)])
def test_q4_refuses(lib, bad):
    assert _q4(lib, **bad) == gemm.ERR_INVALID_ARG


def test_q4_sizes(lib):
    assert _q4(lib, M=0, X=None, Y=None) == gemm.OK
    assert _q4(lib, N=0, Q=None, S=None, Y=None) == gemm.OK
    assert _q4(lib, K=1 << 31, ldx=1 << 31, ldq=1 << 30) == gemm.ERR_UNSUPPORTED
    # gated: both matrices are checked, zero points come in pairs
    def gated(act=0, Qu=P, Zg=None, Zu=None, Su=P):
        return lib.q4_gated(0, act, 2, 3, 9, P, 9, P, 5, P, Zg, Qu, 5, Su, Zu, 32, P, 3, None)
    assert gated(act=7) == gemm.ERR_INVALID_ARG
    assert gated(Qu=None) == gemm.ERR_INVALID_ARG
    assert gated(Su=None) == gemm.ERR_INVALID_ARG
    assert gated(Zg=P) == gemm.ERR_INVALID_ARG
    assert gated(Zu=P) == gemm.ERR_INVALID_ARG
    if not torch.cuda.is_available():
        assert _q4(lib) == gemm.ERR_NO_DEVICE
        assert gated() == gemm.ERR_NO_DEVICE


def _clip(lib, count=1, dtypes=(0,), grads=(P,), outs=(P,), sizes=(4,), max_norm=1.0, norm=P,
          ws=None, wsb=0):
    arr = lambda t, v: None if v is None else (t * max(len(v), 1))(*v)  # noqa: E731
    return lib.grad_norm_clip(count, arr(ctypes.c_int, dtypes), arr(ctypes.c_void_p, grads),
                              arr(ctypes.c_void_p, outs), arr(ctypes.c_int64, sizes), max_norm,
                              norm, ws, wsb, None)


@pytest.mark.parametrize("bad", [
    dict(count=-1), dict(dtypes=None), dict(grads=None), dict(sizes=None), dict(dtypes=(7,)),
    dict(sizes=(-1,)), dict(grads=(None,)), dict(outs=(None,)), dict(grads=(P + 2,)),
    dict(outs=(P + 2,)), dict(dtypes=(1,), grads=(P + 1,)), dict(norm=None), dict(norm=P + 2),
    dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(ws=P + 8, wsb=1 << 20)])
def test_clip_refuses(lib, bad):
    assert _clip(lib, **bad) == gemm.ERR_INVALID_ARG


def test_clip_workspace(lib):
    assert lib.grad_norm_clip_workspace(0) == 0
    assert lib.grad_norm_clip_workspace(-3) == 0
    need = [lib.grad_norm_clip_workspace(n) for n in (1, 10, 1000, 100000)]
    assert need == sorted(need) and need[0] > 0
    if not torch.cuda.is_available():
        assert _clip(lib) == gemm.ERR_NO_DEVICE
        assert _clip(lib, outs=None, max_norm=-1.0) == gemm.ERR_NO_DEVICE  # only the norm


def test_binding_refuses_cpu_tensors_and_shapes():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        ff.gated_ff(x, torch.zeros(8, 6), torch.zeros(8, 6))
    with pytest.raises(ValueError):
        ff.gated_ff(x, torch.zeros(8, 6), torch.zeros(8, 6), act="swish2")
    with pytest.raises(ValueError):
        ff.q4_matmul(x, torch.zeros(3, 4, dtype=torch.uint8), torch.zeros(3, 1))
    with pytest.raises(ValueError):
        ff.clip_grad_norm([x], 1.0)
    with pytest.raises(ValueError):
        ff._act("swish2")


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
def test_reference_gradient_against_differences(act):
    """Central differences in 64 bits: an error of order h^2 (third derivatives
    of order 1 on these inputs) plus 2^-52 / h."""
    g = torch.Generator().manual_seed(3)
    X, Wg, Wu, dH = (torch.randn(s, generator=g, dtype=torch.float64)
                     for s in ((5, 7), (7, 6), (7, 6), (5, 6)))
    f = ref.forward(X.float(), Wg.float(), Wu.float(), act)
    X, Wg, Wu, dH = (t.float().double() for t in (X, Wg, Wu, dH))
    b = ref.backward(dH.float(), X.float(), Wg.float(), Wu.float(), f["G"][0].float(),
                     f["U"][0].float(), act)
    # G and U were rounded to float for the reference: relative 2^-24 on each

    def loss(x, wg, wu):
        a, _ = ref.act_both(x @ wg, act)
        return float((dH * a * (x @ wu)).sum())
    h = 1e-5
    for k, name in enumerate(("dX", "dWg", "dWu")):
        base = [X, Wg, Wu]
        v = torch.randn(base[k].shape, generator=g, dtype=torch.float64)
        hi, lo = list(base), list(base)
        hi[k], lo[k] = base[k] + h * v, base[k] - h * v
        num = (loss(*hi) - loss(*lo)) / (2 * h)
        want = float((b[name][0] * v).sum())
        assert abs(num - want) <= 1e-5 * float((b[name][0].abs() * v.abs()).sum()) + 1e-6
