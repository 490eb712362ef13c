"""Host side of orthogonalised updates, without a GPU: refusals before any device work, workspace
sizes, and the tests' reference against the singular values' own polynomial."""
import ctypes

import pytest
import torch

from tests import ortho_reference as ref
from roofline_gb300 import build, feedforward as ff, gemm

P = 256  # a well-aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gemm.load()


def _call(lib, dtype=0, batch=1, M=4, N=6, G=P, ldg=6, sg=24, O=P, ldo=6, so=24, steps=2,
          abc=ref.MUON * 2, eps=1e-7, ws=None, wsb=0):
    c = None if abc is None else (ctypes.c_float * len(abc))(*abc)
    return lib.orthogonalize(dtype, batch, M, N, G, ldg, sg, O, ldo, so, steps, c, eps, ws, wsb,
                             None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(batch=-1), dict(M=-1), dict(N=-1), dict(G=None), dict(O=None),
    dict(G=P + 2), dict(dtype=1, O=P + 1), dict(ldg=5), dict(ldo=5), dict(ldg=1 << 40),
    dict(batch=2, so=23), dict(batch=2, sg=-1), dict(batch=2, so=-(1 << 62)),
    dict(batch=2, M=1 << 30, N=1, ldo=1 << 36, so=1 << 40), dict(steps=0), dict(steps=-1), dict(abc=None),
    dict(abc=(1.0, NAN, 0.0) * 2), dict(abc=(1.0, 0.0, INF) * 2), dict(eps=-1.0), dict(eps=NAN),
    dict(eps=INF), dict(ws=P + 16, wsb=1 << 30)])
def test_refuses(lib, bad):
    assert _call(lib, **bad) == gemm.ERR_INVALID_ARG


@pytest.mark.parametrize("abc", [
    (2.0, 0.0, 0.0) * 2 + (1.0, 0.0, 0.0),  # singular values of 4 in a factor
    (3.0, 3.0, 3.0) * 2, (-4.0, 0.0, 0.0) * 2,
    (1.0, -300.0, 299.0) * 2,            # b A + c A A of -75
    (1.0, 0.0, -100.0) * 2, (2.0, -1e30, 1e30) * 2,
    (2.0, -1.5, 0.5, 0.0, 200.0, -200.0)])
def test_coefficients_beyond_the_factors_range(lib, abc):
    assert _call(lib, steps=len(abc) // 3, abc=abc) == gemm.ERR_UNSUPPORTED


@pytest.mark.parametrize("abc", [
    ref.MUON * 2, (2.0, -1.5, 0.5) * 2, (1.5, -0.5, 0.0) * 2, (1.875, -1.25, 0.375) * 2,
    (8.28721201814563, -23.595886519098837, 17.300387312530933,
     4.107059111542203, -2.9478499167379106, 0.5448431082926601), (0.0, 0.0, 0.0) * 2])
def test_coefficients_in_use(lib, abc):
    if not torch.cuda.is_available():
        assert _call(lib, abc=abc) == gemm.ERR_NO_DEVICE


def test_sizes(lib):
    for empty in (dict(batch=0), dict(M=0), dict(N=0, ldg=1, ldo=1)):
        assert _call(lib, G=None, O=None, **empty) == gemm.OK
    big = 1 << 21
    assert _call(lib, M=big, N=big, ldg=big, ldo=big) == gemm.ERR_UNSUPPORTED
    assert _call(lib, N=1 << 31, ldg=1 << 31, ldo=1 << 31) == gemm.ERR_UNSUPPORTED
    assert _call(lib, batch=65536) == gemm.ERR_UNSUPPORTED
    assert _call(lib, steps=65, abc=(1.0, 0.0, 0.0) * 65) == gemm.ERR_UNSUPPORTED
    out = ctypes.c_uint64(7)
    assert lib.orthogonalize_workspace(0, 1, 4, 6, None) == gemm.ERR_INVALID_ARG
    assert lib.orthogonalize_workspace(3, 1, 4, 6, out) == gemm.ERR_INVALID_ARG
    assert lib.orthogonalize_workspace(0, 1, big, big, out) == gemm.ERR_UNSUPPORTED
    assert ff.orthogonalize_workspace(0, 5, ff.DT_F32) == 0
    # matrices with a side of up to 128 stay on chip
    assert ff.orthogonalize_workspace(100, 300, ff.DT_BF16) == 0
    one = ff.orthogonalize_workspace(200, 300, ff.DT_BF16)
    assert one == ff.orthogonalize_workspace(300, 200, ff.DT_BF16) >= 200 * 300 * 8
    assert ff.orthogonalize_workspace(200, 300, ff.DT_F32) > one
    assert ff.orthogonalize_workspace(200, 300, ff.DT_BF16, batch=4) > 3 * one
    assert ff.orthogonalize_workspace(100, 10_000, ff.DT_F32) > 0
    assert ff.orthogonalize_workspace(100, 300, ff.DT_F32, batch=1000) > 0


def test_binding_refuses():
    with pytest.raises(ValueError):
        ff.orthogonalize(torch.zeros(4, 6))
    for c in ((1.0, 2.0), [(1.0, 2.0, 3.0)] * 4, (), [(1.0, 2.0)] * 5):
        with pytest.raises(ValueError):
            ff.orthogonalize(torch.zeros(4, 6), coefficients=c)


@pytest.mark.parametrize("shape", [(7, 12), (12, 7), (9, 9), (3, 5, 8)], ids=str)
def test_reference(shape):
    """The steps act on the singular values alone, each by a x + b x^3 + c x^5, and the shifted
    form that the kernel takes is the same function."""
    g = torch.Generator().manual_seed(3)
    G = torch.randn(shape, generator=g)
    U, s, V = torch.linalg.svd(G.double(), full_matrices=False)
    s = s / (torch.sqrt((s * s).sum(-1, keepdim=True)) + 1e-7)
    for a, b, c in ref._steps(ref.MUON, 5):
        s = a * s + b * s ** 3 + c * s ** 5
    want = (U * s[..., None, :]) @ V
    got = ref.exact(G)
    # 64-bit sums, amplified by at most 4^5
    assert float((got - want).abs().max()) <= 1e-11
    shifted = ref.emulate(G, 5, ref.MUON, 1e-7, False, False)
    assert float((got - shifted).abs().max()) <= 1e-11
    one, bound = ref.one_step(G)
    assert float((one - ref.exact(G, 1)).abs().max()) <= 1e-12
    assert bool((bound < 1e-4).all())


class _Taken:
    """A native module that keeps the coefficients it is given."""

    def orthogonalize(self, G, steps, coefficients, *rest):
        self.got = [float(x) for x in coefficients]


@pytest.fixture
def taken(monkeypatch):
    module = _Taken()
    monkeypatch.setattr(ff, "_module", module)
    return module


ROWS = [(1.0, 2.0, 3.0), [4.0, 5.0, 6.0]]


@pytest.mark.parametrize("steps, c, want", [
    (5, (1.0, 2.0, 3.0), [1.0, 2.0, 3.0]), (3, [1, 2, 3], [1.0, 2.0, 3.0]),
    (3, torch.tensor([1.0, 2.0, 3.0]), [1.0, 2.0, 3.0]),
    (1, (torch.tensor(1.0), 2.0, 3.0), [1.0, 2.0, 3.0]),
    (1, [(1.0, 2.0, 3.0)], [1.0, 2.0, 3.0]), (2, ROWS, [1.0, 2.0, 3.0, 4.0, 5.0, 6.0]),
    (2, ROWS[0] + tuple(ROWS[1]), [1.0, 2.0, 3.0, 4.0, 5.0, 6.0]),
    (2, iter(ROWS), [1.0, 2.0, 3.0, 4.0, 5.0, 6.0]),
    (2, torch.tensor(ROWS[1:] + ROWS[:1]), [4.0, 5.0, 6.0, 1.0, 2.0, 3.0]),
    (3, ROWS + ROWS[:1], [1.0, 2.0, 3.0, 4.0, 5.0, 6.0, 1.0, 2.0, 3.0])], ids=str)
def test_forms_of_coefficients(taken, steps, c, want):
    ff.orthogonalize(None, steps=steps, coefficients=c)
    assert taken.got == want


@pytest.mark.parametrize("steps, c", [
    # rows of other lengths, whose numbers add up to what a call may have
    (3, [(1.0,), (2.0,), (3.0,)]), (2, [(1.0, 2.0), (3.0, 4.0, 5.0, 6.0)]),
    (2, [(), (1.0, 2.0, 3.0, 4.0, 5.0, 6.0)]), (2, [(), (1.0, 2.0, 3.0)]),
    (3, torch.ones(3, 1)), (1, torch.ones(1, 9)),
    # numbers and rows side by side
    (2, [1.0, (2.0, 3.0)]), (3, [1.0, (2.0, 3.0), 4.0]), (3, [1.0, 2.0, (3.0,)]),
    # neither numbers nor rows
    (1, ()), (0, ()), (1, 1.0), (1, None),
    (1, torch.tensor(1.0)), (2, [(1.0, 2.0, 3.0)] * 3), (2.5, ROWS), ("all", ROWS),
    (1, "abc")], ids=str)
def test_forms_of_coefficients_refused(taken, steps, c):
    with pytest.raises(ValueError):
        ff.orthogonalize(None, steps=steps, coefficients=c)
    assert not hasattr(taken, "got")


def test_matrices_of_the_result_share_nothing(lib):
    """The call takes the strides of a stack whose matrices have no element in common, rows side by
    side included, and no others."""
    if torch.cuda.is_available():
        pytest.skip("what is taken would run, on addresses that are none")
    taken = 0
    for batch in (1, 2, 3, 5):
        for M in (1, 2, 3):
            for N in (1, 2, 3):
                for ldo in range(N, 9):
                    for so in range(26):
                        places = [z * so + i * ldo + j for z in range(batch) for i in range(M)
                                  for j in range(N)]
                        apart = len(set(places)) == len(places)
                        taken += apart
                        want = gemm.ERR_NO_DEVICE if apart else gemm.ERR_INVALID_ARG
                        got = _call(lib, batch=batch, M=M, N=N, ldg=N, sg=0, ldo=ldo, so=so)
                        assert got == want, (batch, M, N, ldo, so)
    assert taken > 1000
    far = 1 << 62  # three such strides are more than 64 bits hold
    assert _call(lib, batch=4, so=far) == gemm.ERR_NO_DEVICE
    assert _call(lib, batch=65535, M=300, N=4, ldg=4, sg=0, ldo=4 * 65535, so=4) == \
        gemm.ERR_NO_DEVICE
    assert _call(lib, batch=65535, M=300, N=4, ldg=4, sg=0, ldo=4 * 65535 - 1, so=4) == \
        gemm.ERR_INVALID_ARG


# A step's limits one by one: s^2 <= 15, |b| + 3 |c| s^2 <= 250, a span of 60 of b y + c y^2
@pytest.mark.parametrize("beyond, inside", [
    ((3.88, 0.0, 0.0, 0.5, 0.0, 0.0), (3.86, 0.0, 0.0, 0.5, 0.0, 0.0)),
    # singular values of 0.1: b A is 3 at most
    ((0.1, 0.0, 0.0, 0.0, 300.0, 0.0), (0.1, 0.0, 0.0, 0.0, 249.0, 0.0)),
    ((0.1, 0.0, 0.0, 0.0, 0.0, 8400.0), (0.1, 0.0, 0.0, 0.0, 0.0, 8200.0)),
    # |b| + 3 |c| is 61 and 183 at most
    ((1.0, -61.0, 0.0), (1.0, -59.0, 0.0)), ((1.0, 0.0, 61.0), (1.0, 0.0, 59.0)),
    # |b| + 3 |c| of 261 and 247, spans of 49 and 44
    ((1.0, -31.0, 76.5), (1.0, -31.0, 72.0))], ids=str)
def test_each_limit_of_the_coefficients(lib, beyond, inside):
    assert _call(lib, steps=len(beyond) // 3, abc=beyond) == gemm.ERR_UNSUPPORTED
    if not torch.cuda.is_available():
        assert _call(lib, steps=len(inside) // 3, abc=inside) == gemm.ERR_NO_DEVICE


def test_range_of_the_default_coefficients():
    """Singular values from 0.01 to 1 after five steps."""
    s = torch.logspace(-2, 0, 200_001, dtype=torch.float64)
    for a, b, c in ref._steps(ff.NEWTON_SCHULZ, 5):
        s = ((c * s * s + b) * s * s + a) * s
    assert 0.68 <= float(s.min()) < 0.69 and 1.13 < float(s.max()) <= 1.14
