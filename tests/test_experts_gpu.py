"""A mixture layer's tokens sorted by expert, gathered, brought back with weights, and the
gradients, on the GPU against their formulas in 64 bits (experts_reference has the bounds)."""
import pytest
import torch

from tests import experts_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ff():
    from roofline_gb300 import build, feedforward
    build.build()
    return feedforward


def _choices(g, T, k, E, left=0.0, dtype=torch.int64):
    """Experts of a skewed router, some choices left out by ids on either side."""
    p = torch.rand(E, generator=g).pow(3) + 1e-3
    e = torch.multinomial(p, max(T * k, 1), replacement=True, generator=g)[:T * k].view(T, k)
    gone = torch.rand((T, k), generator=g) < left
    far = [-1, E, E + 1, -E, 2 ** 31 - 1] + ([2 ** 32, 2 ** 32 + 1, -2 ** 63, 2 ** 63 - 1]
                                             if dtype == torch.int64 else [-2 ** 31])
    out = torch.tensor(far)[torch.randint(0, len(far), (T, k), generator=g)]
    return torch.where(gone, out, e).to(dtype)


def _mat(g, rows, cols, dt, pad=0, off=0):
    return torch.randn((rows, cols + pad), generator=g).to(dt).cuda()[:, off:off + cols]


SORTS = [(0, 2, 4), (5, 0, 3), (1, 1, 1), (1, 8, 256), (31, 1, 7), (33, 3, 16), (300, 4, 1024),
         (1000, 2, 1000), (1025, 4, 64), (4096, 1, 2), (4097, 1, 33), (2731, 6, 200),
         (9001, 8, 128), (65537, 4, 8), (70000, 2, 1024)]


@pytest.mark.parametrize("dtype", [torch.int64, torch.int32], ids=["i64", "i32"])
@pytest.mark.parametrize("left", [0.0, 0.2, 1.0])
@pytest.mark.parametrize("size", SORTS)
def test_sort(ff, size, left, dtype):
    T, k, E = size
    g = torch.Generator().manual_seed(T + k + E)
    e = _choices(g, T, k, E, left, dtype)
    want = ref.sort(e, E)
    wide = torch.full((T, k + 3), -7, dtype=dtype, device="cuda")  # and as rows of a wider one
    wide[:, 1:k + 1] = e.cuda()
    for ids in (e.cuda(), wide[:, 1:k + 1]):
        got = ff.expert_sort(ids, E)
        for a, b in zip(got, want):
            assert a.dtype == torch.int32 and torch.equal(a.cpu(), b)


def test_sort_one_expert_takes_all(ff):
    for T in (100, 40000):
        e = torch.full((T, 3), 5, device="cuda")
        place, offsets, order = ff.expert_sort(e, 9)
        n = torch.arange(3 * T, dtype=torch.int32, device="cuda")
        assert torch.equal(place.view(-1), n) and torch.equal(order, n)
        assert offsets.tolist() == [0] * 6 + [3 * T] * 4


SIZES = [(1, 1, 1), (1, 8, 4096), (3, 2, 7), (5, 9, 8), (17, 3, 64), (33, 17, 129), (64, 8, 777),
         (130, 1, 1000), (300, 4, 2056), (700, 8, 24), (2000, 2, 40)]
PADS = [(0, 0), (8, 0), (3, 1), (8, 4)]


def _make(ff, seed, T, k, D, dt, pad=0, off=0, left=0.15, E=11):
    g = torch.Generator().manual_seed(seed)
    ids = _choices(g, T, k, E, left).cuda()
    place, offsets, order = ff.expert_sort(ids, E)
    X, dO = _mat(g, T, D, dt, pad, off), _mat(g, T, D, dt, pad, off)
    Y = _mat(g, T * k, D, dt, pad, off)
    w = torch.rand((T, k + 1), generator=g).cuda()[:, :k]
    return X, dO, Y, w, place, offsets, order


@pytest.mark.parametrize("pad", PADS, ids=str)
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_gather(ff, size, dt, pad):
    T, k, D = size
    X, _, _, _, place, offsets, _ = _make(ff, sum(size), *size, dt, *pad)
    n = int(offsets[-1])
    for rows in (None, 0, n // 2, n, T * k + 5):
        want = ref.gather(X, place, n, T * k if rows is None else rows)
        got = ff.expert_gather(X, place, offsets, rows=rows)
        assert torch.equal(got.double().cpu(), want)
    # into rows of a wider buffer, whose other columns stay
    wide = torch.full((T * k, D + 5), 3.0, dtype=dt, device="cuda")
    out = ff.expert_gather(X, place, offsets, out=wide[:, 2:2 + D])
    assert torch.equal(out.double().cpu(), ref.gather(X, place, n, T * k))
    assert bool((wide[:, :2] == 3).all()) and bool((wide[:, 2 + D:] == 3).all())


@pytest.mark.parametrize("weights", ["f32", "bf16", "none"])
@pytest.mark.parametrize("pad", PADS, ids=str)
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_combine_and_its_gradients(ff, size, dt, pad, weights):
    T, k, D = size
    _, dO, Y, w, place, offsets, _ = _make(ff, sum(size), *size, dt, *pad)
    w = {"f32": w, "bf16": w.to(BF16), "none": None}[weights]
    n = int(offsets[-1])
    Y[n:] = float("nan")  # rows of no choice are not read
    got = ff.expert_combine(Y, place, w)
    assert got.dtype == dt and ref.worst(got, ref.combine(Y, place, w)) <= 1.0
    wide = torch.full((T, D + 5), 3.0, dtype=dt, device="cuda")
    out = ff.expert_combine(Y, place, w, out=wide[:, 2:2 + D])
    assert torch.equal(out, got)
    assert bool((wide[:, :2] == 3).all()) and bool((wide[:, 2 + D:] == 3).all())

    (dy, dyb), dw = ref.combine_backward(dO, Y, place, w)
    dY, dW = ff.expert_combine_backward(dO, Y, place, offsets, w)
    at = place.cpu().long()
    on = at >= 0
    assert ref.worst(dY[at[on].cuda()], (dy[on], dyb[on])) <= 1.0
    assert bool((dY[n:] == 0).all())
    if w is None:
        assert dW is None
    else:
        assert dW.dtype == w.dtype and ref.worst(dW, dw) <= 1.0
        only_w = ff.expert_combine_backward(dO, Y, place, offsets, w, need_dy=False)
        assert only_w[0] is None and torch.equal(only_w[1], dW)
    only_y = ff.expert_combine_backward(dO, Y, place, offsets, w, need_dw=False)
    assert only_y[1] is None and torch.equal(only_y[0], dY)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_rows_of_fewer_than_the_choices(ff, dt):
    """Places beyond the rows that a buffer has add nothing and are not written."""
    X, dO, Y, w, place, offsets, _ = _make(ff, 3, 40, 4, 72, dt)
    for rows in (0, 1, 50):
        cut = Y[:rows]
        assert ref.worst(ff.expert_combine(cut, place, w), ref.combine(cut, place, w)) <= 1.0
        dY, dW = ff.expert_combine_backward(dO, cut, place, offsets, w)
        (dy, dyb), dw = ref.combine_backward(dO, cut, place, w)
        assert dY.shape == cut.shape and ref.worst(dW, dw) <= 1.0
        at = place.cpu().long()
        on = (at >= 0) & (at < rows)
        assert ref.worst(dY[at[on].cuda()], (dy[on], dyb[on])) <= 1.0


def test_places_from_elsewhere_stay_inside(ff):
    """Places and a number of routed rows that no sort gave are bounded by the buffers."""
    g = torch.Generator().manual_seed(1)
    T, k, D = 6, 2, 16
    X = _mat(g, T, D, F32)
    buf = torch.full((T * k + 8, D), 5.0, device="cuda")
    out = buf[4:-4]
    place = torch.tensor([[0, 12], [-5, 1], [2 ** 31 - 1, 2], [-2 ** 31, 3], [13, 4], [11, 5]],
                         dtype=torch.int32, device="cuda")
    for routed in (12, 2 ** 31 - 1, 0, -3, 7):
        buf.fill_(5.0)
        offsets = torch.tensor([0, routed], dtype=torch.int32, device="cuda")
        ff.expert_gather(X, place, offsets, out=out)
        assert bool((buf[:4] == 5).all()) and bool((buf[-4:] == 5).all())
    assert torch.equal(ff.expert_combine(out, place).isfinite().all().cpu(), torch.tensor(True))


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_inf_and_nan_stay_with_their_rows(ff, dt):
    g = torch.Generator().manual_seed(2)
    T, k, D, E = 50, 3, 40, 6
    ids = _choices(g, T, k, E, 0.3).cuda()
    place, offsets, _ = ff.expert_sort(ids, E)
    X, Y, w = _mat(g, T, D, dt), _mat(g, T * k, D, dt), torch.rand((T, k), generator=g).cuda()
    X[3, 4], X[5, 6], Y[7, 8], Y[9, 1] = float("nan"), float("inf"), -float("inf"), float("nan")
    w[11, 0] = float("inf")
    n = int(offsets[-1])
    got = ff.expert_gather(X, place, offsets).double().cpu()
    want = ref.gather(X, place, n, T * k)
    assert torch.equal(got.nan_to_num(nan=1e300), want.nan_to_num(nan=1e300))
    v, b = ref.combine(Y, place, w)
    assert ref.worst(ff.expert_combine(Y, place, w), (v, b.nan_to_num(nan=1.0, posinf=1.0))) <= 1.0
    _, dW = ff.expert_combine_backward(X, Y, place, offsets, w)
    v, b = ref.combine_backward(X, Y, place, w)[1]
    assert ref.worst(dW, (v, b.nan_to_num(nan=1.0, posinf=1.0))) <= 1.0


def test_empty_extents(ff):
    e = torch.empty((0, 4), dtype=torch.int64, device="cuda")
    place, offsets, order = ff.expert_sort(e, 3)
    assert place.shape == (0, 4) and offsets.tolist() == [0] * 4 and order.shape == (0,)
    x = torch.empty((0, 8), device="cuda")
    assert ff.expert_gather(x, place, offsets).shape == (0, 8)
    assert bool((ff.expert_gather(x, place, offsets, rows=3) == 0).all())
    assert ff.expert_combine(x, place).shape == (0, 8)
    dY, dW = ff.expert_combine_backward(x, x, place, offsets, torch.empty((0, 4), device="cuda"))
    assert dY.shape == (0, 8) and dW.shape == (0, 4)
    # no choices at all: sums of nothing
    place, offsets, _ = ff.expert_sort(torch.empty((5, 0), dtype=torch.int32, device="cuda"), 2)
    assert bool((ff.expert_combine(x, place) == 0).all())
    # no width
    place, offsets, _ = ff.expert_sort(torch.zeros((5, 2), dtype=torch.int32, device="cuda"), 2)
    w = torch.ones((5, 2), device="cuda")
    z = torch.empty((10, 0), device="cuda")
    dY, dW = ff.expert_combine_backward(z[:5], z, place, offsets, w)
    assert dY.shape == (10, 0) and bool((dW == 0).all())


def _time(f):
    """Milliseconds of the fastest of some calls."""
    times = []
    for _ in range(6):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b))
    return min(times[1:])


@pytest.mark.parametrize("T", [0, 1, 3])
def test_long_buffers_of_few_tokens(ff, T):
    """Rows behind the routed ones are cleared by the whole device, not by the tokens' blocks: half
    a gigabyte takes about what torch's own zeros take (by one block some 60 times as long)."""
    k, D, rows = 8, 4096, 65536
    g = torch.Generator().manual_seed(T)
    X, w = _mat(g, T, D, BF16), torch.rand((T, k), generator=g).cuda()
    place, offsets, order = ff.expert_sort(_choices(g, T, k, 16, 0.3).cuda(), 16)
    n = int(offsets[-1])
    buf = torch.full((rows, D), 7.0, dtype=BF16, device="cuda")
    zeros = _time(buf.zero_)
    buf.fill_(7.0)
    ff.expert_gather(X, place, offsets, out=buf)
    assert torch.equal(buf[:n], X[order[:n].long() // k]) and not bool(buf[n:].any())
    assert _time(lambda: ff.expert_gather(X, place, offsets, out=buf)) < 5 * zeros
    dY, dw = ff.expert_combine_backward(X, buf, place, offsets, w)
    (want, bound), dots = ref.combine_backward(X, buf, place, w)
    at = place.cpu().long()
    on = at >= 0
    assert ref.worst(dY[at[on].cuda()], (want[on], bound[on])) <= 1.0 and not bool(dY[n:].any())
    assert ref.worst(dw, dots) <= 1.0
    del dY
    assert _time(lambda: ff.expert_combine_backward(X, buf, place, offsets, w)) < 5 * zeros


def test_offsets_beyond_32_bits(ff):
    """Rows of the sorted buffer more than 2^32 bytes and 2^31 elements from its start."""
    T, k, D = 70000, 8, 4096
    g = torch.Generator(device="cuda").manual_seed(5)
    X = torch.randn((T, D), generator=g, device="cuda").to(BF16)
    ids = torch.rand((T, 16), generator=g, device="cuda").topk(k, 1)[1]
    place, offsets, order = ff.expert_sort(ids, 16)
    Y = ff.expert_gather(X, place, offsets)
    at = torch.randint(0, T * k, (4096,), generator=g, device="cuda")
    at[-1] = T * k - 1
    assert torch.equal(Y[at], X[order[at].long() // k])
    # powers of two: every sum is exact
    w = 2.0 ** -torch.arange(1, k + 1, device="cuda").float().expand(T, k).contiguous()
    w[:, -1] *= 2
    assert torch.equal(ff.expert_combine(Y, place, w), X)
    del X
    dO = torch.ones((T, D), dtype=BF16, device="cuda")
    dY, dW = ff.expert_combine_backward(dO, Y, place, offsets, w)
    assert torch.equal(dY[at, 7].float(), w.view(-1)[order[at].long()])
    del dY
    want = Y[at].double().sum(1)
    tol = 1.01 * D * ref.E32 * Y[at].double().abs().sum(1)
    assert bool(((dW.view(-1)[order[at].long()].double() - want).abs() <= tol).all())


def test_equal_calls_give_equal_bits(ff):
    X, dO, Y, w, place, offsets, _ = _make(ff, 9, 3000, 8, 520, BF16)
    first = [ff.expert_combine(Y, place, w), *ff.expert_combine_backward(dO, Y, place, offsets, w)]
    for _ in range(3):
        again = [ff.expert_combine(Y, place, w),
                 *ff.expert_combine_backward(dO, Y, place, offsets, w)]
        assert all(torch.equal(a, b) for a, b in zip(first, again))


# ------------------------------------------------------------------ refusals, streams, graphs

def test_refusals(ff):
    from roofline_gb300 import gemm
    X, dO, Y, w, place, offsets, _ = _make(ff, 4, 6, 2, 8, F32)
    one = torch.ones((1, 1), device="cuda")
    bad = [
        lambda: ff.expert_sort(torch.zeros(6, dtype=torch.int64, device="cuda"), 4),
        lambda: ff.expert_sort(torch.zeros((6, 2), device="cuda"), 4),
        lambda: ff.expert_sort(torch.zeros((6, 4), dtype=torch.int32, device="cuda")[:, ::2], 4),
        lambda: ff.expert_sort(torch.zeros((1, 1), dtype=torch.int32, device="cuda").expand(6, 1), 4),
        lambda: ff.expert_sort(torch.zeros((6, 2), dtype=torch.int32, device="cuda"), 0),
        lambda: ff.expert_sort(torch.zeros((6, 2), dtype=torch.int32, device="cuda"), 2 ** 32 + 4),
        lambda: ff.expert_gather(X[:5], place, offsets),
        lambda: ff.expert_gather(X.half(), place, offsets),
        lambda: ff.expert_gather(X, place.long(), offsets),
        lambda: ff.expert_gather(X, place.cpu(), offsets),
        lambda: ff.expert_gather(X, place[:, :1], offsets),
        lambda: ff.expert_gather(X, place, offsets.long()),
        lambda: ff.expert_gather(X, place, offsets[:0]),
        lambda: ff.expert_gather(X, place, offsets[::2]),
        lambda: ff.expert_gather(X, place, offsets, rows=-1),
        lambda: ff.expert_gather(X, place, offsets, rows=2 ** 40),
        lambda: ff.expert_gather(X, place, offsets, rows=5, out=torch.empty((6, 8), device="cuda")),
        lambda: ff.expert_gather(X, place, offsets, out=torch.empty((12, 7), device="cuda")),
        lambda: ff.expert_gather(X, place, offsets, out=torch.empty((12, 8), device="cuda").half()),
        lambda: ff.expert_gather(one.expand(6, 1), place, offsets),
        lambda: ff.expert_combine(Y, place, w[:5]),
        lambda: ff.expert_combine(Y, place, w.double()),
        lambda: ff.expert_combine(Y, place, w.t().contiguous().t()),
        lambda: ff.expert_combine(Y, place, w, out=torch.empty((6, 9), device="cuda")),
        lambda: ff.expert_combine(Y.t(), place, w),
        lambda: ff.expert_combine(one.expand(12, 1), place, w),
        lambda: ff.expert_combine_backward(dO[:5], Y, place, offsets, w),
        lambda: ff.expert_combine_backward(dO.to(BF16), Y, place, offsets, w),
        lambda: ff.expert_combine_backward(dO, Y.cpu(), place, offsets, w),
        lambda: ff.expert_combine_backward(dO, Y, place, None, w),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("not refused:", i)
    with pytest.raises(gemm.GemmError):
        ff.expert_sort(torch.zeros((6, 2), dtype=torch.int32, device="cuda"), 1025)


def test_too_many_experts_take_no_memory(ff):
    from roofline_gb300 import gemm
    ids = torch.zeros((6, 2), dtype=torch.int32, device="cuda")
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.max_memory_allocated()
    for count in (1025, 10 ** 8, 2 ** 31 - 1):
        with pytest.raises(gemm.GemmError) as refused:
            ff.expert_sort(ids, count)
        assert refused.value.code == gemm.ERR_UNSUPPORTED
    assert torch.cuda.max_memory_allocated() == before
    ids[1, 1] = 1023
    assert ff.expert_sort(ids, 1024)[1].tolist() == [0] + 1023 * [11] + [12]


def test_on_another_stream_and_in_a_graph(ff):
    X, dO, Y, w, place, offsets, order = _make(ff, 6, 500, 4, 264, BF16)
    g = torch.Generator().manual_seed(8)
    ids = _choices(g, 500, 4, 11, 0.15).cuda()

    def step(stream=None):
        p, o, r = ff.expert_sort(ids, 11, stream=stream)
        rows = ff.expert_gather(X, p, o, stream=stream)
        out = ff.expert_combine(rows, p, w, stream=stream)
        return [p, o, r, rows, out, *ff.expert_combine_backward(dO, rows, p, o, w, stream=stream)]
    want = step()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = step(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kept = step()
    ids.copy_(_choices(g, 500, 4, 11, 0.4).cuda())
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, step()))


def test_new_outputs_on_another_stream(ff):
    """Memory that the current stream is still to write is not given to a call on another one."""
    X, dO, Y, w, place, offsets, order = _make(ff, 7, 300, 4, 520, BF16)
    ids = _choices(torch.Generator().manual_seed(8), 300, 4, 11, 0.15).cuda()
    calls = [lambda s: ff.expert_sort(ids, 11, stream=s),
             lambda s: (ff.expert_gather(X, place, offsets, stream=s),),
             lambda s: (ff.expert_combine(Y, place, w, stream=s),),
             lambda s: ff.expert_combine_backward(dO, Y, place, offsets, w, stream=s)]
    side = torch.cuda.Stream()
    for call in calls:
        want = call(None)
        torch.cuda.synchronize()
        blocks = [torch.empty(t.untyped_storage().nbytes(), dtype=torch.uint8, device="cuda")
                  for t in want]
        torch.cuda._sleep(50_000_000)
        for b in blocks:
            b.fill_(7)
        del blocks, b
        got = call(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_behind_pending_work(ff):
    """The kernels' launches overlap, but each waits for what is before it in the stream."""
    g = torch.Generator().manual_seed(12)
    ids, X = _choices(g, 3000, 4, 40, 0.1).cuda(), _mat(g, 3000, 264, BF16)
    dO, w = _mat(g, 3000, 264, BF16), torch.rand((3000, 4), generator=g).cuda()

    def step(ids, X, w):
        p, o, r = ff.expert_sort(ids, 40)
        rows = ff.expert_gather(X, p, o)
        return [p, o, r, rows, ff.expert_combine(rows, p, w),
                *ff.expert_combine_backward(dO, rows, p, o, w)]
    want = step(ids, X, w)
    late = [torch.zeros_like(t) for t in (ids, X, w)]
    for _ in range(3):
        for t in late:
            t.zero_()
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        for t, s in zip(late, (ids, X, w)):
            t.copy_(s)
        got = step(*late)
        for t in late:
            t.fill_(-1)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_out_counts_as_modified(ff):
    X, dO, Y, w, place, offsets, _ = _make(ff, 6, 20, 2, 16, F32)
    rows, out = torch.zeros((40, 16), device="cuda"), torch.zeros((20, 16), device="cuda")
    before = rows._version, out._version
    ff.expert_gather(X, place, offsets, out=rows)
    ff.expert_combine(Y, place, w, out=out)
    assert rows._version > before[0] and out._version > before[1]
