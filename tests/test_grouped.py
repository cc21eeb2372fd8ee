"""Grouped expert products (moe_grouped_matmul) and their weight gradient (moe_grouped_wgrad)
against plain float64 products, segment by segment.

Tolerance, per element: the sum's own error plus the rounding of the result.  The tensor cores
add 16 products a step into an fp32 accumulator and may truncate: at most 2^-23 of the running
sum's magnitude per step, and as much again for aligning the step's products, so
2 (n / 16 + 1) 2^-23 * sum |a b| over a reduction of n.  bf16 results are off by half a step of
bf16 more, 2^-8 of the value; fp32 ones by a few 2^-24."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mixture_experts_layer_48_b200 as moe

BF16, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -22}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(BF16)


def _offsets(counts, first=0):
    o = [first]
    for c in counts:
        o.append(o[-1] + c)
    return o, torch.tensor(o, dtype=torch.int32, device="cuda")


def _check(got, ref, mag, n, what):
    tol = HALF_STEP[got.dtype] * ref.abs() + 2 * (n / 16 + 1) * 2.0 ** -23 * mag
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), what
    assert (err <= tol).all(), f"{what}: worst {((err - tol).max()).item():.3g} over"


def _matmul_case(counts, K, N, transpose, out_dtype, first=0, tail=0, seed=0):
    E = len(counts)
    o, offsets = _offsets(counts, first)
    R = o[-1] + tail
    g = _gen(seed)
    x = _normal(g, R, N if transpose else K)
    W = _normal(g, E, K, N)
    out = torch.full((R, K if transpose else N), 7.0, dtype=out_dtype, device="cuda")
    # rows outside the segments hold NaN: no result may see them
    x[:first] = float("nan")
    x[o[-1]:] = float("nan")
    layer = moe.Moe(E, 64, 64, 1)
    got = layer.grouped_matmul(x, W, offsets, transpose=transpose, out=out)
    assert got is out and layer.sync_status() == moe.MOE_OK
    assert (out[:first] == 7).all() and (out[o[-1]:] == 7).all(), "rows outside the segments"
    for e in range(E):
        if counts[e] == 0:
            continue
        a, b = x[o[e]:o[e + 1]].double(), W[e].double()
        b = b.t() if transpose else b
        _check(out[o[e]:o[e + 1]], a @ b, a.abs() @ b.abs(), a.shape[1], f"expert {e}")


# row counts that reach every kernel shape: few rows per expert (split reductions), a tile of 128,
# the CTA pairs; empty experts, one row, rows around every tile edge
COUNTS = {
    "one": [1],
    "few": [0, 1, 2, 0, 15, 16, 17, 3],
    "small": [33, 1, 0, 32, 31, 0, 5, 64],
    "mid": [100, 0, 127, 129, 1, 128, 40, 90],
    "many": [255, 256, 257, 0, 300, 511, 513, 1],
    "one expert long": [1500],
    "skewed": [0, 0, 0, 0, 0, 0, 0, 2100],
}


@pytest.mark.parametrize("out_dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("transpose", [False, True], ids=["product", "transposed"])
@pytest.mark.parametrize("counts", list(COUNTS), ids=lambda c: c.replace(" ", "-"))
@pytest.mark.parametrize("K,N", [(64, 64), (72, 200), (256, 320), (8, 8), (1000, 264)])
def test_matmul(counts, K, N, transpose, out_dtype):
    _matmul_case(COUNTS[counts], K, N, transpose, out_dtype, seed=K + N)


@pytest.mark.parametrize("transpose", [False, True], ids=["product", "transposed"])
@pytest.mark.parametrize("counts", ["few", "mid", "many"])
def test_matmul_rows_outside_the_segments(counts, transpose):
    _matmul_case(COUNTS[counts], 136, 152, transpose, BF16, first=5, tail=9, seed=1)


@pytest.mark.parametrize("counts,K,N,transpose,out_dtype", [
    ([1, 0, 1, 1, 0, 0, 1, 0] * 4, 2880, 2880, False, F32),       # a few tokens, split reductions
    ([2, 3, 1, 2, 0, 4, 2, 2] * 4, 2880, 5760, False, BF16),      # a decode batch, 20b gate/up
    ([60, 70, 64, 1], 2880, 2880, True, BF16),                    # one tile per expert
    ([700, 900], 2880, 5760, True, F32),                          # gradient of the layer input
    ([300] * 16, 2880, 1440, False, BF16),
    ([5, 200], 16384, 128, False, F32),                           # a long reduction, in pieces
    ([900] * 8, 128, 16384, True, F32),                           # the same on the CTA pairs
])
def test_matmul_layer_sizes(counts, K, N, transpose, out_dtype):
    _matmul_case(counts, K, N, transpose, out_dtype, seed=2)


def test_matmul_256_experts_and_no_rows():
    counts = [(7 * i) % 5 for i in range(256)]
    _matmul_case(counts, 64, 128, False, BF16)
    layer = moe.Moe(256, 64, 64, 1)
    W = torch.zeros((256, 64, 128), dtype=BF16, device="cuda")
    o = torch.zeros((257,), dtype=torch.int32, device="cuda")
    assert layer.grouped_matmul(torch.empty((0, 64), dtype=BF16, device="cuda"), W, o).shape == (0, 128)
    # rows, but none in a segment
    out = torch.full((3, 128), 5.0, dtype=BF16, device="cuda")
    layer.grouped_matmul(torch.zeros((3, 64), dtype=BF16, device="cuda"), W, o, out=out)
    assert (out == 5).all() and layer.sync_status() == moe.MOE_OK


def _wgrad_case(counts, K, N, out_dtype, first=0, tail=0, seed=0):
    E = len(counts)
    o, offsets = _offsets(counts, first)
    R = o[-1] + tail
    g = _gen(seed)
    x, dy = _normal(g, R, K), _normal(g, R, N)
    for t in (x, dy):
        t[:first] = float("nan")
        t[o[-1]:] = float("inf")
    out = torch.full((E, K, N), float("nan"), dtype=out_dtype, device="cuda")
    layer = moe.Moe(E, 64, 64, 1)
    assert layer.grouped_wgrad(x, dy, offsets, out=out) is out
    assert layer.sync_status() == moe.MOE_OK
    for e in range(E):
        a, b = x[o[e]:o[e + 1]].double(), dy[o[e]:o[e + 1]].double()
        n = min(counts[e], 6144) if out_dtype == F32 else counts[e]
        _check(out[e], a.t() @ b, a.abs().t() @ b.abs(), n, f"expert {e}")


@pytest.mark.parametrize("out_dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("counts", list(COUNTS), ids=lambda c: c.replace(" ", "-"))
@pytest.mark.parametrize("K,N", [(64, 64), (72, 200), (256, 320), (8, 8), (520, 264)])
def test_wgrad(counts, K, N, out_dtype):
    _wgrad_case(COUNTS[counts], K, N, out_dtype, seed=K + N)


@pytest.mark.parametrize("counts,K,N,out_dtype", [
    ([64, 128, 1, 0, 77, 200], 2880, 1440, BF16),
    ([20000, 3], 128, 256, F32),                 # a long reduction, in pieces
    ([6144, 6145, 6143, 6208], 256, 256, F32),   # around the length of a piece
    ([63, 64, 65, 448, 449, 447, 0, 1, 1, 1, 2, 1], 256, 512, F32),
    ([5000], 520, 264, BF16),                    # few tiles: the rows split over four CTA pairs
    ([4097, 0, 70], 304, 72, F32),
    ([2600], 64, 64, F32),
    ([9001, 2], 1000, 1000, BF16),               # over two
    ([100], 264, 2000, F32),
])
def test_wgrad_sizes(counts, K, N, out_dtype):
    _wgrad_case(counts, K, N, out_dtype, seed=3)


@pytest.mark.parametrize("K,N", [(32768, 8), (8, 32768), (32768, 72), (136, 32768)])
def test_longest_rows(K, N):
    for transpose in (False, True):
        _matmul_case([3, 0, 130], K, N, transpose, BF16, seed=4)
    _matmul_case([3, 0, 130], K, N, False, F32, seed=5)
    _wgrad_case([3, 0, 130], K, N, BF16, seed=6)


@pytest.mark.parametrize("rows", [1, 40])
def test_256_experts(rows):
    counts = [rows if i % 3 else 0 for i in range(256)]
    _matmul_case(counts, 128, 136, True, F32, first=2, tail=1, seed=7)
    _wgrad_case(counts, 136, 64, BF16, first=2, tail=1, seed=8)


def test_results_past_2_to_the_31_elements():
    R, K, N = 70001, 8, 32768
    g = _gen(9)
    x, W = _normal(g, R, K), _normal(g, 2, K, N)
    offsets = torch.tensor([0, 35000, R], dtype=torch.int32, device="cuda")
    layer = moe.Moe(2, 64, 64, 1)
    out = layer.grouped_matmul(x, W, offsets)
    for r in (0, 34999, 35000, 65535, 65536, 66000, R - 1):
        w = W[int(r >= 35000)].double()
        _check(out[r:r + 1], x[r:r + 1].double() @ w, x[r:r + 1].double().abs() @ w.abs(), K, f"row {r}")
    dW = layer.grouped_wgrad(x, out, offsets, out_dtype=F32)   # reads dy past 2^31 elements too
    a, b = x[35000:].double(), out[35000:, -64:].double()
    _check(dW[1][:, -64:], a.t() @ b, a.abs().t() @ b.abs(), 6144, "dW")


def test_wgrad_rows_outside_the_segments():
    _wgrad_case(COUNTS["many"], 136, 152, BF16, first=5, tail=9)
    _wgrad_case(COUNTS["few"], 136, 152, F32, first=70, tail=70)


def test_wgrad_keeps_an_experts_nan_to_itself():
    counts = [5, 40, 0, 70]
    o, offsets = _offsets(counts)
    g = _gen(4)
    x, dy = _normal(g, o[-1], 64), _normal(g, o[-1], 128)
    x[o[1]] = float("nan")       # the first row after expert 0's ragged end
    dy[o[1]] = float("inf")
    layer = moe.Moe(4, 64, 64, 1)
    dW = layer.grouped_wgrad(x, dy, offsets, out_dtype=F32)
    for e in (0, 2, 3):
        assert torch.isfinite(dW[e]).all()
        ref = x[o[e]:o[e + 1]].double().t() @ dy[o[e]:o[e + 1]].double()
        assert (dW[e].double() - ref).abs().max() < 1e-3
    assert torch.isnan(dW[1]).any()


def test_wgrad_without_rows_is_zero():
    layer = moe.Moe(3, 64, 64, 1)
    o = torch.zeros((4,), dtype=torch.int32, device="cuda")
    for R in (0, 7):
        x = torch.ones((R, 64), dtype=BF16, device="cuda")
        out = torch.full((3, 64, 72), 3.0, device="cuda")
        layer.grouped_wgrad(x, torch.ones((R, 72), dtype=BF16, device="cuda"), o, out=out)
        assert (out == 0).all()
    assert layer.sync_status() == moe.MOE_OK


@pytest.mark.parametrize("bad", [[0, 5, 3, 20], [0, 5, 10, 21], [-1, 5, 10, 20]],
                         ids=["decreasing", "past-R", "negative"])
@pytest.mark.parametrize("R", [20, 400, 2000])
def test_bad_offsets_are_reported_and_contained(bad, R):
    """Segments with bad ends count as empty; nothing outside the buffers is touched."""
    scale = R // 20
    o = torch.tensor([v if v < 0 else v * scale for v in bad], dtype=torch.int32, device="cuda")
    layer = moe.Moe(3, 64, 64, 1)
    g = _gen(5)
    x, W = _normal(g, R, 64), _normal(g, 3, 64, 128)
    out = torch.full((R, 128), 9.0, dtype=BF16, device="cuda")
    layer.grouped_matmul(x, W, o, out=out)
    assert layer.sync_status() == moe.MOE_ERR_ARG and layer.sync_status() == moe.MOE_OK
    dW = layer.grouped_wgrad(x, _normal(g, R, 128), o, out_dtype=F32)
    assert layer.sync_status() == moe.MOE_ERR_ARG
    for e in range(3):
        if not 0 <= o[e] <= o[e + 1] <= R:
            assert (dW[e] == 0).all()


def test_same_call_twice_gives_the_same_bits():
    for counts in ("few", "mid", "many"):
        o, offsets = _offsets(COUNTS[counts])
        g = _gen(6)
        x, W, dy = _normal(g, o[-1], 1000), _normal(g, 8, 1000, 264), _normal(g, o[-1], 264)
        layer = moe.Moe(8, 64, 64, 1)
        for f in (lambda: layer.grouped_matmul(x, W, offsets, out_dtype=F32),
                  lambda: layer.grouped_matmul(dy, W, offsets, transpose=True),
                  lambda: layer.grouped_wgrad(x, dy, offsets, out_dtype=F32)):
            assert torch.equal(f(), f())


def test_captured_and_on_another_stream():
    """A captured call reads new rows and new offsets at replay; two handles on two streams."""
    o, offsets = _offsets(COUNTS["few"])
    g = _gen(7)
    R, K, N = 200, 256, 320
    x, W = _normal(g, R, K), _normal(g, 8, K, N)
    layer, other = moe.Moe(8, 64, 64, 1), moe.Moe(8, 64, 64, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ref = layer.grouped_matmul(x, W, offsets)[:o[-1]].clone()
    got = other.grouped_matmul(x, W, offsets, stream=side)[:o[-1]]
    dW = other.grouped_wgrad(x, x, offsets, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(ref, got) and torch.equal(dW, layer.grouped_wgrad(x, x, offsets))
    out = torch.zeros((R, N), dtype=BF16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.grouped_matmul(x, W, offsets, out=out)
        dWg = layer.grouped_wgrad(x, out, offsets, out_dtype=F32)
    counts2 = [20, 0, 30, 1, 0, 99, 2, 48]
    o2, offsets2 = _offsets(counts2)
    x.copy_(_normal(g, R, K))
    offsets.copy_(offsets2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, layer.grouped_matmul(x, W, offsets2))
    assert torch.equal(dWg, layer.grouped_wgrad(x, out, offsets2, out_dtype=F32))
    assert layer.sync_status() == moe.MOE_OK


def test_calls_side_by_side():
    """Kernels of every shape on four streams at once, each with its own handle."""
    g = _gen(10)
    work = []
    for i, counts in enumerate(["few", "mid", "many", "one expert long"]):
        o, offsets = _offsets(COUNTS[counts])
        E = len(COUNTS[counts])
        work.append((moe.Moe(E, 64, 64, 1), _normal(g, o[-1], 520), _normal(g, E, 520, 264), offsets, torch.cuda.Stream()))
    want = [(h.grouped_matmul(x, W, o), h.grouped_wgrad(x, x, o, out_dtype=F32)) for h, x, W, o, _ in work]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got.append([(h.grouped_matmul(x, W, o, stream=s), h.grouped_wgrad(x, x, o, out_dtype=F32, stream=s))
                    for h, x, W, o, s in work])
    torch.cuda.synchronize()
    for run in got:
        for (y, dW), (yw, dWw) in zip(run, want):
            assert torch.equal(y, yw) and torch.equal(dW, dWw)
    assert all(h.sync_status() == moe.MOE_OK for h, *_ in work)


def test_gradients_are_those_of_the_product():
    """<dy, y(x + d, W + D) - y(x, W)> against <dx, d> + <dW, D> for float64 differences: the three
    calls are one function and its two derivatives."""
    counts = [3, 0, 40, 17]
    o, offsets = _offsets(counts)
    g = _gen(8)
    K, N = 128, 192
    x, W, dy = _normal(g, o[-1], K), _normal(g, 4, K, N), _normal(g, o[-1], N)
    layer = moe.Moe(4, 64, 64, 1)
    dx = layer.grouped_matmul(dy, W, offsets, transpose=True, out_dtype=F32).double()
    dW = layer.grouped_wgrad(x, dy, offsets, out_dtype=F32).double()
    expert = torch.repeat_interleave(torch.arange(4, device="cuda"), torch.tensor(counts, device="cuda"))
    f = lambda a, b: torch.einsum("rk,rkn->rn", a, b[expert])  # noqa: E731
    d, D = torch.randn_like(dx), torch.randn_like(dW)
    h = 1e-4   # f is bilinear: a central difference is exact up to rounding
    num = ((f(x.double() + h * d, W.double() + h * D) - f(x.double() - h * d, W.double() - h * D))
           * dy.double()).sum() / (2 * h)
    ana = (dx * d).sum() + (dW * D).sum()
    # each entry of dx, dW carries at most (K / 16 + 1) 2^-22 of its sum of magnitudes (~K): against
    # the norm of a sum of this many independent terms, 1e-4 of the size of the terms is ample
    size = torch.sqrt((dx * d).square().sum() + (dW * D).square().sum())
    assert (num - ana).abs() <= 1e-4 * size + 1e-9 * num.abs()


def test_refusals():
    layer = moe.Moe(4, 64, 64, 1)
    o = torch.zeros((5,), dtype=torch.int32, device="cuda")
    x = torch.zeros((6, 64), dtype=BF16, device="cuda")
    W = torch.zeros((4, 64, 72), dtype=BF16, device="cuda")
    layer.grouped_matmul(x, W, o)
    for bad in (dict(x_rows=x.float()), dict(W=W.float()), dict(offsets=o.long()), dict(offsets=o[:4]),
                dict(W=W[:3]), dict(x_rows=x[:, :32]), dict(x_rows=x[:, ::2]), dict(x_rows=x.cpu()),
                dict(out=torch.zeros((6, 64), dtype=BF16, device="cuda")), dict(transpose=True),
                dict(out_dtype=torch.float16), dict(out=torch.zeros((6, 72), dtype=torch.float16, device="cuda"))):
        with pytest.raises(ValueError):
            layer.grouped_matmul(**{**dict(x_rows=x, W=W, offsets=o), **bad})
    with pytest.raises(ValueError):
        layer.grouped_wgrad(x, x[:5], o)
    with pytest.raises(moe.MoeError):   # 12 columns: not a multiple of 8
        layer.grouped_matmul(x, torch.zeros((4, 64, 12), dtype=BF16, device="cuda"), o)
    with pytest.raises(moe.MoeError):   # a row length of 2 bytes' alignment
        layer.grouped_matmul(torch.zeros((6 * 64 + 1,), dtype=BF16, device="cuda")[1:].view(6, 64), W, o)
    # offsets and per-row arrays may be parts of larger ones
    many = torch.zeros((3, 5), dtype=torch.int32, device="cuda")
    layer.grouped_matmul(x, W, many[1])
    layer.grouped_wgrad(x, x, many[1])
    p = lambda t: t.data_ptr()  # noqa: E731
    out = torch.zeros((6, 72), dtype=BF16, device="cuda")
    call = lambda *a: moe.moe_grouped_matmul(layer.handle, *a, None)  # noqa: E731
    assert call(6, 64, 72, 0, p(o), p(x), p(W), p(out), 0) == moe.MOE_OK
    assert call(-1, 64, 72, 0, p(o), p(x), p(W), p(out), 0) == moe.MOE_ERR_ARG
    assert call(6, 64, 72, 0, p(o), p(x), p(W), p(out), 2) == moe.MOE_ERR_ARG
    assert call(6, 64, 32776, 0, p(o), p(x), p(W), p(out), 0) == moe.MOE_ERR_ARG
    assert call(6, 64, 72, 0, 0, p(x), p(W), p(out), 0) == moe.MOE_ERR_ARG
    assert call(6, 64, 72, 0, p(o), p(x), p(W), 0, 0) == moe.MOE_ERR_ARG
    assert call(0, 64, 72, 0, 0, 0, 0, 0, 0) == moe.MOE_OK
    assert layer.sync_status() == moe.MOE_OK
