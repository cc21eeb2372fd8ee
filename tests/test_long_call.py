"""A weight gradient that runs for longer than any wait of a kernel may last (2 s), with its only ragged
segment at the very end: the warps that wait for that end wait through all of it."""
import time

import pytest
import torch

from test_grouped_sums import _near

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mixture_experts_layer_48_b200 as moe


def test_the_last_segment_of_a_long_call():
    N, long = 32768, 64 * 25000
    R = long + 3
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 2 * N * (R + 2 * N) + (4 << 30):
        pytest.skip("needs 113 GB of free device memory")
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    x = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
    for r in range(0, R, 1 << 14):
        x[r:r + (1 << 14)].uniform_(0.5, 1.0, generator=g)
    o = torch.tensor([0, long, R], dtype=torch.int32, device="cuda")
    layer = moe.Moe(2, 64, 64, 1)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    dW = layer.grouped_wgrad(x, x, o)
    assert layer.sync_status() == moe.MOE_OK
    assert time.perf_counter() - t0 > 2.0, "not the case that this test is for"
    for c in (slice(0, 64), slice(N - 64, N)):      # blocks of dW with a float64 product
        for e, (lo, hi) in enumerate(((0, long), (long, R))):
            ref = sum(x[r:min(r + (1 << 18), hi), c].double().t() @ x[r:min(r + (1 << 18), hi), -64:].double()
                      for r in range(lo, hi, 1 << 18))
            _near(dW[e][c, -64:], ref, hi - lo, f"expert {e}")
    del x, dW
    torch.cuda.empty_cache()


@pytest.mark.parametrize("transpose", [False, True], ids=["product", "transposed"])
def test_products_of_the_most_rows(transpose):
    """2^28 rows, the first and last outside of the segments: offsets near the end of 32 bits' reach."""
    R, n = 1 << 28, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.empty((R, n), dtype=torch.bfloat16, device="cuda").uniform_(0.5, 1.0, generator=g)
    W = torch.empty((3, n, n), dtype=torch.bfloat16, device="cuda").uniform_(0.5, 1.0, generator=g)
    bounds = [1, R // 2 + 77, R // 2 + 77, R - 1]
    o = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    out = torch.full((R, n), 7.0, dtype=torch.bfloat16, device="cuda")
    layer = moe.Moe(3, 64, 64, 1)
    layer.grouped_matmul(x, W, o, transpose=transpose, out=out)
    assert layer.sync_status() == moe.MOE_OK
    assert (out[0] == 7).all() and (out[-1] == 7).all()
    for e in range(3):
        w = W[e].double().t() if transpose else W[e].double()
        for lo in range(bounds[e], bounds[e + 1], 1 << 24):
            hi = min(lo + (1 << 24), bounds[e + 1])
            _near(out[lo:hi], x[lo:hi].double() @ w, n, f"expert {e}, rows from {lo}")
