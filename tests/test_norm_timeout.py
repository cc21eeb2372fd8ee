"""A copy that does not arrive in a norm's ring is an error that the host reads, in the forward and the
backward call: the kernels report it, end, and leave the context and the handle as usable as before."""
import ctypes

import pytest
import torch

BF16, F32 = torch.bfloat16, torch.float32

if torch.cuda.is_available():
    import mixture_experts_layer_48_b200 as moe


def test_bound_and_refused_without_a_handle():
    import __graft_entry__
    __graft_entry__.load_builder().build()
    import mixture_experts_layer_48_b200 as m
    assert m.moe_selftest_norm_timeout(ctypes.c_void_p(None), 0) == m.MOE_ERR_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("resid_type", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,H,from_rows", [(1, 2880, (0,)), (5, 64, (0, 1)), (700, 256, (0, 690)), (4000, 2880, (0, 1, 1500, 3999)),
                                           (9000, 64, (0, 5000, 8990)), (3000, 8192, (0, 149, 2900)), (600, 4096, (0, 300))])
def test_reported_and_usable_afterwards(T, H, from_rows, resid_type):
    g = torch.Generator(device="cuda")
    g.manual_seed(T + H)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    resid, y, w = rnd(T, H).to(resid_type), rnd(T, H).to(BF16), 1 + 0.1 * rnd(H)
    layer = moe.Moe(1, H, 64, 1)
    kw = dict(w_post=w, gate=w, scale=0.5, w_next=w)
    fwd = lambda: layer.block_norm(resid, y, **kw)  # noqa: E731
    f = fwd()
    bwd = lambda: layer.block_norm_backward(resid, f["x"], f["resid"], y, f["rstd_post"], f["rstd_next"], **kw)  # noqa: E731
    b = bwd()
    assert layer.sync_status() == moe.MOE_OK
    for row in from_rows:
        for call in (fwd, bwd):
            layer.selftest_norm_timeout(row)
            call()
            assert layer.sync_status() == moe.MOE_ERR_TIMEOUT, (call is fwd, row)
            layer.selftest_norm_timeout(-1)
            # the next kernels use the same shared memory and find nothing landing in it
            for got, want in ((fwd(), f), (bwd(), b)):
                for key in want:
                    assert torch.equal(got[key], want[key]), (key, row)
            assert layer.sync_status() == moe.MOE_OK
    layer.selftest_norm_timeout(T)   # no such row
    assert all(torch.equal(fwd()[key], f[key]) for key in f)
    assert layer.sync_status() == moe.MOE_OK
