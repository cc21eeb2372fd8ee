"""Kernels that follow each other on a stream start before the one in front has ended, so each has
to wait before it reads what the one in front writes.  Here the norm writes the tensor that the
router reads: a captured chain finds other values in it before every replay, and its routing has to
be that of the values the norm left there."""
import pytest
import torch

import moe_inputs as mi

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mixture_experts_layer_48_b200 as moe

BF16, F32 = torch.bfloat16, torch.float32
ROUTE = ("topk_idx", "topk_w", "expert_offsets", "perm", "inv_perm")


def _setup(T, E, dtype, H=2880, I=64, k=4):
    d = mi.make_inputs(T, H, E, k, I, seed=T + E, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return moe.Moe(E, H, I, k), d, rnd(T, H).to(dtype), 1 + 0.2 * rnd(H)


def _captured(f):
    f()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f()
    return graph, out


SIZES = [(1, 32), (16, 32), (300, 32), (8192, 32), (1, 128), (7, 12), (65, 8)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,E", SIZES)
def test_route_reads_what_the_norm_wrote(T, E, dtype):
    layer, d, resid, w = _setup(T, E, dtype)

    def f():
        n = layer.block_norm(resid, w_next=w)
        return n["x"], layer.route(n["x"], d["W_router"], d["b_router"])

    graph, (x, r) = _captured(f)
    want_x = layer.block_norm(resid, w_next=w)["x"]
    want = layer.route(want_x, d["W_router"], d["b_router"])
    for i in range(100):
        x.copy_(-want_x if i % 2 else want_x.flip(1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want_x)
        for key in ROUTE:
            assert torch.equal(r[key], want[key]), f"{key}, replay {i}"
    assert layer.sync_status() == moe.MOE_OK


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,E", SIZES)
def test_blocks_in_a_row(T, E, dtype):
    layer, d, resid, w = _setup(T, E, dtype)
    args = (d["W_router"], d["b_router"], d["W_gate_up"], d["W_down"])
    kw = dict(w_post=w, scale=0.5, w_next=w)

    def f():
        n = layer.block_norm(resid, w_next=w)
        a = layer.block(resid, n["x"], *args, **kw)
        return n, a, layer.block(a["resid"], a["x"], *args, **kw)

    graph, (n, a, b) = _captured(f)
    poison = [torch.randn_like(t) for t in (n["x"], a["x"])]
    for i in range(30):
        n["x"].copy_(poison[0])
        a["x"].copy_(poison[1])
        graph.replay()
        torch.cuda.synchronize()
        # The layer of the same x takes the same experts; its fp32 sums may be added in another
        # order, at most 4 experts' rows of 64 products each: 2^-14 of the norm's unit rows.  That may
        # move the residual by a step of its bf16, and x by that and one of its own.
        for before, x, after in ((resid, n["x"], a), (a["resid"], a["x"], b)):
            again = layer.block(before, x, *args, **kw)
            for key in ("resid", "x"):
                got, want = after[key].double(), again[key].double()
                assert ((got - want).abs() <= 2.0 ** -6 * want.abs() + 2.0 ** -8).all(), f"{key}, replay {i}"
    assert layer.sync_status() == moe.MOE_OK
