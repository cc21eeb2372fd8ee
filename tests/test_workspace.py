"""Whose memory a layer's own workspaces are: a captured call's stay the graph's, whatever calls follow,
and a call on another stream takes its own from that stream."""
import pytest
import torch

import moe_inputs as mi

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mixture_experts_layer_48_b200 as moe

H, E, k, I = 256, 8, 2, 256


def _layer(T, seed):
    d = mi.make_inputs(T, H, E, k, I, seed=seed, device="cuda")
    return moe.Moe(E, H, I, k), d, (d["W_router"], d["b_router"], d["W_gate_up"], d["W_down"])


def _calls(layer, args, w):
    return {"forward": lambda x, **kw: layer.forward(x, *args, **kw),
            "block": lambda x, **kw: layer.block(x, x, *args, w_post=w, w_next=w, **kw)["resid"],
            "route": lambda x, **kw: layer.route(x, *args[:2], **kw)["topk_w"]}


def _span(t):
    return t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()


def _overlap(a, b):
    return a[0] < b[1] and b[0] < a[1]


@pytest.mark.parametrize("name", ["forward", "block", "route"])
def test_a_captured_call_keeps_its_workspace(name):
    T = 4000
    layer, d, args = _layer(T, 1)
    w = torch.ones(H, device="cuda")
    call = _calls(layer, args, w)[name]
    x = d["x"][:500].contiguous()
    call(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(x)
    graphs, n = _span(layer._ws), layer._ws.numel()
    call(d["x"])                       # a larger call: a workspace of its own
    taken = [torch.full((n,), 77, dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert not any(_overlap(_span(t), graphs) for t in taken)
    assert not _overlap(_span(layer._ws), graphs)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all((t == 77).all() for t in taken)
    want = call(x)
    assert (out.double() - want.double()).abs().max() <= 2.0 ** -6 * want.abs().max()   # fp32 atomics, bf16 steps
    assert layer.sync_status() == moe.MOE_OK


@pytest.mark.parametrize("name", ["forward", "block", "route"])
def test_a_call_on_another_stream_takes_that_streams_memory(name):
    layer, d, args = _layer(4000, 2)
    call = _calls(layer, args, torch.ones(H, device="cuda"))[name]
    x = d["x"][:500].contiguous()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call(x, stream=side)
    sides, n = _span(layer._ws), layer._ws.numel()
    side.synchronize()
    call(d["x"])                       # on the current stream: the side stream's goes back to it
    torch.cuda.synchronize()
    taken = [torch.empty((n,), dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert not any(_overlap(_span(t), sides) for t in taken)
    assert layer.sync_status() == moe.MOE_OK


def test_calls_of_one_size_share_one_workspace():
    layer, d, args = _layer(300, 3)
    layer.forward(d["x"], *args)
    first = layer._ws.data_ptr()
    for _ in range(3):
        layer.forward(d["x"], *args)
        assert layer._ws.data_ptr() == first
    assert max(layer.last_dispatch(300)) > 0     # read from the last call's, still there


def test_tensors_of_the_host_are_still_refused():
    layer, d, args = _layer(8, 4)
    for call in (layer.forward, lambda x, *a: layer.route(x, *a[:2])):
        with pytest.raises(ValueError):
            call(d["x"].cpu(), *args)
        call(d["x"], *args)
    assert layer.sync_status() == moe.MOE_OK


@pytest.mark.parametrize("name", ["forward", "block", "route"])
def test_workspaces_that_are_not_plain_device_memory_are_refused(name):
    layer, d, args = _layer(8, 5)
    call = _calls(layer, args, torch.ones(H, device="cuda"))[name]
    n = max(layer.workspace_bytes(8), layer.route_workspace_bytes(8))
    call(d["x"], workspace=torch.empty((n,), dtype=torch.uint8, device="cuda"))
    for bad in (torch.empty((n,), dtype=torch.uint8), torch.empty((1,), dtype=torch.uint8, device="cuda").expand(n),
                torch.empty((n, 2), dtype=torch.uint8, device="cuda")[:, 0]):
        with pytest.raises(ValueError):
            call(d["x"], workspace=bad)
    with pytest.raises(moe.MoeError):
        call(d["x"], workspace=torch.empty((16,), dtype=torch.uint8, device="cuda"))
    assert layer.sync_status() == moe.MOE_OK


def test_workspaces_of_the_norms_backward_pass_that_are_not_plain_device_memory_are_refused():
    layer = moe.Moe(1, H, 64, 1)
    r, w = torch.randn((4, H), device="cuda"), torch.ones((H,), device="cuda")
    f = layer.block_norm(r, w_next=w)
    call = lambda ws: layer.block_norm_backward(r, f["x"], r, rstd_next=f["rstd_next"], w_next=w, workspace=ws)  # noqa: E731
    n = layer.block_norm_workspace_bytes(4)
    call(torch.empty((n,), dtype=torch.uint8, device="cuda"))
    for bad in (torch.empty((n,), dtype=torch.uint8), torch.empty((1,), dtype=torch.uint8, device="cuda").expand(n)):
        with pytest.raises(ValueError):
            call(bad)
    assert layer.sync_status() == moe.MOE_OK
