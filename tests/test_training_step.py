"""The operators around the layer together, as a program uses them: a training step of one
transformer block (norm, routing, expert products, combine, norm into the residual, and all
gradients back), and the serving path of the same block, against float64."""
import pytest
import torch

import moe_inputs as mi

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mixture_experts_layer_48_b200 as moe

BF16, F32 = torch.bfloat16, torch.float32
EPS, SCALE = 1e-5, 0.5


def _setup(T, H, E, k, I, seed=0):
    d = mi.make_inputs(T, H, E, k, I, seed=seed, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    v = dict(resid=rnd(T, H).to(BF16), w_in=1 + 0.2 * rnd(H), w_post=1 + 0.2 * rnd(H), gate=1 + 0.2 * rnd(H),
             w_next=1 + 0.2 * rnd(H), dres=0.3 * rnd(T, H), dx=(0.3 * rnd(T, H)).to(BF16))
    return d, v


def _step(layer, d, v):
    """One forward and backward pass through the library; the routing is not differentiated here
    (its weights' gradients come out as dw)."""
    Wgu, Wd = d["W_gate_up"], d["W_down"]
    f0 = layer.block_norm(v["resid"], w_next=v["w_in"], eps=EPS)
    r = layer.route(f0["x"], d["W_router"], d["b_router"])
    off = r["expert_offsets"]
    x_rows, row_w = layer.permute(f0["x"], r)
    gu = layer.grouped_matmul(x_rows, Wgu, off)
    h = layer.swiglu(gu, row_w)
    y = layer.combine(r["inv_perm"], layer.grouped_matmul(h, Wd, off, out_dtype=F32))
    f1 = layer.block_norm(v["resid"], y, w_post=v["w_post"], gate=v["gate"], scale=SCALE, w_next=v["w_next"], eps=EPS)
    b1 = layer.block_norm_backward(v["dres"].to(BF16), v["dx"], f1["resid"], y, rstd_post=f1["rstd_post"],
                                   rstd_next=f1["rstd_next"], w_post=v["w_post"], gate=v["gate"], scale=SCALE,
                                   w_next=v["w_next"])
    dy_rows, _ = layer.permute(b1["dy"], r)
    dh = layer.grouped_matmul(dy_rows, Wd, off, transpose=True)
    dWd = layer.grouped_wgrad(h, dy_rows, off, out_dtype=F32)
    dgu, drow_w = layer.swiglu_backward(dh, gu, row_w)
    dx_rows = layer.grouped_matmul(dgu, Wgu, off, transpose=True, out_dtype=F32)
    dWgu = layer.grouped_wgrad(x_rows, dgu, off, out_dtype=F32)
    dx0 = layer.combine(r["inv_perm"], dx_rows)
    b0 = layer.block_norm_backward(b1["dresid"], dx0.to(BF16), v["resid"], rstd_next=f0["rstd_next"], w_next=v["w_in"])
    return dict(resid=f1["resid"], x=f1["x"], dresid=b0["dresid"], dw_in=b0["dw_next"], dw_post=b1["dw_post"],
                dgate=b1["dgate"], dw_next=b1["dw_next"], dWgu=dWgu, dWd=dWd,
                dw=drow_w[r["inv_perm"].long()]), r


def _reference(d, v, r, E, I):
    """The same block in float64 with autograd, with the step's routing."""
    leaf = lambda t: t.double().clone().requires_grad_()  # noqa: E731
    resid, w_in, w_post, gate, w_next = (leaf(v[n]) for n in ("resid", "w_in", "w_post", "gate", "w_next"))
    Wgu, Wd, w = leaf(d["W_gate_up"]), leaf(d["W_down"]), leaf(r["topk_w"])
    norm = lambda t, q: t / torch.sqrt(t.square().mean(1, keepdim=True) + EPS) * q  # noqa: E731
    x = norm(resid, w_in)
    y = torch.zeros_like(x)
    idx = r["topk_idx"].long()
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if len(t):
            gu = x[t] @ Wgu[e]
            h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
            y = y.index_add(0, t, w[t, j][:, None] * (h @ Wd[e]))
    r1 = resid + SCALE * gate * norm(y, w_post)
    x1 = norm(r1, w_next)
    ((r1 * v["dres"].to(BF16).double()).sum() + (x1 * v["dx"].double()).sum()).backward()
    return dict(resid=r1, x=x1, dresid=resid.grad, dw_in=w_in.grad, dw_post=w_post.grad, dgate=gate.grad,
                dw_next=w_next.grad, dWgu=Wgu.grad, dWd=Wd.grad, dw=w.grad)


@pytest.mark.parametrize("T,H,E,k,I", [(5, 256, 8, 2, 256), (300, 256, 8, 2, 320), (1200, 320, 4, 2, 192)])
def test_training_step_against_autograd(T, H, E, k, I):
    d, v = _setup(T, H, E, k, I, seed=T)
    layer = moe.Moe(E, H, I, k)
    got, r = _step(layer, d, v)
    assert layer.sync_status() == moe.MOE_OK
    ref = _reference(d, v, r, E, I)
    # Between leaf and result lie at most eight tensors kept in bf16, each off by half a step
    # (2^-8 of each value, independent): in the norm at most 8 * 2^-8 = 3 %.
    for key, want in ref.items():
        want = want.detach()
        rel = (got[key].double() - want).norm() / want.norm()
        assert rel <= 8 * 2.0 ** -8, f"{key}: {rel.item():.3g}"


def test_training_step_captured_and_replayed():
    T, H, E, k, I = 200, 256, 8, 2, 256
    d, v = _setup(T, H, E, k, I, seed=7)
    layer = moe.Moe(E, H, I, k)
    _step(layer, d, v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(layer, d, v)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, _ = _step(layer, d, v)
    _, other = _setup(T, H, E, k, I, seed=8)
    for key in v:
        v[key].copy_(other[key])
    graph.replay()
    torch.cuda.synchronize()
    want, _ = _step(layer, d, v)
    for key in got:
        assert torch.equal(got[key], want[key]), key


@pytest.mark.parametrize("T", [1, 16, 300])
def test_block_serves_the_layer_in_its_residual_stream(T):
    H, E, k, I = 256, 8, 2, 256
    d, v = _setup(T, H, E, k, I, seed=20 + T)
    layer = moe.Moe(E, H, I, k)
    x = layer.block_norm(v["resid"], w_next=v["w_in"], eps=EPS)["x"]
    args = (d["W_router"], d["b_router"], d["W_gate_up"], d["W_down"])
    got = layer.block(v["resid"], x, *args, w_post=v["w_post"], gate=v["gate"], scale=SCALE, w_next=v["w_next"], eps=EPS)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = moe.Moe(E, H, I, k)
    on_side = other.block(v["resid"], x, *args, w_post=v["w_post"], gate=v["gate"], scale=SCALE, w_next=v["w_next"],
                          eps=EPS, stream=side)
    side.synchronize()
    assert layer.sync_status() == moe.MOE_OK and other.sync_status() == moe.MOE_OK
    y = layer.forward(x, *args).double()   # fp32 atomics: two calls agree to ~1e-4
    norm = lambda t, w: t / torch.sqrt(t.square().mean(1, keepdim=True) + EPS) * w.double()  # noqa: E731
    r = v["resid"].double() + SCALE * v["gate"].double() * norm(y, v["w_post"])
    for out in (got, on_side):
        assert ((out["resid"].double() - r).abs() <= 2.0 ** -8 * r.abs() + 1e-3).all()
        want = norm(out["resid"].double(), v["w_next"])
        assert ((out["x"].double() - want).abs() <= 2.0 ** -7 * want.abs()).all()
