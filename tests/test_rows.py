"""SwiGLU rows and the norms around the block, forward and backward, against float64.

Tolerances: a bf16 result is off by half a step of bf16 (2^-8 of the value), an fp32 one by a few
2^-24.  A reciprocal norm: each thread adds at most 32 squares, then 9 levels of pairs and at most
16 warps, under 64 roundings of 2^-24 in the sum, half of that in its root, and 2 steps of rsqrt:
32 2^-24 + 2^-22 < 2^-18.  What a sum multiplies or is subtracted from carries its error times the
sum of the magnitudes that went into it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mixture_experts_layer_48_b200 as moe

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
SUM = 2.0 ** -18


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _near(got, ref, tol, what):
    assert got.shape == ref.shape and torch.isfinite(got).all(), what
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), f"{what}: {(err - tol).max().item():.3g} over, |ref| up to {ref.abs().max().item():.3g}"


# ---- SwiGLU ------------------------------------------------------------------------------------

def _swiglu_case(R, I, weighted, seed=0, std=2.0):
    g = _gen(seed)
    gu, dh = _normal(g, (R, 2 * I), std), _normal(g, (R, I))
    w = torch.rand((R,), generator=g, device="cuda") + 0.1 if weighted else None
    layer = moe.Moe(1, 64, I, 1)
    h = layer.swiglu(gu, w)
    dgu, dw = layer.swiglu_backward(dh, gu, w)
    assert layer.sync_status() == moe.MOE_OK
    a, b, d = gu[:, :I].double(), gu[:, I:].double(), dh.double()
    ww = 1.0 if w is None else w.double()[:, None]
    s = torch.sigmoid(a)
    # the sigmoid in fp32: exp's argument is rounded (|g| 2^-24) and a few steps follow
    rel = (a.abs() + 8) * 2.0 ** -23
    # and a sigmoid below 2^-126 may come out as 0
    tiny = 2.0 ** -125
    ref = ww * a * s * b
    _near(h, ref, (HALF[BF16] + 2 * rel) * ref.abs() + tiny * (1 + (ww * a * b).abs()), "h")
    du = ww * d * a * s
    _near(dgu[:, I:], du, (HALF[BF16] + 2 * rel) * du.abs() + tiny * (1 + (ww * a * d).abs()), "du")
    dg = ww * d * b * s * (1 + a * (1 - s))
    # 1 + g (1 - s) cancels near g = -1.28: the error is that of its two parts
    mag = (ww * d * b * s).abs() * (1 + a.abs() * (1 - s))
    _near(dgu[:, :I], dg, HALF[BF16] * dg.abs() + 4 * rel * mag + tiny * (1 + (ww * d * b).abs() * (1 + a.abs())), "dg")
    if weighted:
        terms = d * a * s * b
        _near(dw, terms.sum(1), (SUM + 2 * rel.amax(1)) * terms.abs().sum(1), "drow_w")
    else:
        assert dw is None


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("R,I", [(1, 64), (3, 128), (64, 2880), (1000, 704), (129, 832), (5, 1536), (33, 1600),
                                 (7, 4096), (6, 6208), (3, 12288), (2, 12352), (2, 16384), (2049, 64)])
def test_swiglu(R, I, weighted):
    _swiglu_case(R, I, weighted, seed=R + I)


def test_swiglu_large_gates():
    """Saturated sigmoids: gates up to +-1e4 give finite results."""
    _swiglu_case(40, 256, True, seed=5, std=3e3)


def test_swiglu_past_2_to_the_31_elements():
    R, I = 70001, 16384
    g = _gen(7)
    gu = torch.empty((R, 2 * I), dtype=BF16, device="cuda")
    gu.normal_(generator=g)
    dh = torch.empty((R, I), dtype=BF16, device="cuda").normal_(generator=g)
    w = torch.rand((R,), generator=g, device="cuda")
    layer = moe.Moe(1, 64, I, 1)
    h = layer.swiglu(gu, w)
    dgu, dw = layer.swiglu_backward(dh, gu, w)
    rows = [0, 65535, 65536, R - 1]
    part = [t[rows].contiguous() for t in (gu, dh, w)]
    small = layer.swiglu(part[0], part[2])
    d_small, dw_small = layer.swiglu_backward(part[1], part[0], part[2])
    assert torch.equal(h[rows], small) and torch.equal(dgu[rows], d_small) and torch.equal(dw[rows], dw_small)


def test_swiglu_gradient_is_that_of_the_function():
    I = 128
    g = _gen(6)
    gu, dh = _normal(g, (9, 2 * I)), _normal(g, (9, I))
    w = torch.rand((9,), generator=g, device="cuda") + 0.1
    layer = moe.Moe(1, 64, I, 1)
    dgu, dw = layer.swiglu_backward(dh, gu, w)
    a, ww = gu.double(), w.double()
    f = lambda v, q: q[:, None] * v[:, :I] / (1 + torch.exp(-v[:, :I])) * v[:, I:]  # noqa: E731
    for _ in range(4):
        da, dq = torch.randn_like(a), torch.randn_like(ww)
        h = 1e-5
        num = ((f(a + h * da, ww + h * dq) - f(a - h * da, ww - h * dq)) * dh.double()).sum() / (2 * h)
        parts = torch.cat([(dgu.double() * da).flatten(), dw.double() * dq])
        # every entry is off by at most half a step of bf16; the differences by h^2 and 1e-16 / h
        assert (num - parts.sum()).abs() <= HALF[BF16] * parts.abs().sum() + 1e-6 * parts.abs().sum()


def test_swiglu_out_argument_and_refusals():
    layer = moe.Moe(1, 64, 128, 1)
    gu = torch.zeros((4, 256), dtype=BF16, device="cuda")
    out = torch.ones((4, 128), dtype=BF16, device="cuda")
    assert layer.swiglu(gu, out=out) is out and (out == 0).all()
    w = torch.ones((4,), device="cuda")
    for bad in (dict(gu=gu.float()), dict(gu=gu[:, :128]), dict(gu=gu, row_w=w[:3]), dict(gu=gu, row_w=w.half()),
                dict(gu=gu, out=out[:2]), dict(gu=gu.cpu())):
        with pytest.raises(ValueError):
            layer.swiglu(**bad)
    with pytest.raises(ValueError):
        layer.swiglu_backward(out[:3], gu)
    assert torch.equal(layer.swiglu(gu, torch.ones((5,), device="cuda")[1:]), layer.swiglu(gu, w))
    assert layer.swiglu(gu[:0]).shape == (0, 128)
    d, dw = layer.swiglu_backward(out[:0], gu[:0], w[:0])
    assert d.shape == (0, 256) and dw.shape == (0,)
    # a gradient of weights that are not there
    assert moe.moe_swiglu_backward(layer.handle, 4, out.data_ptr(), gu.data_ptr(), None,
                                   gu.clone().data_ptr(), w.data_ptr(), None) == moe.MOE_ERR_ARG


# ---- the norms around the block --------------------------------------------------------------------

EPS = 1e-5


def _inputs(T, H, rt, yt, post, gate, nxt, seed):
    g = _gen(seed)
    vec = lambda on: 1 + 0.3 * torch.randn((H,), generator=g, device="cuda") if on else None  # noqa: E731
    return dict(resid=_normal(g, (T, H), 2.0, rt), y=None if yt is None else _normal(g, (T, H), 0.7, yt),
                w_post=vec(post), gate=vec(gate), w_next=vec(nxt)), g


def _forward_case(T, H, rt, yt, post, gate, nxt, scale=0.5, seed=0, inplace=False):
    a, _ = _inputs(T, H, rt, yt, post, gate, nxt, seed)
    layer = moe.Moe(1, H, 64, 1)
    before = a["resid"].double()
    r = layer.block_norm(**a, scale=scale, eps=EPS, resid_out=a["resid"] if inplace else None)
    assert layer.sync_status() == moe.MOE_OK
    if yt is None:
        assert r["resid"] is a["resid"] and torch.equal(r["resid"].double(), before)
    else:
        n = a["y"].double()
        if post:
            rstd = 1 / torch.sqrt(n.square().mean(1) + EPS)
            _near(r["rstd_post"], rstd, SUM * rstd, "rstd_post")
            n = n * rstd[:, None] * a["w_post"].double()
        b = scale * n * (1 if a["gate"] is None else a["gate"].double())
        ref = before + b
        _near(r["resid"], ref, HALF[rt] * ref.abs() + (SUM + 2.0 ** -22) * b.abs() + 2.0 ** -24 * before.abs(), "resid")
    assert (r["rstd_post"] is not None) == post and (r["x"] is not None) == (r["rstd_next"] is not None) == nxt
    if nxt:   # x is the norm of the new residual as it is stored
        q = r["resid"].double()
        rstd = 1 / torch.sqrt(q.square().mean(1) + EPS)
        _near(r["rstd_next"], rstd, SUM * rstd, "rstd_next")
        ref = q * rstd[:, None] * a["w_next"].double()
        _near(r["x"], ref, (HALF[BF16] + 2 * SUM) * ref.abs(), "x")


TYPES = [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)]
WHAT = [(False, False, True), (True, False, True), (False, True, False), (True, True, True), (False, False, False)]
SIZES = [(1, 64), (3, 768), (130, 832), (257, 2880), (5, 1536), (66, 1600), (9, 4160), (3, 6208), (2, 12288), (3, 16384)]


@pytest.mark.parametrize("rt,yt", TYPES)
@pytest.mark.parametrize("post,gate,nxt", WHAT)
@pytest.mark.parametrize("T,H", SIZES)
def test_block_norm(T, H, rt, yt, post, gate, nxt):
    _forward_case(T, H, rt, yt, post, gate, nxt, seed=T + H)


@pytest.mark.parametrize("rt", [BF16, F32])
@pytest.mark.parametrize("T,H", SIZES)
def test_norm_before_the_first_block(T, H, rt):
    _forward_case(T, H, rt, None, False, False, True, seed=T)


# more rows than the persistent blocks hold at once, several times over: every ring slot is refilled
LONG = [(20011, 64), (15013, 192), (9001, 384), (6007, 640), (5003, 1088), (6001, 2880), (3001, 6016), (1501, 8128)]


@pytest.mark.parametrize("rt,yt", [(BF16, F32), (BF16, BF16), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("post,nxt", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("T,H", LONG)
def test_block_norm_many_rows(T, H, rt, yt, post, nxt):
    _forward_case(T, H, rt, yt, post, True, nxt, seed=T)


@pytest.mark.parametrize("rt", [BF16, F32])
def test_block_norm_in_place(rt):
    _forward_case(77, 2880, rt, F32, True, True, True, seed=3, inplace=True)


def test_block_norm_extreme_rows():
    """A row of zeros (the norm is eps alone), tiny rows and rows of large values."""
    H = 256
    layer = moe.Moe(1, H, 64, 1)
    resid = torch.zeros((4, H), device="cuda")
    resid[1], resid[2], resid[3] = 1e-20, 1e15, -3e4
    w = torch.ones((H,), device="cuda")
    r = layer.block_norm(resid, w_next=w, eps=1e-6)
    assert (r["x"][0] == 0).all() and torch.isfinite(r["x"].float()).all()
    ref = resid.double() / torch.sqrt(resid.double().square().mean(1, keepdim=True) + 1e-6)
    _near(r["x"], ref, (HALF[BF16] + 2 * SUM) * ref.abs() + 1e-38, "x")


def _backward_case(T, H, rt, yt, post, gate, nxt, dyt=BF16, scale=0.5, seed=0, direct=True):
    a, g = _inputs(T, H, rt, yt, post, gate, nxt, seed)
    layer = moe.Moe(1, H, 64, 1)
    f = layer.block_norm(**a, scale=scale, eps=EPS) if yt is not None or nxt else None
    dres = _normal(g, (T, H), 0.3, rt) if direct else None
    dx = _normal(g, (T, H), 0.3) if nxt else None
    b = layer.block_norm_backward(dres, dx, f["resid"], a["y"], rstd_post=f["rstd_post"], rstd_next=f["rstd_next"],
                                  w_post=a["w_post"], gate=a["gate"], scale=scale, w_next=a["w_next"],
                                  dy_dtype=dyt)
    assert layer.sync_status() == moe.MOE_OK
    D = lambda t: None if t is None else t.double()  # noqa: E731
    zero = torch.zeros((T, H), dtype=F64, device="cuda")
    d = zero if dres is None else D(dres)
    mag = d.abs()          # magnitudes that went into d: its fp32 error is SUM of them
    if nxt:
        q, r = D(f["rstd_next"])[:, None], D(f["resid"])
        rh, t = r * q, D(dx) * D(a["w_next"])
        d = d + q * (t - rh * (t * rh).mean(1, keepdim=True))
        mag = mag + q * (t.abs() + rh.abs() * (t * rh).abs().mean(1, keepdim=True))
        ref, m = (D(dx) * rh).sum(0), (D(dx) * rh).abs().sum(0)
        _near(b["dw_next"], ref, SUM * m + T * 2.0 ** -26 * m, "dw_next")
    _near(b["dresid"], d, HALF[rt] * d.abs() + SUM * mag, "dresid")
    if yt is None:
        assert b["dy"] is None
        return
    v, db, m = D(a["y"]), scale * d, scale * mag
    q = D(f["rstd_post"])[:, None] if post else 1.0
    yh = v * q
    if gate:
        n = yh * D(a["w_post"]) if post else yh
        _near(b["dgate"], (db * n).sum(0), (SUM + T * 2.0 ** -26) * (m * n.abs()).sum(0), "dgate")
        db, m = db * D(a["gate"]), m * D(a["gate"]).abs()
    if post:
        _near(b["dw_post"], (db * yh).sum(0), (SUM + T * 2.0 ** -26) * (m * yh.abs()).sum(0), "dw_post")
        t, tm = db * D(a["w_post"]), m * D(a["w_post"]).abs()
        db = q * (t - yh * (t * yh).mean(1, keepdim=True))
        m = q * (tm + yh.abs() * (tm * yh.abs()).mean(1, keepdim=True))
    assert b["dy"].dtype == dyt
    _near(b["dy"], db, HALF[dyt] * db.abs() + 2 * SUM * m, "dy")


@pytest.mark.parametrize("rt,yt", TYPES)
@pytest.mark.parametrize("post,gate,nxt", WHAT)
@pytest.mark.parametrize("T,H", SIZES)
def test_block_norm_backward(T, H, rt, yt, post, gate, nxt):
    _backward_case(T, H, rt, yt, post, gate, nxt, dyt=BF16 if T % 2 else F32, seed=T + H)


@pytest.mark.parametrize("rt,yt", [(BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("post,nxt", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("T,H", LONG)
def test_block_norm_backward_many_rows(T, H, rt, yt, post, nxt):
    _backward_case(T, H, rt, yt, post, post, nxt, seed=T)


@pytest.mark.parametrize("rt", [BF16, F32])
@pytest.mark.parametrize("T,H", [(1, 64), (1000, 2880), (3001, 128), (5, 16384)])
def test_backward_of_the_norm_before_the_first_block(T, H, rt):
    _backward_case(T, H, rt, None, False, False, True, seed=T)
    _backward_case(T, H, rt, None, False, False, True, seed=T, direct=False)


def test_backward_without_a_direct_gradient():
    """The last block: nothing reads the residual but the final norm."""
    _backward_case(301, 2880, BF16, F32, True, True, True, seed=1, direct=False)


def test_backward_of_many_rows_twice_gives_the_same_bits():
    T, H = 5000, 704
    _backward_case(T, H, F32, BF16, True, True, True, seed=2)
    a, g = _inputs(T, H, F32, F32, True, True, True, 9)
    layer = moe.Moe(1, H, 64, 1)
    f = layer.block_norm(**a)
    dres, dx = _normal(g, (T, H), 0.3, F32), _normal(g, (T, H))
    kw = dict(rstd_post=f["rstd_post"], rstd_next=f["rstd_next"], w_post=a["w_post"], gate=a["gate"], w_next=a["w_next"])
    b1 = layer.block_norm_backward(dres, dx, f["resid"], a["y"], **kw)
    b2 = layer.block_norm_backward(dres, dx, f["resid"], a["y"], **kw)
    for key in b1:
        assert torch.equal(b1[key], b2[key]), key


def test_backward_is_the_gradient_of_the_forward():
    """Against float64 differences of the two results along random directions."""
    T, H, scale = 6, 128, 0.7
    a, g = _inputs(T, H, F32, F32, True, True, True, 11)
    layer = moe.Moe(1, H, 64, 1)
    f = layer.block_norm(**a, scale=scale, eps=EPS)
    dres, dx = _normal(g, (T, H), 1.0, F32), _normal(g, (T, H))
    b = layer.block_norm_backward(dres, dx, f["resid"], a["y"], rstd_post=f["rstd_post"], rstd_next=f["rstd_next"],
                                  w_post=a["w_post"], gate=a["gate"], scale=scale, w_next=a["w_next"], dy_dtype=F32)

    def loss(resid, y, w_post, gate, w_next):
        n = y / torch.sqrt(y.square().mean(1, keepdim=True) + EPS) * w_post
        r = resid + scale * gate * n
        x = r / torch.sqrt(r.square().mean(1, keepdim=True) + EPS) * w_next
        return (r * dres.double()).sum() + (x * dx.double()).sum()

    names = ["resid", "y", "w_post", "gate", "w_next"]
    grads = [b["dresid"], b["dy"], b["dw_post"], b["dgate"], b["dw_next"]]
    at = [a[n].double() for n in names]
    h = 1e-5
    for i, (name, grad) in enumerate(zip(names, grads)):
        v = torch.randn_like(at[i])
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * v, at[i] - h * v
        num = (loss(*up) - loss(*down)) / (2 * h)
        part = (grad.double() * v).flatten()
        # fp32 gradients: SUM of the terms; the difference: h^2 and 1e-16 / h of the loss
        assert (num - part.sum()).abs() <= 1e-5 * part.abs().sum() + 1e-6, name


def test_norm_past_2_to_the_31_elements():
    T, H = 140001, 16384
    g = _gen(12)
    resid = torch.empty((T, H), dtype=BF16, device="cuda").normal_(generator=g)
    y = torch.empty((T, H), dtype=BF16, device="cuda").normal_(generator=g)
    w = 1 + 0.1 * torch.randn((H,), generator=g, device="cuda")
    layer = moe.Moe(1, H, 64, 1)
    f = layer.block_norm(resid, y, w_post=w, gate=w, w_next=w)
    rows = [0, 131071, 131072, T - 1]
    s = layer.block_norm(resid[rows].contiguous(), y[rows].contiguous(), w_post=w, gate=w, w_next=w)
    assert torch.equal(f["x"][rows], s["x"]) and torch.equal(f["resid"][rows], s["resid"])
    kw = dict(w_post=w, gate=w, w_next=w)
    b = layer.block_norm_backward(resid, f["x"], f["resid"], y, rstd_post=f["rstd_post"], rstd_next=f["rstd_next"], **kw)
    c = layer.block_norm_backward(resid[rows].contiguous(), s["x"], s["resid"], y[rows].contiguous(),
                                  rstd_post=s["rstd_post"], rstd_next=s["rstd_next"], **kw)
    assert torch.equal(b["dresid"][rows], c["dresid"]) and torch.equal(b["dy"][rows], c["dy"])
    assert layer.sync_status() == moe.MOE_OK


def test_norm_captured_and_on_another_stream():
    T, H = 700, 2880
    a, g = _inputs(T, H, BF16, F32, True, True, True, 13)
    dres, dx = _normal(g, (T, H)), _normal(g, (T, H))
    layer = moe.Moe(1, H, 64, 1)

    def step(stream=None):
        f = layer.block_norm(**a, stream=stream)
        b = layer.block_norm_backward(dres, dx, f["resid"], a["y"], rstd_post=f["rstd_post"], rstd_next=f["rstd_next"],
                                      w_post=a["w_post"], gate=a["gate"], w_next=a["w_next"], stream=stream)
        return list(f.values()) + list(b.values())

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    # two captured graphs, replayed in turn and at once on two streams: workspaces of their own
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step())
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(p, q) for p, q in zip(o, want))


def test_no_rows():
    H = 128
    layer = moe.Moe(1, H, 64, 1)
    e, w = torch.empty((0, H), device="cuda"), torch.ones((H,), device="cuda")
    r = layer.block_norm(e, e, w_post=w, gate=w, w_next=w)
    assert r["x"].shape == (0, H)
    b = layer.block_norm_backward(e, r["x"], r["resid"], e, rstd_post=r["rstd_post"], rstd_next=r["rstd_next"],
                                  w_post=w, gate=w, w_next=w)
    for key in ("dw_post", "dgate", "dw_next"):
        assert (b[key] == 0).all()


def test_norm_refusals():
    H, T = 128, 4
    layer = moe.Moe(1, H, 64, 1)
    r, w = torch.zeros((T, H), device="cuda"), torch.ones((H,), device="cuda")
    y = torch.zeros((T, H), dtype=BF16, device="cuda")
    for bad in (dict(resid=r.half(), w_next=w), dict(resid=r, y=y.half()), dict(resid=r, y=y[:2]), dict(resid=r, w_next=w[:64]),
                dict(resid=r, w_next=w.to(BF16)), dict(resid=r[:, :64], w_next=w), dict(resid=r.cpu(), w_next=w),
                dict(resid=r, y=y, resid_out=y)):
        with pytest.raises(ValueError):
            layer.block_norm(**bad)
    for bad in (dict(resid=r), dict(resid=r, w_post=w, w_next=w), dict(resid=r, gate=w, w_next=w),
                dict(resid=r, w_next=w, eps=0.0), dict(resid=r, w_next=w, eps=float("nan")),
                dict(resid=r, y=y, scale=float("inf")), dict(resid=r, w_next=w, resid_out=torch.zeros_like(r))):
        with pytest.raises(moe.MoeError) as e:
            layer.block_norm(**bad)
        assert e.value.status == moe.MOE_ERR_ARG
    f = layer.block_norm(r, y, w_post=w, w_next=w)
    good = dict(dresid=r, dx=f["x"], resid=f["resid"], y=y, rstd_post=f["rstd_post"], rstd_next=f["rstd_next"],
                w_post=w, w_next=w)
    layer.block_norm_backward(**good)
    for bad in (dict(dx=None), dict(rstd_next=None), dict(rstd_post=None), dict(y=None), dict(y=None, block=True),
                dict(w_next=None), dict(w_post=None), dict(resid=None), dict(block=False)):
        with pytest.raises(moe.MoeError) as e:
            layer.block_norm_backward(**{**good, **bad})
        assert e.value.status == moe.MOE_ERR_ARG
    with pytest.raises(moe.MoeError) as e:
        layer.block_norm_backward(**good, workspace=torch.empty((16,), dtype=torch.uint8, device="cuda"))
    assert e.value.status == moe.MOE_ERR_WORKSPACE
    assert layer.sync_status() == moe.MOE_OK
