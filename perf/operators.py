"""What is measured of the operators around the MoE layer that training and the transformer block need.

Four operators, each with its plain form (elementary torch operations in 32 bits) and the library's call:

  matmul   grouped products of ragged expert segments, y[r] = x[r] W[e(r)], and with `transpose`
           the product that the gradient of x takes, dx[r] = dy[r] W[e(r)]^T
  wgrad    the gradient of the expert weights, dW[e] = sum over e's rows of x[r]^T dy[r]
  swiglu   h[r] = w[r] silu(g[r]) u[r] on rows [g | u], and its backward pass
  norm     the RMS norms before and after the block with its gate and residual scale:
             r' = r + s * gate * (y / rms(y) * w_post),   x = r' / rms(r') * w_next
           and its backward pass

Sizes are those of the 20b layer (32 experts, hidden 2880), the 120b layer (128 experts) and the
tiny layer of this repository, at one token, a decode batch, a prefill and a long packed sequence.
"""
import functools
import math

import torch

own = False  # set by the tools: the library's kernels instead of the plain forms

EPS = 1e-5
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
TYPES = {"bf16": BF16, "f32": F32}


def listed():
    return [
        # gate/up projection of a decode batch of 16 tokens: 64 rows over 32 experts
        dict(name="matmul up decode", op="matmul", tokens=16, k=4, E=32, K=2880, N=5760, transpose=False, out="bf16", skew=0.0, tail=0),
        # down projection of one token on the 128-expert layer, fp32 for the combine
        dict(name="matmul down one token", op="matmul", tokens=1, k=4, E=128, K=2880, N=2880, transpose=False, out="f32", skew=0.0, tail=0),
        # mid-size training microbatch, gradient of h through W_down: about 64 rows an expert
        dict(name="matmul down dx mid", op="matmul", tokens=509, k=4, E=32, K=2880, N=2880, transpose=True, out="bf16", skew=0.3, tail=7),
        # gradient of the layer input through W_gate_up, 8192-token step
        dict(name="matmul up dx 8k", op="matmul", tokens=8192, k=4, E=32, K=2880, N=5760, transpose=True, out="bf16", skew=0.3, tail=0),
        # gate/up projection of a long packed sequence with skewed routing
        dict(name="matmul up 32k skewed", op="matmul", tokens=32768, k=4, E=32, K=2880, N=5760, transpose=False, out="bf16", skew=0.5, tail=0),
        # weight gradient of the tiny layer's gate/up projection
        dict(name="wgrad tiny", op="wgrad", tokens=64, k=2, E=8, K=256, N=512, out="f32", skew=0.0, tail=0),
        # weight gradient of W_gate_up, 8192-token step
        dict(name="wgrad up 8k", op="wgrad", tokens=8192, k=4, E=32, K=2880, N=5760, out="bf16", skew=0.3, tail=0),
        # activation between the two projections of a decode batch
        dict(name="swiglu decode", op="swiglu", rows=64, I=2880, backward=False, weighted=False),
        # its backward pass in an 8192-token step, with the routing weights' gradient
        dict(name="swiglu bwd 8k", op="swiglu", rows=32768, I=2880, backward=True, weighted=True),
        # norm after the block and before the next one, one decoded token
        dict(name="norm one token", op="norm", T=1, H=2880, resid="bf16", y="f32", post=False, gate=False, next=True, backward=False),
        # the same with a post norm and a gate in an 8192-token prefill, ragged
        dict(name="norm 8k", op="norm", T=8189, H=2880, resid="bf16", y="f32", post=True, gate=True, next=True, backward=False),
        # backward pass of the whole thing with an fp32 residual stream, long sequence
        dict(name="norm bwd 32k", op="norm", T=32768, H=2880, resid="f32", y="f32", post=True, gate=True, next=True, backward=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matmul", "wgrad", "swiglu", "norm"])
    if op in ("matmul", "wgrad"):
        E = rng.choice([1, 3, 8, 32, 48, 128])
        k = min(E, rng.choice([1, 2, 4, 6]))
        K, N = 8 * _log_int(rng, 8, 720), 8 * _log_int(rng, 8, 720)
        while K * N > 2880 * 5760 or E * K * N > 32 * 2880 * 5760:
            K, N = 8 * _log_int(rng, 8, 720), 8 * _log_int(rng, 8, 720)
        tokens = _log_int(rng, 1, min(16384, 131072 // k))
        c = dict(op=op, tokens=tokens, k=k, E=E, K=K, N=N, out=rng.choice(["bf16", "f32"]),
                 skew=rng.choice([0.0, 0.3, 0.8]), tail=rng.choice([0, 0, 1, 37]))
        if op == "matmul":
            c["transpose"] = rng.random() < 0.5
        return c
    if op == "swiglu":
        return dict(op=op, rows=_log_int(rng, 1, 32768), I=64 * rng.randint(1, 64), backward=rng.random() < 0.5,
                    weighted=rng.random() < 0.5)
    H = 64 * rng.randint(1, 80)
    block = rng.random() < 0.75   # without: the first norm of a model, no block before it
    return dict(op=op, T=_log_int(rng, 1, 32768 * 2880 // max(H, 2880)), H=H, resid=rng.choice(["bf16", "f32"]),
                y=rng.choice(["bf16", "f32"]) if block else "", post=block and rng.random() < 0.5,
                gate=block and rng.random() < 0.5, next=not block or rng.random() < 0.75, backward=rng.random() < 0.5)


def _segments(c, g):
    """Row counts of the experts for `tokens` tokens that pick k distinct experts each, with a
    popularity that falls off as rank^-skew."""
    T, E, k = c["tokens"], c["E"], c["k"]
    rank = torch.randperm(E, generator=g, device="cuda") + 1
    score = torch.rand((T, E), generator=g, device="cuda").clamp_min(1e-9).log().neg().log().neg()
    score -= c["skew"] * rank.log()
    counts = torch.bincount(score.topk(k, dim=1).indices.reshape(-1), minlength=E)
    return counts.tolist()


def _normal(g, shape, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=g, device="cuda", dtype=F32) * std).to(dtype)


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=c)
    if c["op"] in ("matmul", "wgrad"):
        counts = _segments(c, g)
        bounds = [0]
        for n in counts:
            bounds.append(bounds[-1] + n)
        R, K, N, E = bounds[-1] + c["tail"], c["K"], c["N"], c["E"]
        s["bounds"] = bounds
        s["offsets"] = torch.tensor(bounds, dtype=torch.int32, device="cuda")
        if c["op"] == "wgrad":
            s["x"], s["dy"] = _normal(g, (R, K)), _normal(g, (R, N))
            return s
        s["W"] = torch.empty((E, K, N), dtype=BF16, device="cuda")
        fan_in = N if c["transpose"] else K
        for e in range(E):
            s["W"][e] = _normal(g, (K, N), 1.0 / math.sqrt(fan_in))
        s["x"] = _normal(g, (R, N if c["transpose"] else K))
        # the caller's result buffer: rows behind the last segment stay as they are
        s["out"] = torch.zeros((R, K if c["transpose"] else N), dtype=TYPES[c["out"]], device="cuda")
    elif c["op"] == "swiglu":
        R, I = c["rows"], c["I"]
        s["gu"] = _normal(g, (R, 2 * I))
        s["w"] = torch.rand((R,), generator=g, device="cuda") * 0.9 + 0.05 if c["weighted"] else None
        if c["backward"]:
            s["dh"] = _normal(g, (R, I), 0.1)
    else:
        T, H = c["T"], c["H"]
        vec = lambda: 1.0 + 0.2 * torch.randn((H,), generator=g, device="cuda")  # noqa: E731
        s["scale"] = 0.5 if c["y"] else 1.0
        s["resid"] = _normal(g, (T, H), 2.0, TYPES[c["resid"]])
        s["y"] = _normal(g, (T, H), 0.5, TYPES[c["y"]]) if c["y"] else None
        s["w_post"] = vec() if c["post"] else None
        s["gate"] = vec() if c["gate"] else None
        s["w_next"] = vec() if c["next"] else None
        if c["backward"]:
            # what the forward pass kept: the new residual and the two reciprocal norms
            r = s["resid"].float()
            s["rstd_post"] = s["rstd_next"] = None
            if c["y"]:
                y = s["y"].float()
                if c["post"]:
                    s["rstd_post"] = (y.square().mean(1) + EPS).rsqrt()
                    y = y * s["rstd_post"][:, None] * s["w_post"]
                r = r + s["scale"] * (y if s["gate"] is None else y * s["gate"])
            s["resid"] = r.to(TYPES[c["resid"]])
            if c["next"]:
                s["rstd_next"] = (s["resid"].float().square().mean(1) + EPS).rsqrt()
                s["dx"] = _normal(g, (T, H), 0.1)
            else:
                s["dx"] = None
            s["dresid"] = _normal(g, (T, H), 0.1, TYPES[c["resid"]])
    return s


# ---- the plain forms ----------------------------------------------------------------------------

def _plain_matmul(s):
    c, o = s["case"], s["bounds"]
    for e in range(c["E"]):
        if o[e + 1] > o[e]:
            W = s["W"][e].float()
            s["out"][o[e]:o[e + 1]] = s["x"][o[e]:o[e + 1]].float() @ (W.t() if c["transpose"] else W)
    return s["out"]


def _plain_wgrad(s):
    c, o = s["case"], s["bounds"]
    dW = torch.empty((c["E"], c["K"], c["N"]), dtype=TYPES[c["out"]], device="cuda")
    for e in range(c["E"]):
        dW[e] = s["x"][o[e]:o[e + 1]].float().t() @ s["dy"][o[e]:o[e + 1]].float()
    return dW


def _plain_swiglu(s):
    c, I = s["case"], s["case"]["I"]
    g, u = s["gu"][:, :I].float(), s["gu"][:, I:].float()
    sig = 1.0 / (1.0 + (-g).exp())
    if not c["backward"]:
        h = g * sig * u
        return (h if s["w"] is None else h * s["w"][:, None]).to(BF16)
    dh = s["dh"].float()
    dw = None if s["w"] is None else (dh * (g * sig * u)).sum(1)
    if s["w"] is not None:
        dh = dh * s["w"][:, None]
    dgu = torch.empty_like(s["gu"])
    dgu[:, :I] = dh * u * (sig * (1.0 + g * (1.0 - sig)))
    dgu[:, I:] = dh * (g * sig)
    return [dgu] if dw is None else [dgu, dw]


def _plain_norm(s):
    r, out = s["resid"].float(), {}
    if s["y"] is not None:
        b = s["y"].float()
        if s["w_post"] is not None:
            out["rstd_post"] = (b.square().mean(1) + EPS).rsqrt()
            b = b * out["rstd_post"][:, None] * s["w_post"]
        if s["gate"] is not None:
            b = b * s["gate"]
        out["resid"] = (r + s["scale"] * b).to(s["resid"].dtype)
        r = out["resid"].float()
    if s["w_next"] is not None:
        out["rstd_next"] = (r.square().mean(1) + EPS).rsqrt()
        out["x"] = (r * out["rstd_next"][:, None] * s["w_next"]).to(BF16)
    return out


def _plain_norm_backward(s):
    dr, out = s["dresid"].float(), {}
    if s["w_next"] is not None:
        dx, rhat = s["dx"].float(), s["resid"].float() * s["rstd_next"][:, None]
        out["dw_next"] = (dx * rhat).sum(0)
        t = dx * s["w_next"]
        dr = dr + s["rstd_next"][:, None] * (t - rhat * (t * rhat).mean(1, keepdim=True))
    out["dresid"] = dr.to(s["resid"].dtype)
    if s["y"] is not None:
        y, db = s["y"].float(), s["scale"] * dr
        yhat = y if s["w_post"] is None else y * s["rstd_post"][:, None]
        if s["gate"] is not None:
            out["dgate"] = (db * (yhat if s["w_post"] is None else yhat * s["w_post"])).sum(0)
            db = db * s["gate"]
        if s["w_post"] is not None:
            out["dw_post"] = (db * yhat).sum(0)
            t = db * s["w_post"]
            db = s["rstd_post"][:, None] * (t - yhat * (t * yhat).mean(1, keepdim=True))
        out["dy"] = db.to(BF16)
    return out


# ---- the library's calls ----------------------------------------------------------------------------

@functools.lru_cache(maxsize=None)
def _layer(E, H, I, k):
    from mixture_experts_layer_48_b200 import Moe
    return Moe(E=E, H=H, I=I, k=k)


def _own(s):
    c = s["case"]
    if c["op"] == "matmul":
        layer = _layer(c["E"], 64, 64, c["k"])
        return layer.grouped_matmul(s["x"], s["W"], s["offsets"], transpose=c["transpose"], out=s["out"])
    if c["op"] == "wgrad":
        layer = _layer(c["E"], 64, 64, c["k"])
        return layer.grouped_wgrad(s["x"], s["dy"], s["offsets"], out_dtype=TYPES[c["out"]])
    if c["op"] == "swiglu":
        layer = _layer(1, 64, c["I"], 1)
        if not c["backward"]:
            return layer.swiglu(s["gu"], s["w"])
        dgu, dw = layer.swiglu_backward(s["dh"], s["gu"], s["w"])
        return [dgu] if dw is None else [dgu, dw]
    layer = _layer(1, c["H"], 64, 1)
    if not c["backward"]:
        r = layer.block_norm(s["resid"], s["y"], w_post=s["w_post"], gate=s["gate"], scale=s["scale"],
                             w_next=s["w_next"], eps=EPS)
        if s["y"] is None:
            r.pop("resid")   # nothing was added: the residual is the caller's own
    else:
        r = layer.block_norm_backward(s["dresid"], s["dx"], s["resid"], s["y"], rstd_post=s["rstd_post"],
                                      rstd_next=s["rstd_next"], w_post=s["w_post"], gate=s["gate"],
                                      scale=s["scale"], w_next=s["w_next"], dy_dtype=BF16)
    return {key: v for key, v in r.items() if v is not None}


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "norm":
        return _plain_norm_backward(state) if c["backward"] else _plain_norm(state)
    return {"matmul": _plain_matmul, "wgrad": _plain_wgrad, "swiglu": _plain_swiglu}[c["op"]](state)


# ---- from the definitions, in 64 bits ---------------------------------------------------------------

def _exact_norm(s):
    c, out = s["case"], {}
    r = s["resid"].double()
    gate = 1.0 if s["gate"] is None else s["gate"].double()
    if s["y"] is not None:
        y = s["y"].double()
        n = y
        if c["post"]:
            rms = torch.sqrt((y * y).sum(1) / c["H"] + EPS)
            out["rstd_post"] = 1.0 / rms
            n = y / rms[:, None] * s["w_post"].double()
        # the new residual is kept in its own type, and the next norm reads it so
        out["resid"] = r + s["scale"] * gate * n
        r = out["resid"].to(s["resid"].dtype).double()
    if c["next"]:
        rms = torch.sqrt((r * r).sum(1) / c["H"] + EPS)
        out["rstd_next"] = 1.0 / rms
        out["x"] = r / rms[:, None] * s["w_next"].double()
    return out


def _exact_norm_backward(s):
    """The vector-Jacobian products of v -> w v / rms(v), written with the kept reciprocal norms:
    d v = (w d - v <w d, v> / (H rms^2)) / rms."""
    c, out = s["case"], {}
    d = s["dresid"].double()
    if c["next"]:
        q, v, dx = s["rstd_next"].double()[:, None], s["resid"].double(), s["dx"].double()
        out["dw_next"] = torch.einsum("th,th->h", dx, v * q)
        wd = dx * s["w_next"].double()
        d = d + q * wd - v * q ** 3 * torch.einsum("th,th->t", wd, v)[:, None] / c["H"]
    out["dresid"] = d
    if s["y"] is not None:
        v, d = s["y"].double(), s["scale"] * d
        gate = 1.0 if s["gate"] is None else s["gate"].double()
        if c["post"]:
            q, w = s["rstd_post"].double()[:, None], s["w_post"].double()
            if s["gate"] is not None:
                out["dgate"] = torch.einsum("th,th->h", d, v * q) * w
            out["dw_post"] = torch.einsum("th,th->h", d, v * q) * gate
            wd = d * gate * w
            out["dy"] = q * wd - v * q ** 3 * torch.einsum("th,th->t", wd, v)[:, None] / c["H"]
        else:
            if s["gate"] is not None:
                out["dgate"] = torch.einsum("th,th->h", d, v)
            out["dy"] = d * gate
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "matmul":
        out = torch.zeros(s["out"].shape, dtype=F64, device="cuda")
        expert = torch.bucketize(torch.arange(s["bounds"][-1], device="cuda"), s["offsets"][1:].long(), right=True)
        for e in expert.unique().tolist():
            rows = (expert == e).nonzero().squeeze(1)
            out[rows] = torch.einsum("rn,kn->rk" if c["transpose"] else "rk,kn->rn", s["x"][rows].double(), s["W"][e].double())
        return out
    if c["op"] == "wgrad":
        o = s["bounds"]
        return torch.stack([torch.einsum("rk,rn->kn", s["x"][a:b].double(), s["dy"][a:b].double()) for a, b in zip(o, o[1:])])
    if c["op"] == "swiglu":
        g, u = s["gu"].double().chunk(2, dim=1)
        w = torch.ones((), dtype=F64, device="cuda") if s["w"] is None else s["w"].double()[:, None]
        sig = torch.sigmoid(g)
        if not c["backward"]:
            return w * g * sig * u
        dh = s["dh"].double()
        dgu = torch.cat([w * dh * u * (sig + g * sig * (1 - sig)), w * dh * g * sig], dim=1)
        return [dgu] if s["w"] is None else [dgu, torch.einsum("ri,ri->r", dh, g * sig * u)]
    return _exact_norm_backward(s) if c["backward"] else _exact_norm(s)


# ---- what one pass cannot do without ---------------------------------------------------------------

def work(case):
    c = case
    if c["op"] in ("matmul", "wgrad"):
        R, K, N, E = c["tokens"] * c["k"], c["K"], c["N"], c["E"]
        size = 2 if c["out"] == "bf16" else 4
        flops = 2.0 * R * K * N
        if c["op"] == "wgrad":
            return dict(bytes=2.0 * R * (K + N) + size * float(E) * K * N, flops=flops)
        touched = E * (1.0 - (1.0 - c["k"] / E) ** c["tokens"])   # experts with a row, evenly spread routing
        ins, outs = (N, K) if c["transpose"] else (K, N)
        return dict(bytes=2.0 * touched * K * N + 2.0 * R * ins + size * R * outs, flops=flops)
    if c["op"] == "swiglu":
        R, I = c["rows"], c["I"]
        b = R * I * (10.0 if c["backward"] else 6.0) + (4.0 * R * (2 if c["backward"] else 1) if c["weighted"] else 0)
        return dict(bytes=b, flops=R * I * (16.0 if c["backward"] else 6.0))
    n, T = c["T"] * c["H"], c["T"]
    r, y = (2 if c["resid"] == "bf16" else 4), {"": 0, "bf16": 2, "f32": 4}[c["y"]]
    vecs = 4.0 * c["H"] * (c["post"] + c["gate"] + c["next"])
    stats = 4.0 * T * (c["post"] + c["next"])
    if not c["backward"]:
        return dict(bytes=n * (r + (y + r if y else 0) + (2 if c["next"] else 0)) + vecs + stats, flops=10.0 * n)
    # reads the gradient of the new residual, dx with the residual, y; writes dresid, dy, the sums
    # (a block that has neither post norm nor gate needs no y)
    b = 2.0 * n * r + (n * (2 + r) if c["next"] else 0) + (n * 2 + (n * y if c["post"] or c["gate"] else 0) if y else 0)
    return dict(bytes=b + 2 * vecs + stats, flops=20.0 * n)
