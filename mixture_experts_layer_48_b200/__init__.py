"""Python binding of the B200 MoE layer library (libmoe.so, C ABI in include/moe.h).

Argument marshalling only: every step of the layer runs in the library's CUDA kernels.
PyTorch provides device memory and the current stream.  The module refuses to load without
the compiled library -- there is no CPU fallback.

    from mixture_experts_layer_48_b200 import Moe
    layer = Moe(E=32, H=2880, I=2880, k=4)
    out = layer.forward(x, W_router, b_router, W_gate_up, W_down)   # out [T, H] fp32
    r = layer.route(x, W_router, b_router)   # topk_idx, topk_w, expert_offsets, perm, inv_perm

The pieces of a training step (grouped_matmul, grouped_wgrad, swiglu, swiglu_backward) and the
norms around the block (block_norm, block_norm_backward, block) are methods of the same class.  No
method records anything for autograd: arguments may require a gradient, results never do, and the
backward methods are called by name (from a torch.autograd.Function, for instance).
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python mixture_experts_layer_48_b200/build.py` "
        "(or __graft_entry__.build()); this package has no fallback")

_lib = ctypes.CDLL(LIB_PATH)

MOE_OK, MOE_ERR_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE = 0, 1, 2, 3
MOE_ERR_CUDA, MOE_ERR_TIMEOUT, MOE_ERR_DEVICE = 4, 5, 6
MOE_PATH_AUTO, MOE_PATH_STREAM, MOE_PATH_GEMM, MOE_PATH_TILE = 0, 1, 2, 3
MOE_PROFILE_KINDS = 10
MOE_BF16, MOE_F32 = 0, 1

# Every entry point of include/moe.h: name -> (restype, argtypes)
_c_int, _vp, _sz = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
_c_float = ctypes.c_float
_SIGS = {
    "moe_create": (_c_int, [_c_int, _c_int, _c_int, _c_int, ctypes.POINTER(_vp)]),
    "moe_destroy": (_c_int, [_vp]),
    "moe_workspace_bytes": (_sz, [_vp, _c_int]),
    "moe_route_workspace_bytes": (_sz, [_vp, _c_int]),
    "moe_route": (_c_int, [_vp, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_forward": (_c_int, [_vp, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_workspace_bytes_mxfp4": (_sz, [_vp, _c_int]),
    "moe_forward_mxfp4": (_c_int, [_vp, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                   _sz, _vp]),
    "moe_set_path": (_c_int, [_vp, _c_int, _c_int]),
    "moe_get_path": (_c_int, [_vp, ctypes.POINTER(_c_int), ctypes.POINTER(_c_int)]),
    "moe_set_dispatch": (_c_int, [_vp, _c_int, _c_int, _c_int]),
    "moe_get_dispatch": (_c_int, [_vp, ctypes.POINTER(_c_int), ctypes.POINTER(_c_int),
                                  ctypes.POINTER(_c_int)]),
    "moe_tune_workspace_bytes": (_sz, [_vp, _c_int]),
    "moe_tune": (_c_int, [_vp, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp,
                          ctypes.POINTER(_c_int)]),
    "moe_sync_status": (_c_int, [_vp, _vp]),
    "moe_status_string": (ctypes.c_char_p, [_c_int]),
    "moe_launch_count": (ctypes.c_uint64, [_vp]),
    "moe_profile_begin": (_c_int, [_vp, _c_int]),
    "moe_profile_end": (_c_int, [_vp, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(_c_int),
                                 _c_int]),
    "moe_profile_kind_name": (ctypes.c_char_p, [_c_int]),
    "moe_selftest_timeout": (_c_int, [_vp, _c_int, _vp]),
    "moe_permute": (_c_int, [_vp, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_experts_workspace_bytes": (_sz, [_vp, _c_int, _c_int]),
    "moe_experts": (_c_int, [_vp, _c_int, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_combine": (_c_int, [_vp, _c_int, _vp, _vp, _vp, _vp]),
    "moe_last_dispatch": (_c_int, [_vp, _c_int, _c_int, _vp, _sz, _vp, _vp]),
    "moe_route_static_max_bytes": (_sz, []),
    "moe_grouped_matmul": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp, _c_int,
                                    _vp]),
    "moe_grouped_wgrad": (_c_int, [_vp, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp, _c_int, _vp]),
    "moe_swiglu": (_c_int, [_vp, _c_int, _vp, _vp, _vp, _vp]),
    "moe_swiglu_backward": (_c_int, [_vp, _c_int, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_block_norm": (_c_int, [_vp, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp, _c_float, _vp,
                                _c_float, _vp, _vp, _vp, _vp, _vp]),
    "moe_block_norm_workspace_bytes": (_sz, [_vp, _c_int]),
    "moe_block_norm_backward": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp,
                                         _vp, _vp, _vp, _vp, _c_float, _vp, _vp, _vp, _vp, _vp, _vp,
                                         _vp, _sz, _vp]),
    "moe_selftest_norm_timeout": (_c_int, [_vp, _c_int]),
    "moe_route_static": (_c_int, [_vp, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype, _f.argtypes = _res, _args
    globals()[_name] = _f

EXPORTED = tuple(_SIGS)


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {moe_status_string(status).decode()} (status {status})")


def _check(status: int, what: str) -> None:
    if status != MOE_OK:
        raise MoeError(status, what)


def _ptr(t: torch.Tensor | None, dtype: torch.dtype, name: str, shape=None) -> int:
    if t is None:
        return 0
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _scratch(ws: torch.Tensor, device) -> torch.Tensor:
    """A caller's workspace, which the kernels take for numel() bytes on the device of their tensors."""
    if ws.device != device or not ws.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}, got one on {ws.device}")
    return ws


# The current stream's handle; torch's own short way to it where it has one (a tenth of a
# microsecond instead of three for a Stream object).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


_DTYPES = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}


def _dtype(t, name: str) -> int:
    """moe_dtype of a tensor or a torch.dtype."""
    d = t.dtype if isinstance(t, torch.Tensor) else t
    if d not in _DTYPES:
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, got {d}")
    return _DTYPES[d]


class Moe:
    """One MoE layer shape (E experts, hidden H, intermediate I, top-k) bound to the current device."""

    def __init__(self, E: int, H: int, I: int, k: int):
        self.E, self.H, self.I, self.k = E, H, I, k
        h = _vp()
        _check(moe_create(E, H, I, k, ctypes.byref(h)), "moe_create")
        self._h = h
        self._ws = self._ws_key = None
        self._device_index = torch.cuda.current_device()

    # -- lifetime --------------------------------------------------------------------
    def close(self):
        if getattr(self, "_h", None):
            moe_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    # -- settings --------------------------------------------------------------------
    def set_path(self, path: int, crossover_T: int = -1) -> None:
        """Path; crossover_T >= 0 also sets the largest call AUTO streams (see include/moe.h)."""
        _check(moe_set_path(self._h, path, crossover_T), "moe_set_path")

    def get_path(self) -> tuple[int, int]:
        p, c = _c_int(), _c_int()
        _check(moe_get_path(self._h, ctypes.byref(p), ctypes.byref(c)), "moe_get_path")
        return p.value, c.value

    def set_dispatch(self, stream_rows: int = -1, tile_rows: int = -1, per_expert: int = -1) -> None:
        """AUTO thresholds in rows of one expert and the per-expert switch (negative: keep);
        see include/moe.h."""
        _check(moe_set_dispatch(self._h, stream_rows, tile_rows, int(per_expert)),
               "moe_set_dispatch")

    def get_dispatch(self) -> tuple[int, int, bool]:
        """(stream_rows, tile_rows, per_expert)."""
        s_, t_, p_ = _c_int(), _c_int(), _c_int()
        _check(moe_get_dispatch(self._h, ctypes.byref(s_), ctypes.byref(t_), ctypes.byref(p_)),
               "moe_get_dispatch")
        return s_.value, t_.value, bool(p_.value)

    def workspace_bytes(self, T: int) -> int:
        return moe_workspace_bytes(self._h, T)

    def route_workspace_bytes(self, T: int) -> int:
        return moe_route_workspace_bytes(self._h, T)

    def _workspace(self, nbytes: int, device, stream) -> torch.Tensor:
        """A call's workspace, of the stream that it runs on.  The last call's serves again on the same
        stream if it is large enough; a call that is being captured takes one of its graph's, which no
        later call is given."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self._workspace(nbytes, device, None)
        alone = device.type != "cuda" or torch.cuda.is_current_stream_capturing()
        key = None if alone else (device, _raw_stream(device.index))
        if alone or self._ws is None or self._ws_key != key or self._ws.numel() < nbytes:
            self._ws = None     # back to its stream or graph before the next one is taken
            self._ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
            self._ws_key = key
        return self._ws

    # -- the layer -------------------------------------------------------------------
    def route(self, x, W_router, b_router, stream=None, workspace=None) -> dict:
        T = x.shape[0]
        E, H, k = self.E, self.H, self.k
        dev = x.device
        out = dict(
            topk_idx=torch.empty((T, k), dtype=torch.int32, device=dev),
            topk_w=torch.empty((T, k), dtype=torch.float32, device=dev),
            expert_offsets=torch.empty((E + 1,), dtype=torch.int32, device=dev),
            perm=torch.empty((T * k,), dtype=torch.int32, device=dev),
            inv_perm=torch.empty((T, k), dtype=torch.int32, device=dev),
        )
        need = self.route_workspace_bytes(T)
        ws = self._workspace(need, dev, stream) if workspace is None else _scratch(workspace, dev)
        st = moe_route(self._h, T, _ptr(x, torch.bfloat16, "x", (T, H)),
                       _ptr(W_router, torch.bfloat16, "W_router", (H, E)),
                       _ptr(b_router, torch.float32, "b_router", (E,)),
                       out["topk_idx"].data_ptr(), out["topk_w"].data_ptr(),
                       out["expert_offsets"].data_ptr(), out["perm"].data_ptr(),
                       out["inv_perm"].data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream))
        _check(st, "moe_route")
        return out

    def forward(self, x, W_router, b_router, W_gate_up, W_down, out=None, stream=None,
                workspace=None) -> torch.Tensor:
        T = x.shape[0]
        E, H, I = self.E, self.H, self.I
        if out is None:
            out = torch.empty((T, H), dtype=torch.float32, device=x.device)
        need = self.workspace_bytes(T)
        ws = self._workspace(need, x.device, stream) if workspace is None else _scratch(workspace, x.device)
        st = moe_forward(self._h, T, _ptr(x, torch.bfloat16, "x", (T, H)),
                         _ptr(W_router, torch.bfloat16, "W_router", (H, E)),
                         _ptr(b_router, torch.float32, "b_router", (E,)),
                         _ptr(W_gate_up, torch.bfloat16, "W_gate_up", (E, H, 2 * I)),
                         _ptr(W_down, torch.bfloat16, "W_down", (E, I, H)),
                         _ptr(out, torch.float32, "out", (T, H)),
                         ws.data_ptr(), ws.numel(), _stream(stream))
        _check(st, "moe_forward")
        return out

    __call__ = forward

    # -- expert parallelism: device work on either side of the exchange (include/moe.h) --
    def permute(self, x, r: dict, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
        """Rows in expert order and their routing weights, from moe_route's outputs."""
        T = x.shape[0]
        R = T * self.k
        x_perm = torch.empty((R, self.H), dtype=torch.bfloat16, device=x.device)
        row_w = torch.empty((R,), dtype=torch.float32, device=x.device)
        st = moe_permute(self._h, T, _ptr(x, torch.bfloat16, "x", (T, self.H)),
                         _ptr(r["perm"], torch.int32, "perm", (R,)),
                         _ptr(r["inv_perm"], torch.int32, "inv_perm", (T, self.k)),
                         _ptr(r["topk_w"], torch.float32, "topk_w", (T, self.k)),
                         x_perm.data_ptr(), row_w.data_ptr(), _stream(stream))
        _check(st, "moe_permute")
        return x_perm, row_w

    def experts(self, x_rows, row_w, seg_counts, W_gate_up, W_down, stream=None,
                workspace=None) -> torch.Tensor:
        """The expert half on rows grouped as seg_counts [S, E] segments (source-major)."""
        R = x_rows.shape[0]
        S = seg_counts.shape[0]
        y = torch.empty((R, self.H), dtype=torch.float32, device=x_rows.device)
        if R == 0:
            return y
        need = moe_experts_workspace_bytes(self._h, R, S)
        if need == 0:
            raise ValueError("moe_experts: unsupported R or S")
        ws = self._workspace(need, x_rows.device, stream) if workspace is None else _scratch(workspace, x_rows.device)
        st = moe_experts(self._h, R, S, _ptr(seg_counts, torch.int32, "seg_counts", (S, self.E)),
                         _ptr(x_rows, torch.bfloat16, "x_rows", (R, self.H)),
                         _ptr(row_w, torch.float32, "row_w", (R,)),
                         _ptr(W_gate_up, torch.bfloat16, "W_gate_up", (self.E, self.H, 2 * self.I)),
                         _ptr(W_down, torch.bfloat16, "W_down", (self.E, self.I, self.H)),
                         y.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream))
        _check(st, "moe_experts")
        return y

    def combine(self, inv_perm, y_rows, out=None, stream=None) -> torch.Tensor:
        """out[t] = sum_j y_rows[inv_perm[t, j]] (slot order)."""
        T = inv_perm.shape[0]
        if out is None:
            out = torch.empty((T, self.H), dtype=torch.float32, device=y_rows.device)
        st = moe_combine(self._h, T, _ptr(inv_perm, torch.int32, "inv_perm", (T, self.k)),
                         _ptr(y_rows, torch.float32, "y_rows", (T * self.k, self.H)),
                         _ptr(out, torch.float32, "out", (T, self.H)), _stream(stream))
        _check(st, "moe_combine")
        return out

    # -- training and the block around the layer (include/moe.h) ------------------------
    # A call with stream= runs as one inside torch.cuda.stream(stream): what it allocates (results,
    # workspaces) belongs to the stream it enqueues on.  Its arguments are the caller's to order
    # and to keep for that stream, as for any torch operation.  Tensors must be on the handle's
    # device, which must be the current one.
    def _arg(self, t, dtype, name: str, shape) -> int:
        """Address of an argument after its checks; 0 for None."""
        if t is None:
            return 0
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
        if t.get_device() != self._device_index:
            raise ValueError(f"{name} must be on cuda:{self._device_index}, got {t.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    def _current(self) -> int:
        return _raw_stream(self._device_index)

    def grouped_matmul(self, x_rows, W, offsets, transpose: bool = False, out=None,
                       out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
        """x_rows[r] @ W[e] (transpose: @ W[e].T) for the rows offsets[e] <= r < offsets[e+1] of
        every expert e.  W [E, K, N]; offsets [E + 1] int32.  `out` (bf16 or fp32) keeps its rows
        outside the segments; without it they are not set."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.grouped_matmul(x_rows, W, offsets, transpose, out, out_dtype)
        if W.dim() != 3 or x_rows.dim() != 2:
            raise ValueError("x_rows must be [R, K] (transpose: [R, N]) and W [E, K, N]")
        E, K, N = W.shape
        ins, outs = (N, K) if transpose else (K, N)
        R, bf16 = x_rows.shape[0], torch.bfloat16
        px = self._arg(x_rows, bf16, "x_rows", (R, ins))
        pw = self._arg(W, bf16, "W", (self.E, K, N))
        po = self._arg(offsets, torch.int32, "offsets", (self.E + 1,))
        kind = _dtype(out_dtype if out is None else out, "out")
        if out is None:
            out = x_rows.new_empty((R, outs), dtype=out_dtype)
        st = moe_grouped_matmul(self._h, R, K, N, int(transpose), po, px, pw,
                                self._arg(out, out.dtype, "out", (R, outs)), kind, self._current())
        _check(st, "moe_grouped_matmul")
        return out

    def grouped_wgrad(self, x_rows, dy_rows, offsets, out=None, out_dtype=torch.bfloat16,
                      stream=None) -> torch.Tensor:
        """dW [E, K, N]: dW[e] = x_rows[rows of e].T @ dy_rows[rows of e], zeros without rows."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.grouped_wgrad(x_rows, dy_rows, offsets, out, out_dtype)
        if x_rows.dim() != 2 or dy_rows.dim() != 2:
            raise ValueError("x_rows must be [R, K] and dy_rows [R, N]")
        (R, K), N = x_rows.shape, dy_rows.shape[1]
        px = self._arg(x_rows, torch.bfloat16, "x_rows", (R, K))
        pdy = self._arg(dy_rows, torch.bfloat16, "dy_rows", (R, N))
        po = self._arg(offsets, torch.int32, "offsets", (self.E + 1,))
        kind = _dtype(out_dtype if out is None else out, "out")
        if out is None:
            out = x_rows.new_empty((self.E, K, N), dtype=out_dtype)
        st = moe_grouped_wgrad(self._h, R, K, N, po, px, pdy,
                               self._arg(out, out.dtype, "out", (self.E, K, N)), kind,
                               self._current())
        _check(st, "moe_grouped_wgrad")
        return out

    def swiglu(self, gu, row_w=None, out=None, stream=None) -> torch.Tensor:
        """row_w[r] * silu(gu[r, :I]) * gu[r, I:] -> [R, I] bf16 (row_w None: 1)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.swiglu(gu, row_w, out)
        R, I, bf16 = gu.shape[0], self.I, torch.bfloat16
        pg = self._arg(gu, bf16, "gu", (R, 2 * I))
        pw = self._arg(row_w, torch.float32, "row_w", (R,))
        if out is None:
            out = gu.new_empty((R, I))
        st = moe_swiglu(self._h, R, pg, pw, self._arg(out, bf16, "out", (R, I)), self._current())
        _check(st, "moe_swiglu")
        return out

    def swiglu_backward(self, dh, gu, row_w=None, stream=None) -> tuple:
        """(dgu [R, 2I] bf16, drow_w [R] fp32, or None without row_w) from dh [R, I]."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.swiglu_backward(dh, gu, row_w)
        R, I, bf16 = gu.shape[0], self.I, torch.bfloat16
        pd = self._arg(dh, bf16, "dh", (R, I))
        pg = self._arg(gu, bf16, "gu", (R, 2 * I))
        pw = self._arg(row_w, torch.float32, "row_w", (R,))
        dgu = gu.new_empty((R, 2 * I))
        dw = None if row_w is None else row_w.new_empty((R,))
        st = moe_swiglu_backward(self._h, R, pd, pg, pw, dgu.data_ptr(),
                                 0 if dw is None else dw.data_ptr(), self._current())
        _check(st, "moe_swiglu_backward")
        return dgu, dw

    def block_norm(self, resid, y=None, w_post=None, gate=None, scale: float = 1.0, w_next=None,
                   eps: float = 1e-5, resid_out=None, stream=None) -> dict:
        """The norm after a block, its gate and scale, the residual and the norm before the next
        block in one pass.  Returns resid (the new residual: resid + scale * gate * norm(y), in
        resid's type; resid itself without y), x (its norm, bf16; None without w_next) and
        rstd_post, rstd_next for the backward pass."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.block_norm(resid, y, w_post, gate, scale, w_next, eps, resid_out)
        T, H, f32 = resid.shape[0], self.H, torch.float32
        pr = self._arg(resid, resid.dtype, "resid", (T, H))
        py = self._arg(y, None if y is None else y.dtype, "y", (T, H))
        pp = self._arg(w_post, f32, "w_post", (H,))
        pg = self._arg(gate, f32, "gate", (H,))
        pn = self._arg(w_next, f32, "w_next", (H,))
        rt, yt = _dtype(resid, "resid"), MOE_F32 if y is None else _dtype(y, "y")
        if resid_out is None and y is not None:
            resid_out = resid.new_empty((T, H))
        x = rp = rn = None
        if w_post is not None:
            rp = w_post.new_empty((T,))
        if w_next is not None:
            x = resid.new_empty((T, H), dtype=torch.bfloat16)
            rn = w_next.new_empty((T,))
        st = moe_block_norm(
            self._h, T, rt, yt, pr, py, pp, pg, scale, pn, eps,
            self._arg(resid_out, resid.dtype, "resid_out", (T, H)), 0 if x is None else x.data_ptr(),
            0 if rp is None else rp.data_ptr(), 0 if rn is None else rn.data_ptr(), self._current())
        _check(st, "moe_block_norm")
        return dict(resid=resid if y is None else resid_out, x=x, rstd_post=rp, rstd_next=rn)

    def block_norm_workspace_bytes(self, T: int) -> int:
        return moe_block_norm_workspace_bytes(self._h, T)

    def block_norm_backward(self, dresid, dx, resid, y=None, rstd_post=None, rstd_next=None,
                            w_post=None, gate=None, scale: float = 1.0, w_next=None,
                            block: bool | None = None, dy_dtype=torch.bfloat16, stream=None,
                            workspace=None) -> dict:
        """Gradients of block_norm: dresid and dx are those of its two results (either may be None
        where nothing flows), resid, rstd_post and rstd_next its results.  Returns dresid (the
        gradient of the old residual), dy (None for the norm before a first block: `block` False,
        the default without y), dw_post, dgate and dw_next (None where the vector is)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.block_norm_backward(dresid, dx, resid, y, rstd_post, rstd_next, w_post,
                                                gate, scale, w_next, block, dy_dtype, None, workspace)
        like = dresid if dresid is not None else resid
        T, H, f32, rtype = like.shape[0], self.H, torch.float32, like.dtype
        has_block = (y is not None) if block is None else block
        args = (self._arg(dresid, rtype, "dresid", (T, H)),
                self._arg(dx, torch.bfloat16, "dx", (T, H)),
                self._arg(resid, rtype, "resid", (T, H)),
                self._arg(y, None if y is None else y.dtype, "y", (T, H)),
                self._arg(rstd_post, f32, "rstd_post", (T,)),
                self._arg(rstd_next, f32, "rstd_next", (T,)),
                self._arg(w_post, f32, "w_post", (H,)), self._arg(gate, f32, "gate", (H,)))
        pn = self._arg(w_next, f32, "w_next", (H,))
        types = (_dtype(rtype, "dresid"), MOE_F32 if y is None else _dtype(y, "y"),
                 _dtype(dy_dtype, "dy_dtype"))
        vec = lambda v: None if v is None else v.new_empty((H,))  # noqa: E731
        out = dict(dresid=like.new_empty((T, H)),
                   dy=like.new_empty((T, H), dtype=dy_dtype) if has_block else None,
                   dw_post=vec(w_post), dgate=vec(gate), dw_next=vec(w_next))
        ws = workspace
        if ws is None and not (w_post is None and gate is None and w_next is None):
            ws = like.new_empty((self.block_norm_workspace_bytes(T),), dtype=torch.uint8)
        elif ws is not None:
            _scratch(ws, like.device)
        ptr = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
        st = moe_block_norm_backward(
            self._h, T, *types, *args, scale, pn, ptr(out["dresid"]), ptr(out["dy"]),
            ptr(out["dw_post"]), ptr(out["dgate"]), ptr(out["dw_next"]), ptr(ws),
            0 if ws is None else ws.numel() * ws.element_size(), self._current())
        _check(st, "moe_block_norm_backward")
        return out

    def block(self, resid, x, W_router, b_router, W_gate_up, W_down, w_post=None, gate=None,
              scale: float = 1.0, w_next=None, eps: float = 1e-5, resid_out=None, stream=None,
              workspace=None) -> dict:
        """The layer inside its transformer block: x is the normed residual (block_norm of the
        previous block, or block_norm(resid, w_next=...) before the first), the layer's output goes
        through block_norm into the residual.  Returns block_norm's dict."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.block(resid, x, W_router, b_router, W_gate_up, W_down, w_post, gate,
                                  scale, w_next, eps, resid_out, None, workspace)
        y = self.forward(x, W_router, b_router, W_gate_up, W_down, workspace=workspace)
        return self.block_norm(resid, y, w_post=w_post, gate=gate, scale=scale, w_next=w_next,
                               eps=eps, resid_out=resid_out)

    def workspace_bytes_mxfp4(self, T: int) -> int:
        return moe_workspace_bytes_mxfp4(self._h, T)

    def forward_mxfp4(self, x, W_router, b_router, gu_codes, gu_scales, dn_codes, dn_scales,
                      out=None, stream=None, workspace=None) -> torch.Tensor:
        """The layer with MXFP4 experts (uint8 codes and E8M0 scales, see include/moe.h)."""
        T = x.shape[0]
        E, H, I = self.E, self.H, self.I
        if out is None:
            out = torch.empty((T, H), dtype=torch.float32, device=x.device)
        need = self.workspace_bytes_mxfp4(T)
        ws = self._workspace(need, x.device, stream) if workspace is None else _scratch(workspace, x.device)
        st = moe_forward_mxfp4(self._h, T, _ptr(x, torch.bfloat16, "x", (T, H)),
                               _ptr(W_router, torch.bfloat16, "W_router", (H, E)),
                               _ptr(b_router, torch.float32, "b_router", (E,)),
                               _ptr(gu_codes, torch.uint8, "gu_codes", (E, 2 * I, H // 2)),
                               _ptr(gu_scales, torch.uint8, "gu_scales", (E, H // 32, 2 * I)),
                               _ptr(dn_codes, torch.uint8, "dn_codes", (E, H, I // 2)),
                               _ptr(dn_scales, torch.uint8, "dn_scales", (E, I // 32, H)),
                               _ptr(out, torch.float32, "out", (T, H)),
                               ws.data_ptr(), ws.numel(), _stream(stream))
        _check(st, "moe_forward_mxfp4")
        return out

    def tune(self, x, W_router, b_router, W_gate_up, W_down, stream=None) -> int:
        T = x.shape[0]
        out = torch.empty((T, self.H), dtype=torch.float32, device=x.device)
        need = moe_tune_workspace_bytes(self._h, T)
        ws = self._workspace(need, x.device, stream)
        c = _c_int()
        st = moe_tune(self._h, T, _ptr(x, torch.bfloat16, "x"), _ptr(W_router, torch.bfloat16, "W_router"),
                      _ptr(b_router, torch.float32, "b_router"), _ptr(W_gate_up, torch.bfloat16, "W_gate_up"),
                      _ptr(W_down, torch.bfloat16, "W_down"), out.data_ptr(), ws.data_ptr(), ws.numel(),
                      _stream(stream), ctypes.byref(c))
        _check(st, "moe_tune")
        return c.value

    def last_dispatch(self, T: int, workspace=None, mxfp4: bool = False, stream=None) -> tuple:
        """Work-list entries per family (streaming, expert tiles, row tiles; -1: not launched)
        of the last forward call of T tokens on `workspace` (default: the layer's own)."""
        ws = self._ws if workspace is None else workspace
        out = (ctypes.c_int32 * 3)()
        _check(moe_last_dispatch(self._h, T, int(mxfp4), ws.data_ptr(), ws.numel(), out,
                                 _stream(stream)), "moe_last_dispatch")
        return tuple(out)

    # -- status and measurement --------------------------------------------------------
    def sync_status(self, stream=None) -> int:
        return moe_sync_status(self._h, _stream(stream))

    def launch_count(self) -> int:
        return moe_launch_count(self._h)

    def profile_begin(self, max_calls: int) -> None:
        _check(moe_profile_begin(self._h, max_calls), "moe_profile_begin")

    def profile_end(self) -> dict:
        ms = (ctypes.c_float * MOE_PROFILE_KINDS)()
        n = (_c_int * MOE_PROFILE_KINDS)()
        _check(moe_profile_end(self._h, ms, n, MOE_PROFILE_KINDS), "moe_profile_end")
        return {moe_profile_kind_name(i).decode(): (ms[i], n[i]) for i in range(MOE_PROFILE_KINDS)}

    def selftest_timeout(self, limit_us: int, stream=None) -> None:
        _check(moe_selftest_timeout(self._h, limit_us, _stream(stream)), "moe_selftest_timeout")

    def selftest_norm_timeout(self, from_row: int) -> None:
        _check(moe_selftest_norm_timeout(self._h, from_row), "moe_selftest_norm_timeout")
