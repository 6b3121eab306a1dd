"""Python binding of the operators around the selective scan (include/selscan_ops.h).

Argument marshalling only, as for the scan: tensors are checked for device, dtype, shape and
layout, their data pointers and torch's current HIP stream are passed to the C ABI, and the
computation runs in the library's HIP kernels. Every call runs on the device of its tensors,
whichever is current. With an explicit ``stream`` the outputs and the workspace are allocated
on that stream; the caller orders it against the streams that made the inputs and that use
the outputs.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import SS_BF16, SS_F32, SelscanError, lib

GLR_CKPT = 64    # SS_GLR_CKPT
Q8_BLOCK = 128   # columns that share a scale

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_F32 = torch.float32
_Q8 = torch.float8_e4m3fn


class ss_glr_dims(ctypes.Structure):
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("d", _i64), ("io_dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class ss_view(ctypes.Structure):
    _fields_ = [("p", _vp), ("batch_stride", _i64), ("token_stride", _i64)]


class ss_glr_args(ctypes.Structure):
    _fields_ = [("x", ss_view), ("r", ss_view), ("i", ss_view)] + [(n, _vp) for n in ("A", "reset", "y", "state", "ckpt")]


class ss_glr_grads(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("dy", "dstate_final", "dx", "dr", "di", "dA", "dstate_init")]


class ss_q8_dims(ctypes.Structure):
    _fields_ = [("rows", _i64), ("cols", _i64), ("io_dtype", ctypes.c_int32), ("square", ctypes.c_int32),
                ("eps", ctypes.c_float), ("reserved", ctypes.c_int32)]


class ss_norm_q8_args(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("x", "residual", "w", "q", "scale", "sum")]


class ss_gemm_q8_dims(ctypes.Structure):
    _fields_ = [("m", _i64), ("n", _i64), ("k", _i64), ("y_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class ss_gemm_q8_args(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("xq", "xs", "wq", "ws", "residual", "y")]


def _declare():
    P = ctypes.POINTER
    lib.ss_glr_workspace_bytes.argtypes = [P(ss_glr_dims), ctypes.c_int]
    lib.ss_glr_workspace_bytes.restype = ctypes.c_size_t
    lib.ss_glr_fwd.argtypes = [P(ss_glr_dims), P(ss_glr_args), _vp, ctypes.c_size_t, _vp]
    lib.ss_glr_step.argtypes = [P(ss_glr_dims), P(ss_glr_args), _vp]
    lib.ss_glr_bwd.argtypes = [P(ss_glr_dims), P(ss_glr_args), P(ss_glr_grads), _vp, ctypes.c_size_t, _vp]
    lib.ss_quant_q8.argtypes = [P(ss_q8_dims), _vp, _vp, _vp, _vp]
    lib.ss_norm_q8.argtypes = [P(ss_q8_dims), P(ss_norm_q8_args), _vp]
    lib.ss_gemm_q8.argtypes = [P(ss_gemm_q8_dims), P(ss_gemm_q8_args), _vp]
    for name in ("ss_glr_fwd", "ss_glr_step", "ss_glr_bwd", "ss_quant_q8", "ss_norm_q8", "ss_gemm_q8"):
        getattr(lib, name).restype = ctypes.c_int


_declare()


def _check(status: int):
    if status != 0:
        raise SelscanError(status, lib.ss_last_error().decode())


def _io(t: torch.Tensor, name: str) -> int:
    if t.dtype is torch.bfloat16:
        return SS_BF16
    if t.dtype is _F32:
        return SS_F32
    raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")


def _same(t: torch.Tensor, shape, dtype, device, name: str) -> int:
    """The data pointer of a contiguous tensor of this shape, dtype and device."""
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} must be on {device}, a GPU" if t.is_cuda else f"{name} must be a device tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _opt(t: Optional[torch.Tensor], shape, dtype, device, name: str) -> Optional[int]:
    return None if t is None else _same(t, shape, dtype, device, name)


class _On:
    """The device and stream of a call: the device is made current where it is not, outputs
    are allocated on an explicit stream."""
    __slots__ = ("handle", "_ctx")

    def __init__(self, device: torch.device, stream):
        ctx = []
        if device.type != "cuda":
            raise ValueError(f"the tensors must be on a GPU, got {device}")
        if stream is not None:
            if stream.device != device:
                raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
            ctx.append(torch.cuda.stream(stream))
            self.handle = stream.cuda_stream or None
        else:
            self.handle = torch.cuda.current_stream(device).cuda_stream or None
            if device.index != torch.cuda.current_device():
                ctx.append(torch.cuda.device(device))
        self._ctx = ctx

    def __enter__(self):
        for c in self._ctx:
            c.__enter__()
        return self.handle

    def __exit__(self, *e):
        for c in reversed(self._ctx):
            c.__exit__(*e)


def _workspace(given: Optional[torch.Tensor], need: int, device) -> Optional[torch.Tensor]:
    if given is None:
        return torch.empty(need, dtype=torch.uint8, device=device) if need else None
    if not given.is_cuda or given.device != device:
        raise ValueError(f"workspace must be on {device}")
    if not given.is_contiguous() or given.numel() * given.element_size() < need:
        raise ValueError(f"workspace must be contiguous, of at least {need} bytes")
    return given


def _ws_args(ws: Optional[torch.Tensor]):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


# ---------------------------------------------------------------------------
# gated linear recurrence

def _view(t: torch.Tensor, shape, dtype, device, name: str) -> ss_view:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: channels must be contiguous (last stride 1)")
    return ss_view(t.data_ptr(), st[0], st[1] if len(st) == 3 else 0)


def _glr_args(x, r, i, A, reset, y, state, ckpt, dims: ss_glr_dims):
    shape, dt, dev = x.shape, x.dtype, x.device
    B, D = shape[0], shape[-1]
    lead = shape[:-1]
    if reset is not None and reset.dtype is torch.bool:
        reset = reset.view(torch.uint8)
    return ss_glr_args(
        _view(x, shape, dt, dev, "x"), _view(r, shape, dt, dev, "r"), _view(i, shape, dt, dev, "i"),
        _same(A, (D,), _F32, dev, "A"), _opt(reset, lead, torch.uint8, dev, "reset"),
        _opt(y, shape, dt, dev, "y"), _opt(state, (B, D), _F32, dev, "state"),
        _opt(ckpt, glr_ckpt_shape(B, shape[1], D), _F32, dev, "ckpt") if len(shape) == 3 else None)


def _glr_dims(x: torch.Tensor, dim: int) -> ss_glr_dims:
    if x.dim() != dim:
        raise ValueError("x must be [batch, seqlen, d]" if dim == 3 else "x must be [streams, d]")
    return ss_glr_dims(x.shape[0], x.shape[1] if dim == 3 else 1, x.shape[-1], _io(x, "x"), 0)


def glr_ckpt_shape(batch: int, seqlen: int, d: int) -> tuple:
    """Shape of the recurrence's checkpoints (float32): the state before every 64th token."""
    return (batch, -(-seqlen // GLR_CKPT), d)


def ss_glr_workspace_bytes(dims: ss_glr_dims, backward: bool = False) -> int:
    return int(lib.ss_glr_workspace_bytes(ctypes.byref(dims), int(bool(backward))))


def ss_glr_fwd(x: torch.Tensor, r: torch.Tensor, i: torch.Tensor, A: torch.Tensor, *,
               state: Optional[torch.Tensor] = None, reset: Optional[torch.Tensor] = None,
               ckpt: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gated linear recurrence over whole sequences:

        s = sigmoid(r), a = exp(A s), h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t, y = h

    x, r, i: [B,L,D] (float32 or bfloat16, one dtype; channels contiguous, any strides
    otherwise); A [D] float32, not positive; state [B,D] float32, updated in place when given
    (zero initial state otherwise); reset [B,L] uint8 or bool: a_t = 0 at its nonzero tokens,
    where a new document starts; ckpt: float32 tensor of glr_ckpt_shape that receives the
    checkpoints ss_glr_bwd needs. Returns y [B,L,D] in the I/O dtype. Asynchronous."""
    dims = _glr_dims(x, 3)
    with _On(x.device, stream) as handle:
        if y is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        args = _glr_args(x, r, i, A, reset, y, state, ckpt, dims)
        dref = ctypes.byref(dims)
        ws, ws_bytes = _ws_args(_workspace(workspace, lib.ss_glr_workspace_bytes(dref, 0), x.device))
        _check(lib.ss_glr_fwd(dref, ctypes.byref(args), ws, ws_bytes, handle))
    return y


def ss_glr_step(x: torch.Tensor, r: torch.Tensor, i: torch.Tensor, A: torch.Tensor, state: torch.Tensor, *,
                reset: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token of each stream: x, r, i [S,D] (rows at any stride); state [S,D] float32,
    updated in place; reset [S]. Returns y [S,D]."""
    dims = _glr_dims(x, 2)
    with _On(x.device, stream) as handle:
        if y is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        args = _glr_args(x, r, i, A, reset, y, state, None, dims)
        _check(lib.ss_glr_step(ctypes.byref(dims), ctypes.byref(args), handle))
    return y


def ss_glr_bwd(x: torch.Tensor, r: torch.Tensor, i: torch.Tensor, A: torch.Tensor, ckpt: torch.Tensor,
               dy: torch.Tensor, *, reset: Optional[torch.Tensor] = None,
               dstate_final: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream=None) -> dict:
    """Gradients of ss_glr_fwd for the same inputs; ckpt as that call wrote it (its first row
    is the initial state). dy [B,L,D] in the I/O dtype, dstate_final [B,D] float32 the
    gradient of the returned state. Returns a dict of new tensors: dx, dr, di (I/O dtype), dA
    [D] and dstate_init [B,D] (float32). Asynchronous."""
    dims = _glr_dims(x, 3)
    B, _, D = shape = x.shape
    dt, dev = x.dtype, x.device
    with _On(dev, stream) as handle:
        out = {k: torch.empty(shape, dtype=dt, device=dev) for k in ("dx", "dr", "di")}
        out["dA"] = torch.empty(D, dtype=_F32, device=dev)
        out["dstate_init"] = torch.empty(B, D, dtype=_F32, device=dev)
        args = _glr_args(x, r, i, A, reset, None, None, ckpt, dims)
        g = ss_glr_grads(_same(dy, shape, dt, dev, "dy"), _opt(dstate_final, (B, D), _F32, dev, "dstate_final"),
                         *(out[k].data_ptr() for k in ("dx", "dr", "di", "dA", "dstate_init")))
        dref = ctypes.byref(dims)
        ws, ws_bytes = _ws_args(_workspace(workspace, lib.ss_glr_workspace_bytes(dref, 1), dev))
        _check(lib.ss_glr_bwd(dref, ctypes.byref(args), ctypes.byref(g), ws, ws_bytes, handle))
    return out


# ---------------------------------------------------------------------------
# 8-bit floating point with block scales

def _rows(x: torch.Tensor, name: str) -> tuple:
    """(rows, columns) of a contiguous tensor whose last dimension is the row."""
    if not x.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if x.dim() < 1 or not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous, with at least one dimension")
    K = x.shape[-1]
    return (x.numel() // K if K else 0), K


def ss_quant_q8(x: torch.Tensor, *, square: bool = False, q: Optional[torch.Tensor] = None,
                scale: Optional[torch.Tensor] = None, stream=None) -> tuple:
    """Round x [..., K] (float32 or bfloat16, contiguous) to 8-bit floating point. Returns (q,
    scale): q of x's shape in torch.float8_e4m3fn and float32 scales of blocks of 128 columns,
    [..., ceil(K/128)]; with square (x [N,K]) of 128 x 128, [ceil(N/128), ceil(K/128)]. x stands
    for scale * q. q and scale are allocated where not given. Asynchronous."""
    M, K = _rows(x, "x")
    KB, dev = -(-K // Q8_BLOCK), x.device
    if square and x.dim() != 2:
        raise ValueError("a square rounding takes x [N, K]")
    sshape = (-(-M // Q8_BLOCK), KB) if square else x.shape[:-1] + (KB,)
    with _On(dev, stream) as handle:
        if q is None:
            q = torch.empty(x.shape, dtype=_Q8, device=dev)
        if scale is None:
            scale = torch.empty(sshape, dtype=_F32, device=dev)
        dims = ss_q8_dims(M, K, _io(x, "x"), int(bool(square)), 0.0, 0)
        _check(lib.ss_quant_q8(ctypes.byref(dims), x.data_ptr(), _same(q, x.shape, _Q8, dev, "q"),
                               _same(scale, sshape, _F32, dev, "scale"), handle))
    return q, scale


def ss_norm_q8(x: torch.Tensor, w: torch.Tensor, *, residual: Optional[torch.Tensor] = None, eps: float = 1e-5,
               q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
               sum_out: Optional[torch.Tensor] = None, stream=None) -> tuple:
    """RMS norm of s = x + residual (s = x without one), times w, rounded to 8-bit floating
    point in blocks of 128 columns: x, residual [..., K] (float32 or bfloat16, contiguous), w [K]
    float32. Returns (q, scale, s): q and scale as from ss_quant_q8, s in x's dtype (None
    without a residual). sum_out receives s; it may be x or residual itself. Asynchronous."""
    M, K = _rows(x, "x")
    shape, dt, dev = x.shape, x.dtype, x.device
    sshape = shape[:-1] + (-(-K // Q8_BLOCK),)
    if residual is None and sum_out is not None:
        raise ValueError("sum_out given without a residual")
    with _On(dev, stream) as handle:
        if q is None:
            q = torch.empty(shape, dtype=_Q8, device=dev)
        if scale is None:
            scale = torch.empty(sshape, dtype=_F32, device=dev)
        if residual is not None and sum_out is None:
            sum_out = torch.empty(shape, dtype=dt, device=dev)
        dims = ss_q8_dims(M, K, _io(x, "x"), 0, eps, 0)
        args = ss_norm_q8_args(x.data_ptr(), _opt(residual, shape, dt, dev, "residual"), _same(w, (K,), _F32, dev, "w"),
                               _same(q, shape, _Q8, dev, "q"), _same(scale, sshape, _F32, dev, "scale"),
                               _opt(sum_out, shape, dt, dev, "sum_out"))
        _check(lib.ss_norm_q8(ctypes.byref(dims), ctypes.byref(args), handle))
    return q, scale, sum_out


def ss_gemm_q8(xq: torch.Tensor, xs: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor, *,
               residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """y = X W^T (+ residual) of 8-bit matrices: xq [..., K] and xs [..., ceil(K/128)] as from
    ss_quant_q8 or ss_norm_q8, wq [N,K] and ws [ceil(N/128), ceil(K/128)] as from
    ss_quant_q8(square=True); K a multiple of 16. Returns y [..., N] in out_dtype (float32 or
    bfloat16; out's own where given); residual has y's shape and dtype and may be out itself.
    Asynchronous."""
    M, K = _rows(xq, "xq")
    if wq.dim() != 2:
        raise ValueError("wq must be [N, K]")
    N, dev, lead, KB = wq.shape[0], xq.device, xq.shape[:-1], -(-K // Q8_BLOCK)
    with _On(dev, stream) as handle:
        if out is None:
            out = torch.empty(lead + (N,), dtype=out_dtype, device=dev)
        yshape, dt = lead + (N,), out.dtype
        dims = ss_gemm_q8_dims(M, N, K, _io(out, "out"), 0)
        args = ss_gemm_q8_args(_same(xq, xq.shape, _Q8, dev, "xq"), _same(xs, lead + (KB,), _F32, dev, "xs"),
                               _same(wq, (N, K), _Q8, dev, "wq"), _same(ws, (-(-N // Q8_BLOCK), KB), _F32, dev, "ws"),
                               _opt(residual, yshape, dt, dev, "residual"), _same(out, yshape, dt, dev, "out"))
        _check(lib.ss_gemm_q8(ctypes.byref(dims), ctypes.byref(args), handle))
    return out


__all__ = ["GLR_CKPT", "ss_glr_dims", "ss_view", "ss_glr_args", "ss_glr_grads", "glr_ckpt_shape",
           "ss_glr_workspace_bytes", "ss_glr_fwd", "ss_glr_step", "ss_glr_bwd", "Q8_BLOCK", "ss_q8_dims",
           "ss_norm_q8_args", "ss_gemm_q8_dims", "ss_gemm_q8_args", "ss_quant_q8", "ss_norm_q8", "ss_gemm_q8"]
