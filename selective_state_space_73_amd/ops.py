"""Python binding of the operators around the selective scan (include/selscan_ops.h).

Argument marshalling only, as for the scan: tensors are checked for device, dtype, shape and
layout, their data pointers and torch's current HIP stream are passed to the C ABI, and the
computation runs in the library's HIP kernels. For the recurrence and the 8-bit calls, of which
a decode step makes many small ones, that is done by the C extension csrc/binding.cpp, which the
first such call loads. Every call runs on the device of its tensors, whichever is current. With an explicit ``stream`` the outputs and the workspace are allocated
on that stream; the caller orders it against the streams that made the inputs and that use
the outputs.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional

import torch

from . import (SS_BF16, SS_EULER, SS_F32, SS_ZOH, SelscanError, block_dims, lib, ss_block_dims,
               ss_block_weights)

GLR_CKPT = 64    # SS_GLR_CKPT
GDR_CHUNK = 64   # SS_GDR_CHUNK
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


class ss_block_q8_weights(ctypes.Structure):
    _fields_ = [("w", ss_block_weights), ("S_in", _vp), ("S_out", _vp)]


class ss_gdr_dims(ctypes.Structure):
    _fields_ = [("batch", _i64), ("seqlen", _i64)] + [(n, ctypes.c_int32) for n in ("k_heads", "heads", "dk", "dv", "io_dtype")] + \
               [("scale", ctypes.c_float), ("eps", ctypes.c_float), ("reserved", ctypes.c_int32)]


class ss_head_view(ctypes.Structure):
    _fields_ = [("p", _vp), ("batch_stride", _i64), ("token_stride", _i64), ("head_stride", _i64)]


class ss_gdr_args(ctypes.Structure):
    _fields_ = [(n, ss_head_view) for n in ("q", "k", "v")] + [(n, _vp) for n in ("g", "beta", "reset", "y", "state", "ckpt")]


class ss_gdr_grads(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("dy", "dstate_final", "dq", "dk", "dv", "dg", "dbeta", "dstate_init")]


class ss_gnorm_dims(ctypes.Structure):
    _fields_ = [("rows", _i64), ("cols", _i64), ("group", _i64), ("io_dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class ss_gnorm_args(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("y", "w", "gate", "residual", "scale", "w_next", "s", "n")]


class ss_gnorm_grads(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("ds", "dn", "dy", "dgate", "dresidual", "dw", "dscale", "dw_next")]


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
    lib.ss_block_q8_workspace_bytes.argtypes = [P(ss_block_dims), ctypes.c_int]
    lib.ss_block_q8_workspace_bytes.restype = ctypes.c_size_t
    block = [P(ss_block_dims), P(ss_block_q8_weights), _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
    lib.ss_block_q8_fwd.argtypes = lib.ss_block_q8_step.argtypes = block
    lib.ss_gdr_ckpt_floats.argtypes = [P(ss_gdr_dims)]
    lib.ss_gdr_workspace_bytes.argtypes = [P(ss_gdr_dims), ctypes.c_int]
    lib.ss_gdr_fwd.argtypes = [P(ss_gdr_dims), P(ss_gdr_args), _vp, ctypes.c_size_t, _vp]
    lib.ss_gdr_step.argtypes = [P(ss_gdr_dims), P(ss_gdr_args), _vp]
    lib.ss_gdr_bwd.argtypes = [P(ss_gdr_dims), P(ss_gdr_args), P(ss_gdr_grads), _vp, ctypes.c_size_t, _vp]
    lib.ss_gnorm_workspace_bytes.argtypes = [P(ss_gnorm_dims)]
    lib.ss_gnorm_fwd.argtypes = [P(ss_gnorm_dims), P(ss_gnorm_args), _vp]
    lib.ss_gnorm_bwd.argtypes = [P(ss_gnorm_dims), P(ss_gnorm_args), P(ss_gnorm_grads), _vp, ctypes.c_size_t, _vp]
    for name in ("ss_gdr_ckpt_floats", "ss_gdr_workspace_bytes", "ss_gnorm_workspace_bytes"):
        getattr(lib, name).restype = ctypes.c_size_t
    for name in ("ss_glr_fwd", "ss_glr_step", "ss_glr_bwd", "ss_quant_q8", "ss_norm_q8", "ss_gemm_q8", "ss_block_q8_fwd",
                 "ss_block_q8_step", "ss_gdr_fwd", "ss_gdr_step", "ss_gdr_bwd", "ss_gnorm_fwd", "ss_gnorm_bwd"):
        getattr(lib, name).restype = ctypes.c_int


_declare()


def _check(status: int):
    if status != 0:
        raise SelscanError(status, lib.ss_last_error().decode())


_EXTENSION = ("glr_fwd", "glr_step", "glr_bwd", "quant", "norm", "gemm", "gdr_fwd", "gdr_step", "gdr_bwd", "gnorm_fwd",
              "gnorm_bwd")


def _of_extension(name: str):
    """A call of the C extension, which its first use loads: the scan and the blocks need
    libselscan.so alone, whatever Python and torch the extension was built for."""
    def first(*args):
        try:
            from . import _binding
        except ImportError as e:
            raise ImportError("the operators' extension _binding.so is missing or was built for another Python or "
                              "torch: run __graft_entry__.build()") from e
        for n in _EXTENSION:
            globals()["_" + n] = getattr(_binding, n)
        return globals()["_" + name](*args)
    return first


(_glr_fwd, _glr_step, _glr_bwd, _quant, _norm, _gemm, _gdr_fwd, _gdr_step, _gdr_bwd, _gnorm_fwd,
 _gnorm_bwd) = map(_of_extension, _EXTENSION)


def _done(result):
    """A binding call's result; an int is the status of a refused call."""
    if type(result) is int:
        _check(result)
    return result


def _io(t: torch.Tensor, name: str) -> int:
    if t.dtype is torch.bfloat16:
        return SS_BF16
    if t.dtype is _F32:
        return SS_F32
    raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")


def _gpu(t: torch.Tensor, name: str) -> int:
    """The index of the GPU a tensor is on."""
    idx = t.get_device()
    if idx < 0 or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor, got {t.device}")
    return idx


def _elsewhere(idx: int, stream) -> bool:
    """Whether a call has to move to another device or to an explicit stream first."""
    return stream is not None or idx != torch._C._cuda_getDevice()


@contextlib.contextmanager
def _placed(idx: int, stream):
    if stream is not None and stream.device.index != idx:
        raise ValueError(f"stream is on {stream.device}, the tensors are on cuda:{idx}")
    with torch.cuda.device(idx):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def _wrong(t: torch.Tensor, shape, dtype, idx: int, name: str):
    if t.get_device() != idx:
        raise ValueError(f"{name} must be on cuda:{idx}, got {t.device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}, contiguous")


def _same(t: torch.Tensor, shape, dtype, idx: int, name: str) -> int:
    """The data pointer of a contiguous tensor of this shape, dtype and device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != idx or not t.is_contiguous():
        _wrong(t, shape, dtype, idx, name)
    return t.data_ptr()


def _opt(t: Optional[torch.Tensor], shape, dtype, idx: int, name: str) -> int:
    return 0 if t is None else _same(t, shape, dtype, idx, name)


def _workspace(given: Optional[torch.Tensor], need: int, like: torch.Tensor):
    """(tensor to keep alive, pointer, bytes)."""
    if given is None:
        if not need:
            return None, None, 0
        given = like.new_empty(need, dtype=torch.uint8)
    elif given.get_device() != like.get_device():
        raise ValueError(f"workspace must be on {like.device}")
    elif not given.is_contiguous() or given.numel() * given.element_size() < need:
        raise ValueError(f"workspace must be contiguous, of at least {need} bytes")
    return given, given.data_ptr(), given.numel() * given.element_size()


# ---------------------------------------------------------------------------
# gated linear recurrence

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
    if stream is not None:
        with _placed(_gpu(x, "x"), stream):
            return ss_glr_fwd(x, r, i, A, state=state, reset=reset, ckpt=ckpt, y=y, workspace=workspace)
    return _done(_glr_fwd(x, r, i, A, state, reset, ckpt, y, workspace))


def ss_glr_step(x: torch.Tensor, r: torch.Tensor, i: torch.Tensor, A: torch.Tensor, state: torch.Tensor, *,
                reset: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token of each stream: x, r, i [S,D] (rows at any stride); state [S,D] float32,
    updated in place; reset [S]. Returns y [S,D]."""
    if stream is not None:
        with _placed(_gpu(x, "x"), stream):
            return ss_glr_step(x, r, i, A, state, reset=reset, y=y)
    return _done(_glr_step(x, r, i, A, state, reset, y))


def ss_glr_bwd(x: torch.Tensor, r: torch.Tensor, i: torch.Tensor, A: torch.Tensor, ckpt: torch.Tensor,
               dy: torch.Tensor, *, reset: Optional[torch.Tensor] = None,
               dstate_final: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream=None) -> dict:
    """Gradients of ss_glr_fwd for the same inputs; ckpt as that call wrote it (its first row
    is the initial state). dy [B,L,D] in the I/O dtype, dstate_final [B,D] float32 the
    gradient of the returned state. Returns a dict of new tensors: dx, dr, di (I/O dtype), dA
    [D] and dstate_init [B,D] (float32). Asynchronous."""
    if stream is not None:
        with _placed(_gpu(x, "x"), stream):
            return ss_glr_bwd(x, r, i, A, ckpt, dy, reset=reset, dstate_final=dstate_final, workspace=workspace)
    return dict(zip(("dx", "dr", "di", "dA", "dstate_init"),
                    _done(_glr_bwd(x, r, i, A, ckpt, dy, reset, dstate_final, workspace))))


# ---------------------------------------------------------------------------
# 8-bit floating point with block scales

def ss_quant_q8(x: torch.Tensor, *, square: bool = False, q: Optional[torch.Tensor] = None,
                scale: Optional[torch.Tensor] = None, stream=None) -> tuple:
    """Round x [..., K] (float32 or bfloat16, contiguous) to 8-bit floating point. Returns (q,
    scale): q of x's shape in torch.float8_e4m3fn and float32 scales of blocks of 128 columns,
    [..., ceil(K/128)]; with square (x [N,K]) of 128 x 128, [ceil(N/128), ceil(K/128)]. x stands
    for scale * q. q and scale are allocated where not given. Asynchronous."""
    if stream is not None:
        with _placed(_gpu(x, "x"), stream):
            return ss_quant_q8(x, square=square, q=q, scale=scale)
    return _done(_quant(x, square, q, scale))


def ss_norm_q8(x: torch.Tensor, w: torch.Tensor, *, residual: Optional[torch.Tensor] = None, eps: float = 1e-5,
               q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
               sum_out: Optional[torch.Tensor] = None, stream=None) -> tuple:
    """RMS norm of s = x + residual (s = x without one), times w, rounded to 8-bit floating
    point in blocks of 128 columns: x, residual [..., K] (float32 or bfloat16, contiguous), w [K]
    float32. Returns (q, scale, s): q and scale as from ss_quant_q8, s in x's dtype (None
    without a residual). sum_out receives s; it may be x or residual itself. Asynchronous."""
    if stream is not None:
        with _placed(_gpu(x, "x"), stream):
            return ss_norm_q8(x, w, residual=residual, eps=eps, q=q, scale=scale, sum_out=sum_out)
    return _done(_norm(x, w, residual, eps, q, scale, sum_out))


def ss_gemm_q8(xq: torch.Tensor, xs: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor, *,
               residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """y = X W^T (+ residual) of 8-bit matrices: xq [..., K] and xs [..., ceil(K/128)] as from
    ss_quant_q8 or ss_norm_q8, wq [N,K] and ws [ceil(N/128), ceil(K/128)] as from
    ss_quant_q8(square=True); K a multiple of 16. Returns y [..., N] in out_dtype (float32 or
    bfloat16; out's own where given); residual has y's shape and dtype and may be out itself.
    Asynchronous."""
    if stream is not None:
        with _placed(_gpu(xq, "xq"), stream):
            return ss_gemm_q8(xq, xs, wq, ws, residual=residual, out=out, out_dtype=out_dtype)
    return _done(_gemm(xq, xs, wq, ws, residual, out, out_dtype))


# ---------------------------------------------------------------------------
# the block with 8-bit projections

def block_q8_weights(W: dict, *, stream=None) -> dict:
    """The block's weights with its two wide projections rounded to 8 bits: W as ss_block_fwd
    takes it (BLOCK_WEIGHTS) -> a dict whose W_in and W_out are float8_e4m3fn and whose S_in
    and S_out hold their scales; the other entries are W's own tensors. Done once per model."""
    out = dict(W)
    for name, scale in (("W_in", "S_in"), ("W_out", "S_out")):
        out[name], out[scale] = ss_quant_q8(W[name], square=True, stream=stream)
    return out


def ss_block_q8_workspace_bytes(dims: ss_block_dims, step: bool = False) -> int:
    return int(lib.ss_block_q8_workspace_bytes(ctypes.byref(dims), int(bool(step))))


def _block_q8(step, x, W, dt_rank, ssm_state, conv_state, out, workspace, norm_eps, zoh, stream):
    idx = _gpu(x, "x")
    if _elsewhere(idx, stream):
        with _placed(idx, stream):
            return _block_q8(step, x, W, dt_rank, ssm_state, conv_state, out, workspace, norm_eps, zoh, None)
    if x.dim() != (2 if step else 3):
        raise ValueError("x must be [streams, d_model]" if step else "x must be [batch, seqlen, d_model]")
    io, shape = x.dtype, x.shape
    B, L, dm = shape[0], 1 if step else shape[1], shape[-1]
    if W["W_in"].dim() != 2 or W["A"].dim() != 2:
        raise ValueError("W_in must be [2 d_inner, d_model] and A [d_inner, d_state]")
    di, N, R = W["W_in"].shape[0] // 2, W["A"].shape[1], dt_rank
    KM, KI = -(-dm // Q8_BLOCK), -(-di // Q8_BLOCK)
    dims = block_dims(B, L, dm, di, N, R, _io(x, "x"), norm_eps, SS_ZOH if zoh else SS_EULER)

    def given(name, shape, dtype, key=None):
        return _same(W[key or name], shape, dtype, idx, name)

    def maybe(name, shape, key=None):
        return _opt(W.get(key or name), shape, _F32, idx, name)

    w = ss_block_q8_weights(ss_block_weights(
        norm_w=given("norm_w", (dm,), _F32), W_in=given("W_in", (2 * di, dm), _Q8), conv_w=given("conv_w", (di, 4), _F32),
        conv_b=maybe("conv_b", (di,)), W_x=given("W_x", (R + 2 * N, di), io), W_dt=given("W_dt", (di, R), io),
        dt_bias=maybe("dt_bias", (di,)), A=given("A", (di, N), _F32), Dskip=maybe("D", (di,)),
        W_out=given("W_out", (dm, di), _Q8)),
        given("S_in", (-(-2 * di // Q8_BLOCK), KM), _F32), given("S_out", (KM, KI), _F32))
    xp = _same(x, shape, io, idx, "x")
    if out is None:
        out = x.new_empty(shape)
    keep, ws, ws_bytes = _workspace(workspace, ss_block_q8_workspace_bytes(dims, step), x)
    fn = lib.ss_block_q8_step if step else lib.ss_block_q8_fwd
    _check(fn(ctypes.byref(dims), ctypes.byref(w), xp, _same(out, shape, io, idx, "out"),
              _opt(ssm_state, (B, di, N), _F32, idx, "ssm_state") or None,
              _opt(conv_state, (B, di, 3), _F32, idx, "conv_state") or None, ws, ws_bytes,
              torch._C._cuda_getCurrentRawStream(idx)))
    return out


def ss_block_q8_fwd(x: torch.Tensor, W: dict, dt_rank: int, *, ssm_state: Optional[torch.Tensor] = None,
                    conv_state: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, norm_eps: float = 1e-5, zoh: bool = False,
                    stream=None) -> torch.Tensor:
    """ss_block_fwd with 8-bit input and output projections: x [B,L,d_model] (float32 or
    bfloat16, contiguous) -> out, same shape; W from block_q8_weights; d_model and d_inner
    multiples of 16. States float32, read and updated when given; out may be x. Asynchronous."""
    return _block_q8(False, x, W, dt_rank, ssm_state, conv_state, out, workspace, norm_eps, zoh, stream)


def ss_block_q8_step(x: torch.Tensor, W: dict, dt_rank: int, ssm_state: torch.Tensor, conv_state: torch.Tensor, *,
                     out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     norm_eps: float = 1e-5, zoh: bool = False, stream=None) -> torch.Tensor:
    """One token per stream through the block with 8-bit projections: x [S,d_model] -> out
    [S,d_model]; both states required and updated in place."""
    return _block_q8(True, x, W, dt_rank, ssm_state, conv_state, out, workspace, norm_eps, zoh, stream)


# ---------------------------------------------------------------------------
# gated delta rule

def _gdr_dims(batch, seqlen, heads, dk, dv):
    return ss_gdr_dims(batch, seqlen, 1, heads, dk, dv, SS_F32, 1.0, 0.0, 0)


def gdr_ckpt_shape(batch: int, seqlen: int, heads: int, dk: int, dv: int) -> tuple:
    """Shape of the delta rule's checkpoints (float32): the states before every 64th token and what
    each token writes, one behind the other."""
    n = int(lib.ss_gdr_ckpt_floats(ctypes.byref(_gdr_dims(batch, seqlen, heads, dk, dv))))
    if not n and seqlen:
        raise ValueError(f"no such delta rule: {lib.ss_last_error().decode()}")
    return (n,)


def ss_gdr_workspace_bytes(dims: ss_gdr_dims, backward: bool = False) -> int:
    return int(lib.ss_gdr_workspace_bytes(ctypes.byref(dims), int(bool(backward))))


def ss_gdr_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor, *,
               scale: Optional[float] = None, eps: Optional[float] = 1e-6, state: Optional[torch.Tensor] = None,
               reset: Optional[torch.Tensor] = None, ckpt: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gated delta rule over whole sequences, with a state S [dk, dv] per head:

        S' = exp(g_t) S_{t-1}, u = beta_t (v_t - S'^T k_t), S_t = S' + k_t u^T, y_t = scale S_t^T q_t

    q, k: [B,L,k_heads,dk], v [B,L,H,dv] (float32 or bfloat16, one dtype; the last dimension
    contiguous, any strides otherwise; H a multiple of k_heads, whose keys and queries H / k_heads
    neighbouring heads of v share; dk up to 256, dv up to 512); g (the logarithm of the decay) and
    beta [B,L,H] float32. q and k are divided by their lengths, sqrt(sum x^2 + eps) with eps > 0,
    unless eps is None. scale: 1 / sqrt(dk) by default. state [B,H,dk,dv] float32, updated in place when given
    (zero initial state otherwise); reset [B,L] uint8 or bool: the state in front of its nonzero
    tokens counts as zero; ckpt: float32 tensor of gdr_ckpt_shape that receives what
    ss_gdr_bwd needs. Returns y [B,L,H,dv] in the I/O dtype. Asynchronous."""
    if stream is not None:
        with _placed(_gpu(q, "q"), stream):
            return ss_gdr_fwd(q, k, v, g, beta, scale=scale, eps=eps, state=state, reset=reset, ckpt=ckpt, y=y, workspace=workspace)
    return _done(_gdr_fwd(q, k, v, g, beta, scale, eps, state, reset, ckpt, y, workspace))


def ss_gdr_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                state: torch.Tensor, *, scale: Optional[float] = None, eps: Optional[float] = 1e-6,
                reset: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token of each stream: q, k [S,k_heads,dk], v [S,H,dv] (any strides but the last), g, beta
    [S,H]; state [S,H,dk,dv] float32, updated in place; reset [S]. Returns y [S,H,dv]."""
    if stream is not None:
        with _placed(_gpu(q, "q"), stream):
            return ss_gdr_step(q, k, v, g, beta, state, scale=scale, eps=eps, reset=reset, y=y)
    return _done(_gdr_step(q, k, v, g, beta, scale, eps, state, reset, y))


def ss_gdr_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor, ckpt: torch.Tensor,
               dy: torch.Tensor, *, scale: Optional[float] = None, eps: Optional[float] = 1e-6,
               reset: Optional[torch.Tensor] = None, dstate_final: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of ss_gdr_fwd for the same inputs; ckpt as that call wrote it. dy [B,L,H,dv] in the I/O
    dtype, dstate_final [B,H,dk,dv] float32 the gradient of the returned state. Returns a dict of new
    tensors: dq, dk (summed over the heads that share them), dv (I/O dtype), dg, dbeta [B,L,H] and
    dstate_init [B,H,dk,dv] (float32). Asynchronous."""
    if stream is not None:
        with _placed(_gpu(q, "q"), stream):
            return ss_gdr_bwd(q, k, v, g, beta, ckpt, dy, scale=scale, eps=eps, reset=reset, dstate_final=dstate_final,
                              workspace=workspace)
    return dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dstate_init"),
                    _done(_gdr_bwd(q, k, v, g, beta, scale, eps, ckpt, dy, reset, dstate_final, workspace))))


# ---------------------------------------------------------------------------
# the norms around a layer

def ss_gnorm_workspace_bytes(dims: ss_gnorm_dims) -> int:
    return int(lib.ss_gnorm_workspace_bytes(ctypes.byref(dims)))


def ss_gnorm_fwd(y: torch.Tensor, w: torch.Tensor, *, gate: Optional[torch.Tensor] = None,
                 residual: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                 w_next: Optional[torch.Tensor] = None, eps: float = 1e-5, s: Optional[torch.Tensor] = None,
                 n: Optional[torch.Tensor] = None, stream=None) -> tuple:
    """The norms behind a layer and before the next, with its gate, its scale and the residual, in one pass:

        p = y / rms(y) w,  h = p silu(gate),  s = residual + scale h,  n = s / rms(s) w_next

    y, gate, residual [..., K] (float32 or bfloat16, contiguous, K up to 16384); w [group] float32, group a
    divisor of K: y is normed in groups of so many columns (heads), each with the same weights; scale, w_next
    [K] float32. Without a gate h = p, without scale 1, without residual 0, without w_next n is not made.
    Returns (s, n) in y's dtype (n None without w_next); s may be y, gate or residual itself. Asynchronous."""
    if stream is not None:
        with _placed(_gpu(y, "y"), stream):
            return ss_gnorm_fwd(y, w, gate=gate, residual=residual, scale=scale, w_next=w_next, eps=eps, s=s, n=n)
    return _done(_gnorm_fwd(y, w, gate, residual, scale, w_next, eps, s, n))


def ss_gnorm_bwd(y: torch.Tensor, w: torch.Tensor, ds: Optional[torch.Tensor], *, dn: Optional[torch.Tensor] = None,
                 gate: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                 scale: Optional[torch.Tensor] = None, w_next: Optional[torch.Tensor] = None, eps: float = 1e-5,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of ss_gnorm_fwd for the same inputs (as they were: not where s was written over one of them);
    ds and dn are those of s and n (None: zero; one is required). Returns a dict of new tensors: dy, dgate,
    dresidual (y's dtype), dw [group], dscale, dw_next [K] (float32); None for what was not given. Asynchronous."""
    if stream is not None:
        with _placed(_gpu(y, "y"), stream):
            return ss_gnorm_bwd(y, w, ds, dn=dn, gate=gate, residual=residual, scale=scale, w_next=w_next, eps=eps,
                                workspace=workspace)
    return dict(zip(("dy", "dw", "dgate", "dresidual", "dscale", "dw_next"),
                    _done(_gnorm_bwd(y, w, gate, residual, scale, w_next, eps, ds, dn, workspace))))


__all__ = ["GLR_CKPT", "ss_glr_dims", "ss_view", "ss_glr_args", "ss_glr_grads", "glr_ckpt_shape",
           "ss_glr_workspace_bytes", "ss_glr_fwd", "ss_glr_step", "ss_glr_bwd", "Q8_BLOCK", "ss_q8_dims",
           "ss_norm_q8_args", "ss_gemm_q8_dims", "ss_gemm_q8_args", "ss_quant_q8", "ss_norm_q8", "ss_gemm_q8",
           "ss_block_q8_weights", "block_q8_weights", "ss_block_q8_workspace_bytes", "ss_block_q8_fwd", "ss_block_q8_step",
           "GDR_CHUNK", "ss_gdr_dims", "ss_head_view", "ss_gdr_args", "ss_gdr_grads", "gdr_ckpt_shape", "ss_gdr_workspace_bytes",
           "ss_gdr_fwd", "ss_gdr_step", "ss_gdr_bwd", "ss_gnorm_dims", "ss_gnorm_args", "ss_gnorm_grads",
           "ss_gnorm_workspace_bytes", "ss_gnorm_fwd", "ss_gnorm_bwd"]
