"""The operators between the FP8 linears of a feed-forward or expert block.

Like the package's other calls these only marshal arguments to the C-ABI
library (include/fp8linear.h has the formulas): outputs that are not given
are allocated on the inputs' device, everything runs in the library's
kernels on the current device, where all tensors have to be, and its current
stream.  With stream= (torch's object or a raw handle)
a call is what it is under torch.cuda.stream(stream): its outputs are of that
stream's memory, and a use on another stream waits as for any other tensor.

  fp8_norm_fwd, fp8_norm_bwd      norms before and after a block, gate, residual scale
  fp8_gemm_act, fp8_act_bwd       FP8 GEMM with bias, activation and residual in its epilogue
  fp8_moe_plan, fp8_moe_permute, fp8_moe_unpermute, fp8_moe_unpermute_bwd
                                  tokens sorted by expert and back
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import NamedTuple, Optional

import torch

from . import (_U8, _here, _ptr, _raw_stream, _stream, _under, _vp, E4M3, Fp8Error, GRAN_ROW, GRAN_TENSOR, OUT_BF16, OUT_F32,
               fp8_last_error)
from . import lib as _base_lib

__all__ = [
    "NORM_RMS", "NORM_LAYER", "ACT_NONE", "ACT_RELU", "ACT_SILU", "ACT_GELU", "ACT_GELU_TANH",
    "NormFwd", "NormBwd", "GemmAct", "ActBwd", "MoePlan",
    "fp8_norm_fwd", "fp8_norm_bwd", "fp8_norm_bwd_workspace_size", "fp8_gemm_act", "fp8_act_bwd",
    "fp8_act_bwd_workspace_size", "fp8_moe_rows", "fp8_moe_workspace_size", "fp8_moe_plan",
    "fp8_moe_permute", "fp8_moe_unpermute", "fp8_moe_unpermute_bwd",
]

NORM_RMS, NORM_LAYER = 0, 1
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH = 0, 1, 2, 3, 4

_BF16, _F32, _I32, _BYTE = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_OUT = {_BF16: OUT_BF16, _F32: OUT_F32}
_i32, _i64, _f32, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


class NormFwdArgsC(ctypes.Structure):
    """fp8_norm_fwd_args_t"""
    _fields_ = [("rows", _i64), ("width", _i64), ("kind", _i32), ("stream_type", _i32),
                ("eps", _f32), ("alpha", _f32), ("x", _vp), ("h", _vp), ("gate", _vp),
                ("gate_rows", _i64), ("post_norm", _i32), ("w_post", _vp), ("b_post", _vp),
                ("w_pre", _vp), ("b_pre", _vp), ("x_out", _vp), ("y", _vp), ("q", _vp),
                ("q_format", _i32), ("q_granularity", _i32), ("pow2", _i32), ("q_scale", _vp),
                ("q_scale_inv", _vp), ("amax", _vp), ("stats", _vp)]


class NormBwdArgsC(ctypes.Structure):
    """fp8_norm_bwd_args_t"""
    _fields_ = [("rows", _i64), ("width", _i64), ("kind", _i32), ("stream_type", _i32),
                ("alpha", _f32), ("dy", _vp), ("x_out", _vp), ("dx_out", _vp), ("h", _vp),
                ("gate", _vp), ("gate_rows", _i64), ("post_norm", _i32), ("w_post", _vp),
                ("b_post", _vp), ("w_pre", _vp), ("stats", _vp), ("dx", _vp), ("dh", _vp),
                ("dw_pre", _vp), ("db_pre", _vp), ("dw_post", _vp), ("db_post", _vp),
                ("dgate", _vp), ("accumulate", _i32)]


class GemmActArgsC(ctypes.Structure):
    """fp8_gemm_act_args_t"""
    _fields_ = [("A", _vp), ("B", _vp), ("fa", _i32), ("fb", _i32), ("M", _i64), ("N", _i64),
                ("K", _i64), ("ga", _i32), ("gb", _i32), ("scale_inv_a", _vp),
                ("scale_inv_b", _vp), ("act", _i32), ("gated", _i32), ("bias", _vp),
                ("residual", _vp), ("z", _vp), ("d", _vp), ("q", _vp), ("q_format", _i32),
                ("q_scale", _vp), ("amax", _vp), ("offsets", _vp), ("experts", _i32)]


class ActBwdArgsC(ctypes.Structure):
    """fp8_act_bwd_args_t"""
    _fields_ = [("M", _i64), ("N", _i64), ("act", _i32), ("gated", _i32), ("dD", _vp), ("z", _vp),
                ("dz", _vp), ("q", _vp), ("q_format", _i32), ("q_scale", _vp), ("amax", _vp),
                ("dbias", _vp), ("accumulate", _i32), ("offsets", _vp), ("experts", _i32)]


# A call's arguments are packed to the C struct's bytes in one go, which takes
# a third of the time of filling a ctypes.Structure field by field.
_CODE = {_i32: "i", _i64: "q", _f32: "f", _vp: "P"}


def _packer(args):
    return struct.Struct("@" + "".join(_CODE[t] for _, t in args._fields_)).pack


_pack_norm_fwd, _pack_norm_bwd = _packer(NormFwdArgsC), _packer(NormBwdArgsC)
_pack_gemm_act, _pack_act_bwd = _packer(GemmActArgsC), _packer(ActBwdArgsC)


class NormFwd(NamedTuple):
    x_out: Optional[torch.Tensor]
    y: Optional[torch.Tensor]
    q: Optional[torch.Tensor]
    q_scale_inv: Optional[torch.Tensor]
    amax: Optional[torch.Tensor]
    stats: Optional[torch.Tensor]


class NormBwd(NamedTuple):
    dx: Optional[torch.Tensor]
    dh: Optional[torch.Tensor]
    dw_pre: Optional[torch.Tensor]
    db_pre: Optional[torch.Tensor]
    dw_post: Optional[torch.Tensor]
    db_post: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]


class GemmAct(NamedTuple):
    d: Optional[torch.Tensor]
    z: Optional[torch.Tensor]
    q: Optional[torch.Tensor]
    amax: Optional[torch.Tensor]


class ActBwd(NamedTuple):
    dz: Optional[torch.Tensor]
    q: Optional[torch.Tensor]
    amax: Optional[torch.Tensor]
    dbias: Optional[torch.Tensor]


class MoePlan(NamedTuple):
    offsets: torch.Tensor
    counts: torch.Tensor
    row_of: torch.Tensor
    src: torch.Tensor


_ready = None


def _check(status):
    if status:
        raise Fp8Error(status, fp8_last_error())


def _lib():
    """The library with these calls' signatures declared."""
    global _ready
    if _ready is None:
        L = _base_lib()
        i = ctypes.c_int
        L.fp8_norm_fwd.argtypes = [_vp, _vp]
        L.fp8_norm_bwd.argtypes = [_vp, _vp, _sz, _vp]
        L.fp8_norm_bwd_workspace_size.argtypes = [_i64, _i64, _i64]
        L.fp8_norm_bwd_workspace_size.restype = _sz
        L.fp8_gemm_act.argtypes = [_vp, _vp]
        L.fp8_act_bwd.argtypes = [_vp, _vp, _sz, _vp]
        L.fp8_act_bwd_workspace_size.argtypes = [_i64, _i64, i]
        L.fp8_act_bwd_workspace_size.restype = _sz
        L.fp8_act_bwd_experts_workspace_size.argtypes = [_i64, _i64, i, i]
        L.fp8_act_bwd_experts_workspace_size.restype = _sz
        L.fp8_moe_rows.argtypes = [_i64, i, i, i]
        L.fp8_moe_rows.restype = _i64
        L.fp8_moe_workspace_size.argtypes = [_i64, i, i]
        L.fp8_moe_workspace_size.restype = _sz
        L.fp8_moe_plan.argtypes = [_vp, _i64, i, i, i, _vp, _vp, _vp, _vp, _i64, _vp, _sz, _vp]
        L.fp8_moe_permute.argtypes = [_vp, _vp, _i64, i, _i64, _vp, _vp, _i64, _vp, _vp, _vp]
        L.fp8_moe_unpermute.argtypes = [_vp, i, _vp, _vp, _i64, i, _i64, _i64, _vp, _vp]
        L.fp8_moe_unpermute_bwd.argtypes = [_vp, _vp, i, _vp, _vp, _vp, _i64, i, _i64, _i64, _vp,
                                            _vp, _vp]
        for name in ("fp8_norm_fwd", "fp8_norm_bwd", "fp8_gemm_act", "fp8_act_bwd", "fp8_moe_plan",
                     "fp8_moe_permute", "fp8_moe_unpermute", "fp8_moe_unpermute_bwd"):
            getattr(L, name).restype = i
        _ready = L
    return _ready


def _given(t, what, dtype, shape, on):
    """The address of a tensor that has to be of this type and shape and on
    the device that _here() gave."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous()
                and (on is None or t.get_device() == on)):
            return t.data_ptr()
    except AttributeError:
        pass
    p = _ptr(t, what, _U8 if dtype is _BYTE else dtype)   # says what is wrong
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if on is not None and t.get_device() != on:
        raise ValueError(f"{what}: on cuda:{t.get_device()}, not where the other tensors are")
    return p


def _on(device):
    """The handle of the current stream of the device that _here() gave."""
    return _raw_stream(device or 0) if _raw_stream is not None else _stream(None)


def _rows(t, what):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what} must be 2-D")
    return shape


def _workspace(workspace, need, device, on):
    """(address, bytes, tensor) of the given workspace or of a new one."""
    if workspace is not None:
        return _given(workspace, "workspace", _BYTE, workspace.shape, on), workspace.numel(), workspace
    workspace = torch.empty(need if need > 16 else 16, dtype=_BYTE, device=device)
    return workspace.data_ptr(), workspace.numel(), workspace


# ------------------------------------------------------------------ norms

def fp8_norm_fwd(x, h=None, kind: int = NORM_RMS, eps: float = 1e-5, alpha: float = 1.0, gate=None,
                 post_norm: bool = False, w_post=None, b_post=None, w_pre=None, b_pre=None,
                 want_y: bool = True, want_stats: bool = False, q_fmt: int | None = None,
                 q_gran: int = GRAN_TENSOR, q_scale=None, pow2: bool = False,
                 want_amax: bool = False, x_out=None, y=None, q=None, q_scale_inv=None, amax=None,
                 stats=None, want_x_out: bool = True, stream=None) -> NormFwd:
    """x' = alpha x + gate * p with p = N(h; w_post, b_post) (post_norm) or h,
    then y = N(x'; w_pre, b_pre).  x [T, C] bf16 or fp32 (None: 0), h [T, C]
    bf16 (None: x' = alpha x), gate [G, C] bf16 with G dividing T.  y comes as
    bf16 (want_y) and, with q_fmt, as FP8 codes: per tensor with q_scale (and
    max|y|, want_amax) or per row (GRAN_ROW, q_scale_inv [T]).  stats [4, T]
    (want_stats) is what fp8_norm_bwd needs.  x_out may be x."""
    if stream is not None:
        return _under(stream, fp8_norm_fwd, locals())
    ref = x if x is not None else h
    if ref is None:
        raise ValueError("x and h are None")
    T, C = shape = _rows(ref, "x")
    dev, on = ref.device, _here(ref)
    dt = x.dtype if x is not None else (x_out.dtype if x_out is not None else _BF16)
    if dt not in _OUT:
        raise TypeError(f"x: dtype {dt}, expected bfloat16 or float32")
    p_xo = p_y = p_q = p_inv = p_amax = p_stats = 0
    if x_out is not None:
        p_xo = _given(x_out, "x_out", dt, shape, on)
    elif want_x_out:
        x_out = torch.empty_like(x) if x is not None else torch.empty(T, C, dtype=dt, device=dev)
        p_xo = x_out.data_ptr()
    if y is not None:
        p_y = _given(y, "y", _BF16, shape, on)
    elif want_y:
        y = (torch.empty_like(h) if h is not None else torch.empty_like(x) if dt is _BF16 else
             torch.empty(T, C, dtype=_BF16, device=dev))
        p_y = y.data_ptr()
    if q_fmt is not None or q is not None:
        if q is None:
            q = torch.empty(T, C, dtype=torch.uint8, device=dev)
        p_q = _given(q, "q", _BYTE, shape, on)
        if q_gran == GRAN_ROW and q_scale_inv is None:
            q_scale_inv = torch.empty(T, dtype=_F32, device=dev)
    if q_scale_inv is not None:
        p_inv = _given(q_scale_inv, "q_scale_inv", _F32, (T,), on)
    if want_amax and amax is None:
        amax = torch.empty(1, dtype=_F32, device=dev)
    if amax is not None:
        p_amax = _given(amax, "amax", _F32, (1,), on)
    if stats is not None:
        p_stats = _given(stats, "stats", _F32, (4, T), on)
    elif want_stats:
        stats = torch.empty(4, T, dtype=_F32, device=dev)
        p_stats = stats.data_ptr()
    gate_rows = 0 if gate is None else _rows(gate, "gate")[0]
    vec = (C,)
    a = _pack_norm_fwd(
        T, C, kind, _OUT[dt], eps, alpha, 0 if x is None else _given(x, "x", dt, shape, on),
        0 if h is None else _given(h, "h", _BF16, shape, on),
        0 if gate is None else _given(gate, "gate", _BF16, (gate_rows, C), on), gate_rows,
        1 if post_norm else 0, 0 if w_post is None else _given(w_post, "w_post", _F32, vec, on),
        0 if b_post is None else _given(b_post, "b_post", _F32, vec, on),
        0 if w_pre is None else _given(w_pre, "w_pre", _F32, vec, on),
        0 if b_pre is None else _given(b_pre, "b_pre", _F32, vec, on), p_xo, p_y, p_q,
        E4M3 if q_fmt is None else q_fmt, q_gran, 1 if pow2 else 0,
        0 if q_scale is None else _given(q_scale, "q_scale", _F32, (1,), on), p_inv, p_amax, p_stats)
    _check((_ready or _lib()).fp8_norm_fwd(a, _on(on)))
    return NormFwd(x_out, y, q, q_scale_inv, amax, stats)


def fp8_norm_bwd_workspace_size(rows: int, width: int, gate_rows: int = 0) -> int:
    return int((_ready or _lib()).fp8_norm_bwd_workspace_size(rows, width, gate_rows))


def fp8_norm_bwd(dy, x_out, stats, dx_out=None, h=None, kind: int = NORM_RMS, alpha: float = 1.0,
                 gate=None, post_norm: bool = False, w_post=None, b_post=None, w_pre=None,
                 b_pre=None, dx=None, dh=None, dw_pre=None, db_pre=None, dw_post=None,
                 db_post=None, dgate=None, accumulate: bool = False, workspace=None,
                 stream=None) -> NormBwd:
    """Gradients of fp8_norm_fwd from dy (None: 0) and dx_out, the gradient
    that x' gets from its other use (None: 0; the stream's type).  x_out and
    stats are the forward's.  dx and dh come where their inputs were; the
    vectors' gradients (fp32) where the vectors were given, added to the given
    outputs with accumulate.  dx may be dx_out."""
    if stream is not None:
        return _under(stream, fp8_norm_bwd, locals())
    ref = x_out if x_out is not None else dx_out if dx_out is not None else dy
    if ref is None:
        raise ValueError("dy and dx_out are None")
    T, C = shape = _rows(ref, "x_out")
    dev, on = ref.device, _here(ref)
    dt = x_out.dtype if x_out is not None else dx_out.dtype if dx_out is not None else _BF16
    if dt not in _OUT:
        raise TypeError(f"x_out: dtype {dt}, expected bfloat16 or float32")
    want = [dw_pre is None and w_pre is not None and dy is not None,
            db_pre is None and b_pre is not None and dy is not None,
            dw_post is None and w_post is not None, db_post is None and b_post is not None]
    if accumulate and (any(want) or (dgate is None and gate is not None)):
        raise ValueError("accumulate adds to given outputs")
    vec = (C,)
    if dx is None:
        dx = torch.empty_like(ref) if ref.dtype is dt else torch.empty(T, C, dtype=dt, device=dev)
    if dh is None and h is not None:
        dh = torch.empty_like(h)
    gate_rows = 0 if gate is None else _rows(gate, "gate")[0]
    if want[0]:
        dw_pre = torch.empty(C, dtype=_F32, device=dev)
    if want[1]:
        db_pre = torch.empty(C, dtype=_F32, device=dev)
    if want[2]:
        dw_post = torch.empty(C, dtype=_F32, device=dev)
    if want[3]:
        db_post = torch.empty(C, dtype=_F32, device=dev)
    if dgate is None and gate is not None:
        dgate = torch.empty(gate_rows, C, dtype=_F32, device=dev)
    ws, ws_bytes, workspace = _workspace(workspace, fp8_norm_bwd_workspace_size(T, C, gate_rows), dev, on)
    a = _pack_norm_bwd(
        T, C, kind, _OUT[dt], alpha, 0 if dy is None else _given(dy, "dy", _BF16, shape, on),
        0 if x_out is None else _given(x_out, "x_out", dt, shape, on),
        0 if dx_out is None else _given(dx_out, "dx_out", dt, shape, on),
        0 if h is None else _given(h, "h", _BF16, shape, on),
        0 if gate is None else _given(gate, "gate", _BF16, (gate_rows, C), on), gate_rows,
        1 if post_norm else 0, 0 if w_post is None else _given(w_post, "w_post", _F32, vec, on),
        0 if b_post is None else _given(b_post, "b_post", _F32, vec, on),
        0 if w_pre is None else _given(w_pre, "w_pre", _F32, vec, on),
        0 if stats is None else _given(stats, "stats", _F32, (4, T), on), _given(dx, "dx", dt, shape, on),
        0 if dh is None else _given(dh, "dh", _BF16, shape, on),
        0 if dw_pre is None else _given(dw_pre, "dw_pre", _F32, vec, on),
        0 if db_pre is None else _given(db_pre, "db_pre", _F32, vec, on),
        0 if dw_post is None else _given(dw_post, "dw_post", _F32, vec, on),
        0 if db_post is None else _given(db_post, "db_post", _F32, vec, on),
        0 if dgate is None else _given(dgate, "dgate", _F32, (gate_rows, C), on), 1 if accumulate else 0)
    _check((_ready or _lib()).fp8_norm_bwd(a, ws, ws_bytes, _on(on)))
    return NormBwd(dx, dh, dw_pre, db_pre, dw_post, db_post, dgate)


# ------------------------------------------------------------------ GEMM with an epilogue

def fp8_gemm_act(A, fa: int, B, fb: int, scale_inv_a, scale_inv_b, ga: int = GRAN_TENSOR,
                 gb: int = GRAN_TENSOR, act: int = ACT_NONE, gated: bool = False, bias=None,
                 residual=None, want_z: bool = False, want_d: bool = True, q_fmt: int | None = None,
                 q_scale=None, want_amax: bool = False, z=None, d=None, q=None, amax=None,
                 offsets=None, stream=None) -> GemmAct:
    """D = act(z) + residual with z = s_a s_b A . B^T + bias, or, gated, D =
    act(z[:, :N]) z[:, N:] + residual (B's first N rows are the gate's).  A
    [M, K] and B [N or 2N, K] are FP8 codes.  D comes as bf16 (want_d) and,
    with q_fmt, as FP8 codes of D * q_scale; z (bf16, want_z) is what
    fp8_act_bwd needs.  With offsets [E + 1] (fp8_moe_plan's) B is
    [E, N or 2N, K] and each expert's rows of A take their part of B,
    scale_inv_b and bias; rows that no expert has (past the last offset) are
    left as they are in d, z and q -- of a new tensor, whatever its memory
    held -- so give fp8_act_bwd the same offsets.  d may be residual."""
    if stream is not None:
        return _under(stream, fp8_gemm_act, locals())
    M, K = _rows(A, "A")
    E = 1
    if offsets is not None:
        if B.dim() != 3:
            raise ValueError("B must be [experts, N or 2N, K] with offsets")
        E = B.shape[0]
    elif B.dim() != 2:
        raise ValueError("B must be 2-D")
    rows = B.shape[-2]
    if B.shape[-1] != K:
        raise ValueError("A and B disagree on K")
    if gated and rows % 2:
        raise ValueError("a gated B has an even number of rows")
    N = rows // 2 if gated else rows
    dev, on = A.device, _here(A)
    out = (M, N)
    p_d = p_z = p_q = p_amax = 0
    if d is not None:
        p_d = _given(d, "d", _BF16, out, on)
    elif want_d:
        d = torch.empty(M, N, dtype=_BF16, device=dev)
        p_d = d.data_ptr()
    if z is not None:
        p_z = _given(z, "z", _BF16, (M, rows), on)
    elif want_z:
        z = torch.empty(M, rows, dtype=_BF16, device=dev)
        p_z = z.data_ptr()
    if q is not None:
        p_q = _given(q, "q", _BYTE, out, on)
    elif q_fmt is not None:
        q = torch.empty(M, N, dtype=torch.uint8, device=dev)
        p_q = q.data_ptr()
    if amax is not None:
        p_amax = _given(amax, "amax", _F32, (1,), on)
    elif want_amax:
        amax = torch.empty(1, dtype=_F32, device=dev)
        p_amax = amax.data_ptr()
    per_b = (E,)
    per_row = (E, rows) if offsets is not None else (rows,)
    a = _pack_gemm_act(
        _given(A, "A", _BYTE, (M, K), on), _given(B, "B", _BYTE, B.shape, on), fa, fb, M, N, K, ga, gb,
        _given(scale_inv_a, "scale_inv_a", _F32, (M,) if ga == GRAN_ROW else (1,), on),
        _given(scale_inv_b, "scale_inv_b", _F32, per_row if gb == GRAN_ROW else per_b, on), act,
        1 if gated else 0, 0 if bias is None else _given(bias, "bias", _BF16, per_row, on),
        0 if residual is None else _given(residual, "residual", _BF16, out, on), p_z, p_d, p_q,
        E4M3 if q_fmt is None else q_fmt,
        0 if q_scale is None else _given(q_scale, "q_scale", _F32, (1,), on), p_amax,
        0 if offsets is None else _given(offsets, "offsets", _I32, (E + 1,), on), E)
    _check((_ready or _lib()).fp8_gemm_act(a, _on(on)))
    return GemmAct(d, z, q, amax)


@functools.lru_cache(maxsize=256)
def fp8_act_bwd_workspace_size(M: int, N: int, gated: bool, experts: int = 0) -> int:
    """Bytes for dbias; experts: their number, with offsets (0: without)."""
    L = _ready or _lib()
    if experts:
        return int(L.fp8_act_bwd_experts_workspace_size(M, N, int(bool(gated)), experts))
    return int(L.fp8_act_bwd_workspace_size(M, N, int(bool(gated))))


def fp8_act_bwd(dD, z, act: int, gated: bool = False, want_dz: bool = True, q_fmt: int | None = None,
                q_scale=None, want_amax: bool = False, want_dbias: bool = False, dz=None, q=None,
                amax=None, dbias=None, accumulate: bool = False, workspace=None,
                stream=None, offsets=None) -> ActBwd:
    """dz = dD act'(z) (gated: both halves) from fp8_gemm_act's z, as bf16
    (want_dz) and, with q_fmt, as FP8 codes of dz * q_scale; dbias (fp32,
    want_dbias) is dz's column sum, added to a given one with accumulate.
    With the offsets [E + 1] that fp8_gemm_act had, rows that no expert has are
    neither read nor written nor counted in amax, and dbias is [E, N or 2N]."""
    if stream is not None:
        return _under(stream, fp8_act_bwd, locals())
    M, N = _rows(dD, "dD")
    rows = 2 * N if gated else N
    dev, on = dD.device, _here(dD)
    if accumulate and dbias is None:
        raise ValueError("accumulate adds to a given dbias")
    out = (M, rows)
    p_dz = p_q = p_amax = p_db = 0
    if dz is not None:
        p_dz = _given(dz, "dz", _BF16, out, on)
    elif want_dz:
        dz = torch.empty(M, rows, dtype=_BF16, device=dev)
        p_dz = dz.data_ptr()
    if q is not None:
        p_q = _given(q, "q", _BYTE, out, on)
    elif q_fmt is not None:
        q = torch.empty(M, rows, dtype=_BYTE, device=dev)
        p_q = q.data_ptr()
    if amax is not None:
        p_amax = _given(amax, "amax", _F32, (1,), on)
    elif want_amax:
        amax = torch.empty(1, dtype=_F32, device=dev)
        p_amax = amax.data_ptr()
    p_off, E = 0, 0
    if offsets is not None:
        E = offsets.numel() - 1
        if E < 1:
            raise ValueError("offsets must hold one number an expert and the end")
        p_off = _given(offsets, "offsets", _I32, (E + 1,), on)
    per_col = (rows,) if offsets is None else (E, rows)
    if dbias is None and want_dbias:
        dbias = torch.empty(per_col, dtype=_F32, device=dev)
    ws, ws_bytes = None, 0
    if dbias is not None:
        p_db = _given(dbias, "dbias", _F32, per_col, on)
        ws, ws_bytes, workspace = _workspace(workspace, fp8_act_bwd_workspace_size(M, N, gated, E), dev, on)
    a = _pack_act_bwd(
        M, N, act, 1 if gated else 0, _given(dD, "dD", _BF16, (M, N), on), _given(z, "z", _BF16, out, on),
        p_dz, p_q, E4M3 if q_fmt is None else q_fmt,
        0 if q_scale is None else _given(q_scale, "q_scale", _F32, (1,), on), p_amax, p_db,
        1 if accumulate else 0, p_off, E)
    _check((_ready or _lib()).fp8_act_bwd(a, ws, ws_bytes, _on(on)))
    return ActBwd(dz, q, amax, dbias)


# ------------------------------------------------------------------ tokens by expert

@functools.lru_cache(maxsize=256)
def fp8_moe_rows(tokens: int, slots: int, experts: int, align: int = 1) -> int:
    """Rows that hold any routing of this size."""
    r = int((_ready or _lib()).fp8_moe_rows(tokens, slots, experts, align))
    if r < 0:
        raise ValueError("fp8_moe_rows: slots 1..64, experts 1..1024, align 1..4096, tokens * slots <= 2^30")
    return r


@functools.lru_cache(maxsize=256)
def fp8_moe_workspace_size(tokens: int, slots: int, experts: int) -> int:
    return int((_ready or _lib()).fp8_moe_workspace_size(tokens, slots, experts))


def fp8_moe_plan(ids, experts: int, align: int = 1, rows: int | None = None, offsets=None,
                 counts=None, row_of=None, src=None, workspace=None, stream=None) -> MoePlan:
    """Sort the slots of ids [T, k] (int32; outside 0..experts-1: dropped) by
    expert: offsets [E + 1] and counts [E] of the experts' rows, row_of [T, k]
    the slot's row or -1, src [rows] the row's slot (t * k + j) or -1.  Each
    expert's rows are padded to a multiple of align."""
    if stream is not None:
        return _under(stream, fp8_moe_plan, locals())
    T, k = _rows(ids, "ids")
    dev, on = ids.device, _here(ids)
    if rows is None:
        rows = fp8_moe_rows(T, k, experts, align) if src is None else src.numel()
    if offsets is None:
        offsets = torch.empty(experts + 1, dtype=_I32, device=dev)
        p_off = offsets.data_ptr()
    else:
        p_off = _given(offsets, "offsets", _I32, (experts + 1,), on)
    if counts is None:
        counts = torch.empty(experts, dtype=_I32, device=dev)
        p_cnt = counts.data_ptr()
    else:
        p_cnt = _given(counts, "counts", _I32, (experts,), on)
    if row_of is None:
        row_of = torch.empty_like(ids)
    if src is None:
        src = torch.empty(rows, dtype=_I32, device=dev)
        p_src = src.data_ptr()
    else:
        p_src = _given(src, "src", _I32, (rows,), on)
    ws, ws_bytes, need = None, 0, fp8_moe_workspace_size(T, k, experts)
    if need:
        ws, ws_bytes, workspace = _workspace(workspace, need, dev, on)
    _check((_ready or _lib()).fp8_moe_plan(
        _given(ids, "ids", _I32, (T, k), on), T, k, experts, align, p_off, p_cnt,
        _given(row_of, "row_of", _I32, (T, k), on), p_src, rows, ws, ws_bytes, _on(on)))
    return MoePlan(offsets, counts, row_of, src)


def fp8_moe_permute(x, row_of, src, scale=None, xs=None, scale_s=None, stream=None):
    """xs [rows, C] = x's rows in the plan's order, zeros where there is no
    source; x is of any type (codes go with their per-row factors, scale [T]).
    Returns (xs, scale_s or None)."""
    if stream is not None:
        return _under(stream, fp8_moe_permute, locals())
    T, C = _rows(x, "x")
    k, rows = _rows(row_of, "row_of")[1], src.numel()
    on = _here(x)
    if xs is None:
        xs = torch.empty(rows, C, dtype=x.dtype, device=x.device)
        p_xs = xs.data_ptr()
    else:
        p_xs = _given(xs, "xs", x.dtype, (rows, C), on)
    p_sc = p_ss = 0
    if scale is not None:
        if scale_s is None:
            scale_s = torch.empty(rows, dtype=_F32, device=x.device)
        p_sc = _given(scale, "scale", _F32, (T,), on)
    if scale_s is not None:
        p_ss = _given(scale_s, "scale_s", _F32, (rows,), on)
    _check((_ready or _lib()).fp8_moe_permute(
        _given(x, "x", x.dtype, (T, C), on), p_sc, T, k, C * x.element_size(),
        _given(row_of, "row_of", _I32, (T, k), on), _given(src, "src", _I32, (rows,), on), rows, p_xs, p_ss,
        _on(on)))
    return xs, scale_s


def fp8_moe_unpermute(ys, row_of, weights=None, y=None, stream=None) -> torch.Tensor:
    """y [T, C] = the weighted sum of each token's rows of ys [rows, C] (bf16
    or fp32); weights [T, k] fp32, None: 1 (the gradient of the permutation)."""
    if stream is not None:
        return _under(stream, fp8_moe_unpermute, locals())
    rows, C = _rows(ys, "ys")
    T, k = _rows(row_of, "row_of")
    on = _here(ys)
    if ys.dtype not in _OUT:
        raise TypeError(f"ys: dtype {ys.dtype}, expected bfloat16 or float32")
    if y is None:
        y = torch.empty(T, C, dtype=ys.dtype, device=ys.device)
    _check((_ready or _lib()).fp8_moe_unpermute(
        _given(ys, "ys", ys.dtype, (rows, C), on), _OUT[ys.dtype], _given(row_of, "row_of", _I32, (T, k), on),
        0 if weights is None else _given(weights, "weights", _F32, (T, k), on), T, k, C, rows,
        _given(y, "y", ys.dtype, (T, C), on), _on(on)))
    return y


def fp8_moe_unpermute_bwd(dy, ys, row_of, src, weights=None, dys=None, dweights=None, stream=None):
    """Gradients of fp8_moe_unpermute: (dys [rows, C], dweights [T, k] or None
    without weights)."""
    if stream is not None:
        return _under(stream, fp8_moe_unpermute_bwd, locals())
    rows, C = _rows(ys, "ys")
    T, k = _rows(row_of, "row_of")
    on = _here(ys)
    if ys.dtype not in _OUT:
        raise TypeError(f"ys: dtype {ys.dtype}, expected bfloat16 or float32")
    if dys is None:
        dys = torch.empty(rows, C, dtype=ys.dtype, device=ys.device)
    if dweights is None and weights is not None:
        dweights = torch.empty(T, k, dtype=_F32, device=ys.device)
    _check((_ready or _lib()).fp8_moe_unpermute_bwd(
        _given(dy, "dy", ys.dtype, (T, C), on), _given(ys, "ys", ys.dtype, (rows, C), on), _OUT[ys.dtype],
        _given(row_of, "row_of", _I32, (T, k), on), _given(src, "src", _I32, (rows,), on),
        0 if weights is None else _given(weights, "weights", _F32, (T, k), on), T, k, C, rows,
        _given(dys, "dys", ys.dtype, (rows, C), on),
        0 if dweights is None else _given(dweights, "dweights", _F32, (T, k), on), _on(on)))
    return dys, dweights
