"""Experts, and the activations between two products, in blocks of 128.

Calls of the same kind as block_ops' (include/fp8linear.h has the formulas).
They are a feed-forward block of experts under the block recipe: weights in
128x128 blocks, activations and gradients in 1x128 blocks, what the backward
pass needs of the forward kept in 8 bits, row counts on the device only:

  fp8_gemm_experts      one product per expert, forward and dgrad
  fp8_wgrad_experts     the experts' weight gradients
  fp8_act_block         the activation, to codes, with its checkpoint
  fp8_act_block_bwd     its gradient from the checkpoint: the operands of both backward products
  fp8_block_transpose   a kept input as the wgrad's operand

The weight gradients' offsets are multiples of 128: fp8_moe_plan with
align=128 and rows a multiple of 128.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _here, _under, _vp, E4M3, E5M2, Fp8Error, OUT_BF16, OUT_F32, fp8_last_error
from . import lib as _base_lib
from .block_ops import _BF16, _BYTE, _F32, _I32, _f32, _given, _i32, _i64, _on, _packer, _rows

__all__ = ["ActBlock", "ActBlockBwd", "fp8_gemm_experts", "fp8_wgrad_experts", "fp8_act_block", "fp8_act_block_bwd",
           "fp8_block_transpose"]

_BLOCK = 128


class GemmExpertsArgsC(ctypes.Structure):
    """fp8_gemm_experts_args_t"""
    _fields_ = [("A", _vp), ("B", _vp), ("fa", _i32), ("fb", _i32), ("M", _i64), ("N", _i64), ("K", _i64),
                ("scale_inv_a", _vp), ("scale_inv_b", _vp), ("pow2", _i32), ("out", _i32), ("d", _vp),
                ("offsets", _vp), ("experts", _i32)]


class WgradExpertsArgsC(ctypes.Structure):
    """fp8_wgrad_experts_args_t"""
    _fields_ = [("dY_t", _vp), ("X_t", _vp), ("f_dy", _i32), ("f_x", _i32), ("M", _i64), ("N", _i64), ("K", _i64),
                ("scale_inv_dy", _vp), ("scale_inv_x", _vp), ("pow2", _i32), ("accumulate", _i32), ("dW", _vp),
                ("offsets", _vp), ("experts", _i32)]


class ActBlockArgsC(ctypes.Structure):
    """fp8_act_block_args_t"""
    _fields_ = [("M", _i64), ("N", _i64), ("act", _i32), ("gated", _i32), ("z", _vp), ("q", _vp), ("scale_inv", _vp),
                ("q_format", _i32), ("pow2", _i32), ("z_q", _vp), ("z_scale_inv", _vp), ("offsets", _vp),
                ("experts", _i32)]


class ActBlockBwdArgsC(ctypes.Structure):
    """fp8_act_block_bwd_args_t"""
    _fields_ = [("M", _i64), ("N", _i64), ("act", _i32), ("gated", _i32), ("dD", _vp), ("z_q", _vp),
                ("z_scale_inv", _vp), ("q", _vp), ("scale_inv", _vp), ("q_t", _vp), ("scale_inv_t", _vp),
                ("q_format", _i32), ("h_t", _vp), ("h_scale_inv_t", _vp), ("h_format", _i32), ("pow2", _i32),
                ("offsets", _vp), ("experts", _i32)]


_pack_gemm, _pack_wgrad = _packer(GemmExpertsArgsC), _packer(WgradExpertsArgsC)
_pack_act, _pack_act_bwd = _packer(ActBlockArgsC), _packer(ActBlockBwdArgsC)


class ActBlock(NamedTuple):
    q: Optional[torch.Tensor]
    scale_inv: Optional[torch.Tensor]
    z_q: Optional[torch.Tensor]
    z_scale_inv: Optional[torch.Tensor]


class ActBlockBwd(NamedTuple):
    q: Optional[torch.Tensor]
    scale_inv: Optional[torch.Tensor]
    q_t: Optional[torch.Tensor]
    scale_inv_t: Optional[torch.Tensor]
    h_t: Optional[torch.Tensor]
    h_scale_inv_t: Optional[torch.Tensor]


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
        for name in ("fp8_gemm_experts", "fp8_wgrad_experts", "fp8_act_block", "fp8_act_block_bwd"):
            f = getattr(L, name)
            f.argtypes, f.restype = [_vp, _vp], i
        L.fp8_block_transpose.argtypes = [_vp, _vp, _i64, _i64, i, i, _vp, _vp, _vp]
        L.fp8_block_transpose.restype = i
        _ready = L
    return _ready


def _blocks(n, what):
    if n % _BLOCK:
        raise ValueError(f"{what} must be a multiple of {_BLOCK}")
    return n // _BLOCK


def _offsets(offsets, on):
    """(address, experts) of the given offsets."""
    if offsets is None:
        return 0, 0
    E = offsets.numel() - 1
    if E < 1:
        raise ValueError("offsets must hold one number an expert and the end")
    return _given(offsets, "offsets", _I32, (E + 1,), on), E


def _codes(t, inv, wanted, shape, inv_shape, what, dev, on):
    """Codes and their factors, the given ones or (wanted) new ones:
    (codes, factors, address, address)."""
    if t is None and inv is None:
        if not wanted:
            return None, None, 0, 0
        t = torch.empty(shape, dtype=_BYTE, device=dev)
        inv = torch.empty(inv_shape, dtype=_F32, device=dev)
        return t, inv, t.data_ptr(), inv.data_ptr()
    if t is None:
        t = torch.empty(shape, dtype=_BYTE, device=dev)
    if inv is None:
        inv = torch.empty(inv_shape, dtype=_F32, device=dev)
    return t, inv, _given(t, what, _BYTE, shape, on), _given(inv, what + "'s factors", _F32, inv_shape, on)


def fp8_gemm_experts(A, fa: int, B, fb: int, scale_inv_a, scale_inv_b, offsets, out: int = OUT_BF16,
                     pow2: bool = False, d=None, stream=None) -> torch.Tensor:
    """D [M, N] = A . B_e^T for the rows of each expert e, offsets[e] ..
    offsets[e + 1]: A [M, K] codes with scale_inv_a [M, K/128], B [E, N, K]
    codes with scale_inv_b [E, N/128, K/128], offsets [E + 1] int32 as
    fp8_moe_plan writes them (any alignment).  out: OUT_BF16 or OUT_F32.  pow2:
    every factor is a power of two (from pow2 casts), which the tensor core
    applies itself.  Rows that no expert has are left as they are in d -- of a
    new tensor, whatever its memory held.  The input gradient is the same call
    with the transposed weight codes and their factors."""
    if stream is not None:
        return _under(stream, fp8_gemm_experts, locals())
    M, K = _rows(A, "A")
    if B.dim() != 3 or B.shape[2] != K:
        raise ValueError("B must be [experts, N, K] with A's K")
    E, N, _ = B.shape
    kb, nb = _blocks(K, "K"), _blocks(N, "N")
    if out not in (OUT_BF16, OUT_F32):
        raise ValueError("out must be OUT_BF16 or OUT_F32")
    dt, dev, on = (_F32 if out == OUT_F32 else _BF16), A.device, _here(A)
    if d is None:
        d = torch.empty(M, N, dtype=dt, device=dev)
    a = _pack_gemm(
        _given(A, "A", _BYTE, (M, K), on), _given(B, "B", _BYTE, (E, N, K), on), fa, fb, M, N, K,
        _given(scale_inv_a, "scale_inv_a", _F32, (M, kb), on), _given(scale_inv_b, "scale_inv_b", _F32, (E, nb, kb), on),
        1 if pow2 else 0, out, _given(d, "d", dt, (M, N), on), _given(offsets, "offsets", _I32, (E + 1,), on), E)
    _check((_ready or _lib()).fp8_gemm_experts(a, _on(on)))
    return d


def fp8_wgrad_experts(dY_t, f_dy: int, X_t, f_x: int, scale_inv_dy, scale_inv_x, offsets, pow2: bool = False,
                      dW=None, accumulate: bool = False, stream=None) -> torch.Tensor:
    """dW [E, N, K] fp32 (+)= dY^T . X over each expert's tokens, offsets[e] ..
    offsets[e + 1], multiples of 128 (otherwise that expert's dW is NaN and
    check_device_status() raises): dY_t [N, M] codes with scale_inv_dy
    [N, M/128], X_t [K, M] codes with scale_inv_x [K, M/128].  An expert without
    tokens gets zeros; accumulate adds to the given dW."""
    if stream is not None:
        return _under(stream, fp8_wgrad_experts, locals())
    N, M = _rows(dY_t, "dY_t")
    K = _rows(X_t, "X_t")[0]
    mb = _blocks(M, "the number of tokens")
    if accumulate and dW is None:
        raise ValueError("accumulate adds to a given dW")
    dev, on = dY_t.device, _here(dY_t)
    p_off, E = _offsets(offsets, on)
    if not E:
        raise ValueError("offsets is None")
    if dW is None:
        dW = torch.empty(E, N, K, dtype=_F32, device=dev)
    a = _pack_wgrad(
        _given(dY_t, "dY_t", _BYTE, (N, M), on), _given(X_t, "X_t", _BYTE, (K, M), on), f_dy, f_x, M, N, K,
        _given(scale_inv_dy, "scale_inv_dy", _F32, (N, mb), on), _given(scale_inv_x, "scale_inv_x", _F32, (K, mb), on),
        1 if pow2 else 0, 1 if accumulate else 0, _given(dW, "dW", _F32, (E, N, K), on), p_off, E)
    _check((_ready or _lib()).fp8_wgrad_experts(a, _on(on)))
    return dW


def fp8_act_block(z, act: int, gated: bool = False, q_fmt: int = E4M3, pow2: bool = False, want_q: bool = True,
                  keep: bool = False, q=None, scale_inv=None, z_q=None, z_scale_inv=None, offsets=None,
                  stream=None) -> ActBlock:
    """h = act(z), gated: act(z[:, :N]) z[:, N:], as codes q [M, N] with factors
    scale_inv [M, N/128] (want_q), and with keep the checkpoint of z [M, N or
    2N] (bf16) in 8 bits: z_q (E4M3) and z_scale_inv, what fp8_act_block_bwd
    takes.  With offsets only the rows of experts are read and written."""
    if stream is not None:
        return _under(stream, fp8_act_block, locals())
    M, W = _rows(z, "z")
    if gated and W % 2:
        raise ValueError("a gated z has an even number of columns")
    N = W // 2 if gated else W
    nb, wb = _blocks(N, "N"), W // _BLOCK
    dev, on = z.device, _here(z)
    q, scale_inv, p_q, p_inv = _codes(q, scale_inv, want_q, (M, N), (M, nb), "q", dev, on)
    z_q, z_scale_inv, p_zq, p_zinv = _codes(z_q, z_scale_inv, keep, (M, W), (M, wb), "z_q", dev, on)
    p_off, E = _offsets(offsets, on)
    a = _pack_act(M, N, act, 1 if gated else 0, _given(z, "z", _BF16, (M, W), on), p_q, p_inv, q_fmt,
                  1 if pow2 else 0, p_zq, p_zinv, p_off, E)
    _check((_ready or _lib()).fp8_act_block(a, _on(on)))
    return ActBlock(q, scale_inv, z_q, z_scale_inv)


def fp8_act_block_bwd(dD, z_q, z_scale_inv, act: int, gated: bool = False, q_fmt: int = E5M2, h_fmt: int = E4M3,
                      pow2: bool = False, want_q: bool = True, want_t: bool = False, want_h_t: bool = False, q=None,
                      scale_inv=None, q_t=None, scale_inv_t=None, h_t=None, h_scale_inv_t=None, offsets=None,
                      stream=None) -> ActBlockBwd:
    """dz from dD [M, N] (bf16) and fp8_act_block's checkpoint: codes q [M, N or
    2N] of its rows (want_q, the dgrad's operand), codes q_t [N or 2N, M] of
    dz^T in blocks of 128 tokens (want_t, the wgrad's), and codes h_t [N, M] of
    h^T (want_h_t, the next product's wgrad operand), h computed again; each
    with its factors, one for 128 elements of a row.  want_t and want_h_t need
    M a multiple of 128.  With offsets only the rows of experts are read and
    written, and blocks of 128 tokens without any are left out."""
    if stream is not None:
        return _under(stream, fp8_act_block_bwd, locals())
    M, N = _rows(dD, "dD")
    nb = _blocks(N, "N")
    W, wb = (2 * N, 2 * nb) if gated else (N, nb)
    dev, on = dD.device, _here(dD)
    tokens = any(t is not None for t in (q_t, scale_inv_t, h_t, h_scale_inv_t))
    mb = _blocks(M, "M") if want_t or want_h_t or tokens else 0
    q, scale_inv, p_q, p_inv = _codes(q, scale_inv, want_q, (M, W), (M, wb), "q", dev, on)
    q_t, scale_inv_t, p_t, p_tinv = _codes(q_t, scale_inv_t, want_t, (W, M), (W, mb), "q_t", dev, on)
    h_t, h_scale_inv_t, p_h, p_hinv = _codes(h_t, h_scale_inv_t, want_h_t, (N, M), (N, mb), "h_t", dev, on)
    p_off, E = _offsets(offsets, on)
    a = _pack_act_bwd(
        M, N, act, 1 if gated else 0, _given(dD, "dD", _BF16, (M, N), on), _given(z_q, "z_q", _BYTE, (M, W), on),
        _given(z_scale_inv, "z_scale_inv", _F32, (M, wb), on), p_q, p_inv, p_t, p_tinv, q_fmt, p_h, p_hinv, h_fmt,
        1 if pow2 else 0, p_off, E)
    _check((_ready or _lib()).fp8_act_block_bwd(a, _on(on)))
    return ActBlockBwd(q, scale_inv, q_t, scale_inv_t, h_t, h_scale_inv_t)


def fp8_block_transpose(q, fmt: int, scale_inv, pow2: bool = False, q_t=None, scale_inv_t=None, stream=None):
    """(q_t [C, T], scale_inv_t [C, T/128]): the transpose of x [T, C], given as
    codes with factors for 1x128 blocks of its rows (scale_inv [T, C/128]), cast
    again in 1x128 blocks along T.  T and C are multiples of 128."""
    if stream is not None:
        return _under(stream, fp8_block_transpose, locals())
    T, C = _rows(q, "q")
    tb, cb = _blocks(T, "the number of rows"), _blocks(C, "the number of columns")
    on = _here(q)
    q_t, scale_inv_t, p_t, p_inv = _codes(q_t, scale_inv_t, True, (C, T), (C, tb), "q_t", q.device, on)
    _check((_ready or _lib()).fp8_block_transpose(
        _given(q, "q", _BYTE, (T, C), on), _given(scale_inv, "scale_inv", _F32, (T, cb), on), T, C, fmt,
        1 if pow2 else 0, p_t, p_inv, _on(on)))
    return q_t, scale_inv_t
