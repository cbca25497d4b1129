"""Rotary positions (include/attn.h): argument checks and marshalling, and tables of frequencies."""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from ._binding import _i64x3, lib
from ._paged import _INT32, _guard, _i64x2, _launch, _packer, _refuse, _refuse_devices


class RotaryParams(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("N", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hk", ctypes.c_int32), ("d", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("interleaved", ctypes.c_int32),
        ("magnitude", ctypes.c_float), ("reserved0", ctypes.c_int32),
        ("positions", ctypes.c_void_p), ("position_stride", _i64x2), ("inv_freq", ctypes.c_void_p),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p),
        ("q_stride", _i64x3), ("k_stride", _i64x3), ("q_out_stride", _i64x3), ("k_out_stride", _i64x3),
    ]


_ROTARY = _packer(RotaryParams)
for _entry in (lib.attn_rotary, lib.attn_rotary_bwd):
    _entry.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    _entry.restype = ctypes.c_int

_TYPES = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}


def rotary_frequencies(rotary_dim: int, *, base: float = 10000.0, linear: float = 1.0, ntk: float = 1.0, by_parts: float = 1.0,
                       context: int = 0, low_turns: float = 1.0, high_turns: float = 32.0, device=None) -> torch.Tensor:
    """Frequencies base^(-2 i / rotary_dim) of the pairs i < rotary_dim / 2, as attn_rotary takes them (fp32), scaled for
    contexts longer than a model was trained on by one of

    - linear: positions divided by the factor;
    - ntk: the base raised so that the lowest frequency is divided by the factor and the highest stays;
    - by_parts: frequencies that make fewer than low_turns turns in the trained context are divided by the factor, those of
      more than high_turns stay, and between the two the share kept grows in proportion to the turns.
    """
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError(f"rotary_dim must be positive and even, got {rotary_dim}")
    if not base > 0 or min(linear, ntk, by_parts) < 1:
        raise ValueError("base must be positive, and factors at least 1")
    if sum(f != 1 for f in (linear, ntk, by_parts)) > 1:
        raise ValueError("only one way of scaling at a time")
    if ntk != 1:
        if rotary_dim == 2:
            raise ValueError("ntk scaling needs more than one frequency")
        base = base * ntk ** (rotary_dim / (rotary_dim - 2))
    freq = base ** (-2.0 * torch.arange(rotary_dim // 2, dtype=torch.float64) / rotary_dim) / linear
    if by_parts != 1:
        if context < 1 or not 0 <= low_turns < high_turns:
            raise ValueError("by_parts needs the trained context, and low_turns below high_turns")
        kept = ((context * freq / (2 * math.pi) - low_turns) / (high_turns - low_turns)).clamp(0, 1)
        freq = freq * (kept + (1 - kept) / by_parts)
    return freq.to(device=device, dtype=torch.float32)


_F32 = torch.float32


def _check_call(q, k, positions, inv_freq, q_out, k_out) -> None:
    """Says what is wrong with the tensors of a call, if anything is."""
    dtype, dims = q.dtype, q.dim()
    if dtype not in _TYPES:
        raise TypeError(f"q must be bfloat16, float16 or float32, got {dtype}")
    if dims not in (3, 4):
        raise ValueError(f"q has shape {tuple(q.shape)}, expected [rows, H, d] or [B, H, N, d]")
    at = (0, 2, 3) if dims == 4 else (0, 2)  # all but the heads
    for name, t in (("k", k), ("q_out", q_out), ("k_out", k_out)):
        if t is None:
            continue
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        like = k if name == "k_out" else q
        if t.dim() != dims or (name == "k" and any(t.shape[i] != q.shape[i] for i in at)) or (name != "k" and t.shape != like.shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, which does not go with {tuple(like.shape)}")
    for name, t in (("q", q), ("k", k), ("q_out", q_out), ("k_out", k_out)):
        if t is not None and t.stride()[-1] != 1 and t.numel() > 0:
            raise ValueError(f"{name} must be contiguous along its last dimension")
    if positions.dtype is not _INT32:
        raise TypeError(f"positions must be {_INT32}, got {positions.dtype}")
    n = q.shape[0] if dims == 3 else q.shape[2]
    if positions.shape != (n,) and (dims == 3 or positions.shape != (q.shape[0], n)):
        raise ValueError(f"positions has shape {tuple(positions.shape)}, expected {(n,)}" +
                         (f" or {(q.shape[0], n)}" if dims == 4 else ""))
    if inv_freq.dtype is not _F32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        _refuse("inv_freq", inv_freq, _F32, (inv_freq.numel(),))


def _strides(t, dims):
    if t is None:
        return 0, 0, 0
    s = t.stride()
    return s[:3] if dims == 4 else (0, s[1], s[0])


def _call(entry, q, k, positions, inv_freq, interleaved, magnitude, q_out, k_out, stream):
    if k is None and k_out is not None:
        raise ValueError("k_out given without k")
    # one condition over plain reads for a ragged batch's rows, as serving has them; what it does not hold for is looked at
    dtype, shape, at, freq = q.dtype, q.shape, positions.shape, inv_freq.shape
    good = len(shape) == 3 and k is not None and q_out is not None and k_out is not None and len(k.shape) == 3 and len(freq) == 1
    if good:
        N, heads, d = shape
        kshape, sq, sk, so, sp = k.shape, q.stride(), k.stride(), q_out.stride(), k_out.stride()
        good = (dtype in _TYPES and k.dtype is dtype and q_out.dtype is dtype and k_out.dtype is dtype and positions.dtype is _INT32
                and inv_freq.dtype is _F32 and kshape[0] == N and kshape[2] == d and q_out.shape == shape and k_out.shape == kshape
                and at == (N,) and sq[2] == 1 and sk[2] == 1 and so[2] == 1 and sp[2] == 1 and inv_freq.is_contiguous())
    if not good:
        _check_call(q, k, positions, inv_freq, q_out, k_out)
    dev = q.get_device()
    if not (dev >= 0 and positions.get_device() == dev and inv_freq.get_device() == dev and (k is None or k.get_device() == dev)
            and (q_out is None or q_out.get_device() == dev) and (k_out is None or k_out.get_device() == dev)):
        _refuse_devices(q, positions, inv_freq, *(t for t in (k, q_out, k_out) if t is not None))
    if good:
        packed = _ROTARY.pack(1, N, heads, kshape[1], d, 2 * freq[0], _TYPES[dtype], 1 if interleaved else 0, magnitude, 0,
                              positions.data_ptr(), 0, positions.stride()[0], inv_freq.data_ptr(), q.data_ptr(), k.data_ptr(),
                              q_out.data_ptr(), k_out.data_ptr(), 0, sq[1], sq[0], 0, sk[1], sk[0], 0, so[1], so[0], 0, sp[1], sp[0])
        guard = _guard(dev, stream)
        if guard is None:
            _launch(entry, dev, packed)
        else:
            with guard:
                _launch(entry, dev, packed)
        return q_out, k_out
    dims = len(shape)
    if dims == 4:
        B, _, N, d = shape
    else:
        (N, _, d), B = shape, 1
    pb, pn = positions.stride() if len(at) == 2 else (0, positions.stride()[0])
    guard = _guard(dev, stream)
    if guard is not None:
        guard.__enter__()
    try:
        if q_out is None:
            q_out = torch.empty(shape, dtype=dtype, device=q.device)
        if k_out is None and k is not None:
            k_out = torch.empty(k.shape, dtype=dtype, device=q.device)
        _launch(entry, dev, _ROTARY.pack(
            B, N, shape[1], 0 if k is None else k.shape[1], d, 2 * freq[0], _TYPES[dtype], 1 if interleaved else 0,
            magnitude, 0, positions.data_ptr(), pb, pn, inv_freq.data_ptr(), q.data_ptr(), 0 if k is None else k.data_ptr(),
            q_out.data_ptr(), 0 if k is None else k_out.data_ptr(), *_strides(q, dims), *_strides(k, dims), *_strides(q_out, dims),
            *_strides(k_out, dims)))
    finally:
        if guard is not None:
            guard.__exit__(None, None, None)
    return q_out, k_out


def attn_rotary(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, inv_freq: torch.Tensor, *,
                interleaved: bool = False, magnitude: float = 1.0, q_out: Optional[torch.Tensor] = None,
                k_out: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Queries and keys turned by their positions; k may be None. Returns (q_out, k_out).

    q [B, Hq, N, d], k [B, Hk, N, d] with positions [N] or [B, N], or rows of a ragged batch q [rows, Hq, d], k [rows, Hk,
    d] with positions [rows]; int32. Pair i of the first 2 * len(inv_freq) columns is turned by positions * inv_freq[i]
    (rotary_frequencies) and multiplied by magnitude; a pair is columns (i, i + len(inv_freq)), or (2 i, 2 i + 1) if
    interleaved. Rows with a negative position are left as they are in the outputs (unset in tensors allocated
    here). q_out and k_out may be q and k themselves."""
    return _call(lib.attn_rotary, q, k, positions, inv_freq, interleaved, magnitude, q_out, k_out, stream)


def attn_rotary_bwd(dq: torch.Tensor, dk: Optional[torch.Tensor], positions: torch.Tensor, inv_freq: torch.Tensor, *,
                    interleaved: bool = False, magnitude: float = 1.0, q_out: Optional[torch.Tensor] = None,
                    k_out: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gradients of attn_rotary's inputs from those of its outputs, dq and dk. Returns (q_out, k_out); all else as there."""
    return _call(lib.attn_rotary_bwd, dq, dk, positions, inv_freq, interleaved, magnitude, q_out, k_out, stream)
