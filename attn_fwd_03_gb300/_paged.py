"""The paged key/value cache's entry points (include/attn.h): argument checks and marshalling.

Shapes, types and devices are checked here (the C ABI sees pointers and sizes only); everything
else is checked by the library, on the host where it can be seen there and in the kernels for the
lengths, pages and slots that live on the device (attn_status reports those).
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import Dict, Optional, Tuple

import torch

from ._binding import _check, _dtype_code, _i64x3, lib

_i64x2 = ctypes.c_int64 * 2
_i32x2 = ctypes.c_int32 * 2


class PagedParams(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32), ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
        ("d", ctypes.c_int32), ("total_q", ctypes.c_int32), ("max_q", ctypes.c_int32), ("num_pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("causal", ctypes.c_int32), ("scale", ctypes.c_float), ("reserved0", _i32x2),
        ("q", ctypes.c_void_p), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p), ("o", ctypes.c_void_p),
        ("lse", ctypes.c_void_p), ("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
        ("q_stride", _i64x2), ("o_stride", _i64x2), ("k_stride", _i64x3), ("v_stride", _i64x3),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class PagesWriteParams(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("d", ctypes.c_int32),
        ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("reserved0", _i32x2),
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("slots", ctypes.c_void_p),
        ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("k_row_stride", _i64x2), ("v_row_stride", _i64x2), ("k_stride", _i64x3), ("v_stride", _i64x3),
    ]


class PagesPlanParams(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32), ("total_q", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("max_pages", ctypes.c_int32), ("free_capacity", ctypes.c_int32), ("reserved0", ctypes.c_int32),
        ("q_len", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
        ("table_stride", ctypes.c_int64), ("free_pages", ctypes.c_void_p), ("free_count", ctypes.c_void_p),
        ("cu_q", ctypes.c_void_p), ("new_len", ctypes.c_void_p), ("slots", ctypes.c_void_p),
        ("positions", ctypes.c_void_p), ("free_left", ctypes.c_void_p),
    ]


class PagesReleaseParams(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("free_capacity", ctypes.c_int32),
        ("done", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
        ("table_stride", ctypes.c_int64), ("free_pages", ctypes.c_void_p), ("free_count", ctypes.c_void_p),
        ("new_len", ctypes.c_void_p), ("free_left", ctypes.c_void_p),
    ]


def _packer(params) -> struct.Struct:
    """Packs a parameter struct from plain numbers, its array fields spelled out (NULL is 0). One pack
    call costs about a tenth of filling the ctypes struct, and a decode step is paced by the host."""
    codes = {ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_float: "f", ctypes.c_void_p: "P", ctypes.c_size_t: "N"}
    fmt = "".join(codes[kind] if kind in codes else codes[kind._type_] * kind._length_ for _, kind in params._fields_)
    packer = struct.Struct("@" + fmt + "0q")
    assert packer.size == ctypes.sizeof(params)
    return packer


_PAGED, _WRITE, _PLAN, _RELEASE = map(_packer, (PagedParams, PagesWriteParams, PagesPlanParams, PagesReleaseParams))

# the struct is passed as packed bytes or by reference
for _entry in (lib.attn_paged, lib.attn_pages_write, lib.attn_pages_plan, lib.attn_pages_release):
    _entry.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    _entry.restype = ctypes.c_int
lib.attn_paged_workspace_size.argtypes = [ctypes.c_void_p]
lib.attn_paged_workspace_size.restype = ctypes.c_size_t

_INT32 = torch.int32
_TYPES = {torch.bfloat16: _dtype_code(torch.bfloat16), torch.float16: _dtype_code(torch.float16)}


def _is_ints(t: torch.Tensor, shape: tuple) -> bool:
    return t.dtype is _INT32 and t.shape == shape and (t.is_contiguous() or t.stride(-1) == 1)


def _is_rows(t: torch.Tensor, dtype: torch.dtype, shape: tuple) -> bool:
    return t.dtype is dtype and t.shape == shape and (t.stride()[-1] == 1 or t.numel() == 0)


def _refuse(name: str, t: torch.Tensor, dtype: torch.dtype, shape) -> None:
    """Says what is wrong with a tensor that one of the checks above turned down."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous along its last dimension")


def _need_dims(name: str, t: torch.Tensor, dims: int) -> None:
    if t.dim() != dims:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {dims} dimensions")


def _type_code(name: str, t: torch.Tensor) -> int:
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    return code


def _device(*tensors: torch.Tensor) -> int:
    """The index of the CUDA device that all tensors are on."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != dev or not t.is_cuda:
            raise ValueError(f"tensors must be on one CUDA device, got {sorted({str(x.device) for x in tensors})}")
    return dev


def _guard(dev: int, stream):
    """What to enter for a call on `stream` (default: the current stream of the tensors' device): that
    stream and its device made current, so that what the call allocates belongs to the stream that uses
    it. None where they are current already."""
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"stream of {stream.device} given for tensors on cuda:{dev}")
        return torch.cuda.stream(stream)
    if dev != torch._C._cuda_getDevice():
        return torch.cuda.device(dev)
    return None


def _guarded(call, dev: int, stream, *args):
    guard = _guard(dev, stream)
    if guard is None:
        return call(dev, *args)
    with guard:
        return call(dev, *args)


def _launch(entry, dev: int, packed: bytes) -> None:
    status = entry(packed, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        _check(status)


def _default_max_q(total_q: int, num_seqs: int) -> int:
    # the longest chunk if every sequence brings at least one row
    return max(1, total_q - num_seqs + 1)


def _pack_paged(q, k_cache, v_cache, block_table, cu_q, kv_len, out, lse, scale, causal, max_q, workspace, nbytes) -> bytes:
    total_q, hq, d = q.shape
    num_seqs, columns = block_table.shape
    pages, hkv, page_size, _ = k_cache.shape
    qr, qh, _ = q.stride()
    orow, oh, _ = out.stride()
    kp, kh, ks, _ = k_cache.stride()
    vp, vh, vs, _ = v_cache.stride()
    return _PAGED.pack(num_seqs, hq, hkv, d, total_q, max_q, pages, page_size, columns, _TYPES[q.dtype],
                       1 if causal else 0, scale, 0, 0, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                       out.data_ptr(), lse.data_ptr(), cu_q.data_ptr(), kv_len.data_ptr(), block_table.data_ptr(),
                       block_table.stride(0), qr, qh, orow, oh, kp, kh, ks, vp, vh, vs, workspace, nbytes)


def paged_workspace_size(q, k_cache, v_cache, block_table, cu_q, kv_len, *, max_q: Optional[int] = None) -> int:
    """Bytes of workspace attn_paged needs for these shapes."""
    if max_q is None:
        max_q = _default_max_q(q.shape[0], block_table.shape[0])
    # out and lse are not read: q stands in for both
    return int(lib.attn_paged_workspace_size(
        _pack_paged(q, k_cache, v_cache, block_table, cu_q, kv_len, q, q, 1.0, False, max_q, 0, 0)))


# (device, d, heads, key/value heads, max_q) -> bytes; all that the size depends on
_workspace_bytes: Dict[tuple, int] = {}


def _attn_paged(dev, q, k_cache, v_cache, block_table, cu_q, kv_len, out, lse, scale, causal, max_q, workspace):
    total_q, hq, d = q.shape
    if out is None:
        out = torch.empty((total_q, hq, d), dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty((hq, total_q), dtype=torch.float32, device=q.device)
    if workspace is None:
        key = (dev, d, hq, k_cache.shape[1], max_q)
        nbytes = _workspace_bytes.get(key)
        if nbytes is None:
            nbytes = paged_workspace_size(q, k_cache, v_cache, block_table, cu_q, kv_len, max_q=max_q)
            if nbytes > 0:  # 0: nothing to do, or a call that will be refused
                _workspace_bytes[key] = nbytes
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    else:
        nbytes = workspace.numel() * workspace.element_size()
    _launch(lib.attn_paged, dev, _pack_paged(q, k_cache, v_cache, block_table, cu_q, kv_len, out, lse, scale, causal,
                                             max_q, workspace.data_ptr(), nbytes))
    return out, lse


def attn_paged(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
               cu_q: torch.Tensor, kv_len: torch.Tensor, *, scale: Optional[float] = None, causal: bool = False,
               max_q: Optional[int] = None, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of a ragged batch of new tokens over a paged cache. Returns (O, LSE).

    q [rows, Hq, d] holds the sequences' new rows one after another, sequence b in rows cu_q[b] ..
    cu_q[b + 1] - 1; k_cache, v_cache [pages, Hkv, page_size, d]; block_table [B, columns], cu_q
    [B + 1] and kv_len [B] int32 on the GPU (kv_len counts the new tokens' keys too). O is [rows, Hq,
    d], LSE fp32 [Hq, rows]. With causal each sequence's rows are its last positions. Rows behind the
    last sequence are left as they are in out and lse (unset in tensors allocated here).

    max_q, the most rows that a sequence is expected to bring, only chooses the tile shape."""
    dtype = q.dtype
    _type_code("q", q)
    _need_dims("q", q, 3)
    _need_dims("k_cache", k_cache, 4)
    _need_dims("block_table", block_table, 2)
    total_q, hq, d = q.shape
    pages, hkv, page_size, _ = k_cache.shape
    num_seqs = block_table.shape[0]
    if q.stride()[2] != 1 and q.numel() > 0:
        _refuse("q", q, dtype, q.shape)
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not _is_rows(t, dtype, (pages, hkv, page_size, d)):
            _refuse(name, t, dtype, (pages, hkv, page_size, d))
    if not _is_ints(block_table, block_table.shape):
        _refuse("block_table", block_table, _INT32, block_table.shape)
    if not _is_ints(cu_q, (num_seqs + 1,)):
        _refuse("cu_q", cu_q, _INT32, (num_seqs + 1,))
    if not _is_ints(kv_len, (num_seqs,)):
        _refuse("kv_len", kv_len, _INT32, (num_seqs,))
    tensors = [q, k_cache, v_cache, block_table, cu_q, kv_len]
    if out is not None:
        if not _is_rows(out, dtype, (total_q, hq, d)):
            _refuse("out", out, dtype, (total_q, hq, d))
        tensors.append(out)
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (hq, total_q):
            _refuse("lse", lse, torch.float32, (hq, total_q))
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")
        tensors.append(lse)
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        tensors.append(workspace)
    return _guarded(_attn_paged, _device(*tensors), stream, q, k_cache, v_cache, block_table, cu_q, kv_len, out, lse,
                    1.0 / math.sqrt(d) if scale is None else float(scale), causal,
                    _default_max_q(total_q, num_seqs) if max_q is None else int(max_q), workspace)


def _attn_pages_write(dev, packed):
    _launch(lib.attn_pages_write, dev, packed)


def attn_pages_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
                     v_cache: torch.Tensor, *, stream=None) -> None:
    """Store k, v [rows, Hkv, d] in the caches [pages, Hkv, page_size, d]: row t goes to slot
    slots[t] % page_size of page slots[t] // page_size; rows with a negative slot are skipped."""
    dtype, code = k.dtype, _type_code("k", k)
    _need_dims("k", k, 3)
    _need_dims("k_cache", k_cache, 4)
    rows, heads, d = k.shape
    pages, _, page_size, _ = k_cache.shape
    if k.stride()[2] != 1 and k.numel() > 0:
        _refuse("k", k, dtype, k.shape)
    if not _is_rows(v, dtype, (rows, heads, d)):
        _refuse("v", v, dtype, (rows, heads, d))
    if not _is_ints(slots, (rows,)):
        _refuse("slots", slots, _INT32, (rows,))
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not _is_rows(t, dtype, (pages, heads, page_size, d)):
            _refuse(name, t, dtype, (pages, heads, page_size, d))
    kr, kh, _ = k.stride()
    vr, vh, _ = v.stride()
    kp, kch, ks, _ = k_cache.stride()
    vp, vch, vs, _ = v_cache.stride()
    _guarded(_attn_pages_write, _device(k, v, slots, k_cache, v_cache), stream, _WRITE.pack(
        rows, heads, d, pages, page_size, code, 0, 0, k.data_ptr(), v.data_ptr(), slots.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), kr, kh, vr, vh, kp, kch, ks, vp, vch, vs))


def _check_tables(name: str, first: torch.Tensor, kv_len: torch.Tensor, block_table: torch.Tensor,
                  free_pages: torch.Tensor, free_count: torch.Tensor) -> int:
    """The checks that plan and release share; `first` has an entry per sequence. Returns the number of
    sequences."""
    _need_dims(name, first, 1)
    _need_dims("block_table", block_table, 2)
    n = first.shape[0]
    if not (_is_ints(first, (n,)) and _is_ints(kv_len, (n,)) and _is_ints(block_table, (n, block_table.shape[1]))
            and _is_ints(free_pages, (free_pages.numel(),)) and _is_ints(free_count, (1,))):
        for what, t, shape in ((name, first, (n,)), ("kv_len", kv_len, (n,)), ("block_table", block_table, (n, block_table.shape[1])),
                               ("free_pages", free_pages, (free_pages.numel(),)), ("free_count", free_count, (1,))):
            if not _is_ints(t, shape):
                _refuse(what, t, _INT32, shape)
    return n


def _attn_pages_plan(dev, q_len, kv_len, block_table, free_pages, free_count, page_size, total_q, outs):
    n, columns = block_table.shape
    where = q_len.device
    outs = cu_q, new_len, slots, positions, free_left = [
        torch.empty(m, dtype=_INT32, device=where) if t is None else t
        for t, m in zip(outs, (n + 1, n, total_q, total_q, 1))]
    _launch(lib.attn_pages_plan, dev, _PLAN.pack(
        n, total_q, page_size, columns, free_pages.shape[0], 0, q_len.data_ptr(), kv_len.data_ptr(),
        block_table.data_ptr(), block_table.stride(0) if n > 1 else columns, free_pages.data_ptr(),
        free_count.data_ptr(), cu_q.data_ptr(), new_len.data_ptr(), slots.data_ptr(), positions.data_ptr(),
        free_left.data_ptr()))
    return tuple(outs)


def attn_pages_plan(q_len: torch.Tensor, kv_len: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                    free_count: torch.Tensor, page_size: int, total_q: int, *, cu_q: Optional[torch.Tensor] = None,
                    new_len: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None,
                    positions: Optional[torch.Tensor] = None, free_left: Optional[torch.Tensor] = None,
                    stream=None) -> Tuple[torch.Tensor, ...]:
    """Tables of one step, from the sequences' new (q_len [B]) and cached (kv_len [B]) tokens.

    Takes the pages that the new tokens open from the top of the stack free_pages[:free_count[0]] and
    enters them in block_table [B, columns], in place. Returns (cu_q [B + 1], new_len [B], slots
    [total_q], positions [total_q], free_left [1]); total_q is the number of query rows, padding
    included, whose slots and positions are -1. All int32 on the GPU. new_len and free_left are the
    next call's kv_len and free_count. free_left < 0: pages were missing."""
    n = _check_tables("q_len", q_len, kv_len, block_table, free_pages, free_count)
    if total_q < 0:
        raise ValueError(f"total_q must not be negative, got {total_q}")
    outs, given = (cu_q, new_len, slots, positions, free_left), []
    for name, t, m in zip(("cu_q", "new_len", "slots", "positions", "free_left"), outs, (n + 1, n, total_q, total_q, 1)):
        if t is not None:
            if not _is_ints(t, (m,)):
                _refuse(name, t, _INT32, (m,))
            given.append(t)
    return _guarded(_attn_pages_plan, _device(q_len, kv_len, block_table, free_pages, free_count, *given), stream, q_len,
                    kv_len, block_table, free_pages, free_count, page_size, total_q, outs)


def _attn_pages_release(dev, done, kv_len, block_table, free_pages, free_count, page_size, new_len, free_left):
    n, columns = block_table.shape
    if new_len is None:
        new_len = torch.empty(n, dtype=_INT32, device=done.device)
    if free_left is None:
        free_left = torch.empty(1, dtype=_INT32, device=done.device)
    _launch(lib.attn_pages_release, dev, _RELEASE.pack(
        n, page_size, columns, free_pages.shape[0], done.data_ptr(), kv_len.data_ptr(), block_table.data_ptr(),
        block_table.stride(0) if n > 1 else columns, free_pages.data_ptr(), free_count.data_ptr(), new_len.data_ptr(),
        free_left.data_ptr()))
    return new_len, free_left


def attn_pages_release(done: torch.Tensor, kv_len: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                       free_count: torch.Tensor, page_size: int, *, new_len: Optional[torch.Tensor] = None,
                       free_left: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Push the pages of the sequences with done[b] != 0 onto the stack free_pages, in place from
    free_count[0] on. Returns (new_len [B], free_left [1]): new_len is 0 for those sequences and kv_len
    for the others. All int32 on the GPU."""
    n = _check_tables("done", done, kv_len, block_table, free_pages, free_count)
    given = []
    for name, t, m in (("new_len", new_len, n), ("free_left", free_left, 1)):
        if t is not None:
            if not _is_ints(t, (m,)):
                _refuse(name, t, _INT32, (m,))
            given.append(t)
    return _guarded(_attn_pages_release, _device(done, kv_len, block_table, free_pages, free_count, *given), stream, done,
                    kv_len, block_table, free_pages, free_count, page_size, new_len, free_left)
