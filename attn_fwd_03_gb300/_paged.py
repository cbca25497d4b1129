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
_INT32_MAX = 2 ** 31 - 1
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


def _refuse_devices(*tensors: torch.Tensor) -> None:
    raise ValueError(f"tensors must be on one CUDA device, got {sorted({str(t.device) for t in tensors})}")


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


def _launch(entry, dev: int, packed: bytes) -> None:
    status = entry(packed, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        _check(status)


# The entry points below are written for the host time of a call that is all right: one condition over plain
# reads of the tensors, and a slower function that finds out what is wrong where it does not hold.

def _default_max_q(total_q: int, num_seqs: int) -> int:
    # the longest chunk if every sequence brings at least one row
    return max(1, total_q - num_seqs + 1)


def _as_int32(x) -> int:
    return min(max(int(x), -_INT32_MAX), _INT32_MAX)


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
    """Bytes of workspace attn_paged needs for these shapes on q's device."""
    _check_paged(q, k_cache, v_cache, block_table, cu_q, kv_len, None, None)
    max_q = _default_max_q(q.shape[0], block_table.shape[0]) if max_q is None else _as_int32(max_q)
    # out and lse are not read: q stands in for both
    packed = _pack_paged(q, k_cache, v_cache, block_table, cu_q, kv_len, q, q, 1.0, False, max_q, 0, 0)
    dev = q.get_device()
    guard = _guard(dev, None) if dev >= 0 else None  # the size goes by the current device's number of SMs
    if guard is None:
        return int(lib.attn_paged_workspace_size(packed))
    with guard:
        return int(lib.attn_paged_workspace_size(packed))


# (device, d, heads, key/value heads, max_q) -> bytes; all that the size depends on. No head group fits more
# than 128 rows in one tile, so it is the same for every max_q beyond, and the table stays small.
_workspace_bytes: Dict[tuple, int] = {}
# device -> workspace of calls on its default stream, which are in order and cannot be captured. An
# allocation costs a decode call about a third of its host time. Calls on other streams allocate: a
# stream's handle may come back for another stream, and a captured graph needs memory of its own.
_default_workspace: Dict[int, torch.Tensor] = {}


def _workspace(dev: int, nbytes: int) -> torch.Tensor:
    if torch._C._cuda_getCurrentRawStream(dev) != 0:
        return torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", dev))
    kept = _default_workspace.get(dev)
    if kept is None or kept.numel() < nbytes:
        kept = _default_workspace[dev] = torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", dev))
    return kept


def _check_paged(q, k_cache, v_cache, block_table, cu_q, kv_len, out, lse) -> None:
    _type_code("q", q)
    _need_dims("q", q, 3)
    _need_dims("k_cache", k_cache, 4)
    _need_dims("block_table", block_table, 2)
    (total_q, hq, d), (pages, hkv, page_size, _), num_seqs = q.shape, k_cache.shape, block_table.shape[0]
    for name, t, shape in (("q", q, (total_q, hq, d)), ("k_cache", k_cache, (pages, hkv, page_size, d)),
                           ("v_cache", v_cache, (pages, hkv, page_size, d)), ("out", out, (total_q, hq, d))):
        if t is not None and not _is_rows(t, q.dtype, shape):
            _refuse(name, t, q.dtype, shape)
    for name, t, shape in (("block_table", block_table, block_table.shape), ("cu_q", cu_q, (num_seqs + 1,)),
                           ("kv_len", kv_len, (num_seqs,))):
        if not _is_ints(t, shape):
            _refuse(name, t, _INT32, shape)
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (hq, total_q):
            _refuse("lse", lse, torch.float32, (hq, total_q))
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")


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

    max_q, the most rows that a sequence is expected to bring, only chooses the tile shape. out may be q
    itself. Without a workspace, calls on the device's default stream keep one for good (the largest
    that was needed, tens of MB), and others allocate one."""
    dtype = q.dtype
    if not (dtype in _TYPES and q.dim() == 3 and k_cache.dim() == 4 and block_table.dim() == 2 and q.stride()[2] == 1
            and k_cache.dtype is dtype and k_cache.shape[3] == q.shape[2] and k_cache.stride()[3] == 1
            and v_cache.dtype is dtype and v_cache.shape == k_cache.shape and v_cache.stride()[3] == 1
            and block_table.dtype is _INT32 and block_table.is_contiguous()
            and cu_q.dtype is _INT32 and cu_q.shape == (block_table.shape[0] + 1,) and cu_q.is_contiguous()
            and kv_len.dtype is _INT32 and kv_len.shape == (block_table.shape[0],) and kv_len.is_contiguous()
            and (out is None or (out.dtype is dtype and out.shape == q.shape and out.stride()[2] == 1))
            and (lse is None or (lse.dtype is torch.float32 and lse.shape == (q.shape[1], q.shape[0]) and lse.is_contiguous()))):
        _check_paged(q, k_cache, v_cache, block_table, cu_q, kv_len, out, lse)
    dev = q.get_device()
    if not (dev >= 0 and k_cache.get_device() == dev and v_cache.get_device() == dev and block_table.get_device() == dev
            and cu_q.get_device() == dev and kv_len.get_device() == dev and (out is None or out.get_device() == dev)
            and (lse is None or lse.get_device() == dev) and (workspace is None or workspace.get_device() == dev)):
        _refuse_devices(q, k_cache, v_cache, block_table, cu_q, kv_len, *(t for t in (out, lse, workspace) if t is not None))
    total_q, hq, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    max_q = _default_max_q(total_q, block_table.shape[0]) if max_q is None else _as_int32(max_q)
    guard = _guard(dev, stream)
    if guard is not None:
        guard.__enter__()
    try:
        where = q.device
        if out is None:
            out = torch.empty((total_q, hq, d), dtype=dtype, device=where)
        if lse is None:
            lse = torch.empty((hq, total_q), dtype=torch.float32, device=where)
        if workspace is None:
            key = (dev, d, hq, k_cache.shape[1], max_q if max_q < 129 else 129)
            nbytes = _workspace_bytes.get(key)
            if nbytes is None:
                nbytes = paged_workspace_size(q, k_cache, v_cache, block_table, cu_q, kv_len, max_q=max_q)
                if nbytes > 0:  # 0: nothing to do, or a call that will be refused
                    _workspace_bytes[key] = nbytes
            workspace = _workspace(dev, max(nbytes, 1))
        elif workspace.is_contiguous():
            nbytes = workspace.numel() * workspace.element_size()
        else:
            raise ValueError("workspace must be contiguous")
        _launch(lib.attn_paged, dev, _pack_paged(q, k_cache, v_cache, block_table, cu_q, kv_len, out, lse, scale, causal,
                                                 max_q, workspace.data_ptr(), nbytes))
    finally:
        if guard is not None:
            guard.__exit__(None, None, None)
    return out, lse


def _check_write(k, v, slots, k_cache, v_cache) -> None:
    _type_code("k", k)
    _need_dims("k", k, 3)
    _need_dims("k_cache", k_cache, 4)
    (rows, heads, d), (pages, _, page_size, _) = k.shape, k_cache.shape
    for name, t, shape in (("k", k, (rows, heads, d)), ("v", v, (rows, heads, d)),
                           ("k_cache", k_cache, (pages, heads, page_size, d)),
                           ("v_cache", v_cache, (pages, heads, page_size, d))):
        if not _is_rows(t, k.dtype, shape):
            _refuse(name, t, k.dtype, shape)
    if not _is_ints(slots, (rows,)):
        _refuse("slots", slots, _INT32, (rows,))


def attn_pages_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
                     v_cache: torch.Tensor, *, stream=None) -> None:
    """Store k, v [rows, Hkv, d] in the caches [pages, Hkv, page_size, d]: row t goes to slot
    slots[t] % page_size of page slots[t] // page_size; rows with a negative slot are skipped."""
    dtype = k.dtype
    if not (dtype in _TYPES and k.dim() == 3 and k_cache.dim() == 4 and k.stride()[2] == 1
            and v.dtype is dtype and v.shape == k.shape and v.stride()[2] == 1
            and k_cache.dtype is dtype and k_cache.shape[1] == k.shape[1] and k_cache.shape[3] == k.shape[2]
            and k_cache.stride()[3] == 1 and v_cache.dtype is dtype and v_cache.shape == k_cache.shape
            and v_cache.stride()[3] == 1
            and slots.dtype is _INT32 and slots.shape == (k.shape[0],) and slots.is_contiguous()):
        _check_write(k, v, slots, k_cache, v_cache)
    dev = k.get_device()
    if not (dev >= 0 and v.get_device() == dev and slots.get_device() == dev and k_cache.get_device() == dev
            and v_cache.get_device() == dev):
        _refuse_devices(k, v, slots, k_cache, v_cache)
    rows, heads, d = k.shape
    pages, _, page_size, _ = k_cache.shape
    kr, kh, _ = k.stride()
    vr, vh, _ = v.stride()
    kp, kch, ks, _ = k_cache.stride()
    vp, vch, vs, _ = v_cache.stride()
    packed = _WRITE.pack(rows, heads, d, pages, page_size, _TYPES[dtype], 0, 0, k.data_ptr(), v.data_ptr(), slots.data_ptr(),
                         k_cache.data_ptr(), v_cache.data_ptr(), kr, kh, vr, vh, kp, kch, ks, vp, vch, vs)
    guard = _guard(dev, stream)
    if guard is None:
        _launch(lib.attn_pages_write, dev, packed)
    else:
        with guard:
            _launch(lib.attn_pages_write, dev, packed)


def _check_tables(name, first, kv_len, block_table, free_pages, free_count) -> int:
    """The checks that plan and release share; `first` has an entry per sequence. Returns the device."""
    shape, dev = first.shape, first.get_device()
    if not (first.dtype is _INT32 and first.dim() == 1 and first.is_contiguous()
            and kv_len.dtype is _INT32 and kv_len.shape == shape and kv_len.is_contiguous()
            and block_table.dtype is _INT32 and block_table.dim() == 2 and block_table.shape[0] == shape[0]
            and block_table.is_contiguous() and free_pages.dtype is _INT32 and free_pages.dim() == 1
            and free_pages.is_contiguous() and free_count.dtype is _INT32 and free_count.shape == (1,)
            and dev >= 0 and kv_len.get_device() == dev and block_table.get_device() == dev
            and free_pages.get_device() == dev and free_count.get_device() == dev):
        _need_dims(name, first, 1)
        _need_dims("block_table", block_table, 2)
        n = shape[0]
        for what, t, want in ((name, first, (n,)), ("kv_len", kv_len, (n,)), ("block_table", block_table, (n, block_table.shape[1])),
                              ("free_pages", free_pages, (free_pages.numel(),)), ("free_count", free_count, (1,))):
            if not _is_ints(t, want):
                _refuse(what, t, _INT32, want)
        if dev < 0 or any(t.get_device() != dev for t in (kv_len, block_table, free_pages, free_count)):
            _refuse_devices(first, kv_len, block_table, free_pages, free_count)
    return dev


def _page_size(page_size) -> int:
    """As the C ABI's int32; the library checks the rest."""
    if not 0 < page_size <= _INT32_MAX or int(page_size) != page_size:
        raise ValueError(f"page_size must be a positive 32-bit integer, got {page_size}")
    return int(page_size)


def _given(name: str, t: torch.Tensor, n: int, like: torch.Tensor) -> torch.Tensor:
    """Checks an output of n entries that the caller brought."""
    if not _is_ints(t, (n,)):
        _refuse(name, t, _INT32, (n,))
    if t.get_device() != like.get_device():
        _refuse_devices(like, t)
    return t


def _plan_call(dev, q_len, kv_len, block_table, free_pages, free_count, page_size, total_q, cu_q, new_len, slots, positions,
               free_left):
    n, columns = block_table.shape
    empty, where = torch.empty, q_len.device
    cu_q = empty(n + 1, dtype=_INT32, device=where) if cu_q is None else _given("cu_q", cu_q, n + 1, q_len)
    new_len = empty(n, dtype=_INT32, device=where) if new_len is None else _given("new_len", new_len, n, q_len)
    slots = empty(total_q, dtype=_INT32, device=where) if slots is None else _given("slots", slots, total_q, q_len)
    positions = (empty(total_q, dtype=_INT32, device=where) if positions is None
                 else _given("positions", positions, total_q, q_len))
    free_left = empty(1, dtype=_INT32, device=where) if free_left is None else _given("free_left", free_left, 1, q_len)
    _launch(lib.attn_pages_plan, dev, _PLAN.pack(
        n, total_q, page_size, columns, free_pages.numel(), 0, q_len.data_ptr(), kv_len.data_ptr(), block_table.data_ptr(),
        block_table.stride()[0] if n > 1 else columns, free_pages.data_ptr(), free_count.data_ptr(), cu_q.data_ptr(),
        new_len.data_ptr(), slots.data_ptr(), positions.data_ptr(), free_left.data_ptr()))
    return cu_q, new_len, slots, positions, free_left


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
    dev = _check_tables("q_len", q_len, kv_len, block_table, free_pages, free_count)
    if not 0 <= total_q <= _INT32_MAX:
        raise ValueError(f"total_q must be a 32-bit integer that is not negative, got {total_q}")
    page_size = _page_size(page_size)
    guard = _guard(dev, stream)
    if guard is None:
        return _plan_call(dev, q_len, kv_len, block_table, free_pages, free_count, page_size, total_q, cu_q, new_len, slots,
                          positions, free_left)
    with guard:
        return _plan_call(dev, q_len, kv_len, block_table, free_pages, free_count, page_size, total_q, cu_q, new_len, slots,
                          positions, free_left)


def _release_call(dev, done, kv_len, block_table, free_pages, free_count, page_size, new_len, free_left):
    n, columns = block_table.shape
    new_len = (torch.empty(n, dtype=_INT32, device=done.device) if new_len is None
               else _given("new_len", new_len, n, done))
    free_left = (torch.empty(1, dtype=_INT32, device=done.device) if free_left is None
                 else _given("free_left", free_left, 1, done))
    _launch(lib.attn_pages_release, dev, _RELEASE.pack(
        n, page_size, columns, free_pages.numel(), done.data_ptr(), kv_len.data_ptr(), block_table.data_ptr(),
        block_table.stride()[0] if n > 1 else columns, free_pages.data_ptr(), free_count.data_ptr(), new_len.data_ptr(),
        free_left.data_ptr()))
    return new_len, free_left


def attn_pages_release(done: torch.Tensor, kv_len: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                       free_count: torch.Tensor, page_size: int, *, new_len: Optional[torch.Tensor] = None,
                       free_left: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Push the pages of the sequences with done[b] != 0 onto the stack free_pages, in place from
    free_count[0] on. Returns (new_len [B], free_left [1]): new_len is 0 for those sequences and kv_len
    for the others. All int32 on the GPU."""
    dev = _check_tables("done", done, kv_len, block_table, free_pages, free_count)
    page_size = _page_size(page_size)
    guard = _guard(dev, stream)
    if guard is None:
        return _release_call(dev, done, kv_len, block_table, free_pages, free_count, page_size, new_len, free_left)
    with guard:
        return _release_call(dev, done, kv_len, block_table, free_pages, free_count, page_size, new_len, free_left)
