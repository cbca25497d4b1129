"""The paged key/value cache's entry points (include/attn.h): argument checks and marshalling.

Shapes, types and devices are checked here (the C ABI sees pointers and sizes only); everything
else is checked by the library, on the host where it can be seen there and in the kernels for the
lengths, pages and slots that live on the device (attn_status reports those).
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

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


for _name, _params in (("attn_paged", PagedParams), ("attn_pages_write", PagesWriteParams),
                       ("attn_pages_plan", PagesPlanParams), ("attn_pages_release", PagesReleaseParams)):
    _entry = getattr(lib, _name)
    _entry.argtypes = [ctypes.POINTER(_params), ctypes.c_void_p]
    _entry.restype = ctypes.c_int
lib.attn_paged_workspace_size.argtypes = [ctypes.POINTER(PagedParams)]
lib.attn_paged_workspace_size.restype = ctypes.c_size_t


def _shape(name: str, t: torch.Tensor, *want: int) -> None:
    """want: one extent per dimension, -1 for any."""
    if t.dim() != len(want) or any(w >= 0 and s != w for s, w in zip(t.shape, want)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected "
                         f"[{', '.join('any' if w < 0 else str(w) for w in want)}]")


def _ints(name: str, t: torch.Tensor, *want: int) -> None:
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32, got {t.dtype}")
    _shape(name, t, *want)
    if t.numel() > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")


def _vectors(name: str, t: torch.Tensor, dtype: torch.dtype, *want: int) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    _shape(name, t, *want)
    if t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")


def _device(first: torch.Tensor, *others: torch.Tensor) -> torch.device:
    dev = first.device
    for t in others:
        if t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device} in one call")
    if dev.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, got {dev}")
    return dev


def _caches(k_cache: torch.Tensor, v_cache: torch.Tensor, dtype: torch.dtype, heads: int, d: int) -> None:
    _vectors("k_cache", k_cache, dtype, -1, heads, -1, d)
    _vectors("v_cache", v_cache, dtype, k_cache.shape[0], heads, k_cache.shape[2], d)


class _Launch:
    """Runs a call on `stream` (default: the current stream of the tensors' device) with that stream
    and its device current, so that what the call allocates belongs to the stream that uses it."""

    def __init__(self, dev: torch.device, stream):
        self.dev, self.stream = dev, stream
        if stream is not None:
            if stream.device != dev:
                raise ValueError(f"stream of {stream.device} given for tensors on {dev}")
            self.guard = torch.cuda.stream(stream)
        elif dev.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(dev)
        else:
            self.guard = None

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        if self.stream is None:
            self.stream = torch.cuda.current_stream()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def empty(self, shape, dtype: torch.dtype) -> torch.Tensor:
        return torch.empty(shape, dtype=dtype, device=self.dev)

    def call(self, entry, params) -> None:
        _check(entry(ctypes.byref(params), ctypes.c_void_p(self.stream.cuda_stream)))


def paged_params(q, k_cache, v_cache, block_table, cu_q, kv_len, out, lse, scale: float, causal: bool,
                 max_q: int) -> PagedParams:
    """Fill attn_paged_params; out and lse may be None (attn_paged_workspace_size reads sizes only)."""
    total_q, hq, d = q.shape
    o = q if out is None else out
    qs, os_, ks, vs = q.stride(), o.stride(), k_cache.stride(), v_cache.stride()
    return PagedParams(
        block_table.shape[0], hq, k_cache.shape[1], d, total_q, max_q, k_cache.shape[0], k_cache.shape[2],
        block_table.shape[1], _dtype_code(q.dtype), 1 if causal else 0, scale, _i32x2(0, 0),
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), o.data_ptr(), q.data_ptr() if lse is None else lse.data_ptr(),
        cu_q.data_ptr(), kv_len.data_ptr(), block_table.data_ptr(), block_table.stride(0) if block_table.shape[0] > 1 else 0,
        _i64x2(qs[0], qs[1]), _i64x2(os_[0], os_[1]), _i64x3(*ks[:3]), _i64x3(*vs[:3]), None, 0)


def _default_max_q(total_q: int, num_seqs: int) -> int:
    # the longest chunk if every sequence brings at least one row
    return max(1, total_q - num_seqs + 1)


def paged_workspace_size(q, k_cache, v_cache, block_table, cu_q, kv_len, *, max_q: Optional[int] = None) -> int:
    """Bytes of workspace attn_paged needs for these shapes."""
    if max_q is None:
        max_q = _default_max_q(q.shape[0], block_table.shape[0])
    return int(lib.attn_paged_workspace_size(ctypes.byref(
        paged_params(q, k_cache, v_cache, block_table, cu_q, kv_len, None, None, 1.0, False, max_q))))


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
    _vectors("q", q, q.dtype, -1, -1, -1)
    total_q, hq, d = q.shape
    _dtype_code(q.dtype)
    _caches(k_cache, v_cache, q.dtype, -1, d)
    if v_cache.shape[1] != k_cache.shape[1]:
        raise ValueError(f"k_cache has {k_cache.shape[1]} heads, v_cache {v_cache.shape[1]}")
    _ints("block_table", block_table, -1, -1)
    num_seqs = block_table.shape[0]
    _ints("cu_q", cu_q, num_seqs + 1)
    _ints("kv_len", kv_len, num_seqs)
    if out is not None:
        _vectors("out", out, q.dtype, total_q, hq, d)
    if lse is not None:
        _vectors("lse", lse, torch.float32, hq, total_q)
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    dev = _device(q, k_cache, v_cache, block_table, cu_q, kv_len, *(t for t in (out, lse, workspace) if t is not None))
    if max_q is None:
        max_q = _default_max_q(total_q, num_seqs)
    with _Launch(dev, stream) as at:
        if out is None:
            out = at.empty((total_q, hq, d), q.dtype)
        if lse is None:
            lse = at.empty((hq, total_q), torch.float32)
        p = paged_params(q, k_cache, v_cache, block_table, cu_q, kv_len, out, lse,
                         1.0 / math.sqrt(d) if scale is None else float(scale), causal, int(max_q))
        if workspace is None:
            workspace = at.empty((max(int(lib.attn_paged_workspace_size(ctypes.byref(p))), 1),), torch.uint8)
        p.workspace, p.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        at.call(lib.attn_paged, p)
    return out, lse


def attn_pages_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
                     v_cache: torch.Tensor, *, stream=None) -> None:
    """Store k, v [rows, Hkv, d] in the caches [pages, Hkv, page_size, d]: row t goes to slot
    slots[t] % page_size of page slots[t] // page_size; rows with a negative slot are skipped."""
    _vectors("k", k, k.dtype, -1, -1, -1)
    rows, heads, d = k.shape
    dtype = _dtype_code(k.dtype)
    _vectors("v", v, k.dtype, rows, heads, d)
    _ints("slots", slots, rows)
    _caches(k_cache, v_cache, k.dtype, heads, d)
    dev = _device(k, v, slots, k_cache, v_cache)
    ks, vs = k.stride(), v.stride()
    p = PagesWriteParams(rows, heads, d, k_cache.shape[0], k_cache.shape[2], dtype, _i32x2(0, 0),
                         k.data_ptr(), v.data_ptr(), slots.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                         _i64x2(ks[0], ks[1]), _i64x2(vs[0], vs[1]), _i64x3(*k_cache.stride()[:3]),
                         _i64x3(*v_cache.stride()[:3]))
    with _Launch(dev, stream) as at:
        at.call(lib.attn_pages_write, p)


def _table(block_table: torch.Tensor, num_seqs: int) -> int:
    """Checks the block table and returns its row stride."""
    _ints("block_table", block_table, num_seqs, -1)
    return block_table.stride(0) if num_seqs > 1 else block_table.shape[1]


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
    num_seqs = q_len.shape[0] if q_len.dim() == 1 else -1
    _ints("q_len", q_len, -1)
    _ints("kv_len", kv_len, num_seqs)
    table_stride = _table(block_table, num_seqs)
    _ints("free_pages", free_pages, -1)
    _ints("free_count", free_count, 1)
    outs = {"cu_q": (cu_q, num_seqs + 1), "new_len": (new_len, num_seqs), "slots": (slots, total_q),
            "positions": (positions, total_q), "free_left": (free_left, 1)}
    given = []
    for name, (t, n) in outs.items():
        if t is not None:
            _ints(name, t, n)
            given.append(t)
    dev = _device(q_len, kv_len, block_table, free_pages, free_count, *given)
    with _Launch(dev, stream) as at:
        if not given:  # one allocation for all: a step's tables are small
            whole = at.empty((2 * num_seqs + 2 + 2 * total_q,), torch.int32)
            outs = whole.split((num_seqs + 1, num_seqs, total_q, total_q, 1))
        else:
            outs = tuple(at.empty((n,), torch.int32) if t is None else t for t, n in outs.values())
        cu_q, new_len, slots, positions, free_left = outs
        at.call(lib.attn_pages_plan, PagesPlanParams(
            num_seqs, total_q, page_size, block_table.shape[1], free_pages.shape[0], 0, q_len.data_ptr(),
            kv_len.data_ptr(), block_table.data_ptr(), table_stride, free_pages.data_ptr(), free_count.data_ptr(),
            cu_q.data_ptr(), new_len.data_ptr(), slots.data_ptr(), positions.data_ptr(), free_left.data_ptr()))
    return outs


def attn_pages_release(done: torch.Tensor, kv_len: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                       free_count: torch.Tensor, page_size: int, *, new_len: Optional[torch.Tensor] = None,
                       free_left: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Push the pages of the sequences with done[b] != 0 onto the stack free_pages, in place from
    free_count[0] on. Returns (new_len [B], free_left [1]): new_len is 0 for those sequences and kv_len
    for the others. All int32 on the GPU."""
    num_seqs = done.shape[0] if done.dim() == 1 else -1
    _ints("done", done, -1)
    _ints("kv_len", kv_len, num_seqs)
    table_stride = _table(block_table, num_seqs)
    _ints("free_pages", free_pages, -1)
    _ints("free_count", free_count, 1)
    if new_len is not None:
        _ints("new_len", new_len, num_seqs)
    if free_left is not None:
        _ints("free_left", free_left, 1)
    dev = _device(done, kv_len, block_table, free_pages, free_count, *(t for t in (new_len, free_left) if t is not None))
    with _Launch(dev, stream) as at:
        new_len = at.empty((num_seqs,), torch.int32) if new_len is None else new_len
        free_left = at.empty((1,), torch.int32) if free_left is None else free_left
        at.call(lib.attn_pages_release, PagesReleaseParams(
            num_seqs, page_size, block_table.shape[1], free_pages.shape[0], done.data_ptr(), kv_len.data_ptr(),
            block_table.data_ptr(), table_stride, free_pages.data_ptr(), free_count.data_ptr(), new_len.data_ptr(),
            free_left.data_ptr()))
    return new_len, free_left
