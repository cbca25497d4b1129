"""The 8-bit paged cache and trees of drafted tokens (include/attn.h): argument checks and marshalling.

As in _paged.py, shapes, types and devices are checked here and everything else by the library.
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import Dict, Optional, Tuple

import torch

from ._binding import lib
from ._paged import (_INT32, _PAGED, _TYPES, PagedParams, _as_int32, _default_max_q, _given, _guard, _i32x2, _i64x2, _i64x3, _is_ints,
                     _is_rows, _launch, _need_dims, _packer, _refuse, _refuse_devices, _type_code, _workspace, _workspace_bytes,
                     paged_workspace_size)


class PagesFp8Params(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("d", ctypes.c_int32),
        ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("reserved0", _i32x2),
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("slots", ctypes.c_void_p),
        ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("k_row_stride", _i64x2), ("v_row_stride", _i64x2), ("k_stride", _i64x3), ("v_stride", _i64x3),
        ("k_scale_stride", _i64x2), ("v_scale_stride", _i64x2),
    ]


class TreePlanParams(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32), ("total_q", ctypes.c_int32), ("words", ctypes.c_int32), ("reserved0", ctypes.c_int32),
        ("parents", ctypes.c_void_p), ("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("mask", ctypes.c_void_p),
        ("mask_stride", ctypes.c_int64), ("positions", ctypes.c_void_p),
    ]


class PagedTreeParams(ctypes.Structure):
    _fields_ = [
        ("f", PagedParams), ("mask", ctypes.c_void_p), ("mask_stride", ctypes.c_int64), ("words", ctypes.c_int32),
        ("reserved1", ctypes.c_int32),
    ]


class PagedFp8Params(ctypes.Structure):
    _fields_ = [
        ("t", PagedTreeParams), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("k_scale_stride", _i64x2), ("v_scale_stride", _i64x2),
    ]


_PAGES_FP8, _TREE_PLAN = _packer(PagesFp8Params), _packer(TreePlanParams)
# what PagedTreeParams adds behind its first field, and PagedFp8Params behind that
_TREE, _SCALES = struct.Struct("@Pqii"), struct.Struct("@PPqqqq")
assert _PAGED.size + _TREE.size == ctypes.sizeof(PagedTreeParams)
assert ctypes.sizeof(PagedTreeParams) + _SCALES.size == ctypes.sizeof(PagedFp8Params)

for _entry in (lib.attn_pages_write_fp8, lib.attn_pages_read_fp8, lib.attn_tree_plan, lib.attn_paged_tree, lib.attn_paged_fp8):
    _entry.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    _entry.restype = ctypes.c_int
lib.attn_paged_fp8_workspace_size.argtypes = [ctypes.c_void_p]
lib.attn_paged_fp8_workspace_size.restype = ctypes.c_size_t

_CODES = (torch.float8_e4m3fn, torch.uint8)
_SCALE_BYTES = (torch.float8_e8m0fnu, torch.uint8)


def _check_codes(name: str, t: torch.Tensor, shape: tuple) -> None:
    if t.dtype not in _CODES:
        raise TypeError(f"{name} must be float8_e4m3fn (or uint8 that holds the codes), got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.stride()[-1] != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")


def _check_scale(name: str, t: torch.Tensor, shape: tuple) -> None:
    if t.dtype not in _SCALE_BYTES:
        raise TypeError(f"{name} must be float8_e8m0fnu (or uint8 that holds exponents + 127), got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.stride()[-1] != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")


def _is_cache(k_cache, v_cache, k_scale, v_scale) -> bool:
    """Whether four tensors are the codes and scales of one cache."""
    shape = k_cache.shape
    return (k_cache.dtype in _CODES and v_cache.dtype in _CODES and k_scale.dtype in _SCALE_BYTES and v_scale.dtype in _SCALE_BYTES
            and len(shape) == 4 and v_cache.shape == shape and k_scale.shape == shape[:3] and v_scale.shape == shape[:3]
            and k_cache.stride()[3] == 1 and v_cache.stride()[3] == 1 and k_scale.stride()[2] == 1 and v_scale.stride()[2] == 1)


def _check_cache(k_cache, v_cache, k_scale, v_scale) -> None:
    _need_dims("k_cache", k_cache, 4)
    shape = k_cache.shape
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _check_codes(name, t, shape)
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        _check_scale(name, t, shape[:3])


# ---------------------------------------------------------------- writes and reads
def _pages_call(entry, k, v, slots, k_cache, v_cache, k_scale, v_scale, stream) -> None:
    # shapes and strides are read once, for the checks and for the struct
    dtype, shape, pages = k.dtype, k.shape, k_cache.shape
    good = len(shape) == 3 and len(pages) == 4 and v.shape == shape and v_cache.shape == pages
    if good:
        rows, heads, d = shape
        num_pages, _, page_size, _ = pages
        kr, kh, ke = k.stride()
        vr, vh, ve = v.stride()
        kp, kch, ks, kce = k_cache.stride()
        vp, vch, vs, vce = v_cache.stride()
        good = (dtype in _TYPES and v.dtype is dtype and k_cache.dtype in _CODES and v_cache.dtype in _CODES
                and k_scale.dtype in _SCALE_BYTES and v_scale.dtype in _SCALE_BYTES and slots.dtype is _INT32
                and ke == 1 and ve == 1 and kce == 1 and vce == 1 and pages[1] == heads and pages[3] == d
                and k_scale.shape == pages[:3] and v_scale.shape == pages[:3] and slots.shape == shape[:1] and slots.is_contiguous())
        if good:
            ksp, ksh, kse = k_scale.stride()
            vsp, vsh, vse = v_scale.stride()
            good = kse == 1 and vse == 1
    if not good:
        _type_code("k", k)
        _need_dims("k", k, 3)
        _need_dims("k_cache", k_cache, 4)
        (rows, heads, d), (num_pages, _, page_size, _) = k.shape, k_cache.shape
        for name, t in (("k", k), ("v", v)):
            if not _is_rows(t, dtype, (rows, heads, d)):
                _refuse(name, t, dtype, (rows, heads, d))
        for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
            _check_codes(name, t, (num_pages, heads, page_size, d))
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            _check_scale(name, t, (num_pages, heads, page_size))
        if not _is_ints(slots, (rows,)):
            _refuse("slots", slots, _INT32, (rows,))
        # empty rows, or strides over an extent of 1, which the conditions above are too strict for
        (kr, kh, _), (vr, vh, _), (kp, kch, ks, _), (vp, vch, vs, _) = k.stride(), v.stride(), k_cache.stride(), v_cache.stride()
        (ksp, ksh, _), (vsp, vsh, _) = k_scale.stride(), v_scale.stride()
    dev = k.get_device()
    if not (dev >= 0 and v.get_device() == dev and slots.get_device() == dev and k_cache.get_device() == dev
            and v_cache.get_device() == dev and k_scale.get_device() == dev and v_scale.get_device() == dev):
        _refuse_devices(k, v, slots, k_cache, v_cache, k_scale, v_scale)
    packed = _PAGES_FP8.pack(rows, heads, d, num_pages, page_size, _TYPES[dtype], 0, 0, k.data_ptr(), v.data_ptr(), slots.data_ptr(),
                             k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), kr, kh, vr, vh, kp, kch, ks,
                             vp, vch, vs, ksp, ksh, vsp, vsh)
    guard = _guard(dev, stream)
    if guard is None:
        _launch(entry, dev, packed)
    else:
        with guard:
            _launch(entry, dev, packed)


def attn_pages_write_fp8(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                         k_scale: torch.Tensor, v_scale: torch.Tensor, *, stream=None) -> None:
    """Store k, v [rows, Hkv, d] in 8 bits: codes in the caches [pages, Hkv, page_size, d] (float8_e4m3fn),
    a power of two for each token and head in the scales [pages, Hkv, page_size] (float8_e8m0fnu, the slots
    contiguous). Row t goes to slot slots[t] % page_size of page slots[t] // page_size; rows with a
    negative slot are skipped. uint8 tensors may stand for either 8-bit type."""
    _pages_call(lib.attn_pages_write_fp8, k, v, slots, k_cache, v_cache, k_scale, v_scale, stream)


def attn_pages_read_fp8(slots: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                        v_scale: torch.Tensor, *, dtype: torch.dtype = torch.bfloat16, k: Optional[torch.Tensor] = None,
                        v: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The keys and values of the given slots [rows] as 16-bit rows (k, v) [rows, Hkv, d], of the type of a given k
    or v, or `dtype`. Rows with a negative slot are left as they are (zeros in tensors allocated here)."""
    if k is None or v is None:
        _need_dims("k_cache", k_cache, 4)
        _need_dims("slots", slots, 1)
        like = k if k is not None else v
        dtype = dtype if like is None else like.dtype
        if dtype not in _TYPES:
            raise TypeError(f"k and v must be bfloat16 or float16, got {dtype}")
        if slots.get_device() < 0:
            _refuse_devices(slots)
        guard = _guard(slots.get_device(), stream)
        if guard is not None:
            guard.__enter__()
        try:
            shape = (slots.shape[0], k_cache.shape[1], k_cache.shape[3])
            k = torch.zeros(shape, dtype=dtype, device=slots.device) if k is None else k
            v = torch.zeros(shape, dtype=dtype, device=slots.device) if v is None else v
        finally:
            if guard is not None:
                guard.__exit__(None, None, None)
    _pages_call(lib.attn_pages_read_fp8, k, v, slots, k_cache, v_cache, k_scale, v_scale, stream)
    return k, v


# ---------------------------------------------------------------- trees
def attn_tree_plan(parents: torch.Tensor, cu_q: torch.Tensor, kv_len: torch.Tensor, max_nodes: int, *,
                   mask: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                   stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Who sees whom in trees of up to max_nodes (at most 1024) drafted tokens, and where they stand.

    parents [rows]: of each node, the number within its sequence of the node it follows, which is below its
    own, or -1 for the context; cu_q [B + 1], kv_len [B] as attn_paged takes them. Returns (mask [rows,
    words], positions [rows]), int32 like the inputs: bit c % 32 of word c // 32 says that a row sees node c.
    Sequences with more rows than the mask has bits are chunks of a prompt: their words are 0, their
    positions consecutive. Rows behind the last sequence get words 0 and position -1."""
    if not 1 <= max_nodes <= 1024 or int(max_nodes) != max_nodes:
        raise ValueError(f"max_nodes must be 1 to 1024, got {max_nodes}")
    words = (int(max_nodes) + 31) // 32
    dev, shape, seqs = parents.get_device(), parents.shape, kv_len.shape
    if not (parents.dtype is _INT32 and cu_q.dtype is _INT32 and kv_len.dtype is _INT32 and len(shape) == 1 and len(seqs) == 1
            and cu_q.shape == (seqs[0] + 1,) and parents.is_contiguous() and cu_q.is_contiguous() and kv_len.is_contiguous()
            and dev >= 0 and cu_q.get_device() == dev and kv_len.get_device() == dev):
        _need_dims("parents", parents, 1)
        _need_dims("kv_len", kv_len, 1)
        n = seqs[0]
        for name, t, want in (("parents", parents, shape), ("cu_q", cu_q, (n + 1,)), ("kv_len", kv_len, (n,))):
            if not _is_ints(t, want):
                _refuse(name, t, _INT32, want)
        if dev < 0 or cu_q.get_device() != dev or kv_len.get_device() != dev:
            _refuse_devices(parents, cu_q, kv_len)
    guard = _guard(dev, stream)
    if guard is None:
        return _tree_call(dev, shape[0], seqs[0], words, parents, cu_q, kv_len, mask, positions)
    with guard:
        return _tree_call(dev, shape[0], seqs[0], words, parents, cu_q, kv_len, mask, positions)


def _tree_call(dev, rows, seqs, words, parents, cu_q, kv_len, mask, positions):
    stride = words
    if mask is None:
        mask = torch.empty((rows, words), dtype=_INT32, device=parents.device)
    else:
        if not _is_ints(mask, (rows, words)):
            _refuse("mask", mask, _INT32, (rows, words))
        if mask.get_device() != dev:
            _refuse_devices(parents, mask)
        if rows > 1:
            stride = mask.stride()[0]
    positions = torch.empty_like(parents) if positions is None else _given("positions", positions, rows, parents)
    _launch(lib.attn_tree_plan, dev, _TREE_PLAN.pack(seqs, rows, words, 0, parents.data_ptr(), cu_q.data_ptr(), kv_len.data_ptr(),
                                                     mask.data_ptr(), stride, positions.data_ptr()))
    return mask, positions


# ---------------------------------------------------------------- attention
def _check_attend(q, k_cache, v_cache, scales, block_table, cu_q, kv_len, tree, out, lse) -> None:
    """Says what is wrong with the tensors of a call, if anything is."""
    _type_code("q", q)
    _need_dims("q", q, 3)
    _need_dims("k_cache", k_cache, 4)
    _need_dims("block_table", block_table, 2)
    (total_q, hq, d), (pages, hkv, page_size, _), num_seqs = q.shape, k_cache.shape, block_table.shape[0]
    for name, t in (("q", q), ("out", out)):
        if t is not None and not _is_rows(t, q.dtype, (total_q, hq, d)):
            _refuse(name, t, q.dtype, (total_q, hq, d))
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if scales:
            _check_codes(name, t, (pages, hkv, page_size, d))
        elif not _is_rows(t, q.dtype, (pages, hkv, page_size, d)):
            _refuse(name, t, q.dtype, (pages, hkv, page_size, d))
    for name, t in zip(("k_scale", "v_scale"), scales):
        _check_scale(name, t, (pages, hkv, page_size))
    for name, t, shape in (("block_table", block_table, block_table.shape), ("cu_q", cu_q, (num_seqs + 1,)),
                           ("kv_len", kv_len, (num_seqs,))):
        if not _is_ints(t, shape):
            _refuse(name, t, _INT32, shape)
    if tree is not None:
        _need_dims("tree", tree, 2)
        if not _is_ints(tree, (total_q, tree.shape[1])):
            _refuse("tree", tree, _INT32, (total_q, tree.shape[1]))
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (hq, total_q):
            _refuse("lse", lse, torch.float32, (hq, total_q))
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")


def _pack(q, k_cache, v_cache, scales, block_table, cu_q, kv_len, tree, out, lse, scale, causal, max_q, workspace, nbytes) -> bytes:
    total_q, hq, d = q.shape
    num_seqs, columns = block_table.shape
    pages, hkv, page_size, _ = k_cache.shape
    qr, qh, _ = q.stride()
    orow, oh, _ = out.stride()
    kp, kh, ks, _ = k_cache.stride()
    vp, vh, vs, _ = v_cache.stride()
    packed = _PAGED.pack(num_seqs, hq, hkv, d, total_q, max_q, pages, page_size, columns, _TYPES[q.dtype],
                         1 if causal else 0, scale, 0, 0, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                         out.data_ptr(), lse.data_ptr(), cu_q.data_ptr(), kv_len.data_ptr(), block_table.data_ptr(),
                         block_table.stride(0), qr, qh, orow, oh, kp, kh, ks, vp, vh, vs, workspace, nbytes)
    if tree is not None:
        packed += _TREE.pack(tree.data_ptr(), tree.stride()[0], tree.shape[1], 0)
    else:
        packed += _TREE.pack(0, 0, 0, 0)
    if scales:
        k_scale, v_scale = scales
        ksp, ksh, _ = k_scale.stride()
        vsp, vsh, _ = v_scale.stride()
        packed += _SCALES.pack(k_scale.data_ptr(), v_scale.data_ptr(), ksp, ksh, vsp, vsh)
    return packed


def paged_fp8_workspace_size(q, k_cache, v_cache, k_scale, v_scale, block_table, cu_q, kv_len, *, tree=None,
                             max_q: Optional[int] = None) -> int:
    """Bytes of workspace attn_paged_fp8 needs for these shapes on q's device."""
    _check_attend(q, k_cache, v_cache, (k_scale, v_scale), block_table, cu_q, kv_len, tree, None, None)
    max_q = _default_max_q(q.shape[0], block_table.shape[0]) if max_q is None else _as_int32(max_q)
    # out and lse are not read: q stands in for both
    packed = _pack(q, k_cache, v_cache, (k_scale, v_scale), block_table, cu_q, kv_len, tree, q, q, 1.0, False, max_q, 0, 0)
    dev = q.get_device()
    guard = _guard(dev, None) if dev >= 0 else None
    if guard is None:
        return int(lib.attn_paged_fp8_workspace_size(packed))
    with guard:
        return int(lib.attn_paged_fp8_workspace_size(packed))


# as _paged._workspace_bytes, of attn_paged_fp8
_fp8_workspace_bytes: Dict[tuple, int] = {}


def _attend(q, k_cache, v_cache, scales, block_table, cu_q, kv_len, tree, scale, causal, max_q, out, lse, workspace, stream):
    dtype = q.dtype
    if not (dtype in _TYPES and q.dim() == 3 and k_cache.dim() == 4 and block_table.dim() == 2 and q.stride()[2] == 1
            and k_cache.shape[3] == q.shape[2]
            and (_is_cache(k_cache, v_cache, *scales) if scales else
                 (k_cache.dtype is dtype and k_cache.stride()[3] == 1 and v_cache.dtype is dtype and v_cache.shape == k_cache.shape
                  and v_cache.stride()[3] == 1))
            and block_table.dtype is _INT32 and block_table.is_contiguous()
            and cu_q.dtype is _INT32 and cu_q.shape == (block_table.shape[0] + 1,) and cu_q.is_contiguous()
            and kv_len.dtype is _INT32 and kv_len.shape == (block_table.shape[0],) and kv_len.is_contiguous()
            and (tree is None or (tree.dtype is _INT32 and tree.dim() == 2 and tree.shape[0] == q.shape[0] and tree.is_contiguous()))
            and (out is None or (out.dtype is dtype and out.shape == q.shape and out.stride()[2] == 1))
            and (lse is None or (lse.dtype is torch.float32 and lse.shape == (q.shape[1], q.shape[0]) and lse.is_contiguous()))):
        _check_attend(q, k_cache, v_cache, scales, block_table, cu_q, kv_len, tree, out, lse)
    dev = q.get_device()
    if not (dev >= 0 and k_cache.get_device() == dev and v_cache.get_device() == dev and block_table.get_device() == dev
            and cu_q.get_device() == dev and kv_len.get_device() == dev and (out is None or out.get_device() == dev)
            and (lse is None or lse.get_device() == dev) and (workspace is None or workspace.get_device() == dev)
            and (tree is None or tree.get_device() == dev) and all(t.get_device() == dev for t in scales)):
        _refuse_devices(q, k_cache, v_cache, block_table, cu_q, kv_len, *scales,
                        *(t for t in (tree, out, lse, workspace) if t is not None))
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
            known = _fp8_workspace_bytes if scales else _workspace_bytes
            nbytes = known.get(key)
            if nbytes is None:
                if scales:
                    nbytes = paged_fp8_workspace_size(q, k_cache, v_cache, *scales, block_table, cu_q, kv_len, max_q=max_q)
                else:
                    nbytes = paged_workspace_size(q, k_cache, v_cache, block_table, cu_q, kv_len, max_q=max_q)
                if nbytes > 0:  # 0: nothing to do, or a call that will be refused
                    known[key] = nbytes
            workspace = _workspace(dev, max(nbytes, 1))
        elif workspace.is_contiguous():
            nbytes = workspace.numel() * workspace.element_size()
        else:
            raise ValueError("workspace must be contiguous")
        _launch(lib.attn_paged_fp8 if scales else lib.attn_paged_tree, dev,
                _pack(q, k_cache, v_cache, scales, block_table, cu_q, kv_len, tree, out, lse, scale, causal, max_q,
                      workspace.data_ptr(), nbytes))
    finally:
        if guard is not None:
            guard.__exit__(None, None, None)
    return out, lse


def attn_paged_tree(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor, cu_q: torch.Tensor,
                    kv_len: torch.Tensor, tree: torch.Tensor, *, scale: Optional[float] = None, max_q: Optional[int] = None,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """attn_paged for trees of drafted tokens. Returns (O, LSE).

    tree [rows, words] int32 (attn_tree_plan's, or any bits): each row sees its sequence's context and those of
    the sequence's new rows whose bits are set. Sequences of more than 32 * words rows are attended to
    causally, as chunks of a prompt. Everything else as attn_paged."""
    if tree is None:
        raise ValueError("tree is None")
    return _attend(q, k_cache, v_cache, (), block_table, cu_q, kv_len, tree, scale, False, max_q, out, lse, workspace, stream)


def attn_paged_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                   block_table: torch.Tensor, cu_q: torch.Tensor, kv_len: torch.Tensor, *, scale: Optional[float] = None,
                   causal: bool = False, tree: Optional[torch.Tensor] = None, max_q: Optional[int] = None,
                   out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """attn_paged over a cache in 8 bits (attn_pages_write_fp8's codes and scales), q in bf16 or fp16. Returns (O, LSE)
    of exactly the values that the cache stands for. With tree, as attn_paged_tree (and causal False)."""
    return _attend(q, k_cache, v_cache, (k_scale, v_scale), block_table, cu_q, kv_len, tree, scale, causal, max_q, out, lse, workspace,
                   stream)
