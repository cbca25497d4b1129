"""The paged key/value cache by its definition, in fp64 and plain Python integers.

Key j of a sequence is slot j % page_size of page table[j // page_size]; each sequence's rows attend
to its own keys as oracle.ref defines attention, query head h with key/value head h // group. The
page functions restate how a step's pages, slots and positions follow from its lengths, one token
after another.
"""
from __future__ import annotations

from typing import List, Sequence, Tuple

import numpy as np

from . import ref


def gather_keys(cache, table_row: Sequence[int], length: int) -> np.ndarray:
    """[heads, length, d] of one sequence from a cache [pages, heads, page_size, d]."""
    cache = np.asarray(cache)
    page_size = cache.shape[2]
    out = np.zeros((cache.shape[1], length, cache.shape[3]), dtype=np.float64)
    for j in range(length):
        out[:, j] = cache[table_row[j // page_size], :, j % page_size]
    return out


def paged_forward(q, k_cache, v_cache, table, cu_q, kv_len, scale: float, causal: bool) -> Tuple[np.ndarray, np.ndarray]:
    """O [rows, Hq, d] and LSE [Hq, rows]; rows behind the last sequence are NaN in both."""
    q = np.asarray(q, dtype=np.float64)
    rows, hq, d = q.shape
    group = hq // np.asarray(k_cache).shape[1]
    o, lse = np.full((rows, hq, d), np.nan), np.full((hq, rows), np.nan)
    for b in range(len(kv_len)):
        r0, r1, n = int(cu_q[b]), int(cu_q[b + 1]), int(kv_len[b])
        if r1 == r0:
            continue
        if n == 0:
            o[r0:r1], lse[:, r0:r1] = 0.0, -np.inf
            continue
        k, v = gather_keys(k_cache, table[b], n), gather_keys(v_cache, table[b], n)
        qs = q[r0:r1].transpose(1, 0, 2)
        ob, lb = ref.decode_forward(qs[None], np.repeat(k, group, 0)[None], np.repeat(v, group, 0)[None], scale, causal)
        o[r0:r1], lse[:, r0:r1] = ob[0].transpose(1, 0, 2), lb[0]
    return o, lse


def plan(q_len, kv_len, table, free_pages, free_count: int, page_size: int, total_q: int):
    """(cu_q, new_len, slots, positions, free_left, table) of one step; a page that the stack could
    not give is -1, and free_left counts below zero then."""
    table = [list(r) for r in table]
    cu_q, new_len, slots, positions, left = [0], [], [], [], int(free_count)
    for b, (n, old) in enumerate(zip(q_len, kv_len)):
        for pos in range(old, old + n):
            if pos % page_size == 0:
                left -= 1
                table[b][pos // page_size] = int(free_pages[left]) if left >= 0 else -1
            page = table[b][pos // page_size]
            slots.append(page * page_size + pos % page_size if page >= 0 else -1)
            positions.append(pos)
        cu_q.append(cu_q[-1] + n)
        new_len.append(old + n)
    pad = [-1] * (total_q - len(slots))
    return cu_q, new_len, slots + pad, positions + pad, left, table


def release(done, kv_len, table, free_pages, free_count: int, page_size: int) -> Tuple[List[int], int, List[int]]:
    """(new_len, free_left, free_pages) after the sequences with done[b] gave their pages back."""
    stack, left, new_len = [int(x) for x in free_pages], int(free_count), []
    for b, n in enumerate(kv_len):
        if done[b]:
            for i in range((n + page_size - 1) // page_size):
                stack[left] = int(table[b][i])
                left += 1
        new_len.append(0 if done[b] else int(n))
    return new_len, left, stack
