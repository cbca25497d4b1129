"""Rotary positions, the 8-bit cache and trees of drafted tokens by their definitions, in fp64 and plain integers."""
from __future__ import annotations

import math
from fractions import Fraction
from typing import List, Sequence, Tuple

import numpy as np

from . import ref
from .paged import gather_keys

# 2 pi to 62 digits
_TURN = Fraction(628318530717958647692528676655900576839433879875021164194988918, 10 ** 62)


def turn_of(position: int, freq: float) -> float:
    """The angle position * freq as a fraction of a turn in [0, 1), exact before its rounding to fp64."""
    x = Fraction(int(position)) * Fraction(float(freq)) / _TURN
    return float(x - math.floor(x))


def rotate(x, positions: Sequence[int], inv_freq: Sequence[float], interleaved: bool, magnitude: float = 1.0,
           backward: bool = False) -> np.ndarray:
    """x [..., N, d] with a position for each of the N rows."""
    x = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    a, b = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else (np.arange(half), np.arange(half) + half)
    for n, pos in enumerate(positions):
        t = np.array([2 * np.pi * turn_of(pos, f) for f in inv_freq])
        c, s = magnitude * np.cos(t), magnitude * np.sin(t) * (-1 if backward else 1)
        xa, xb = x[..., n, a].copy(), x[..., n, b].copy()
        x[..., n, a], x[..., n, b] = xa * c - xb * s, xb * c + xa * s
    return x


def e4m3_values() -> np.ndarray:
    """The values of the codes 0 .. 126, ascending."""
    return ref.decode_e4m3(np.arange(127))


def quantise_row(x: Sequence[float]) -> Tuple[List[int], int]:
    """Codes and exponent of one row: the smallest e in [-119, 119] with max|x| <= 448 * 2^e, codes of the nearest E4M3
    value (ties to the even code), saturated; NaN is code 127 and does not count for e."""
    finite = [abs(v) for v in x if not math.isnan(v)]
    top, e = max(finite, default=0.0), -119
    while e < 119 and top > 448.0 * 2.0 ** e:
        e += 1
    values, codes = e4m3_values(), []
    for v in x:
        if math.isnan(v):
            codes.append(127)
            continue
        m = abs(v) / 2.0 ** e
        if m >= 448.0:
            c = 126
        else:
            hi = int(np.searchsorted(values, m))
            lo = max(hi - 1, 0)
            if values[hi] - m == m - values[lo]:
                c = hi if hi % 2 == 0 else lo
            else:
                c = hi if values[hi] - m < m - values[lo] else lo
        codes.append(c | (128 if math.copysign(1.0, v) < 0 else 0))
    return codes, e


def quantise(x) -> Tuple[np.ndarray, np.ndarray]:
    """Codes (uint8, the shape of x) and exponents + 127 (uint8, without the last dimension)."""
    x = np.asarray(x, dtype=np.float64)
    flat = x.reshape(-1, x.shape[-1])
    codes, exps = np.zeros(flat.shape, dtype=np.uint8), np.zeros(len(flat), dtype=np.uint8)
    for i, row in enumerate(flat):
        c, e = quantise_row(row.tolist())
        codes[i], exps[i] = c, e + 127
    return codes.reshape(x.shape), exps.reshape(x.shape[:-1])


def restore(codes, exps) -> np.ndarray:
    return ref.decode_e4m3(codes) * np.exp2(np.asarray(exps, dtype=np.float64) - 127)[..., None]


def tree_plan(parents: Sequence[int], cu_q: Sequence[int], kv_len: Sequence[int], words: int) -> Tuple[np.ndarray, List[int]]:
    """(mask [rows, words] of 32-bit words as int64, positions), one node after another."""
    rows = len(parents)
    mask, positions = np.zeros((rows, words), dtype=np.int64), [-1] * rows
    for b, length in enumerate(kv_len):
        r0, n = cu_q[b], cu_q[b + 1] - cu_q[b]
        seen, depth = [], []
        for i in range(n):
            up = parents[r0 + i] if n <= 32 * words else i - 1
            if not -1 <= up < i:
                up = -1
            seen.append((seen[up] if up >= 0 else 0) | 1 << i)
            depth.append(depth[up] + 1 if up >= 0 else 0)
            positions[r0 + i] = max(-1, length - n + depth[i])
            if n <= 32 * words:
                mask[r0 + i] = [seen[i] >> 32 * w & 0xFFFFFFFF for w in range(words)]
    return mask, positions


def tree_forward(q, k_cache, v_cache, table, cu_q, kv_len, mask, scale: float) -> Tuple[np.ndarray, np.ndarray]:
    """O [rows, Hq, d] and LSE [Hq, rows]; mask [rows, words] of 32-bit words. Rows behind the last sequence are NaN."""
    q, mask = np.asarray(q, dtype=np.float64), np.asarray(mask, dtype=np.int64) & 0xFFFFFFFF
    rows, hq, d = q.shape
    group, nodes = hq // np.asarray(k_cache).shape[1], 32 * mask.shape[1]
    o, lse = np.full((rows, hq, d), np.nan), np.full((hq, rows), np.nan)
    for b in range(len(kv_len)):
        r0, n, length = int(cu_q[b]), int(cu_q[b + 1] - cu_q[b]), int(kv_len[b])
        if n == 0:
            continue
        sees = np.zeros((n, length), dtype=bool)
        for i in range(n):
            for j in range(length):
                c = j - (length - n)
                sees[i, j] = c <= i if n > nodes else c < 0 or (c < nodes and bool(mask[r0 + i, c // 32] >> (c % 32) & 1))
        k, v = gather_keys(k_cache, table[b], length), gather_keys(v_cache, table[b], length)
        for h in range(hq):
            s = np.where(sees, scale * (q[r0:r0 + n, h] @ k[h // group].T), -np.inf)
            if length == 0:
                o[r0:r0 + n, h], lse[h, r0:r0 + n] = 0.0, -np.inf
                continue
            p, lse[h, r0:r0 + n] = ref.row_softmax(s)
            o[r0:r0 + n, h] = p @ v[h // group]
    return o, lse
