"""The 8-bit paged cache at the ends of its range on the GPU: what attn_paged promises holds for every value that the cache may
stand for, in units of every kind (up to 32 rows, up to 128, two tiles).

Bounds are those of test_paged_fp8.py unless a test derives its own.
"""
import math

import numpy as np
import pytest
import torch

from oracle import paged, ref, serving
from parity_util import assert_close_bf16, assert_lse, to64
from test_paged_fp8 import A, Case, _i32, _ok  # noqa: F401

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


def _codes_of(x):
    """E4M3 codes of values within its range (rounded by torch)."""
    return torch.as_tensor(np.asarray(x), dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def _set(c, x, b, j, values, e):
    """Token j of sequence b: values (over 2^e) of all heads in the keys (x = 0) or values (x = 1), and the scale 2^e."""
    at = (c.table[b, j // c.page], slice(None), j % c.page)
    c.codes[x][at], c.exps[x][at] = _codes_of(values), e + 127


def _restored(c):
    c.values = [serving.restore(codes, np.where(e == 255, 127, e)) for codes, e in zip(c.codes, c.exps)]


def _forward(c, causal, scale, values=None):
    k, v = c.values if values is None else values
    return paged.paged_forward(to64(c.q), k, v, c.table, c.cu, c.kv, scale, causal)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("seqs", [0, 2])
def test_a_batch_without_rows(A, bits, seqs):
    # an idle step: torch's pointer of an empty mask is NULL
    c = Case([1, 1], [20, 30], 1, 2, 64, 16, BF16, 101)
    table, _, kv = (t[:seqs] for t in c.rest())
    cu, q, tree = _i32([0] * (seqs + 1)), c.q.cuda()[:0], _i32(np.zeros((0, 2)))
    if bits == 8:
        o, lse = A.attn_paged_fp8(q, *c.cache(), table, cu, kv, tree=tree)
        assert A.paged_fp8_workspace_size(q, *c.cache(), table, cu, kv, tree=tree) == 0
    else:
        o, lse = A.attn_paged_tree(q, *c.cache16(), table, cu, kv, tree)
    _ok(A)
    assert o.shape == (0, 2, 64) and lse.shape == (2, 0)


# ---------------------------------------------------------------- weights
def _check_columns(c, o, lse, causal, scale):
    """Every column by the sizes of what it sums: a weight and the output are each rounded by at most half a step, values in
    fp16 by half of 2^-24 where they are below 2^-14 (and O, too), the scores by less than 1e-3."""
    O, L = _forward(c, causal, scale)
    size, _ = _forward(c, causal, scale, (c.values[0], np.abs(c.values[1])))
    eps, tiny = torch.finfo(c.dtype).eps, 2.0 ** -24 if c.dtype == F16 else 0.0
    assert_lse(lse, L)
    assert np.all(np.abs(to64(o) - O) <= (eps + 1e-3) * size + tiny)


@pytest.mark.parametrize("dtype,low", [(BF16, -30), (BF16, -100), (F16, -19)])
@pytest.mark.parametrize("kv", [60, 300, 3000])
@pytest.mark.parametrize("n", [1, 6, 40, 150])
def test_columns_of_small_values_beside_rows_of_large_ones(A, n, kv, dtype, low):
    # every other key has values 2^-low times larger, in the first half of the columns only; weights are much alike
    c = Case([n, 2], [kv + n, 40], 2, 2, 64, 16, dtype, 90)
    for b, length in enumerate(c.kv):
        for j in range(length):
            at = (c.table[b, j // 16], slice(None), j % 16)
            if j % 2:
                c.codes[1][at + (slice(32, None),)] = 0
                c.exps[1][at] = 127 - (5 if dtype == F16 else 0)  # within fp16's range
            else:
                c.exps[1][at] = 127 - 5 + low if dtype == F16 else 127 + low
    _restored(c)
    o, lse = A.attn_paged_fp8(*c.args(), causal=True, scale=0.02, max_q=n)
    _ok(A)
    _check_columns(c, o, lse, True, 0.02)


@pytest.mark.parametrize("n", [1, 7, 40, 150])
@pytest.mark.parametrize("kv", [300, 5000])
def test_light_keys_beside_a_heavy_one(A, n, kv):
    # one key of weight 1, zero in half of the columns, among keys of weight 2^-26: a bf16 weight like any other
    c = Case([n], [kv], 1, 2, 64, 16, BF16, 91)
    c.q[:] = 0
    c.q[:, :, 0] = 16.0
    for j in range(kv):
        _set(c, 0, 0, j, np.eye(1, 64) * (9.0 if j == 70 else 0.0), 0)
        _set(c, 1, 0, j, np.where(np.arange(64) < 32, 1.0, 0.0 if j == 70 else 1.0 + (j % 8) / 8)[None], 0)
    _restored(c)
    o, lse = A.attn_paged_fp8(*c.args(), max_q=n)
    _ok(A)
    _check_columns(c, o, lse, False, 0.125)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("group", [16, 40])
def test_the_largest_weight_is_divided_by_what_it_was_rounded_to(A, group, dtype):
    # Scores whose maximum lags behind: key 9 sets it, key 137 is 2^3 to 2^7.9 times heavier, the others have no weight. With
    # w = 2^x that of key 137 and 1 that of key 9, both of the same values v, O = v whatever w is rounded to. 100 sequences over the
    # same pages, so that most are not cut between two tiles.
    c = Case([1], [256], 8, group, 64, 16, dtype, 92)
    for j in range(256):
        _set(c, 0, 0, j, np.eye(1, 64) * {9: 0.0, 137: 1.0}.get(j, 0.0) - np.eye(1, 64, 1) * (0.0 if j in (9, 137) else 448.0), 0)
        _set(c, 1, 0, j, np.full((1, 64), 1.875), 0)
    x = torch.linspace(3.0, 7.9, group)
    c.q = torch.zeros(100, 8, group, 64, dtype=dtype)
    c.q[..., 0], c.q[..., 1] = x, 1.0
    c.q = c.q.view(100, 8 * group, 64)
    c.table, c.kv, c.cu = np.repeat(c.table, 100, 0), [256] * 100, np.arange(101)
    _restored(c)
    o, _ = A.attn_paged_fp8(*c.args(), scale=math.log(2.0), max_q=1)
    _ok(A)
    assert torch.all(o == 1.875)


# ---------------------------------------------------------------- NaN and infinities
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n", [1, 6, 50, 200])
@pytest.mark.parametrize("code", [127, 255])
def test_nan_among_the_values_shows(A, n, code, dtype):
    c = Case([n, n], [200 + n, 130 + n], 1, 2, 64, 16, dtype, 93)
    c.codes[1][c.table[0, 3], 0, 2, 5] = code  # a value of sequence 0 that every row sees
    o, lse = A.attn_paged_fp8(*c.args(), causal=True, max_q=n)
    _ok(A)
    assert torch.isnan(o[:n, :, 5]).all() and torch.isfinite(o[:n, :, :5]).all() and torch.isfinite(o[:n, :, 6:]).all()
    assert torch.isfinite(o[n:]).all() and torch.isfinite(lse).all()
    k, _ = A.attn_pages_read_fp8(_i32([int(c.table[0, 3]) * 16 + 2]), *reversed(c.cache()[:2]), *reversed(c.cache()[2:]), dtype=dtype)
    assert torch.isnan(k[0, 0, 5])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n", [1, 6, 50, 200])
@pytest.mark.parametrize("what", [math.inf, -math.inf, math.nan])
def test_queries_that_are_not_finite_show(A, n, what, dtype):
    c = Case([n, n], [200 + n, 130 + n], 1, 2, 64, 16, dtype, 94)
    c.q[n // 2, 1, 7] = what
    o, lse = A.attn_paged_fp8(*c.args(), causal=True, max_q=n)
    _ok(A)
    bad = torch.zeros(2 * n, 2, dtype=torch.bool)
    bad[n // 2, 1] = True
    assert torch.isnan(o.cpu()).all(-1).equal(bad) and torch.isnan(lse.t().cpu()).equal(bad)
    assert torch.isfinite(o.cpu()[~bad]).all() and torch.isfinite(lse.t().cpu()[~bad]).all()


@pytest.mark.parametrize("n", [6, 40, 200])
def test_rows_without_keys_whatever_the_query(A, n):
    # more rows than keys: the first see none
    c = Case([n], [2], 1, 2, 64, 16, BF16, 95)
    c.q[0, 0, 3], c.q[1, 1, 5], c.q[2] = math.inf, math.nan, 0.0
    o, lse = A.attn_paged_fp8(*c.args(), causal=True, max_q=n)
    _ok(A)
    assert torch.all(o[:n - 2] == 0) and torch.isneginf(lse[:, :n - 2]).all() and torch.isfinite(lse[:, n - 2:]).all()


# ---------------------------------------------------------------- scales of the keys
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 6, 50, 200])
@pytest.mark.parametrize("up,down", [(118, 12), (110, 12), (105, 0), (-100, 0), (-112, 12)])
def test_keys_at_the_ends_of_the_scales(A, n, up, down, d):
    # keys 2^up times as large, queries as much smaller but for 2^down, which is in the scale: ordinary scores
    c = Case([n, 3], [300 + n, 9], 2, 2, d, 16, BF16, 96)
    c.exps[0][c.exps[0] != 255] = np.clip(c.exps[0][c.exps[0] != 255].astype(int) + up, 8, 246)
    c.q = (c.q.float() * 2.0 ** (down - up)).to(BF16)
    _restored(c)
    scale = 2.0 ** -down / math.sqrt(d)
    o, lse = A.attn_paged_fp8(*c.args(), causal=True, scale=scale, max_q=n)
    _ok(A)
    c.check(o, lse, True, scale=scale)


@pytest.mark.parametrize("n", [1, 6, 50, 200])
def test_large_keys_beside_ordinary_ones(A, n):
    # ordinary keys and queries, but that one token's keys reach 2^126 in columns where the queries are 0: its scores are 0
    c = Case([n], [200 + n], 2, 2, 64, 16, BF16, 97)
    c.q[:, :, 32:] = 0
    _set(c, 0, 0, 5, np.where(np.arange(64) < 32, 0.0, 448.0)[None], 118)
    _restored(c)
    o, lse = A.attn_paged_fp8(*c.args(), causal=True, max_q=n)
    _ok(A)
    c.check(o, lse, True)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n", [1, 6, 50, 200])
def test_small_scale_and_rows_of_zeros(A, n, dtype):
    # scores of almost 0 everywhere: each row averages the values that it sees
    c = Case([n], [200 + n], 1, 2, 64, 16, dtype, 98)
    c.q[::2] = 0
    o, lse = A.attn_paged_fp8(*c.args(), causal=True, scale=1e-30, max_q=n)
    _ok(A)
    c.check(o, lse, True, scale=1e-30)


# ---------------------------------------------------------------- entries of a query
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 6, 50, 200])
@pytest.mark.parametrize("ratio", [256, 1024, 2048])
def test_one_large_entry_in_a_query(A, ratio, n, d, dtype):
    # one entry of up to `ratio` times the largest of the others, 4, its keys as much smaller: ordinary scores, to which every entry
    # counts. Entries below 2^-16 of the row's largest, 4 * ratio, are off by 2^-24 of it, 2^-22 * ratio, at most: 2^-11 for 2048,
    # where they are below 2^-3. A tenth of normal entries with a largest of 4 are; with keys of up to 8 and either sign some 10
    # such errors of half that size on the average make 10^0.5 * 2^-12 * 8 / 64^0.5 = 8e-4 of a score's unit at most, of
    # LSE's 1e-3
    c = Case([n], [1000 + n], 1, 2, d, 16, dtype, 99)
    c.q = (c.q.float() * 4.0 / c.q.float().abs().amax()).to(dtype)
    c.q[:, :, 11] *= ratio
    codes = torch.from_numpy(c.codes[0]).view(torch.float8_e4m3fn).float()
    codes[..., 11] /= ratio
    c.codes[0] = codes.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    _restored(c)
    o, lse = A.attn_paged_fp8(*c.args(), causal=True, max_q=n)
    _ok(A)
    c.check(o, lse, True)


# ---------------------------------------------------------------- scales of the values
@pytest.mark.parametrize("n", [1, 6, 50, 200])
def test_fp16_values_whose_scale_is_beyond_its_range(A, n):
    # codes of up to 2^-3 times 2^17, and rows of zeros with any scale: values that fp16 holds
    c = Case([n], [200 + n], 1, 2, 64, 16, F16, 100)
    g = np.random.default_rng(100)
    for j in range(200 + n):
        _set(c, 1, 0, j, g.integers(-7, 8, (1, 64)) * 2.0 ** -(6 + j % 3) if j % 5 else np.zeros((1, 64)), 17 if j % 5 else 100)
    _restored(c)
    o, lse = A.attn_paged_fp8(*c.args(), causal=True, max_q=n)
    _ok(A)
    O, L = _forward(c, True, 0.125)
    # parity_util's bounds over the largest O, which is some 2^14 here
    assert_lse(lse, L)
    assert np.all(np.abs(to64(o) - O) <= 4e-3 * np.abs(O).max())


# ---------------------------------------------------------------- large caches, and rows moved within one
def test_cache_beyond_32_bit_offsets(A):
    # more than 2^32 bytes of codes; the pages in use lie at both ends
    hkv, page, d = 8, 256, 128
    pages = (1 << 32) // (hkv * page * d) + 40
    kv, table = [700, 300], np.array([[pages - 1, 3, pages - 2], [pages - 3, 0, 10 ** 6]])
    cache = [torch.empty(pages, page, hkv, d, dtype=torch.uint8, device="cuda").transpose(1, 2) for _ in range(2)]
    cache += [torch.empty(pages, hkv, page, dtype=torch.uint8, device="cuda") for _ in range(2)]
    slots = _i32([int(table[b, j // page]) * page + j % page for b in range(2) for j in range(kv[b])])
    g = torch.Generator().manual_seed(102)
    rows = [torch.randn(1000, hkv, d, generator=g).to(BF16) for _ in range(2)]
    A.attn_pages_write_fp8(rows[0].cuda(), rows[1].cuda(), slots, *cache)
    held = A.attn_pages_read_fp8(slots, *cache)
    _ok(A)
    for x, got in zip(rows, held):  # a code is off by 2^-4 of its value, or by 2^-10 of a scale, less than 2^-17 of the row's largest
        x, got = to64(x), to64(got)
        assert np.all(np.abs(got - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -17 * np.abs(x).max(-1, keepdims=True))
    q = torch.randn(4, hkv * 2, d, generator=g).to(BF16)
    o, lse = A.attn_paged_fp8(q.cuda(), *cache, _i32(table), _i32([0, 1, 4]), _i32(kv), causal=True)
    _ok(A)
    ks, vs = (to64(x).transpose(1, 0, 2) for x in held)
    for r0, r1, k0, k1 in ((0, 1, 0, 700), (1, 4, 700, 1000)):
        O, L = ref.decode_forward(to64(q[r0:r1]).transpose(1, 0, 2)[None], np.repeat(ks[:, k0:k1], 2, 0)[None],
                                  np.repeat(vs[:, k0:k1], 2, 0)[None], 1 / math.sqrt(d), True)
        assert_close_bf16("O", o[r0:r1], O[0].transpose(1, 0, 2))
        assert_lse(lse[:, r0:r1], L[0])


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_rows_moved_to_other_slots_keep_their_values(A, dtype):
    # the accepted nodes of a tree, read and written to consecutive slots: bf16 holds every value of a cache
    c = Case([1], [90], 2, 1, 64, 16, dtype, 103)
    cache = c.cache()
    slot = lambda j: int(c.table[0, j // 16]) * 16 + j % 16  # noqa: E731
    kept, to = [80, 83, 84, 88], [80, 81, 82, 83]
    A.attn_pages_write_fp8(*A.attn_pages_read_fp8(_i32([slot(j) for j in kept]), *cache), _i32([slot(j) for j in to]), *cache)
    k, v = A.attn_pages_read_fp8(_i32([slot(j) for j in to]), *cache)
    _ok(A)
    for got, x in ((k, c.values[0]), (v, c.values[1])):
        for t, j in enumerate(kept):
            assert np.array_equal(to64(got[t]), x[c.table[0, j // 16], :, j % 16])
