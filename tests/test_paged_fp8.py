"""The 8-bit paged cache and trees of drafted tokens on the GPU against the fp64 oracle (oracle/serving.py, oracle/paged.py).

Codes, scales, rows read back, masks and positions are held to the definition bit for bit. Attention is held to the bounds of
the other forward kernels (parity_util): its inputs are the values that the cache stands for, the products of codes are exact in
fp32, and P and O carry the roundings of the 16-bit kernels. Everything of a cache that a sequence does not hold is NaN (code
127, scale 255), and block-table entries beyond its pages are far out of range, so anything read by mistake shows.
"""
import math

import numpy as np
import pytest
import torch

import workloads as W
from oracle import paged, ref, serving
from parity_util import assert_close_bf16, assert_lse, assert_masked_rows_zero, to64
from test_paged import SHAPES, UNUSED

pytestmark = pytest.mark.gpu
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import attn_fwd_03_gb300 as m
    assert m.attn_status() == m.ATTN_OK
    return m


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _ok(A):
    torch.cuda.synchronize()
    assert A.attn_status() == A.ATTN_OK, A.last_error()


def _quantised(rows, seed, mult=1.0):
    """Codes and exponent bytes of random rows [n, heads, d], by torch (the oracle's are held to it below)."""
    x = W.random_tensor(rows, seed, torch.float32) * mult
    x = x * torch.exp2(torch.randint(-4, 4, rows[:2], generator=torch.Generator().manual_seed(seed)).float())[..., None]
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return (torch.ldexp(x, -e[..., None]).to(F8).view(torch.uint8).numpy(), (e + 127).to(torch.uint8).numpy())


class Case:
    """Random q, caches and tables of a ragged batch; 16-bit caches hold the same values, in bf16 or fp16."""

    def __init__(self, n, kv, hkv, group, d, page, dtype, seed, pad=0, heads_first=False, mult=1.0):
        rng = np.random.default_rng(seed)
        self.n, self.kv, self.page, self.dtype = list(n), list(kv), page, dtype
        self.cu = np.concatenate([[0], np.cumsum(n)]).astype(int)
        rows = int(self.cu[-1]) + pad
        need = [(k + page - 1) // page for k in kv]
        pages = sum(need) + 3
        order = rng.permutation(pages).tolist()
        self.table = np.full((len(n), max(max(need), 1)), UNUSED, dtype=np.int64)
        self.q = W.random_tensor((rows, hkv * group, d), seed, dtype)
        self.heads_first = heads_first
        self.codes = [np.full((pages, hkv, page, d), 127, np.uint8) for _ in range(2)]
        self.exps = [np.full((pages, hkv, page), 255, np.uint8) for _ in range(2)]
        for b, m in enumerate(need):
            for i in range(m):
                at, held = order.pop(), min(page, kv[b] - i * page)
                self.table[b, i] = at
                for x in range(2):
                    c, e = _quantised((held, hkv, d), seed + 7 * at + x, mult if x == 1 else 1.0)
                    self.codes[x][at, :, :held], self.exps[x][at, :, :held] = c.transpose(1, 0, 2), e.T
        self.values = [serving.restore(c, np.where(e == 255, 127, e)) for c, e in zip(self.codes, self.exps)]

    def cache(self):
        out = []
        for c in self.codes:
            t = torch.from_numpy(c).cuda()
            out.append((t if self.heads_first else t.transpose(1, 2).contiguous().transpose(1, 2)).view(F8))
        return out + [torch.from_numpy(e).cuda().view(E8) for e in self.exps]

    def cache16(self):
        return [torch.from_numpy(v).to(self.dtype).cuda() for v in self.values]

    def rest(self):
        return _i32(self.table), _i32(self.cu), _i32(self.kv)

    def args(self):
        return (self.q.cuda(), *self.cache(), *self.rest())

    def check(self, o, lse, causal, mask=None, scale=None):
        # values reach 2^3 times those of the other tests, O up to some 30: a bf16 number from 16 to 32 steps by 2^-3, half of
        # which, 0.0625, is beyond the bound for O of up to 1 (2e-2), so that grows with the largest O
        scale = 1 / math.sqrt(self.q.shape[2]) if scale is None else scale
        rows = int(self.cu[-1])
        if mask is None:
            O, L = paged.paged_forward(to64(self.q), *self.values, self.table, self.cu, self.kv, scale, causal)
        else:
            O, L = serving.tree_forward(to64(self.q), *self.values, self.table, self.cu, self.kv, mask, scale)
        assert_close_bf16("O", o[:rows], O[:rows], relative_max=True)
        assert_lse(lse[:, :rows], L[:, :rows])
        assert_masked_rows_zero(o[:rows].transpose(0, 1), L[:, :rows])


# ---------------------------------------------------------------- writes and reads
SPECIAL = [0.0, -0.0, 1.0, 448.0, 449.0, 460.0, 464.0, 465.0, 1.0625, 1.1875, 2.0 ** -6, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -10, 3e4, -7.0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,heads,page,heads_first", [(64, 1, 16, False), (128, 3, 32, True), (128, 8, 64, False)])
def test_write_and_read_by_the_definition(A, d, heads, page, heads_first, dtype):
    rows, pages = 45, 5
    g = torch.Generator().manual_seed(d + heads)
    k, v = (torch.randn(rows, heads, d, generator=g) * torch.exp(4 * torch.randn(rows, heads, 1, generator=g)) for _ in range(2))
    k[0], v[1] = 0.0, -0.0
    for i, x in enumerate(SPECIAL):
        k[2 + i, 0] = torch.tensor(SPECIAL).repeat(d // 16).roll(i) * (1 if x == 0 else 1.0)
        v[2 + i, 0] = x * torch.linspace(-1, 1, d)
    k[20, 0, 3], v[21, 0, 5], v[22, 0, 7], v[23, 0, 9] = math.nan, math.inf, -math.inf, math.nan
    if dtype == torch.bfloat16:
        k[24, 0], v[24, 0], v[25, 0] = 3.3e38 * torch.linspace(-1, 1, d), 1e-38 * torch.linspace(-1, 1, d), 1e-30
    k, v = k.to(dtype), v.to(dtype)
    slots = torch.randperm(pages * page, generator=g)[:rows].to(torch.int32)
    slots[30] = -1
    shape = (pages, heads, page) if heads_first else (pages, page, heads)
    caches = [torch.full((*shape, d), 99, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((pages, heads, page), 99, dtype=torch.uint8, device="cuda") for _ in range(2)]
    view = lambda t: t if heads_first else t.transpose(1, 2)  # noqa: E731
    A.attn_pages_write_fp8(k.cuda(), v.cuda(), slots.cuda(), *(view(c).view(F8) for c in caches), *(s.view(E8) for s in scales))
    _ok(A)
    back = A.attn_pages_read_fp8(slots.cuda(), *(view(c) for c in caches), *scales, dtype=dtype)
    _ok(A)
    for x, cache, scale, rd in zip((k, v), caches, scales, back):
        want_c, want_e = np.full((pages, heads, page, d), 99, np.uint8), np.full((pages, heads, page), 99, np.uint8)
        codes, exps = serving.quantise(to64(x))
        for t, s in enumerate(slots.tolist()):
            if s >= 0:
                want_c[s // page, :, s % page], want_e[s // page, :, s % page] = codes[t], exps[t]
        got = view(cache).cpu().numpy()
        nan = (want_c & 127) == 127  # either sign of a NaN is one
        assert np.array_equal(np.where(nan, 127, want_c), np.where((got & 127) == 127, 127, got))
        assert np.array_equal(scale.cpu().numpy(), want_e)
        held = torch.from_numpy(serving.restore(codes, exps)).to(dtype)
        held[30] = 0
        assert torch.equal(torch.nan_to_num(rd.cpu().float(), 1.5), torch.nan_to_num(held.float(), 1.5))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_read_repeats_slots_and_leaves_rows(A, dtype):
    c = Case([1], [50], 2, 1, 64, 16, dtype, 3)
    cache = c.cache()
    slot = lambda j: int(c.table[0, j // 16]) * 16 + j % 16  # noqa: E731
    want = [3, 3, None, 49, 0, 3]
    slots = _i32([-1 if j is None else slot(j) for j in want])
    k, v = (torch.full((6, 2, 64), 5.0, dtype=dtype, device="cuda") for _ in range(2))
    got = A.attn_pages_read_fp8(slots, *cache, k=k, v=v)
    _ok(A)
    assert got[0] is k and got[1] is v and torch.all(k[2] == 5) and torch.all(v[2] == 5)
    for t, j in enumerate(want):
        if j is not None:
            for x, out in zip(c.values, (k, v)):
                assert torch.equal(out[t].cpu(), torch.from_numpy(x[c.table[0, j // 16], :, j % 16]).to(dtype))


def test_every_code_and_scale_read_back(A):
    # bf16 holds every code times every scale that a write makes
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(1, 4, 64).expand(15, 4, 64).reshape(1, 60, 1, 64)
    cache = torch.zeros(1, 64, 1, 64, dtype=torch.uint8, device="cuda")
    cache[:, :60] = codes
    for first in range(8, 247, 60):
        scale = torch.arange(first, first + 64, device="cuda").clamp(max=246).to(torch.uint8).view(1, 1, 64)
        k, v = A.attn_pages_read_fp8(_i32(np.arange(64)), cache.transpose(1, 2), cache.transpose(1, 2), scale, scale)
        want = torch.from_numpy(serving.restore(cache.cpu().numpy().reshape(64, 64), scale.cpu().numpy().reshape(64)))
        assert torch.equal(torch.nan_to_num(k.view(64, 64).double().cpu(), 1.5), torch.nan_to_num(want, 1.5)) and torch.equal(
            torch.nan_to_num(k, 1.5), torch.nan_to_num(v, 1.5))


def test_slots_out_of_range_are_reported(A):
    c = Case([1], [20], 1, 1, 64, 16, torch.bfloat16, 4)
    cache = c.cache()
    before = [t.view(torch.uint8).clone() for t in cache]
    bad = _i32([16 * cache[0].shape[0], 2 ** 31 - 1])
    k = torch.ones(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    A.attn_pages_write_fp8(k, k, bad, *cache)
    assert A.attn_status() == A.ATTN_ERR_INVALID
    got = A.attn_pages_read_fp8(bad, *cache, k=k.clone(), v=k.clone())
    assert A.attn_status() == A.ATTN_ERR_INVALID and torch.equal(got[0], k) and torch.equal(got[1], k)
    assert all(torch.equal(t.view(torch.uint8), b) for t, b in zip(cache, before))
    A.attn_pages_write_fp8(k[:0], k[:0], bad[:0], *cache)
    _ok(A)


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_attention_matches_oracle(A, shape, causal, dtype):
    c = Case(*SHAPES[shape], dtype, 40)
    o, lse = A.attn_paged_fp8(*c.args(), causal=causal, max_q=max(max(c.n), 1))
    _ok(A)
    c.check(o, lse, causal)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 8, 9, 16, 17, 32, 33, 64, 65, 128])
def test_rows_of_a_unit(A, rows, d):
    # sequences whose rows fill a tile up to each border between the kernels' ways, cut among many CTAs and whole
    c = Case([rows, 1, rows], [rows + 2000, 130, rows], 1, 1, d, 64, torch.bfloat16, 41)
    o, lse = A.attn_paged_fp8(*c.args(), causal=True, max_q=rows)
    _ok(A)
    c.check(o, lse, True)


@pytest.mark.parametrize("max_q", [None, 1, 3, 17, 40, 5000])
def test_max_q_is_only_a_hint(A, max_q):
    c = Case([1, 45, 0, 9, 1], [300, 77, 12, 513, 5], 2, 4, 128, 32, torch.bfloat16, 50)
    o, lse = A.attn_paged_fp8(*c.args(), causal=True, max_q=max_q)
    _ok(A)
    c.check(o, lse, True)


@pytest.mark.parametrize("dtype,mult", [(torch.bfloat16, 2.0 ** 40), (torch.bfloat16, 2.0 ** -60), (torch.float16, 300.0),
                                        (torch.float16, 2.0 ** -9), (torch.float16, 2.0 ** -17)])
@pytest.mark.parametrize("n", [2, 70])
def test_large_and_small_values(A, n, dtype, mult):
    # scales beyond 2^7 in bf16 and below 2^-24 in fp16 take a second multiplication on chip; O is compared over its largest
    c = Case([n, 1], [300, 5], 2, 2, 64, 16, dtype, 51, mult=mult)
    o, lse = A.attn_paged_fp8(*c.args(), causal=True, max_q=n)
    _ok(A)
    O, L = paged.paged_forward(to64(c.q), *c.values, c.table, c.cu, c.kv, 0.125, True)
    # fp16 values below 2^-14 step by 2^-24, in the cache as used and in O: half a step each on top
    tiny = 2.0 ** -24 if dtype == torch.float16 else 0.0
    top = np.abs(O).max()
    assert np.all(np.abs(to64(o) - O) <= (4e-3 if dtype == torch.float16 else 2e-2) * top + tiny)
    assert_lse(lse, L)


@pytest.mark.parametrize("n", [1, 6, 70])
@pytest.mark.parametrize("kv", [70, 300, 5000])
@pytest.mark.parametrize("order", [(-200, 0, 40), (40, -200, 0), (0, 100, -60)])
def test_values_of_very_different_size(A, order, kv, n):
    # a third of the keys each with values of 2^order, below 2^-128 zeros: a weight counts whatever its value
    c = Case([n, 2], [kv, 40], 2, 2, 64, 16, torch.bfloat16, 55)
    for b, length in enumerate(c.kv):
        for j in range(length):
            at, e = (c.table[b, j // 16], slice(None), j % 16), order[3 * j // length]
            if e < -128:
                c.codes[1][at], c.exps[1][at] = 0, 8
            else:
                c.exps[1][at] += np.uint8(e) if e >= 0 else np.uint8(256 + e)
    c.values[1] = serving.restore(c.codes[1], np.where(c.exps[1] == 255, 127, c.exps[1]))
    o, lse = A.attn_paged_fp8(*c.args(), causal=True)
    _ok(A)
    O, L = paged.paged_forward(to64(c.q), *c.values, c.table, c.cu, c.kv, 0.125, True)
    assert_lse(lse, L)
    # a weight and the output are each rounded by at most 2^-8 of themselves, the scores by less than 1e-3
    size, _ = paged.paged_forward(to64(c.q), c.values[0], np.abs(c.values[1]), c.table, c.cu, c.kv, 0.125, True)
    assert np.all(np.abs(to64(o) - O) <= (2.0 ** -7 + 1e-3) * size + 2.0 ** -70 * np.nanmax(np.abs(c.values[1])))


def test_large_queries_and_keys(A):
    # rows of q of very different size, each split by a factor of its own
    c = Case([3, 40], [200, 90], 1, 2, 128, 16, torch.bfloat16, 52)
    c.q = (c.q.float() * torch.exp2(torch.arange(43.0) - 20)[:, None, None]).to(torch.bfloat16)
    c.q[5] = 0
    o, lse = A.attn_paged_fp8(*c.args(), causal=True, scale=2.0 ** -12, max_q=40)
    _ok(A)
    O, L = paged.paged_forward(to64(c.q), *c.values, c.table, c.cu, c.kv, 2.0 ** -12, True)
    # scores reach 2^22 * 100 / 2^12 = 1e5: fp32 carries them to 2^-24 of that, 6e-3, so the largest are left out of O
    small = np.abs(L).max(0) < 200
    assert small.sum() >= 25
    # a score of up to 200 is off by at most 2^-23 of the sum of its 128 products' sizes, some 20 times itself: 5e-4
    assert_lse(lse[:, torch.from_numpy(small)], L[:, small])
    assert np.all(np.abs(to64(o)[small] - O[small]) <= 2e-2 * np.abs(O).max())


def test_nan_reaches_its_rows_only(A):
    for n in (1, 50):
        c = Case([n, n], [200 + n, 130 + n], 1, 2, 64, 16, torch.bfloat16, 53)
        c.codes[0][c.table[0, 3], 0, 2, 5] = 127  # a key of sequence 0, row 50
        o, lse = A.attn_paged_fp8(*c.args(), causal=True, max_q=n)
        _ok(A)
        r0 = slice(0, n)
        assert torch.isnan(o[r0]).all() and torch.isnan(lse[:, r0]).all()
        assert torch.isfinite(o[n:2 * n]).all() and torch.isfinite(lse[:, n:2 * n]).all()


@pytest.mark.parametrize("n", [1, 60])
def test_heads_first_pages_strided_rows_and_padding(A, n):
    c = Case([n, n], [200, 129], 2, 4, 64, 32, torch.bfloat16, 60, heads_first=True, pad=5)
    q, *cache_and_rest = c.args()
    wide = torch.zeros(q.shape[0], 12, 64, dtype=q.dtype, device="cuda")
    wide[:, :8] = q
    out, lse = torch.full_like(wide, 3.0), torch.full((8, q.shape[0]), 3.0, device="cuda")
    o, _ = A.attn_paged_fp8(wide[:, :8], *cache_and_rest, causal=True, out=out[:, 2:10], lse=lse, max_q=n)
    _ok(A)
    c.check(o, lse, True)
    assert torch.all(out[:, :2] == 3) and torch.all(out[:, 10:] == 3) and torch.all(out[2 * n:] == 3) and torch.all(lse[:, 2 * n:] == 3)


@pytest.mark.parametrize("n", [1, 3, 200])
def test_output_over_q_and_the_same_bits(A, n):
    c = Case([n] * 5, [n + 200, n, 3000, n + 1, n + 130], 2, 3, 128, 16, torch.bfloat16, 66, pad=2)
    args = c.args()
    want, want_lse = A.attn_paged_fp8(*args, causal=True, max_q=n)
    again = A.attn_paged_fp8(*args, causal=True, max_q=n, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    rows = 5 * n
    assert torch.equal(again[0][:rows], want[:rows]) and torch.equal(again[1][:, :rows], want_lse[:, :rows])
    o, lse = A.attn_paged_fp8(*args, causal=True, max_q=n, out=args[0])
    _ok(A)
    assert torch.equal(o[:rows], want[:rows]) and torch.equal(lse[:, :rows], want_lse[:, :rows])
    assert torch.equal(o[rows:].cpu(), c.q[rows:])
    c.check(o, lse, True)


def test_keys_and_values_apart_and_workspace(A):
    c = Case([2, 1], [90, 40], 2, 3, 64, 16, torch.bfloat16, 63)
    q, k, v, ks, vs, *rest = c.args()
    k = k.view(torch.uint8).contiguous().view(F8)
    assert k.stride() != v.stride()
    need = A.paged_fp8_workspace_size(q, k, v, ks, vs, *rest, max_q=2)
    with pytest.raises(A.AttnError) as e:
        A.attn_paged_fp8(q, k, v, ks, vs, *rest, causal=True, max_q=2, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == A.ATTN_ERR_WORKSPACE
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN: nothing of it is read before it is written
    o, lse = A.attn_paged_fp8(q, k, v, ks, vs, *rest, causal=True, max_q=2, workspace=ws)
    _ok(A)
    c.check(o, lse, True)


def test_bad_pages_and_lengths_are_reported(A):
    c = Case([1, 1], [100, 60], 1, 2, 128, 16, torch.bfloat16, 70)
    q, *cache, table, cu, kv = c.args()
    for what, t in (("page", (table.clone(), cu, kv)), ("length", (table, cu, kv.clone())), ("rows", (table, cu.clone(), kv))):
        t[{"page": 0, "length": 2, "rows": 1}[what]].view(-1)[1] = {"page": 10 ** 6, "length": 10 ** 6, "rows": -4}[what]
        o, lse = A.attn_paged_fp8(q, *cache, *t, causal=True, max_q=1)
        assert A.attn_status() == A.ATTN_ERR_INVALID
        if what == "page":  # the other sequence's rows
            O, L = paged.paged_forward(to64(c.q), *c.values, c.table, c.cu, c.kv, 1 / math.sqrt(128), True)
            assert_lse(lse[:, 1:], L[:, 1:])
    o, lse = A.attn_paged_fp8(q, *cache, table, cu, kv, causal=True, max_q=1)
    _ok(A)
    c.check(o, lse, True)


@pytest.mark.parametrize("n", [1, 100])
def test_a_stalled_producer_is_reported_and_the_next_call_is_right(A, n):
    c = Case([n], [60000], 2, 2, 64, 256, torch.bfloat16, 71)  # several tiles for every CTA, so that each one's producers stop
    args = c.args()
    A.set_wait_timeout_ns(5_000_000)
    A.debug_set_producer_stall(1)
    try:
        A.attn_paged_fp8(*args, causal=True, max_q=n)
        assert A.attn_status() == A.ATTN_ERR_TIMEOUT
    finally:
        A.debug_set_producer_stall(0)
        A.set_wait_timeout_ns(2_000_000_000)
    o, lse = A.attn_paged_fp8(*args, causal=True, max_q=n)
    _ok(A)
    c.check(o, lse, True)


# ---------------------------------------------------------------- trees
def _random_tree(n, rng):
    return [int(rng.integers(max(-1, i - 6), i)) if i else -1 for i in range(n)]


@pytest.mark.parametrize("n,words", [([1], 1), ([5, 32, 1, 0, 33, 64], 2), ([31, 70, 3], 1), ([200, 256, 1], 8), ([1000], 32), ([], 1)])
def test_tree_plan(A, n, words):
    rng = np.random.default_rng(sum(n) + words)
    parents = sum((_random_tree(m, rng) for m in n), []) + [5, -1, 3]
    cu, kv = np.concatenate([[0], np.cumsum(n)]).astype(int).tolist(), [m + 10 * i for i, m in enumerate(n)]
    mask, pos = A.attn_tree_plan(_i32(parents), _i32(cu), _i32(kv).view(-1), 32 * words)
    _ok(A)
    want, want_pos = serving.tree_plan(parents, cu, kv, words)
    assert mask.shape == (len(parents), words) and np.array_equal(mask.cpu().numpy().astype(np.int64) & 0xFFFFFFFF, want)
    assert pos.tolist() == want_pos


def test_tree_plan_reports_what_is_no_tree(A):
    for parents, kv in (([0, 0], 5), ([-1, 1], 5), ([-2, 0], 5), ([-1, 0], 1)):
        mask, pos = A.attn_tree_plan(_i32(parents), _i32([0, 2]), _i32([kv]), 32)
        assert A.attn_status() == A.ATTN_ERR_INVALID
        want, want_pos = serving.tree_plan(parents, [0, 2], [kv], 1)
        assert np.array_equal(mask.cpu().numpy(), want) and pos.tolist() == want_pos


def test_tree_plan_into_given_tensors(A):
    mask, pos = torch.full((4, 3), 9, dtype=torch.int32, device="cuda"), torch.full((3,), 9, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = A.attn_tree_plan(_i32([-1, 0, 0]), _i32([0, 3]), _i32([8]), 40, mask=mask[:3, :2], positions=pos, stream=side)
    side.synchronize()
    assert mask.tolist() == [[1, 0, 9], [3, 0, 9], [5, 0, 9], [9, 9, 9]] and pos.tolist() == [5, 6, 6] and got[1] is pos


TREES = {
    "one node": ([1], [1], 1, 1, 64, 16, 1),
    "root alone over a context": ([1, 4], [40, 300], 2, 4, 128, 32, 1),
    "all new rows": ([26, 3], [26, 3], 1, 4, 128, 16, 1),
    "trees and a chunk": ([7, 90, 1, 0, 33], [200, 400, 17, 50, 1000], 2, 2, 64, 16, 2),
    "context ends in a tile": ([30, 30, 30], [128 + 30, 127 + 30, 100 + 30], 1, 5, 128, 64, 1),
    "large trees": ([250, 128], [700, 400], 1, 4, 128, 64, 8),
    "large trees, small head dim": ([250, 61], [700, 3000], 1, 2, 64, 128, 8),
    "more rows than keys": ([20, 5], [3, 0], 2, 2, 64, 16, 1),
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("shape", list(TREES))
def test_attention_of_trees(A, shape, bits, dtype):
    n, kv, hkv, group, d, page, words = TREES[shape]
    c = Case(n, kv, hkv, group, d, page, dtype, 80, pad=2)
    rng = np.random.default_rng(81)
    mask = np.zeros((len(c.q), words), dtype=np.int64)
    mask[:int(c.cu[-1])] = serving.tree_plan(sum((_random_tree(m, rng) for m in n), []), c.cu.tolist(), kv, words)[0][:int(c.cu[-1])]
    tree = torch.from_numpy(mask.astype(np.uint32).view(np.int32)).cuda()
    table, cu, lens = c.rest()
    if bits == 8:
        o, lse = A.attn_paged_fp8(c.q.cuda(), *c.cache(), table, cu, lens, tree=tree, max_q=max(n))
    else:
        o, lse = A.attn_paged_tree(c.q.cuda(), *c.cache16(), table, cu, lens, tree, max_q=max(n))
    _ok(A)
    c.check(o, lse, False, mask)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_any_bits_are_masks(A, bits, d):
    # bits above a row's own, rows without any, a first row of all; without a context rows may see nothing
    n, kv = [40, 64, 3], [40, 300, 3]
    c = Case(n, kv, 1, 3, d, 16, torch.bfloat16, 82)
    rng = np.random.default_rng(83)
    mask = rng.integers(0, 2 ** 32, size=(107, 2))
    mask[3], mask[104], mask[106], mask[10] = 0, 0, 0, 2 ** 32 - 1
    tree = torch.from_numpy(mask.astype(np.uint32).view(np.int32)).cuda()
    wide = torch.zeros(107, 5, dtype=torch.int32, device="cuda")
    wide[:, 1:3] = tree
    for t in (tree, wide[:, 1:3]):
        if bits == 8:
            o, lse = A.attn_paged_fp8(*c.args(), tree=t, max_q=64)
        else:
            o, lse = A.attn_paged_tree(c.q.cuda(), *c.cache16(), *c.rest(), t, max_q=64)
        _ok(A)
        c.check(o, lse, False, mask)
    assert torch.isneginf(lse[:, 3]).all() and torch.isneginf(lse[:, 106]).all() and not torch.isneginf(lse[:, 104 - 3]).any()


def test_a_chain_is_causal_attention(A):
    c = Case([30, 12], [500, 12], 2, 4, 128, 32, torch.bfloat16, 84)
    parents = list(range(-1, 29)) + list(range(-1, 11))
    tree, pos = A.attn_tree_plan(_i32(parents), _i32(c.cu), _i32(c.kv), 32)
    assert pos.tolist() == list(range(470, 500)) + list(range(12))
    for args, tree_call in ((c.args(), A.attn_paged_fp8), ((c.q.cuda(), *c.cache16(), *c.rest()), None)):
        if tree_call:
            o, lse = A.attn_paged_fp8(*args, tree=tree, max_q=30)
            want, want_lse = A.attn_paged_fp8(*args, causal=True, max_q=30)
        else:
            o, lse = A.attn_paged_tree(*args, tree, max_q=30)
            want, want_lse = A.attn_paged(*args, causal=True, max_q=30)
        _ok(A)
        assert_close_bf16("O", o, want, relative_max=True)  # as in Case.check
        assert_lse(lse, want_lse)


# ---------------------------------------------------------------- a run of them, as a server makes it
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_drafted_step(A, dtype):
    """plan, positions of the tree, rotation, write in 8 bits, attention; then again as a graph with other lengths."""
    hkv, group, d, page, B = 2, 4, 64, 16, 3
    scale, freq = 1 / math.sqrt(d), A.rotary_frequencies(32, by_parts=4.0, context=4096, device="cuda")
    pages, rng = 40, np.random.default_rng(90)
    cache = [torch.full((pages, page, hkv, d), 127, dtype=torch.uint8, device="cuda").transpose(1, 2) for _ in range(2)]
    cache += [torch.full((pages, hkv, page), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    table, free = torch.full((B, 12), -1, dtype=torch.int32, device="cuda"), _i32(rng.permutation(pages))
    kv_len, count = _i32([0, 0, 0]), _i32([pages])
    held = [np.zeros((0, hkv, d)) for _ in range(2 * B)]  # each sequence's keys and values as the cache holds them

    def step(q_len, parents, rows, seed, kv_len, count):
        q, k, v = (W.random_tensor((rows, h, d), seed + i, dtype) for i, h in enumerate((hkv * group, hkv, hkv)))
        st = dict(q=q.cuda(), k=k.cuda(), v=v.cuda(), q_len=_i32(q_len), parents=_i32(parents + [-1] * (rows - len(parents))),
                  kv_len=kv_len, count=count, host=(q, k, v))
        return st

    def run(st, rows):
        cu, lens, slots, _, left = A.attn_pages_plan(st["q_len"], st["kv_len"], table, free, st["count"], page, rows)
        tree, pos = A.attn_tree_plan(st["parents"], cu, lens, 32)
        qr, kr = A.attn_rotary(st["q"], st["k"], pos, freq, q_out=torch.zeros_like(st["q"]), k_out=torch.zeros_like(st["k"]))
        A.attn_pages_write_fp8(kr, st["v"], slots, *cache)
        o, lse = A.attn_paged_fp8(qr, *cache, table, cu, lens, tree=tree, max_q=32)
        return cu, lens, left, tree, pos, qr, kr, o, lse

    def check(st, q_len, res, old):
        cu, lens, left, tree, pos, qr, kr, o, lse = res
        r = 0
        for b, n in enumerate(q_len):
            for x, rows in ((0, kr[r:r + n]), (1, st["v"][r:r + n])):
                new = serving.restore(*serving.quantise(to64(rows)))
                held[2 * b + x] = np.concatenate([held[2 * b + x][:old[b]], new])
            for h in range(hkv * group):
                s = scale * (to64(qr[r:r + n, h]) @ held[2 * b][:, h // group].T)
                bits = tree[r:r + n, 0].cpu().numpy().astype(np.int64) & 0xFFFFFFFF
                sees = np.ones_like(s, dtype=bool)
                for i in range(n):
                    for c in range(n):
                        sees[i, old[b] + c] = c <= i if n > 32 else bool(bits[i] >> c & 1)
                p, L = ref.row_softmax(np.where(sees, s, -np.inf))
                assert_lse(lse[h, r:r + n], L)
                assert_close_bf16("O", o[r:r + n, h], p @ held[2 * b + 1][:, h // group])
            r += n
        want = serving.rotate(np.moveaxis(to64(st["host"][0]), 0, 1), [max(x, 0) for x in pos.tolist()], freq.tolist(), False)
        assert_close_bf16("q", qr[:r], np.moveaxis(want, 1, 0)[:r])

    # prompts (one longer than a tree may be), then trees over them
    q_len = [50, 20, 33]
    st = step(q_len, list(range(-1, 49)) + list(range(-1, 19)) + list(range(-1, 32)), 110, 91, kv_len, count)
    res = run(st, 110)
    _ok(A)
    check(st, q_len, res, [0, 0, 0])
    kv_len, count = res[1], res[2]
    trees = [[9, 0, 17], [12, 30, 1]]
    parents = [sum((_random_tree(n, rng) for n in t), []) for t in trees]
    st = step(trees[0], parents[0], 44, 95, kv_len.clone(), count.clone())
    st["kv_len"].copy_(kv_len)
    g = torch.cuda.CUDAGraph()
    run(st, 44)  # every kernel's first call, outside the capture; the step is planned again
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        res = run(st, 44)
    for i, t in enumerate(trees):
        new = step(t, parents[i], 44, 95 + 10 * i, kv_len, count)
        for name in ("q", "k", "v", "q_len", "parents"):
            st[name].copy_(new[name])
        st["host"] = new["host"]
        g.replay()
        _ok(A)
        check(st, t, res, kv_len.tolist())  # neither step is taken: both follow the prompts


def test_two_captured_calls_and_an_eager_one_at_once(A):
    cases = [Case([1] * 4, [700, 30, 2000, 5], 2, 4, 64, 16, torch.bfloat16, 100 + i) for i in range(3)]
    args = [c.args() for c in cases]
    graphs, got, side = [], [], [torch.cuda.Stream() for _ in cases]
    for a in args[:2]:
        A.attn_paged_fp8(*a, causal=True, max_q=1)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(A.attn_paged_fp8(*a, causal=True, max_q=1))
        graphs.append(g)
    for _ in range(5):
        for g, s in zip(graphs, side):
            with torch.cuda.stream(s):
                g.replay()
        eager = A.attn_paged_fp8(*args[2], causal=True, max_q=1)
    _ok(A)
    for c, (o, lse) in zip(cases, got + [eager]):
        c.check(o, lse, True)
