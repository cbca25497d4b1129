"""The paged cache on the GPU: attention, writes and tables against the fp64 oracle (oracle/paged.py).

Attention outputs are held to the bounds of the other forward kernels (parity_util): the arithmetic is
the same, 16-bit operands with fp32 accumulation and P rounded to the operand type. Everything of a
cache that a sequence does not hold is NaN (free pages, slots of the last page beyond its length), and
block-table entries beyond its pages are far out of range, so anything read by mistake shows.
"""
import math

import numpy as np
import pytest
import torch

import workloads as W
from oracle import paged, ref
from parity_util import assert_close_bf16, assert_lse, assert_masked_rows_zero, to64

pytestmark = pytest.mark.gpu

UNUSED = 0x7FFFFF00  # a block-table entry that must not be followed


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import attn_fwd_03_gb300 as m
    assert m.attn_status() == m.ATTN_OK
    return m


class Case:
    """Random q, caches and tables of a ragged batch."""

    def __init__(self, n, kv, hkv, group, d, page, dtype, seed, pad=0, heads_first=False, mult=1.0, columns=0):
        rng = np.random.default_rng(seed)
        self.n, self.kv, self.page, self.dtype = list(n), list(kv), page, dtype
        self.cu = np.concatenate([[0], np.cumsum(n)]).astype(int)
        rows = int(self.cu[-1]) + pad
        need = [(k + page - 1) // page for k in kv]
        pages = sum(need) + 3
        order = rng.permutation(pages).tolist()
        cols = max(max(need), 1) + columns
        self.table = np.full((len(n), cols), UNUSED, dtype=np.int64)
        self.q = W.random_tensor((rows, hkv * group, d), seed, dtype) * mult
        shape = (pages, hkv, page, d) if heads_first else (pages, page, hkv, d)
        self.k, self.v = (torch.full(shape, float("nan"), dtype=dtype) for _ in range(2))
        ks, vs = (W.random_tensor(shape, seed + i, dtype) for i in (1, 2))
        for b, m in enumerate(need):
            for i in range(m):
                at, held = order.pop(), min(page, kv[b] - i * page)
                self.table[b, i] = at
                for cache, src in ((self.k, ks), (self.v, vs)):
                    if heads_first:
                        cache[at, :, :held] = src[at, :, :held]
                    else:
                        cache[at, :held] = src[at, :held]
        if not heads_first:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.k = self.k * mult if mult != 1.0 else self.k

    def device(self):
        i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
        dev = lambda t: t.cuda() if t.is_contiguous() else t.transpose(1, 2).cuda().transpose(1, 2)  # noqa: E731
        return dev(self.q), dev(self.k), dev(self.v), i32(self.table), i32(self.cu), i32(self.kv)

    def oracle(self, causal, scale=None):
        scale = 1 / math.sqrt(self.q.shape[2]) if scale is None else scale
        return paged.paged_forward(to64(self.q), to64(self.k), to64(self.v), self.table, self.cu, self.kv, scale, causal)

    def check(self, o, lse, causal, scale=None):
        rows = int(self.cu[-1])
        O, L = self.oracle(causal, scale)
        assert_close_bf16("O", o[:rows], O[:rows])
        assert_lse(lse[:, :rows], L[:, :rows])
        assert_masked_rows_zero(o[:rows].transpose(0, 1), L[:, :rows])


def _ok(A):
    torch.cuda.synchronize()
    assert A.attn_status() == A.ATTN_OK, A.last_error()


SHAPES = {
    "one key": ([1], [1], 1, 1, 64, 16),
    "page and tile ends": ([1] * 9, [1, 15, 16, 17, 127, 128, 129, 255, 256], 2, 4, 128, 16),
    "ragged chunks with empty ones": ([3, 0, 7, 1, 0], [3, 5, 130, 257, 0], 2, 3, 64, 32),
    "one head to a group": ([5, 130, 1], [260, 130, 400], 3, 1, 128, 64),
    "two-tile units": ([300, 70], [700, 70], 2, 4, 128, 64),
    "two-tile units, small head dim": ([300, 70], [700, 333], 2, 4, 64, 128),
    "more rows than keys": ([4, 2, 200], [2, 0, 90], 2, 2, 64, 16),
    "odd group": ([129, 1, 64], [500, 1000, 64], 1, 7, 128, 32),
    "group of 128": ([3, 1], [40, 200], 1, 128, 64, 16),
    "group of 80": ([5, 2], [150, 20], 1, 80, 128, 64),
    "long pages": ([1, 40], [600, 1100], 2, 5, 64, 512),
    "long rows": ([2, 1], [2500, 1900], 1, 8, 128, 256),
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_paged_matches_oracle(A, shape, causal, dtype):
    c = Case(*SHAPES[shape], dtype, 40)
    o, lse = A.attn_paged(*c.device(), causal=causal, max_q=max(max(c.n), 1))
    _ok(A)
    c.check(o, lse, causal)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("max_q", [None, 1, 3, 17, 40, 5000])
def test_max_q_is_only_a_hint(A, max_q, d):
    c = Case([1, 45, 0, 9, 1], [300, 77, 12, 513, 5], 2, 4, d, 32, torch.bfloat16, 50)
    o, lse = A.attn_paged(*c.device(), causal=True, max_q=max_q)
    _ok(A)
    c.check(o, lse, True)


@pytest.mark.parametrize("max_q", [0, -1, -2 ** 40])
def test_max_q_below_one_is_refused(A, max_q):
    args = Case([1], [5], 1, 1, 64, 16, torch.bfloat16, 51).device()
    with pytest.raises(A.AttnError, match="max_q must be at least 1"):
        A.attn_paged(*args, max_q=max_q)
    assert A.paged_workspace_size(*args, max_q=max_q) == 0


@pytest.mark.parametrize("n", [1, 60])
def test_heads_first_pages_and_strided_rows(A, n):
    # pages hold [heads, slots, d]; q is part of a wider row, O is written into one
    c = Case([n, n], [200, 129], 2, 4, 64, 32, torch.bfloat16, 60, heads_first=True, columns=3)
    q, k, v, table, cu, kv = c.device()
    wide = torch.zeros(q.shape[0], 12, 64, dtype=q.dtype, device="cuda")
    wide[:, :8] = q
    out = torch.zeros_like(wide)
    o, lse = A.attn_paged(wide[:, :8], k, v, table[:, :max(1, table.shape[1] - 1)], cu, kv, causal=True, out=out[:, 2:10], max_q=n)
    _ok(A)
    c.check(o, lse, True)
    assert torch.all(out[:, :2] == 0) and torch.all(out[:, 10:] == 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 100])
def test_output_rows_aligned_to_16_bytes_only(A, n, d):
    c = Case([n, 2], [n + 200, 70], 1, 4, d, 32, torch.bfloat16, 62)
    flat = torch.zeros(c.q.numel() + 8, dtype=c.dtype, device="cuda")
    out = flat[8:].view(c.q.shape)
    assert out.data_ptr() % 32 == 16
    o, lse = A.attn_paged(*c.device(), causal=True, out=out, max_q=n)
    _ok(A)
    c.check(o, lse, True)
    assert torch.all(flat[:8] == 0)


@pytest.mark.parametrize("n,max_q", [(1, 1), (3, 3), (3, 2), (200, 200)])
def test_output_over_q(A, n, max_q):
    # the tiles of neighbouring sequences overlap in the rows that they load, not in those that they write
    c = Case([n] * 5, [n + 200, n, 3000, n + 1, n + 130], 2, 3, 128, 16, torch.bfloat16, 66, pad=2)
    args = c.device()
    want, want_lse = A.attn_paged(*args, causal=True, max_q=max_q)
    o, lse = A.attn_paged(*args, causal=True, max_q=max_q, out=args[0])
    _ok(A)
    rows = 5 * n
    assert o is args[0] and torch.equal(o[:rows], want[:rows]) and torch.equal(lse[:, :rows], want_lse[:, :rows])
    assert torch.equal(o[rows:].cpu(), c.q[rows:])
    c.check(o, lse, True)


def test_write_from_other_slots_of_the_cache(A):
    # a page moved within the caches: its rows are k and v, the slots another page's
    kc, vc = (W.random_tensor((4, 16, 3, 64), 67 + i, torch.float16).cuda() for i in range(2))
    before = [t.clone() for t in (kc, vc)]
    A.attn_pages_write(kc[2], vc[2], torch.arange(16, 32, dtype=torch.int32, device="cuda"), kc.transpose(1, 2), vc.transpose(1, 2))
    _ok(A)
    for t, was in zip((kc, vc), before):
        assert torch.equal(t[1], was[2]) and torch.equal(t[[0, 2, 3]], was[[0, 2, 3]])


def test_keys_and_values_in_different_page_orders(A):
    c = Case([2, 1], [90, 40], 2, 3, 64, 16, torch.bfloat16, 63)
    q, k, v, table, cu, kv = c.device()
    o, lse = A.attn_paged(q, k.contiguous(), v, table, cu, kv, causal=True)
    _ok(A)
    assert k.stride() != k.contiguous().stride()
    c.check(o, lse, True)


def test_workspace_of_the_callers(A):
    c = Case([1, 3], [400, 70], 2, 4, 128, 16, torch.float16, 64)
    args = c.device()
    need = A.paged_workspace_size(*args, max_q=3)
    assert need > 0
    with pytest.raises(A.AttnError) as e:
        A.attn_paged(*args, causal=True, max_q=3, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == A.ATTN_ERR_WORKSPACE
    with pytest.raises(A.AttnError) as e:
        A.attn_paged(*args, causal=True, max_q=3, workspace=torch.empty(need + 8, dtype=torch.uint8, device="cuda")[8:])
    assert e.value.status == A.ATTN_ERR_ALIGN
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN everywhere: nothing of it is read before it is written
    o, lse = A.attn_paged(*args, causal=True, max_q=3, workspace=ws)
    _ok(A)
    c.check(o, lse, True)
    with pytest.raises(ValueError):
        A.attn_paged(*args, causal=True, workspace=torch.empty(need, dtype=torch.uint8))


def test_workspace_size_goes_by_max_q_up_to_a_tile(A):
    for group, d in ((1, 64), (3, 128), (128, 64)):
        args = Case([1], [5], 2, group, d, 16, torch.bfloat16, 52).device()
        sizes = [A.paged_workspace_size(*args, max_q=m) for m in (129, 130, 5000, 2 ** 31 - 1)]
        assert sizes[0] > 0 and len(set(sizes)) == 1


def test_keys_and_values_interleaved_in_one_tensor(A):
    c = Case([1, 2], [70, 100], 3, 2, 128, 16, torch.float16, 65)
    q, k, v, table, cu, kv = c.device()
    both = torch.stack([k.transpose(1, 2), v.transpose(1, 2)], dim=1).contiguous()  # [pages, 2, slot, head, d]
    o, lse = A.attn_paged(q, both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2), table, cu, kv, causal=True)
    _ok(A)
    c.check(o, lse, True)


@pytest.mark.parametrize("n", [1, 150])
def test_padding_rows_stay_as_they_were(A, n):
    c = Case([n, 2], [n + 30, 90], 2, 2, 64, 16, torch.bfloat16, 70, pad=9)
    rows = int(c.cu[-1])
    c.q[rows:] = float("nan")
    out = torch.full(c.q.shape, 7.0, dtype=c.dtype, device="cuda")
    lse = torch.full((4, rows + 9), 3.0, device="cuda")
    A.attn_paged(*c.device(), causal=True, out=out, lse=lse, max_q=n)
    _ok(A)
    c.check(out, lse, True)
    assert torch.all(out[rows:] == 7.0) and torch.all(lse[:, rows:] == 3.0)


def test_one_table_for_every_sequence(A):
    # a table stride of 0: all sequences attend to the same pages (an encoder's states)
    c = Case([3, 1, 6], [90, 0, 0], 2, 2, 64, 32, torch.bfloat16, 75)
    c.kv, c.table = [90, 90, 41], np.repeat(c.table[:1], 3, 0)
    q, k, v, table, cu, kv = c.device()
    o, lse = A.attn_paged(q, k, v, table[:1].expand(3, -1), cu, kv)
    _ok(A)
    c.check(o, lse, False)


@pytest.mark.parametrize("n", [2, 140])
def test_large_scores(A, n):
    # q and k times sqrt(30): raw scores reach about +-90, where an unshifted fp32 exp overflows
    c = Case([n, 1], [600, 300], 2, 4, 128, 64, torch.bfloat16, 80, mult=math.sqrt(30.0))
    o, lse = A.attn_paged(*c.device(), causal=True, max_q=n)
    _ok(A)
    c.check(o, lse, True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 150])
@pytest.mark.parametrize("where", ["q", "k"])
def test_nan_scores_stay_nan(A, where, n, d):
    # a row with NaN among its scores is NaN in O and LSE, whether its keys are split over CTAs (3000 keys)
    # or not (90); every other row is as it would be without
    c = Case([n, 1], [3000, 90], 2, 2, d, 32, torch.bfloat16, 82)
    O, L = c.oracle(True)
    spoilt = np.zeros((n + 1, 4), dtype=bool)
    if where == "q":
        spoilt[0, 1] = spoilt[n, 2] = True
        c.q[torch.from_numpy(spoilt)] = float("nan")
    else:  # the last key but one of head 0: its sequence's last two rows see it
        for b, kv in enumerate(c.kv):
            c.k[int(c.table[b, (kv - 2) // 32]), 0, (kv - 2) % 32] = float("nan")
        spoilt[max(n - 2, 0):, :2] = True
    o, lse = A.attn_paged(*c.device(), causal=True, max_q=n)
    _ok(A)
    got, got_lse = to64(o), to64(lse).T
    assert np.all(np.isnan(got[spoilt])) and np.all(np.isnan(got_lse[spoilt]))
    assert_close_bf16("O", got[~spoilt], O[~spoilt])
    assert_lse(got_lse[~spoilt], L.T[~spoilt])


def test_explicit_scale(A):
    c = Case([2], [50], 1, 2, 64, 16, torch.float16, 85)
    o, lse = A.attn_paged(*c.device(), causal=True, scale=0.31)
    _ok(A)
    c.check(o, lse, True, 0.31)


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [3, 40, 200])
def test_rows_without_keys_are_zero_whatever_the_values(A, n, d, value):
    # more rows than keys: the rows before the first key's are 0 though the tile's other rows meet values
    # that are not finite
    c = Case([n, 2], [n // 2, 1], 2, 2, d, 16, torch.float16, 86)
    for b in range(2):
        c.v[int(c.table[b, 0]), :, 0] = value
    o, lse = A.attn_paged(*c.device(), causal=True, max_q=n)
    _ok(A)
    empty = np.array([i < n - n // 2 for i in range(n)] + [True, False])
    assert np.all(to64(o)[empty] == 0) and np.all(np.isneginf(to64(lse)[:, empty]))
    assert not np.isfinite(to64(o)[~empty]).any() and np.isfinite(to64(lse)[:, ~empty]).all()


def test_many_sequences(A):
    rng = np.random.default_rng(3)
    n, kv = rng.integers(0, 3, 700), rng.integers(0, 70, 700)
    c = Case(n.tolist(), kv.tolist(), 1, 2, 64, 16, torch.bfloat16, 90)
    o, lse = A.attn_paged(*c.device(), causal=True, max_q=2)
    _ok(A)
    c.check(o, lse, True)


def test_many_sequences_beside_long_chunks(A):
    # more sequences than the kernel has threads, a few of them in two-tile units
    rng = np.random.default_rng(4)
    n, kv = rng.integers(0, 3, 450), rng.integers(0, 40, 450)
    n[[3, 200, 449]], kv[[3, 200, 449]] = [150, 300, 90], [150, 411, 400]
    c = Case(n.tolist(), kv.tolist(), 1, 4, 128, 16, torch.bfloat16, 91)
    o, lse = A.attn_paged(*c.device(), causal=True, max_q=300)
    _ok(A)
    c.check(o, lse, True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("n", [1, 3, 8])
def test_short_tables(A, n, page, dtype):
    # tables of up to 384 keys at d = 128: 4 to 32 rows, two CTAs to an SM, one to four query tiles ahead
    rng = np.random.default_rng(n + page)
    kv = rng.integers(0, 385, 37)
    kv[:4] = [384, 0, 128, 1]
    c = Case([n] * 36 + [0], kv.tolist(), 3, 4, 128, page, dtype, 93)
    o, lse = A.attn_paged(*c.device(), causal=True, max_q=n)
    _ok(A)
    c.check(o, lse, True)


@pytest.mark.parametrize("max_q", [1, 400])
def test_no_rows_at_all(A, max_q):
    c = Case([0, 0], [40, 0], 1, 2, 64, 16, torch.bfloat16, 92, pad=3)
    out, lse = torch.full(c.q.shape, 5.0, dtype=c.dtype, device="cuda"), torch.full((2, 3), 5.0, device="cuda")
    A.attn_paged(*c.device(), causal=True, max_q=max_q, out=out, lse=lse)
    _ok(A)
    assert torch.all(out == 5.0) and torch.all(lse == 5.0)


@pytest.mark.parametrize("n,kv", [([1] * 8, [4000, 10, 900, 1, 128, 2048, 77, 1500]), ([600, 1, 90], [1900, 2500, 90])])
def test_same_bits_on_every_call_and_stream(A, n, kv):
    c = Case(n, kv, 2, 4, 128, 64, torch.bfloat16, 95)
    args = c.device()
    o, lse = A.attn_paged(*args, causal=True, max_q=max(n))
    _ok(A)
    c.check(o, lse, True)
    side = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(6):  # two streams at once, a workspace to each call
        got.append(A.attn_paged(*args, causal=True, max_q=max(n), stream=side[i % 2]))
    _ok(A)
    for o2, lse2 in got:
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_threads_on_one_stream(A):
    # calls of several host threads on the default stream share the binding's workspace there
    import threading
    cases = [Case([1] * 3, [900, 1300, 40], 2, 4, 64, 16, torch.bfloat16, 97), Case([90, 2], [900, 700], 2, 2, 64, 16, torch.bfloat16, 98)]
    args = [c.device() for c in cases]
    want = [A.attn_paged(*a, causal=True) for a in args]
    _ok(A)
    got = [[], []]

    def calls(k):
        for _ in range(40):
            got[k].append(A.attn_paged(*args[k], causal=True))

    threads = [threading.Thread(target=calls, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    _ok(A)
    for c, w, g in zip(cases, want, got):
        c.check(*w, True)
        assert len(g) == 40 and all(torch.equal(w[0], o) and torch.equal(w[1], l) for o, l in g)


def test_against_attn_fwd_and_decode(A):
    # a whole prompt is the causal forward, its last rows are the causal decode
    B, H, N, d, page = 1, 3, 384, 64, 128
    q, k, v = (W.random_tensor((B, H, N, d), 100 + i, torch.bfloat16).cuda() for i in range(3))
    want, want_lse = A.attn_fwd(q, k, v, causal=True)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    kc, vc = (torch.empty(3, H, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for i, at in enumerate([2, 0, 1]):
        kc[at], vc[at] = k[0, :, i * page:(i + 1) * page], v[0, :, i * page:(i + 1) * page]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    o, lse = A.attn_paged(q[0].transpose(0, 1), kc, vc, table, i32(0, N), i32(N), causal=True)
    od, lsed = A.attn_decode(q[:, :, -5:], k, v, causal=True)
    o5, lse5 = A.attn_paged(q[0, :, -5:].transpose(0, 1), kc, vc, table, i32(0, 5), i32(N), causal=True)
    _ok(A)
    assert_close_bf16("O", o, to64(want[0].transpose(0, 1)))
    assert_lse(lse, want_lse[0])
    assert_close_bf16("O of the last rows", o5, to64(od[0].transpose(0, 1)))
    assert_lse(lse5, lsed[0])


def test_cache_beyond_32_bit_offsets(A):
    # more than 2^32 elements a cache; the pages in use lie at both ends
    hkv, page, d = 8, 256, 128
    pages = (1 << 32) // (hkv * page * d) + 40
    kv, table = [700, 300], np.array([[pages - 1, 3, pages - 2], [pages - 3, 0, UNUSED]])
    k, v = (torch.empty(pages, page, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots, rows = [], []
    for b in range(2):
        slots += [int(table[b, j // page]) * page + j % page for j in range(kv[b])]
    rows = [W.random_tensor((len(slots), hkv, d), 110 + i, torch.bfloat16) for i in range(2)]
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    A.attn_pages_write(rows[0].cuda(), rows[1].cuda(), i32(slots), k.transpose(1, 2), v.transpose(1, 2))
    q = W.random_tensor((4, hkv * 2, d), 112, torch.bfloat16)
    o, lse = A.attn_paged(q.cuda(), k.transpose(1, 2), v.transpose(1, 2), i32(table), i32([0, 1, 4]), i32(kv), causal=True)
    _ok(A)
    ks, vs = to64(rows[0]).transpose(1, 0, 2), to64(rows[1]).transpose(1, 0, 2)
    for b, (r0, r1, k0, k1) in enumerate([(0, 1, 0, 700), (1, 4, 700, 1000)]):
        qs = to64(q[r0:r1]).transpose(1, 0, 2)
        O, L = ref.decode_forward(qs[None], np.repeat(ks[:, k0:k1], 2, 0)[None], np.repeat(vs[:, k0:k1], 2, 0)[None],
                                  1 / math.sqrt(d), True)
        assert_close_bf16("O", o[r0:r1], O[0].transpose(1, 0, 2))
        assert_lse(lse[:, r0:r1], L[0])


def test_captured_call_follows_the_lengths(A):
    c = Case([1, 1, 1], [500, 40, 129], 2, 4, 64, 16, torch.bfloat16, 120)
    q, k, v, table, cu, kv = c.device()
    out, lse = torch.empty_like(q), torch.empty(8, 3, device="cuda")
    ws = torch.empty(A.paged_workspace_size(q, k, v, table, cu, kv, max_q=1), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        A.attn_paged(q, k, v, table, cu, kv, causal=True, max_q=1, out=out, lse=lse, workspace=ws)
    for lengths in ([500, 40, 129], [1, 33, 0], [16, 17, 128]):
        c.kv = lengths
        kv.copy_(torch.tensor(lengths, dtype=torch.int32))
        g.replay()
        _ok(A)
        c.check(out, lse, True)


def test_two_captured_calls_and_an_eager_one_at_once(A):
    # each capture allocates a workspace of its own, and the default stream's is neither
    cases = [Case([1] * 6, [3000, 10, 900, 1, 128, 2048], 2, 4, 64, 32, torch.bfloat16, 121),
             Case([200, 1], [900, 1500], 2, 4, 64, 32, torch.bfloat16, 122)]
    args = [c.device() for c in cases]
    want = [A.attn_paged(*a, causal=True, max_q=max(c.n)) for a, c in zip(args, cases)]
    _ok(A)
    graphs, got, side = [], [], [torch.cuda.Stream() for _ in cases]
    for a, c in zip(args, cases):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(A.attn_paged(*a, causal=True, max_q=max(c.n)))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for o, lse in got:
            o.fill_(9.0)
            lse.fill_(9.0)
        torch.cuda.synchronize()
        for g, s in zip(graphs, side):
            with torch.cuda.stream(s):
                g.replay()
        eager = A.attn_paged(*args[1], causal=True, max_q=200)
        _ok(A)
        for (o, lse), (w, wl) in zip(got + [eager], want + [want[1]]):
            assert torch.equal(o, w) and torch.equal(lse, wl)
    for c, (o, lse) in zip(cases, got):
        c.check(o, lse, True)


def test_longest_table(A):
    # as many keys as a table may have: four pages named over and over. Softmax weights are the pages'
    # multiplicities times exp(s). O's accumulator takes 8 products of 16 keys a tile, each rounded or
    # cut to 2^-23 of it (v > 0, so it only grows), l two additions of 2^-24; P and O round to bf16.
    page, cols, d = 1024, 2 ** 21 - 1, 64
    g = torch.Generator().manual_seed(150)
    k, q = (torch.randn(shape, generator=g).bfloat16() for shape in ((4, 1, page, d), (1, 1, d)))
    v = (1 + torch.rand((4, 1, page, d), generator=g)).bfloat16()
    table = torch.arange(cols, dtype=torch.int32, device="cuda").view(1, -1) % 4
    o, lse = A.attn_paged(q.cuda(), k.cuda(), v.cuda(), table, *(torch.tensor(x, dtype=torch.int32, device="cuda")
                                                                 for x in ([0, 1], [cols * page])), causal=True, max_q=1)
    _ok(A)
    w = np.exp(to64(k)[:, 0] @ to64(q)[0, 0] / math.sqrt(d)) * np.bincount(np.arange(cols) % 4)[:, None]
    want = np.einsum("ps,psd->d", w, to64(v)[:, 0]) / w.sum()
    tiles = cols * page / 128 / torch.cuda.get_device_properties(0).multi_processor_count + 1  # of a CTA, at most
    of_l = tiles * 2 * 2.0 ** -24 + 2.0 ** -20  # and the merge
    assert np.abs(to64(o)[0, 0] / want - 1).max() <= tiles * 8 * 2.0 ** -23 + of_l + 2 * 2.0 ** -8
    assert abs(float(lse[0, 0]) - math.log(w.sum())) <= of_l + 32 * 2.0 ** -24


def test_longest_table_every_page_counts(A):
    # 64 pages that differ in V alone, page p 1 in column p and 0 elsewhere, each named for a 64th of the table in
    # turn: column p of O is that page's share. The keys are the same on every page, so that a CTA's sums grow
    # evenly and the n roundings of a running sum (2^-24 each; 8 of 2^-23 a tile in the accumulator) weigh half of
    # what they do at its end. Keys of one CTA that were left out would take 10 % or more from some column.
    page, cols, d = 1024, 2 ** 21 - 1, 64
    g = torch.Generator().manual_seed(151)
    k1, q = (torch.randn(shape, generator=g).bfloat16() for shape in ((1, 1, page, d), (1, 1, d)))
    k = k1.expand(64, -1, -1, -1).contiguous()
    v = torch.eye(64)[:, None, None, :].expand(-1, 1, page, -1).bfloat16().contiguous()
    table = torch.arange(cols, dtype=torch.int64) * 64 // cols
    o, lse = A.attn_paged(q.cuda(), k.cuda(), v.cuda(), table.int().view(1, -1).cuda(), _i32([0, 1]), _i32([cols * page]),
                          causal=True, max_q=1)
    _ok(A)
    share = np.bincount(table.numpy()) / cols
    tiles = cols * page / 128 / torch.cuda.get_device_properties(0).multi_processor_count + 9  # of a CTA, at most
    of_l = (tiles / 2 + 48) * 2.0 ** -24  # and 35 additions inside a tile, 10 in the merge
    assert np.abs(to64(o)[0, 0] / share - 1).max() <= tiles / 2 * 8 * 2.0 ** -23 + of_l + 2 * 2.0 ** -8
    want = math.log(np.exp(to64(k1)[0, 0] @ to64(q)[0, 0] / math.sqrt(d)).sum() * cols)
    assert abs(float(lse[0, 0]) - want) <= of_l + 2.0 ** -18


@pytest.mark.parametrize("n", [1, 200])
def test_bad_lengths_and_pages_are_reported(A, n):
    # a page out of range, a length that the table cannot hold: no access follows them, attn_status
    # tells, and the other sequences are right
    c = Case([n, 1, n], [300, 90, 210], 2, 2, 64, 32, torch.bfloat16, 130)
    q, k, v, table, cu, kv = c.device()
    for spoil in ("page", "negative page", "length", "negative length"):
        t2, kv2 = table.clone(), kv.clone()
        if "page" in spoil:
            t2[0, 2] = -5 if "negative" in spoil else k.shape[0]
        else:
            kv2[0] = -3 if "negative" in spoil else table.shape[1] * 32 + 1
        o, lse = A.attn_paged(q, k, v, t2, cu, kv2, causal=True, max_q=n)
        torch.cuda.synchronize()
        assert A.attn_status() == A.ATTN_ERR_INVALID and "out of range" in A.last_error()
        assert A.attn_status() == A.ATTN_OK
        O, L = c.oracle(True)
        rest = slice(int(c.cu[1]), int(c.cu[3]))
        assert_close_bf16("O", o[rest], O[rest])
        assert_lse(lse[:, rest], L[:, rest])


@pytest.mark.parametrize("n", [1, 200])
@pytest.mark.parametrize("entry,value,right", [(0, 1, [1, 2]), (0, -1, [0, 1, 2]), (1, -4, [2]), (1, 2 ** 31 - 1, []), (2, 0, []),
                                               (3, 10 ** 6, [0, 1, 2]), (3, -2 ** 31, [0, 1])])
def test_bad_row_offsets_are_reported(A, n, entry, value, right):
    # cu_q that does not begin at 0, decreases or passes the rows of q: nothing outside out and lse is written,
    # attn_status tells, and the sequences whose rows no other one claims are right
    c = Case([n, 1, n], [300, 90, 210], 2, 2, 64, 32, torch.bfloat16, 131)
    q, k, v, table, cu, kv = c.device()
    cu[entry] = value
    room = torch.full((len(q) + 2, 4, 64), 7.0, dtype=c.dtype, device="cuda")
    flat = torch.full((4 * len(q) + 128,), 7.0, device="cuda")
    out, lse = room[1:-1], flat[64:-64].view(4, len(q))
    A.attn_paged(q, k, v, table, cu, kv, max_q=n, out=out, lse=lse)
    torch.cuda.synchronize()
    assert A.attn_status() == A.ATTN_ERR_INVALID and A.attn_status() == A.ATTN_OK
    assert torch.all(room[[0, -1]] == 7.0) and torch.all(flat[:64] == 7.0) and torch.all(flat[-64:] == 7.0)
    O, L = c.oracle(False)
    for b in right:
        rows = slice(int(c.cu[b]), int(c.cu[b + 1]))
        assert_close_bf16("O", out[rows], O[rows])
        assert_lse(lse[:, rows], L[:, rows])


# ---------------------------------------------------------------- writes
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,hkv,d,page,heads_first", [(1, 1, 64, 16, False), (7, 1, 128, 32, True), (300, 3, 64, 16, True),
                                                         (1000, 8, 128, 64, False), (65, 5, 128, 128, False), (9, 16, 128, 16, True)])
def test_write_stores_rows_in_their_slots(A, rows, hkv, d, page, heads_first, dtype):
    pages = rows // page + 5
    shape = (pages, hkv, page, d) if heads_first else (pages, page, hkv, d)
    fused = W.random_tensor((rows, hkv + 2, 2 * d), 200, dtype).cuda()  # k and v as parts of wider rows
    k, v = fused[:, 1:hkv + 1, :d], fused[:, :hkv, d:]
    k[0, 0, 0] = float("nan")
    g = torch.Generator().manual_seed(rows)
    slots = torch.randperm(pages * page, generator=g)[:rows].to(torch.int32)
    slots[rows // 2::5] = -1
    caches = [torch.full(shape, 9.0, dtype=dtype, device="cuda") for _ in range(2)]
    views = [c if heads_first else c.transpose(1, 2) for c in caches]
    A.attn_pages_write(k, v, slots.cuda(), *views)
    _ok(A)
    for src, got in ((k, views[0]), (v, views[1])):
        want = torch.full((pages * page, hkv, d), 9.0, dtype=dtype)
        keep = slots >= 0
        want[slots[keep].long()] = src.cpu()[keep]
        want = want.view(pages, page, hkv, d).transpose(1, 2)
        assert torch.equal(got.cpu().contiguous().view(torch.int16), want.contiguous().view(torch.int16))


def test_write_skips_and_reports_slots_beyond_the_cache(A):
    k, v = (W.random_tensor((3, 2, 64), 210 + i, torch.bfloat16).cuda() for i in range(2))
    caches = [torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    A.attn_pages_write(k, v, torch.tensor([5, 64, 2 ** 31 - 1], dtype=torch.int32, device="cuda"), *caches)
    torch.cuda.synchronize()
    assert A.attn_status() == A.ATTN_ERR_INVALID
    assert torch.equal(caches[0][0, :, 5], k[0]) and torch.equal(caches[1][0, :, 5], v[0])
    assert int((caches[0] != 0).any(-1).sum()) == 2


# ---------------------------------------------------------------- tables
def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _filled_table(rng, lengths, page, cols, spare):
    need = [(n + page - 1) // page for n in lengths]
    order = rng.permutation(sum(need) + spare)
    table, at = np.full((len(lengths), cols), -1, dtype=np.int64), 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    return table, order[at:].tolist()


@pytest.mark.parametrize("seqs,most,page,pad", [(1, 1, 16, 0), (5, 3, 16, 4), (64, 40, 32, 0), (257, 9, 16, 300),
                                                (600, 30, 64, 1), (3, 5000, 128, 17)])
def test_plan_matches_oracle(A, seqs, most, page, pad):
    rng = np.random.default_rng(seqs)
    q_len, old = rng.integers(0, most + 1, seqs), rng.integers(0, 500, seqs)
    old[rng.random(seqs) < 0.3] //= page
    cols = int(max((old + q_len).max() + page - 1, page) // page) + 1
    table, free = _filled_table(rng, old, page, cols, int(((q_len + page - 1) // page + 1).sum()))
    total = int(q_len.sum()) + pad
    want = paged.plan(q_len.tolist(), old.tolist(), table, free, len(free), page, total)
    args = [_i32(q_len), _i32(old), _i32(table), _i32(free + [77, 78]), _i32([len(free)])]
    for _ in range(2):  # the inputs stay as they are, so a second call gives the same
        got = A.attn_pages_plan(*args, page, total)
        _ok(A)
        for name, g, w in zip(("cu_q", "new_len", "slots", "positions", "free_left"), got, want):
            assert g.cpu().tolist() == (w if isinstance(w, list) else [w]), name
        assert args[2].cpu().tolist() == [[int(x) for x in r] for r in want[5]]


def test_plan_without_sequences_or_rows(A):
    empty = _i32([]).view(-1)
    cu, new, slots, pos, left = A.attn_pages_plan(empty, empty, _i32(np.zeros((0, 3))), _i32([4, 5]), _i32([2]), 16, 3)
    _ok(A)
    assert cu.tolist() == [0] and new.numel() == 0 and slots.tolist() == [-1] * 3 and pos.tolist() == [-1] * 3
    assert left.tolist() == [2]
    cu, new, slots, pos, left = A.attn_pages_plan(_i32([0, 0]), _i32([3, 0]), _i32([[1], [-1]]), empty, _i32([0]), 16, 0)
    _ok(A)
    assert cu.tolist() == [0, 0, 0] and new.tolist() == [3, 0] and slots.numel() == 0 and left.tolist() == [0]


def test_plan_that_runs_out_of_pages(A):
    args = ([20, 40, 1], [10, 0, 5], [[2, -1, -1], [-1, -1, -1], [0, -1, -1]], [8, 6])
    want = paged.plan(*args, 2, 16, 61)
    table = _i32(args[2])
    got = A.attn_pages_plan(_i32(args[0]), _i32(args[1]), table, _i32(args[3]), _i32([2]), 16, 61)
    _ok(A)
    assert want[4] == -2 and got[4].tolist() == [-2]
    assert got[2].tolist() == want[2] and table.tolist() == want[5]


def test_plan_reports_lengths_out_of_range(A):
    table, free = [[0, 1]], _i32([2, 3])
    for q_len, old, total in ([40], [0], 40), ([-1], [4], 4), ([1], [-2], 4), ([5], [0], 3), ([2 ** 31 - 1], [2 ** 31 - 1], 8):
        t = _i32(table)
        A.attn_pages_plan(_i32(q_len), _i32(old), t, free, _i32([2]), 16, total)
        torch.cuda.synchronize()
        assert A.attn_status() == A.ATTN_ERR_INVALID
    # a stack pointer beyond the stack, a page that the table does not name
    for count, t, old in (9, [[0, 1]], 3), (2, [[-1, 1]], 3):
        A.attn_pages_plan(_i32([14]), _i32([old]), _i32(t), free, _i32([count]), 16, 14)
        torch.cuda.synchronize()
        assert A.attn_status() == A.ATTN_ERR_INVALID


def test_plan_reports_pages_below_zero_on_the_stack(A):
    # as a release of a sequence that was never given all its pages leaves them
    table = _i32([[-1, -1], [-1, -1]])
    cu, new, slots, pos, left = A.attn_pages_plan(_i32([17, 2]), _i32([0, 0]), table, _i32([5, -1, 7]), _i32([3]), 16, 19)
    torch.cuda.synchronize()
    assert A.attn_status() == A.ATTN_ERR_INVALID and A.attn_status() == A.ATTN_OK
    assert slots.tolist() == list(range(7 * 16, 8 * 16)) + [-1] + [80, 81] and left.tolist() == [0]
    assert table.tolist() == [[7, -1], [5, -1]]


def test_tables_into_given_tensors_on_another_stream(A):
    side = torch.cuda.Stream()
    lens, table, free, count = _i32([5, 16]), _i32([[3, -1], [2, -1]]), _i32([0, 1, 4, 0]), _i32([3])
    outs = {n: _i32([9] * m) for n, m in (("cu_q", 3), ("new_len", 2), ("slots", 5), ("positions", 5), ("free_left", 1))}
    side.wait_stream(torch.cuda.current_stream())
    got = A.attn_pages_plan(_i32([2, 1]), lens, table, free, count, 16, 5, stream=side, **outs)
    new, left = A.attn_pages_release(_i32([0, 1]), got[1], table, free, got[4], 16, new_len=_i32([8, 8]), stream=side)
    _ok(A)
    assert all(g is outs[n] for g, n in zip(got, outs))
    assert [outs[n].tolist() for n in outs] == [[0, 2, 3], [7, 17], [53, 54, 64, -1, -1], [5, 6, 16, -1, -1], [2]]
    assert table.tolist() == [[3, -1], [2, 4]] and new.tolist() == [7, 0] and left.tolist() == [4]
    assert free.tolist() == [0, 1, 2, 4]


def test_arrays_between_the_rows_of_a_wider_table(A):
    # the counts lie in the columns that the table leaves over: no overlap
    wide = _i32([[3, -1, 3, 9], [2, -1, 9, 9], [0, -1, 9, 9]])
    table, count, left = wide[:, :2], wide[0, 2:3], wide[1, 3:4]
    cu, new, slots, _, got = A.attn_pages_plan(_i32([2, 1, 1]), _i32([15, 16, 3]), table, _i32([4, 5, 6]), count, 16, 4, free_left=left)
    _ok(A)
    assert got is left and wide.tolist() == [[3, 6, 3, 9], [2, 5, 9, 1], [0, -1, 9, 9]]
    assert slots.tolist() == [63, 96, 80, 3]
    stack = _i32([4, 0, 0, 0])
    A.attn_pages_release(_i32([0, 1, 1]), new, table, stack, left, 16, new_len=new.clone(), free_left=wide[0, 3:4])
    _ok(A)
    assert stack.tolist() == [4, 2, 5, 0] and wide[0].tolist() == [3, 6, 3, 4]


@pytest.mark.parametrize("seqs,page,every", [(1, 16, 1), (9, 32, 2), (777, 16, 3), (5000, 16, 7), (40, 256, 1), (6, 16, 99)])
def test_release_matches_oracle(A, seqs, page, every):
    rng = np.random.default_rng(seqs + 1)
    lengths = rng.integers(0, 900 if seqs < 1000 else 60, seqs)
    cols = int(max(lengths.max() + page - 1, page) // page)
    table, free = _filled_table(rng, lengths, page, cols, 11)
    done = (np.arange(seqs) % every == every - 1).astype(int) * 3
    room = int((table >= 0).sum())
    want = paged.release(done, lengths, table, free + [0] * room, len(free), page)
    stack = _i32(free + [0] * room)
    new, left = A.attn_pages_release(_i32(done), _i32(lengths), _i32(table), stack, _i32([len(free)]), page)
    _ok(A)
    assert new.tolist() == want[0] and left.tolist() == [want[1]] and stack.tolist() == want[2]


def test_release_reports_pages_that_were_never_given(A):
    stack = _i32([5, 0, 0, 0])
    A.attn_pages_release(_i32([1]), _i32([40]), _i32([[1, -1, -1]]), stack, _i32([1]), 16)
    torch.cuda.synchronize()
    assert A.attn_status() == A.ATTN_ERR_INVALID


def test_release_reports_a_stack_that_cannot_hold_the_pages(A):
    stack = _i32([5, 0, 0])
    A.attn_pages_release(_i32([1]), _i32([64]), _i32([[1, 2, 3, 4]]), stack, _i32([1]), 16)
    torch.cuda.synchronize()
    assert A.attn_status() == A.ATTN_ERR_INVALID and stack.tolist() == [5, 1, 2]
    empty = _i32([]).view(-1)
    new, left = A.attn_pages_release(empty, empty, _i32(np.zeros((0, 2))), stack, _i32([3]), 16)
    _ok(A)
    assert new.numel() == 0 and left.tolist() == [3]


# ---------------------------------------------------------------- all of it, as a server runs it
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
def test_serving_steps_match_attention_over_the_whole_sequences(A, d, page):
    """Prompts come in chunks, sequences decode, end, and give their pages to new ones; after each
    step every sequence's rows are checked against attention over all of its keys."""
    hkv, group, columns, pages = 2, 3, 400 // page, 40 * 16 // page
    dev = "cuda"
    rng = np.random.default_rng(d)
    k_cache, v_cache = (torch.full((pages, page, hkv, d), float("nan"), dtype=torch.bfloat16, device=dev).transpose(1, 2)
                        for _ in range(2))
    table, lens = _i32(np.full((3, columns), -1)), _i32([0, 0, 0])
    free, count = _i32(rng.permutation(pages)), _i32([pages])
    keys = [[np.zeros((hkv, 0, d))] * 2 for _ in range(3)]
    for step, (q_len, done) in enumerate([([130, 0, 3], None), ([50, 20, 1], None), ([1, 1, 1], [0, 0, 1]), ([1, 1, 60], None),
                                          ([1, 0, 1], [1, 0, 0]), ([90, 5, 1], None), ([1, 1, 1], None)]):
        rows = sum(q_len) + step % 3
        cu, lens, slots, pos, count = A.attn_pages_plan(_i32(q_len), lens, table, free, count, page, rows)
        q, k, v = (W.random_tensor((rows, hkv * (group if i == 0 else 1), d), 300 + 10 * step + i, torch.bfloat16) for i in range(3))
        A.attn_pages_write(k.to(dev), v.to(dev), slots, k_cache, v_cache)
        o, lse = A.attn_paged(q.to(dev), k_cache, v_cache, table, cu, lens, causal=True, max_q=max(q_len))
        _ok(A)
        r0 = 0
        for b, n in enumerate(q_len):
            keys[b] = [np.concatenate([old, to64(x[r0:r0 + n]).transpose(1, 0, 2)], 1) for old, x in zip(keys[b], (k, v))]
            if n:
                O, L = ref.decode_forward(to64(q[r0:r0 + n]).transpose(1, 0, 2)[None], np.repeat(keys[b][0], group, 0)[None],
                                          np.repeat(keys[b][1], group, 0)[None], 1 / math.sqrt(d), True)
                assert_close_bf16(f"O step {step}", o[r0:r0 + n], O[0].transpose(1, 0, 2))
                assert_lse(lse[:, r0:r0 + n], L[0])
            r0 += n
        assert lens.tolist() == [x[0].shape[1] for x in keys]
        if done is not None:
            lens, count = A.attn_pages_release(_i32(done), lens, table, free, count, page)
            for b in range(3):
                if done[b]:
                    keys[b] = [x[:, :0] for x in keys[b]]
        held = sum((x[0].shape[1] + page - 1) // page for x in keys)
        _ok(A)
        assert count.tolist() == [pages - held]


def test_captured_decode_loop(A):
    """One captured step (plan, write, attend, take the step) replayed across page ends."""
    hkv, group, d, page, seqs = 1, 2, 64, 16, 3
    rng = np.random.default_rng(8)
    pages, start, steps = 30, [14, 31, 0], 20
    k_cache, v_cache = (torch.full((pages, hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table, lens = _i32(np.full((seqs, 8), -1)), _i32([0] * seqs)
    free, count = _i32(rng.permutation(pages)), _i32([pages])
    fill = [W.random_tensor((sum(start), hkv, d), 400 + i, torch.bfloat16) for i in range(2)]
    _, lens2, slots, _, count2 = A.attn_pages_plan(_i32(start), lens, table, free, count, page, sum(start))
    A.attn_pages_write(fill[0].cuda(), fill[1].cuda(), slots, k_cache, v_cache)
    lens.copy_(lens2)
    count.copy_(count2)
    ones = _i32([1] * seqs)
    q, k, v = (torch.zeros(seqs, hkv * (group if i == 0 else 1), d, dtype=torch.bfloat16, device="cuda") for i in range(3))

    def one_step():
        cu, new, slots, _, left = A.attn_pages_plan(ones, lens, table, free, count, page, seqs)
        A.attn_pages_write(k, v, slots, k_cache, v_cache)
        o, lse = A.attn_paged(q, k_cache, v_cache, table, cu, new, causal=True, max_q=1)
        lens.copy_(new)
        count.copy_(left)
        return o, lse

    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = one_step()
    at, keys = 0, []
    for b in range(seqs):
        keys.append([to64(x[at:at + start[b]]).transpose(1, 0, 2) for x in fill])
        at += start[b]
    for step in range(steps):
        new = [W.random_tensor(t.shape, 410 + 3 * step + i, torch.bfloat16) for i, t in enumerate((q, k, v))]
        for t, x in zip((q, k, v), new):
            t.copy_(x)
        g.replay()
        _ok(A)
        for b in range(seqs):
            keys[b] = [np.concatenate([old, to64(x[b:b + 1]).transpose(1, 0, 2)], 1) for old, x in zip(keys[b], new[1:])]
            O, L = ref.decode_forward(to64(new[0][b:b + 1]).transpose(1, 0, 2)[None], np.repeat(keys[b][0], group, 0)[None],
                                      np.repeat(keys[b][1], group, 0)[None], 1 / math.sqrt(d), True)
            assert_close_bf16("O", o[b:b + 1], O[0].transpose(1, 0, 2))
            assert_lse(lse[:, b:b + 1], L[0])
    assert lens.tolist() == [s + steps for s in start]
