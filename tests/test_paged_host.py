"""The paged cache without a GPU: the oracle's pins, the C structs against their ctypes mirrors, and
the refusals of the C entry points and of the binding."""
import ctypes
import math
import os
import subprocess
import tempfile

import numpy as np
import pytest
import torch

from oracle import paged, ref
from test_abi import _build_library

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def A():
    _build_library()
    import attn_fwd_03_gb300 as m
    return m


# ---------------------------------------------------------------- the oracle
def _scatter(k, page_size, order, num_pages):
    """A cache [pages, heads, page_size, d] that holds k [heads, n, d] in pages `order`; NaN elsewhere."""
    cache = np.full((num_pages, k.shape[0], page_size, k.shape[2]), np.nan)
    for j in range(k.shape[1]):
        cache[order[j // page_size], :, j % page_size] = k[:, j]
    return cache


@pytest.mark.parametrize("causal", [False, True])
def test_oracle_equals_contiguous_decode(causal):
    rng = np.random.default_rng(5)
    hkv, group, n, nk, d, page = 2, 3, 5, 37, 8, 16
    q, k, v = rng.normal(size=(n, hkv * group, d)), rng.normal(size=(hkv, nk, d)), rng.normal(size=(hkv, nk, d))
    order = [4, 0, 2]
    o, lse = paged.paged_forward(np.concatenate([q, q[:1]]), _scatter(k, page, order, 5), _scatter(v, page, order, 5),
                                 [order], [0, n], [nk], 0.3, causal)
    for h in range(hkv * group):
        O, L = ref.decode_forward(q[None, None, :, h], k[None, None, h // group], v[None, None, h // group], 0.3, causal)
        np.testing.assert_allclose(o[:n, h], O[0, 0], rtol=0, atol=1e-14)
        np.testing.assert_allclose(lse[h, :n], L[0, 0], rtol=0, atol=1e-14)
    assert np.isnan(o[n:]).all() and np.isnan(lse[:, n:]).all()


def test_oracle_rows_without_keys():
    q = np.ones((4, 1, 2))
    cache = np.ones((1, 1, 16, 2))
    o, lse = paged.paged_forward(q, cache, cache, [[0], [0]], [0, 3, 4], [1, 0], 1.0, True)
    assert np.all(o[:2] == 0) and np.all(np.isneginf(lse[0, :2]))  # 3 rows, 1 key: the last row alone sees it
    assert np.all(o[2] == 1) and math.isclose(lse[0, 2], 2.0)
    assert np.all(o[3] == 0) and np.isneginf(lse[0, 3])


def test_oracle_plan_worked_example():
    # pages of 16; sequence 0 has 15 tokens in page 7 and gets 2; sequence 1 is new and gets 17; sequence 2 rests
    cu, new, slots, pos, left, table = paged.plan([2, 17, 0], [15, 0, 3], [[7, -1], [-1, -1], [1, -1]],
                                                  [10, 11, 12, 13], 4, 16, 21)
    assert cu == [0, 2, 19, 19] and new == [17, 17, 3] and left == 1
    assert table == [[7, 13], [12, 11], [1, -1]]
    assert slots == [7 * 16 + 15, 13 * 16] + [12 * 16 + i for i in range(16)] + [11 * 16, -1, -1]
    assert pos == [15, 16] + list(range(17)) + [-1, -1]


def test_oracle_release_undoes_plan():
    free, table = [3, 5, 8, 9], [[-1, -1], [-1, -1]]
    _, new, _, _, left, table = paged.plan([20, 5], [0, 0], table, free, 4, 16, 25)
    new2, back, stack = paged.release([1, 0], new, table, free, left, 16)
    assert new2 == [0, 5] and back == 3
    assert set(stack[:3]) | {table[1][0]} == set(free)


# ---------------------------------------------------------------- structs
def test_struct_layout_matches_c(A):
    fields = {
        "attn_paged_params": (A.PagedParams, ["q", "table_stride", "q_stride", "v_stride", "workspace_bytes", "scale"]),
        "attn_pages_write_params": (A.PagesWriteParams, ["k", "slots", "k_row_stride", "v_stride", "reserved0"]),
        "attn_pages_plan_params": (A.PagesPlanParams, ["q_len", "table_stride", "free_count", "free_left"]),
        "attn_pages_release_params": (A.PagesReleaseParams, ["done", "table_stride", "free_pages", "free_left"]),
    }
    lines, want = [], []
    for c, (mirror, names) in fields.items():
        lines.append(f'printf("%zu\\n", sizeof({c}));')
        want.append(ctypes.sizeof(mirror))
        for n in names:
            lines.append(f'printf("%zu\\n", offsetof({c}, {n}));')
            want.append(getattr(mirror, n).offset)
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "attn.h"\nint main(void) {' + "\n".join(lines) + "return 0; }"
    with tempfile.TemporaryDirectory() as td:
        c, exe = os.path.join(td, "l.c"), os.path.join(td, "l")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == want


# ---------------------------------------------------------------- refusals at the C entry points
FAKE = 1 << 20  # never dereferenced: every case below fails a check first


def _filled(struct, **kw):
    p = struct()
    for name, kind in struct._fields_:
        if kind is ctypes.c_void_p:
            setattr(p, name, FAKE)
    for name, value in kw.items():
        arr = dict(struct._fields_)[name]
        setattr(p, name, arr(*value) if isinstance(value, tuple) else value)
    return p


def _paged(A, **kw):
    base = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, d=64, total_q=10, max_q=1, num_pages=9, page_size=16, max_pages=4,
                dtype=A.ATTN_BF16, causal=1, scale=0.125, table_stride=4, q_stride=(512, 64), o_stride=(512, 64),
                k_stride=(2048, 64, 128), v_stride=(2048, 64, 128), workspace=FAKE, workspace_bytes=1 << 40)
    return _filled(A.PagedParams, **{**base, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(num_seqs=-1), "ATTN_ERR_INVALID"),
    (dict(total_q=-1), "ATTN_ERR_INVALID"),
    (dict(num_kv_heads=0), "ATTN_ERR_INVALID"),
    (dict(num_q_heads=7), "ATTN_ERR_INVALID"),
    (dict(num_q_heads=258, num_kv_heads=2), "ATTN_ERR_UNSUPPORTED"),
    (dict(num_q_heads=65536, num_kv_heads=65536), "ATTN_ERR_UNSUPPORTED"),
    (dict(d=256), "ATTN_ERR_UNSUPPORTED"),
    (dict(dtype=1), "ATTN_ERR_UNSUPPORTED"),
    (dict(dtype=3), "ATTN_ERR_UNSUPPORTED"),
    (dict(dtype=9), "ATTN_ERR_INVALID"),
    (dict(causal=2), "ATTN_ERR_INVALID"),
    (dict(scale=0.0), "ATTN_ERR_INVALID"),
    (dict(scale=float("inf")), "ATTN_ERR_INVALID"),
    (dict(max_q=0), "ATTN_ERR_INVALID"),
    (dict(reserved0=(0, 1)), "ATTN_ERR_INVALID"),
    (dict(page_size=0), "ATTN_ERR_INVALID"),
    (dict(page_size=8), "ATTN_ERR_UNSUPPORTED"),
    (dict(page_size=48), "ATTN_ERR_UNSUPPORTED"),
    (dict(max_pages=0), "ATTN_ERR_INVALID"),
    (dict(max_pages=1 << 27), "ATTN_ERR_UNSUPPORTED"),
    (dict(max_pages=(1 << 27) - 1), "ATTN_ERR_UNSUPPORTED"),
    (dict(page_size=512, max_pages=(1 << 22) - 1), "ATTN_ERR_UNSUPPORTED"),
    (dict(num_pages=0), "ATTN_ERR_INVALID"),
    (dict(num_pages=1 << 27), "ATTN_ERR_UNSUPPORTED"),
    (dict(table_stride=-1), "ATTN_ERR_INVALID"),
    (dict(q=0), "ATTN_ERR_INVALID"),
    (dict(lse=0), "ATTN_ERR_INVALID"),
    (dict(block_table=0), "ATTN_ERR_INVALID"),
    (dict(cu_q=FAKE + 2), "ATTN_ERR_ALIGN"),
    (dict(v_cache=FAKE + 8), "ATTN_ERR_ALIGN"),
    (dict(q_stride=(516, 64)), "ATTN_ERR_ALIGN"),
    (dict(k_stride=(2048, 0, 128)), "ATTN_ERR_INVALID"),
    (dict(o_stride=(1 << 38, 64)), "ATTN_ERR_UNSUPPORTED"),
])
def test_paged_refusals(A, kw, status):
    p = _paged(A, **kw)
    assert A.lib.attn_paged(ctypes.byref(p), None) == getattr(A, status)
    assert A.last_error() != ""
    assert A.lib.attn_paged_workspace_size(ctypes.byref(p)) == 0


@pytest.mark.parametrize("kw", [dict(num_seqs=0), dict(total_q=0)])
def test_paged_empty_is_a_no_op(A, kw):
    p = _paged(A, **kw, q=0, o=0, lse=0, cu_q=0, kv_len=0, block_table=0, workspace=0)
    assert A.lib.attn_paged(ctypes.byref(p), None) == A.ATTN_OK
    assert A.lib.attn_paged_workspace_size(ctypes.byref(p)) == 0


def _write(A, **kw):
    base = dict(rows=3, num_kv_heads=2, d=64, num_pages=4, page_size=16, dtype=A.ATTN_F16, k_row_stride=(128, 64),
                v_row_stride=(128, 64), k_stride=(2048, 64, 128), v_stride=(2048, 64, 128))
    return _filled(A.PagesWriteParams, **{**base, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), "ATTN_ERR_INVALID"),
    (dict(num_kv_heads=0), "ATTN_ERR_INVALID"),
    (dict(d=80), "ATTN_ERR_UNSUPPORTED"),
    (dict(dtype=1), "ATTN_ERR_UNSUPPORTED"),
    (dict(page_size=24), "ATTN_ERR_UNSUPPORTED"),
    (dict(num_pages=0), "ATTN_ERR_INVALID"),
    (dict(slots=0), "ATTN_ERR_INVALID"),
    (dict(k=FAKE + 4), "ATTN_ERR_ALIGN"),
    (dict(k_cache=0), "ATTN_ERR_INVALID"),
    (dict(v_row_stride=(100, 64)), "ATTN_ERR_ALIGN"),
    (dict(reserved0=(1, 0)), "ATTN_ERR_INVALID"),
])
def test_write_refusals(A, kw, status):
    p = _write(A, **kw)
    assert A.lib.attn_pages_write(ctypes.byref(p), None) == getattr(A, status)
    assert A.last_error() != ""


def test_write_of_nothing_is_a_no_op(A):
    p = _write(A, rows=0, k=0, v=0, slots=0, k_cache=0, v_cache=0)
    assert A.lib.attn_pages_write(ctypes.byref(p), None) == A.ATTN_OK


def _plan(A, **kw):
    base = dict(num_seqs=2, total_q=5, page_size=16, max_pages=4, free_capacity=8, table_stride=4, q_len=FAKE + 64,
                kv_len=FAKE + 128, new_len=FAKE + 256, free_left=FAKE + 512)
    return _filled(A.PagesPlanParams, **{**base, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(num_seqs=-2), "ATTN_ERR_INVALID"),
    (dict(total_q=-2), "ATTN_ERR_INVALID"),
    (dict(free_capacity=-1), "ATTN_ERR_INVALID"),
    (dict(page_size=10), "ATTN_ERR_UNSUPPORTED"),
    (dict(max_pages=0), "ATTN_ERR_INVALID"),
    (dict(table_stride=3), "ATTN_ERR_INVALID"),
    (dict(free_left=FAKE), "ATTN_ERR_INVALID"),     # free_count itself
    (dict(new_len=FAKE + 128), "ATTN_ERR_INVALID"),  # kv_len itself
    (dict(q_len=0), "ATTN_ERR_INVALID"),
    (dict(slots=0), "ATTN_ERR_INVALID"),
    (dict(positions=FAKE + 1), "ATTN_ERR_ALIGN"),
    (dict(free_pages=0), "ATTN_ERR_INVALID"),
    (dict(reserved0=7), "ATTN_ERR_INVALID"),
])
def test_plan_refusals(A, kw, status):
    p = _plan(A, **kw)
    assert A.lib.attn_pages_plan(ctypes.byref(p), None) == getattr(A, status)
    assert A.last_error() != ""


@pytest.mark.parametrize("kw,status", [
    (dict(num_seqs=-2), "ATTN_ERR_INVALID"),
    (dict(page_size=-16), "ATTN_ERR_INVALID"),
    (dict(table_stride=1), "ATTN_ERR_INVALID"),
    (dict(free_left=FAKE), "ATTN_ERR_INVALID"),
    (dict(new_len=FAKE + 128), "ATTN_ERR_INVALID"),
    (dict(done=0), "ATTN_ERR_INVALID"),
    (dict(block_table=FAKE + 3), "ATTN_ERR_ALIGN"),
])
def test_release_refusals(A, kw, status):
    base = dict(num_seqs=2, page_size=16, max_pages=4, free_capacity=8, table_stride=4, done=FAKE + 64, kv_len=FAKE + 128,
                new_len=FAKE + 256, free_left=FAKE + 512)
    p = _filled(A.PagesReleaseParams, **{**base, **kw})
    assert A.lib.attn_pages_release(ctypes.byref(p), None) == getattr(A, status)
    assert A.last_error() != ""


# a plan's or release's arrays: entries, and whether the call writes them (2 sequences of 4 table columns, 5 rows)
ARRAYS = {
    "plan": dict(q_len=(2, False), kv_len=(2, False), block_table=(8, True), free_pages=(8, False), free_count=(1, False),
                 cu_q=(3, True), new_len=(2, True), slots=(5, True), positions=(5, True), free_left=(1, True)),
    "release": dict(done=(2, False), kv_len=(2, False), block_table=(8, False), free_pages=(8, True), free_count=(1, False),
                    new_len=(2, True), free_left=(1, True)),
}


@pytest.mark.parametrize("call,first,second", [(call, a, b) for call, arrays in ARRAYS.items() for a in arrays for b in arrays
                                               if a != b and arrays[a][1]])
def test_overlapping_table_arrays_are_refused(A, call, first, second):
    # the second array starts at the first one's last entry, or ends in its first one
    arrays = ARRAYS[call]
    for ends in (False, True):
        at = {name: FAKE + 64 * i for i, name in enumerate(arrays)}
        at[second] = at[first] - 4 * (arrays[second][0] - 1) if ends else at[first] + 4 * (arrays[first][0] - 1)
        sizes = dict(num_seqs=2, page_size=16, max_pages=4, free_capacity=8, table_stride=4)
        if call == "plan":
            p = _filled(A.PagesPlanParams, total_q=5, **sizes, **at)
        else:
            p = _filled(A.PagesReleaseParams, **sizes, **at)
        assert getattr(A.lib, f"attn_pages_{call}")(ctypes.byref(p), None) == A.ATTN_ERR_INVALID
        assert "overlap" in A.last_error() and first in A.last_error() and second in A.last_error()


@pytest.mark.parametrize("name,entries", [("free_left", [0, 3, 7, 10, 14, 17]), ("cu_q", [-3, 0, 4, 10, 11, 17])])
def test_overlap_with_a_row_of_a_wider_table_is_refused(A, name, entries):
    # 3 rows of 4 columns, 7 entries apart; free_left has 1 entry, cu_q 4
    for entry in entries:
        table = FAKE + 4096
        p = _plan(A, num_seqs=3, table_stride=7, block_table=table, **{name: table + 4 * entry})
        assert A.lib.attn_pages_plan(ctypes.byref(p), None) == A.ATTN_ERR_INVALID
        assert f"block_table and {name} overlap" in A.last_error()


@pytest.mark.parametrize("num_seqs", [2 ** 31 - 1023, 2 ** 31 - 1])
def test_too_many_sequences_or_rows_are_refused(A, num_seqs):
    # the kernels' 32-bit loops over the sequences and over a sequence's rows would wrap and not end
    assert A.lib.attn_paged(ctypes.byref(_paged(A, total_q=num_seqs)), None) == A.ATTN_ERR_UNSUPPORTED
    assert "total_q" in A.last_error()
    release = _filled(A.PagesReleaseParams, num_seqs=num_seqs, page_size=16, max_pages=4, free_capacity=8, table_stride=4)
    for name, p in (("attn_paged", _paged(A, num_seqs=num_seqs)), ("attn_pages_plan", _plan(A, num_seqs=num_seqs)),
                    ("attn_pages_release", release)):
        assert getattr(A.lib, name)(ctypes.byref(p), None) == A.ATTN_ERR_UNSUPPORTED
        assert "num_seqs" in A.last_error()


def test_null_params(A):
    for name in ("attn_paged", "attn_pages_write", "attn_pages_plan", "attn_pages_release"):
        assert getattr(A.lib, name)(None, None) == A.ATTN_ERR_INVALID
    assert A.lib.attn_paged_workspace_size(None) == 0


# ---------------------------------------------------------------- refusals of the binding
def _attend_args(**kw):
    a = dict(q=torch.zeros(3, 4, 64, dtype=torch.bfloat16), k=torch.zeros(5, 2, 16, 64, dtype=torch.bfloat16),
             v=torch.zeros(5, 2, 16, 64, dtype=torch.bfloat16), table=torch.zeros(2, 3, dtype=torch.int32),
             cu=torch.zeros(3, dtype=torch.int32), n=torch.zeros(2, dtype=torch.int32))
    opts = {k: kw.pop(k) for k in list(kw) if k not in a}
    a.update(kw)
    return tuple(a.values()), opts


@pytest.mark.parametrize("kw,error", [
    (dict(), ValueError),  # all well but on the CPU
    (dict(q=torch.zeros(3, 4, 64)), TypeError),
    (dict(k=torch.zeros(5, 2, 16, 64, dtype=torch.float16)), TypeError),
    (dict(v=torch.zeros(5, 1, 16, 64, dtype=torch.bfloat16)), ValueError),
    (dict(v=torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)), ValueError),
    (dict(k=torch.zeros(5, 2, 64, 16, dtype=torch.bfloat16).transpose(2, 3)), ValueError),
    (dict(table=torch.zeros(2, 3, dtype=torch.int64)), TypeError),
    (dict(cu=torch.zeros(2, dtype=torch.int32)), ValueError),
    (dict(n=torch.zeros(4, dtype=torch.int32)[::2]), ValueError),
    (dict(out=torch.zeros(3, 4, 128, dtype=torch.bfloat16)), ValueError),
    (dict(lse=torch.zeros(3, 4)), ValueError),
    (dict(lse=torch.zeros(4, 6)[:, :3]), ValueError),
])
def test_binding_attend_refusals(A, kw, error):
    args, opts = _attend_args(**kw)
    with pytest.raises(error):
        A.attn_paged(*args, **opts)


class _OnDevice(torch.Tensor):
    """A CPU tensor that says it is on cuda:1."""

    def get_device(self):
        return 1


def test_workspace_size_is_asked_on_the_tensors_device(A, monkeypatch):
    import contextlib
    import types

    from attn_fwd_03_gb300 import _paged
    current, asked = [0], []

    @contextlib.contextmanager
    def device(dev):
        before, current[0] = current[0], dev
        yield
        current[0] = before

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(_paged, "lib", types.SimpleNamespace(attn_paged_workspace_size=lambda p: asked.append(current[0]) or 4096))
    args, _ = _attend_args()
    assert A.paged_workspace_size(*args) == 4096
    assert A.paged_workspace_size(args[0].as_subclass(_OnDevice), *args[1:]) == 4096
    assert asked == [0, 1] and current == [0]


def test_binding_write_refusals(A):
    k = torch.zeros(3, 2, 64, dtype=torch.float16)
    cache = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    slots = torch.zeros(3, dtype=torch.int32)
    for args, error in [((k, k, slots, cache, cache), ValueError),  # on the CPU
                        ((k, k[:2], slots, cache, cache), ValueError),
                        ((k, k, slots[:2], cache, cache), ValueError),
                        ((k, k, slots.long(), cache, cache), TypeError),
                        ((k, k, slots, cache.bfloat16(), cache), TypeError),
                        ((k, k, slots, cache[:, :1], cache), ValueError)]:
        with pytest.raises(error):
            A.attn_pages_write(*args)


@pytest.mark.parametrize("page_size", [16.5, 0.5, 0, -16, 2 ** 31, float("nan")])
def test_binding_page_size_refusals(A, page_size):
    from attn_fwd_03_gb300 import _paged
    with pytest.raises(ValueError, match="page_size"):
        _paged._page_size(page_size)
    assert _paged._page_size(16) == 16


def test_binding_tables_refusals(A):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    for args, kw, error in [((i(2), i(2), i(2, 3), i(9), i(1), 16, 4), {}, ValueError),  # on the CPU
                            ((i(2), i(3), i(2, 3), i(9), i(1), 16, 4), {}, ValueError),
                            ((i(2), i(2), i(3, 3), i(9), i(1), 16, 4), {}, ValueError),
                            ((i(2).long(), i(2), i(2, 3), i(9), i(1), 16, 4), {}, TypeError),
                            ((i(2), i(2), i(3, 2).t(), i(9), i(1), 16, 4), {}, ValueError),
                            ((i(2), i(2), i(2, 3), i(9), i(2), 16, 4), {}, ValueError),
                            ((i(2), i(2), i(2, 3), i(9), i(1), 16, 4), {"slots": i(5)}, ValueError)]:
        with pytest.raises(error):
            A.attn_pages_plan(*args, **kw)
    for args, error in [((i(2), i(2), i(2, 3), i(9), i(1), 16), ValueError),
                        ((i(2), i(2), i(2, 3), i(9).long(), i(1), 16), TypeError),
                        ((i(2, 1), i(2), i(2, 3), i(9), i(1), 16), ValueError)]:
        with pytest.raises(error):
            A.attn_pages_release(*args)
