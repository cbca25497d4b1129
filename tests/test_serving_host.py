"""Rotary positions, the 8-bit cache and trees without a GPU: the oracle's pins, the C structs against their ctypes
mirrors, the table of frequencies, and the refusals of the C entry points and of the binding."""
import ctypes
import math
import os
import subprocess
import tempfile

import numpy as np
import pytest
import torch

from oracle import paged, serving
from test_abi import _build_library
from test_paged_host import FAKE, ROOT, _filled, _scatter


@pytest.fixture(scope="module")
def A():
    _build_library()
    import attn_fwd_03_gb300 as m
    return m


# ---------------------------------------------------------------- the oracle
def test_oracle_turns():
    assert serving.turn_of(0, 1.0) == 0.0
    assert math.isclose(serving.turn_of(1, 1.0), 1 / (2 * math.pi), rel_tol=1e-15)
    assert math.isclose(serving.turn_of(7, 1.0), 7 / (2 * math.pi) - 1, rel_tol=1e-14)
    # 355 / 113 is pi to 7 digits: 710 is nearly 113 turns
    assert math.isclose(serving.turn_of(710, 1.0), (710 - 113 * 2 * math.pi) / (2 * math.pi), rel_tol=1e-8)


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rotation_is_a_complex_product_and_its_transpose(interleaved):
    rng = np.random.default_rng(1)
    x, y, freq, pos = rng.normal(size=(3, 10)), rng.normal(size=(3, 10)), [1.0, 0.25, 3e-3], [0, 5, 1000]
    got = serving.rotate(x, pos, freq, interleaved, 1.5)
    z = x[:, :6].reshape(3, 3, 2) if interleaved else np.stack([x[:, :3], x[:, 3:6]], -1)
    w = 1.5 * (z[..., 0] + 1j * z[..., 1]) * np.exp(1j * np.outer(pos, freq))
    want = np.stack([w.real, w.imag], -1).reshape(3, 6) if interleaved else np.concatenate([w.real, w.imag], 1)
    np.testing.assert_allclose(got[:, :6], want, atol=1e-12)
    assert np.array_equal(got[:, 6:], x[:, 6:])
    back = serving.rotate(y, pos, freq, interleaved, 1.5, backward=True)
    assert math.isclose(float((got * y).sum()), float((x * back).sum()), rel_tol=1e-12)


def test_oracle_quantises_by_hand():
    codes, e = serving.quantise_row([448.0, -1.0, 0.0, 2.0 ** -9])
    assert e == 0 and codes == [126, 128 + 56, 0, 1]
    codes, e = serving.quantise_row([448.1, 7.0])
    assert e == 1 and codes[0] == 0x76 and serving.restore(np.array(codes, np.uint8), np.uint8(128))[0] == 448.0
    assert serving.quantise_row([0.0, -0.0]) == ([0, 128], -119)
    assert serving.quantise_row([math.nan, 1.0]) == ([127, 0x78], -8)  # 1 = 256 * 2^-8
    assert serving.quantise_row([math.inf, 1.0]) == ([126, 0], 119)
    # 17 * 2^-4 lies between 16 and 18 sixteenths: to the even code
    assert serving.quantise_row([448.0, 1.0625, 1.1875])[0][1:] == [56, 58]


def test_oracle_codes_are_the_nearest_values():
    rng = np.random.default_rng(2)
    x = rng.normal(size=(50, 64)) * np.exp(rng.normal(size=(50, 1)) * 20)
    codes, exps = serving.quantise(x)
    values = np.concatenate([serving.e4m3_values(), -serving.e4m3_values()])
    scaled = x / np.exp2(exps.astype(float) - 127)[:, None]
    best = np.abs(scaled[..., None] - values).min(-1)
    got = np.abs(serving.restore(codes, np.full(50, 127)) - scaled)
    assert np.array_equal(got, best)
    top = np.abs(x).max(1)
    assert np.all(top <= 448 * np.exp2(exps.astype(float) - 127)) and np.all(top > 224 * np.exp2(exps.astype(float) - 127))


def test_oracle_tree_by_hand():
    # 0 - 1 - 3, 0 - 2, 4 a second root; then a chunk of 33 rows, and padding
    parents = [-1, 0, 0, 1, -1] + [7] * 33 + [9]
    mask, pos = serving.tree_plan(parents, [0, 5, 38], [25, 33], 1)
    assert mask[:5, 0].tolist() == [1, 3, 5, 11, 16] and pos[:5] == [20, 21, 21, 22, 20]
    assert np.all(mask[5:] == 0) and pos[5:38] == list(range(33)) and pos[38] == -1


def test_oracle_chain_is_causal():
    rng = np.random.default_rng(3)
    q, k, v = rng.normal(size=(5, 4, 8)), rng.normal(size=(2, 21, 8)), rng.normal(size=(2, 21, 8))
    kc, vc = _scatter(k, 16, [2, 0], 3), _scatter(v, 16, [2, 0], 3)
    mask, _ = serving.tree_plan([-1, 0, 1, 2, 3], [0, 5], [21], 1)
    o, lse = serving.tree_forward(q, kc, vc, [[2, 0]], [0, 5], [21], mask, 0.4)
    want, want_lse = paged.paged_forward(q, kc, vc, [[2, 0]], [0, 5], [21], 0.4, True)
    np.testing.assert_allclose(o, want, atol=1e-14)
    np.testing.assert_allclose(lse, want_lse, atol=1e-14)


# ---------------------------------------------------------------- frequencies
def test_frequencies(A):
    f = A.rotary_frequencies(8)
    assert f.dtype is torch.float32 and torch.allclose(f.double(), torch.tensor([1, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-7)
    assert torch.allclose(A.rotary_frequencies(8, linear=4.0), f / 4)
    g = A.rotary_frequencies(8, ntk=4.0)
    assert g[0] == 1 and math.isclose(g[3].item(), f[3].item() / 4, rel_tol=1e-6)
    # by parts, context 1000: 159, 15.9, 1.59 and 0.159 turns; kept above 32, divided below 1, in proportion between
    h = A.rotary_frequencies(8, by_parts=4.0, context=1000)
    kept = [(1000 * x / (2 * math.pi) - 1) / 31 for x in (0.1, 0.01)]
    want = [1.0] + [x * (k + (1 - k) / 4) for x, k in zip((0.1, 0.01), kept)] + [0.001 / 4]
    assert torch.allclose(h.double(), torch.tensor(want, dtype=torch.float64), rtol=1e-6)


@pytest.mark.parametrize("kw", [dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, base=0.0), dict(rotary_dim=8, linear=0.5),
                                dict(rotary_dim=8, linear=2.0, ntk=2.0), dict(rotary_dim=8, by_parts=2.0),
                                dict(rotary_dim=8, by_parts=2.0, context=10, low_turns=5.0, high_turns=5.0), dict(rotary_dim=2, ntk=2.0)])
def test_frequencies_refused(A, kw):
    with pytest.raises(ValueError):
        A.rotary_frequencies(**kw)


# ---------------------------------------------------------------- structs
def test_struct_layout_matches_c(A):
    fields = {
        "attn_pages_write_fp8_params": (A.PagesFp8Params, ["k", "slots", "k_scale", "k_row_stride", "v_stride", "v_scale_stride"]),
        "attn_tree_plan_params": (A.TreePlanParams, ["words", "parents", "mask", "mask_stride", "positions"]),
        "attn_paged_tree_params": (A.PagedTreeParams, ["f", "mask", "mask_stride", "words", "reserved1"]),
        "attn_paged_fp8_params": (A.PagedFp8Params, ["t", "k_scale", "v_scale", "k_scale_stride", "v_scale_stride"]),
        "attn_rotary_params": (A.RotaryParams, ["Hk", "magnitude", "positions", "position_stride", "inv_freq", "k", "k_out", "k_out_stride"]),
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
def _run(A, name, p, status):
    assert getattr(A.lib, name)(ctypes.byref(p), None) == getattr(A, status)
    if status != "ATTN_OK":
        assert A.last_error() != ""


def _rotary(A, **kw):
    base = dict(B=2, N=3, Hq=4, Hk=2, d=64, rotary_dim=32, dtype=A.ATTN_BF16, interleaved=0, magnitude=1.0, position_stride=(0, 1),
                **{f"{n}_stride": (768, 64, 256) for n in ("q", "k", "q_out", "k_out")})
    p = _filled(A.RotaryParams, **base)
    p.q_out, p.k_out = FAKE + 4096, FAKE + 8192
    for n, v in kw.items():
        setattr(p, n, dict(p._fields_)[n](*v) if isinstance(v, tuple) else v)
    return p


@pytest.mark.parametrize("name", ["attn_rotary", "attn_rotary_bwd"])
@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), "ATTN_ERR_INVALID"),
    (dict(Hk=-1), "ATTN_ERR_INVALID"),
    (dict(d=0), "ATTN_ERR_INVALID"),
    (dict(d=72), "ATTN_ERR_UNSUPPORTED"),
    (dict(d=272), "ATTN_ERR_UNSUPPORTED"),
    (dict(rotary_dim=0), "ATTN_ERR_INVALID"),
    (dict(rotary_dim=80), "ATTN_ERR_INVALID"),
    (dict(rotary_dim=24), "ATTN_ERR_UNSUPPORTED"),
    (dict(dtype=3), "ATTN_ERR_UNSUPPORTED"),
    (dict(dtype=7), "ATTN_ERR_INVALID"),
    (dict(interleaved=2), "ATTN_ERR_INVALID"),
    (dict(magnitude=0.0), "ATTN_ERR_INVALID"),
    (dict(magnitude=float("nan")), "ATTN_ERR_INVALID"),
    (dict(reserved0=1), "ATTN_ERR_INVALID"),
    (dict(Hq=65536), "ATTN_ERR_UNSUPPORTED"),
    (dict(N=2 ** 31 - 1), "ATTN_ERR_UNSUPPORTED"),
    (dict(positions=0), "ATTN_ERR_INVALID"),
    (dict(positions=FAKE + 2), "ATTN_ERR_ALIGN"),
    (dict(inv_freq=0), "ATTN_ERR_INVALID"),
    (dict(q=0), "ATTN_ERR_INVALID"),
    (dict(k_out=0), "ATTN_ERR_INVALID"),
    (dict(q=FAKE + 8), "ATTN_ERR_ALIGN"),
    (dict(k_stride=(768, 60, 256)), "ATTN_ERR_ALIGN"),
    (dict(q_out_stride=(768, 64, 0)), "ATTN_ERR_INVALID"),
    (dict(q_stride=(1 << 38, 64, 256)), "ATTN_ERR_UNSUPPORTED"),
    (dict(position_stride=(-1, 1)), "ATTN_ERR_INVALID"),
    (dict(q_out=FAKE, q_out_stride=(768, 192, 64)), "ATTN_ERR_INVALID"),  # over its input with other strides
    (dict(N=0, positions=0, q=0), "ATTN_OK"),
    (dict(Hq=0, Hk=0, q=0, k=0), "ATTN_OK"),
])
def test_rotary_refusals(A, name, kw, status):
    _run(A, name, _rotary(A, **kw), status)


def _pages8(A, **kw):
    base = dict(rows=3, num_kv_heads=2, d=64, num_pages=4, page_size=16, dtype=A.ATTN_F16, k_row_stride=(128, 64), v_row_stride=(128, 64),
                k_stride=(2048, 64, 128), v_stride=(2048, 64, 128), k_scale_stride=(32, 16), v_scale_stride=(32, 16))
    return _filled(A.PagesFp8Params, **{**base, **kw})


@pytest.mark.parametrize("name", ["attn_pages_write_fp8", "attn_pages_read_fp8"])
@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), "ATTN_ERR_INVALID"),
    (dict(num_kv_heads=0), "ATTN_ERR_INVALID"),
    (dict(d=256), "ATTN_ERR_UNSUPPORTED"),
    (dict(dtype=1), "ATTN_ERR_UNSUPPORTED"),
    (dict(dtype=3), "ATTN_ERR_UNSUPPORTED"),
    (dict(page_size=24), "ATTN_ERR_UNSUPPORTED"),
    (dict(num_pages=0), "ATTN_ERR_INVALID"),
    (dict(slots=0), "ATTN_ERR_INVALID"),
    (dict(k=FAKE + 4), "ATTN_ERR_ALIGN"),
    (dict(k_cache=0), "ATTN_ERR_INVALID"),
    (dict(v_scale=0), "ATTN_ERR_INVALID"),
    (dict(k_scale=FAKE + 8), "ATTN_ERR_ALIGN"),
    (dict(k_stride=(2048, 64, 72)), "ATTN_ERR_ALIGN"),
    (dict(k_scale_stride=(32, 8)), "ATTN_ERR_ALIGN"),
    (dict(v_scale_stride=(0, 16)), "ATTN_ERR_INVALID"),
    (dict(reserved0=(1, 0)), "ATTN_ERR_INVALID"),
    (dict(rows=2 ** 31 - 1, num_kv_heads=65535), "ATTN_ERR_UNSUPPORTED"),
    (dict(rows=0, k=0, k_cache=0, slots=0), "ATTN_OK"),
])
def test_pages_fp8_refusals(A, name, kw, status):
    _run(A, name, _pages8(A, **kw), status)


@pytest.mark.parametrize("kw,status", [
    (dict(num_seqs=-1), "ATTN_ERR_INVALID"),
    (dict(total_q=-1), "ATTN_ERR_INVALID"),
    (dict(words=0), "ATTN_ERR_INVALID"),
    (dict(words=33), "ATTN_ERR_INVALID"),
    (dict(reserved0=1), "ATTN_ERR_INVALID"),
    (dict(mask_stride=1), "ATTN_ERR_INVALID"),
    (dict(parents=0), "ATTN_ERR_INVALID"),
    (dict(mask=FAKE + 2), "ATTN_ERR_ALIGN"),
    (dict(positions=FAKE), "ATTN_ERR_INVALID"),      # the parents themselves
    (dict(mask=FAKE + 64), "ATTN_ERR_INVALID"),      # cu_q itself
    (dict(positions=FAKE + 256 + 4 * 9), "ATTN_ERR_INVALID"),  # the mask's last row
    (dict(total_q=2 ** 31 - 1), "ATTN_ERR_UNSUPPORTED"),
    (dict(total_q=0, parents=0, mask=0, cu_q=0), "ATTN_OK"),
])
def test_tree_plan_refusals(A, kw, status):
    base = dict(num_seqs=2, total_q=5, words=2, mask_stride=2, cu_q=FAKE + 64, kv_len=FAKE + 128, mask=FAKE + 256, positions=FAKE + 512)
    _run(A, "attn_tree_plan", _filled(A.TreePlanParams, **{**base, **kw}), status)


def _attend(A, tree, f8, **kw):
    es = 1 if f8 else 2
    base = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, d=64, total_q=10, max_q=1, num_pages=9, page_size=16, max_pages=4,
                dtype=A.ATTN_BF16, causal=0, scale=0.125, table_stride=4, q_stride=(512, 64), o_stride=(512, 64),
                k_stride=(2048, 64, 128), v_stride=(2048, 64, 128), workspace=FAKE, workspace_bytes=1 << 40)
    names = {n for n, _ in A.PagedParams._fields_}
    f = _filled(A.PagedParams, **{**base, **{k: v for k, v in kw.items() if k in names}})
    t = A.PagedTreeParams(f, FAKE if tree else None, 2 if tree else 0, 2 if tree else 0, 0)
    p = A.PagedFp8Params(t, FAKE, FAKE, (ctypes.c_int64 * 2)(32, 16), (ctypes.c_int64 * 2)(32, 16)) if f8 else t
    for n, v in kw.items():
        if n not in names:
            holder = p if n in dict(p._fields_) else p.t
            setattr(holder, n, dict(holder._fields_)[n](*v) if isinstance(v, tuple) else v)
    assert es
    return p


COMMON = [(dict(num_q_heads=7), "ATTN_ERR_INVALID"), (dict(d=256), "ATTN_ERR_UNSUPPORTED"), (dict(dtype=3), "ATTN_ERR_UNSUPPORTED"),
          (dict(dtype=1), "ATTN_ERR_UNSUPPORTED"), (dict(max_q=0), "ATTN_ERR_INVALID"), (dict(page_size=8), "ATTN_ERR_UNSUPPORTED"),
          (dict(k_cache=0), "ATTN_ERR_INVALID"), (dict(v_cache=FAKE + 8), "ATTN_ERR_ALIGN"), (dict(lse=0), "ATTN_ERR_INVALID"),
          (dict(num_seqs=2 ** 31 - 1), "ATTN_ERR_UNSUPPORTED"), (dict(q_stride=(516, 64)), "ATTN_ERR_ALIGN"),
          (dict(num_seqs=0, q=0, k_cache=0), "ATTN_OK"), (dict(total_q=0, q=0, k_cache=0), "ATTN_OK")]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(causal=1), "ATTN_ERR_INVALID"),
    (dict(words=0), "ATTN_ERR_INVALID"),
    (dict(words=33), "ATTN_ERR_INVALID"),
    (dict(mask=0), "ATTN_ERR_INVALID"),
    (dict(mask=FAKE + 1), "ATTN_ERR_ALIGN"),
    (dict(mask_stride=-1), "ATTN_ERR_INVALID"),
    (dict(mask_stride=1 << 38), "ATTN_ERR_UNSUPPORTED"),
    (dict(reserved1=1), "ATTN_ERR_INVALID"),
    (dict(k_stride=(2048, 64, 36)), "ATTN_ERR_ALIGN"),
])
def test_paged_tree_refusals(A, kw, status):
    _run(A, "attn_paged_tree", _attend(A, True, False, **kw), status)


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(k_scale=0), "ATTN_ERR_INVALID"),
    (dict(v_scale=FAKE + 4), "ATTN_ERR_ALIGN"),
    (dict(k_scale_stride=(16, 8)), "ATTN_ERR_ALIGN"),
    (dict(v_scale_stride=(32, 0)), "ATTN_ERR_INVALID"),
    (dict(k_stride=(2048, 64, 72)), "ATTN_ERR_ALIGN"),  # bytes
    (dict(words=1), "ATTN_ERR_INVALID"),
    (dict(mask_stride=4), "ATTN_ERR_INVALID"),
    (dict(reserved1=3), "ATTN_ERR_INVALID"),
    (dict(causal=2), "ATTN_ERR_INVALID"),
])
def test_paged_fp8_refusals(A, kw, status):
    p = _attend(A, False, True, **kw)
    _run(A, "attn_paged_fp8", p, status)
    assert A.lib.attn_paged_fp8_workspace_size(ctypes.byref(p)) == 0


@pytest.mark.parametrize("kw", [dict(causal=1), dict(words=0), dict(words=40), dict(mask=FAKE + 2)])
def test_paged_fp8_refusals_with_a_tree(A, kw):
    status = "ATTN_ERR_ALIGN" if "mask" in kw else "ATTN_ERR_INVALID"
    _run(A, "attn_paged_fp8", _attend(A, True, True, **kw), status)


def test_null_params(A):
    for name in ("attn_rotary", "attn_rotary_bwd", "attn_pages_write_fp8", "attn_pages_read_fp8", "attn_tree_plan", "attn_paged_tree",
                 "attn_paged_fp8"):
        assert getattr(A.lib, name)(None, None) == A.ATTN_ERR_INVALID
    assert A.lib.attn_paged_fp8_workspace_size(None) == 0


# ---------------------------------------------------------------- refusals of the binding
I32, BF, F8, E8 = torch.int32, torch.bfloat16, torch.float8_e4m3fn, torch.float8_e8m0fnu


def _t(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=torch.uint8).view(dtype) if dtype in (F8, E8) else torch.zeros(*shape, dtype=dtype)


def _cache():
    return [_t(4, 2, 16, 64, dtype=F8), _t(4, 2, 16, 64, dtype=F8), _t(4, 2, 16, dtype=E8), _t(4, 2, 16, dtype=E8)]


def test_binding_refuses_tensors_that_are_not_on_a_gpu(A):
    k, slots = _t(3, 2, 64), _t(3, dtype=I32)
    q, table, cu, kv, tree = _t(3, 4, 64), _t(2, 2, dtype=I32), _t(3, dtype=I32), _t(2, dtype=I32), _t(3, 1, dtype=I32)
    pages = _t(4, 2, 16, 64)
    for call in (lambda: A.attn_pages_write_fp8(k, k, slots, *_cache()), lambda: A.attn_pages_read_fp8(slots, *_cache()),
                 lambda: A.attn_tree_plan(slots, cu, kv, 32), lambda: A.attn_paged_tree(q, pages, pages, table, cu, kv, tree),
                 lambda: A.attn_paged_fp8(q, *_cache(), table, cu, kv, tree=tree), lambda: A.attn_paged_fp8(q, *_cache(), table, cu, kv),
                 lambda: A.attn_rotary(q, None, slots, torch.ones(32)), lambda: A.attn_rotary_bwd(q, q, slots, torch.ones(32))):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


@pytest.mark.parametrize("at,value,error", [
    (0, _t(4, 2, 16, 64), TypeError), (1, _t(4, 2, 16, 64, dtype=E8), TypeError), (2, _t(4, 2, 16, dtype=F8), TypeError),
    (3, _t(4, 16, 2, dtype=E8), ValueError), (3, _t(4, 16, 2, dtype=E8).transpose(1, 2), ValueError),
    (1, _t(4, 2, 64, 16, dtype=F8).transpose(2, 3), ValueError), (0, _t(4, 3, 16, 64, dtype=F8), ValueError)])
def test_binding_refuses_other_caches(A, at, value, error):
    cache = _cache()
    cache[at] = value
    with pytest.raises(error):
        A.attn_pages_write_fp8(_t(3, 2, 64), _t(3, 2, 64), _t(3, dtype=I32), *cache)
    with pytest.raises((error, ValueError)):
        A.attn_paged_fp8(_t(3, 6, 64), *cache, _t(2, 2, dtype=I32), _t(3, dtype=I32), _t(2, dtype=I32))


def test_binding_refusals(A):
    q, table, cu, kv, tree = _t(3, 4, 64), _t(2, 2, dtype=I32), _t(3, dtype=I32), _t(2, dtype=I32), _t(3, 1, dtype=I32)
    pages, freq = _t(4, 2, 16, 64), torch.ones(32)
    with pytest.raises(ValueError, match="tree is None"):
        A.attn_paged_tree(q, pages, pages, table, cu, kv, None)
    for bad, error in ((_t(3, 1, dtype=torch.int64), TypeError), (_t(2, 1, dtype=I32), ValueError), (_t(3, dtype=I32), ValueError)):
        with pytest.raises(error, match="tree"):
            A.attn_paged_tree(q, pages, pages, table, cu, kv, bad)
    with pytest.raises(TypeError, match="q must be"):
        A.attn_paged_fp8(q.float(), *_cache(), table, cu, kv)
    for nodes in (0, 1025, 1.5):
        with pytest.raises(ValueError, match="max_nodes"):
            A.attn_tree_plan(_t(3, dtype=I32), cu, kv, nodes)
    with pytest.raises(ValueError, match="cu_q"):
        A.attn_tree_plan(_t(3, dtype=I32), _t(2, dtype=I32), kv, 32)
    with pytest.raises(TypeError, match="positions"):
        A.attn_rotary(q, None, _t(3, dtype=torch.int64), freq)
    with pytest.raises(ValueError, match="positions"):
        A.attn_rotary(q, None, _t(4, dtype=I32), freq)
    with pytest.raises(TypeError, match="inv_freq"):
        A.attn_rotary(q, None, _t(3, dtype=I32), freq.double())
    with pytest.raises(TypeError, match="k must be"):
        A.attn_rotary(q, q.float(), _t(3, dtype=I32), freq)
    with pytest.raises(ValueError, match="k has shape"):
        A.attn_rotary(q, _t(4, 2, 64), _t(3, dtype=I32), freq)
    with pytest.raises(ValueError, match="k_out given"):
        A.attn_rotary(q, None, _t(3, dtype=I32), freq, k_out=q)
    with pytest.raises(ValueError, match="q has shape"):
        A.attn_rotary(_t(3, 64), None, _t(3, dtype=I32), freq)
    with pytest.raises(TypeError, match="k and v must be"):
        A.attn_pages_read_fp8(_t(3, dtype=I32), *_cache(), dtype=torch.float32)


# ---------------------------------------------------------------- batches without rows
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("size", [dict(total_q=0), dict(num_seqs=0)])
@pytest.mark.parametrize("stride", [0, 2])
def test_a_tree_call_without_rows_needs_no_mask(A, stride, size, f8):
    p = _attend(A, True, f8, mask=0, mask_stride=stride, **size)
    _run(A, "attn_paged_fp8" if f8 else "attn_paged_tree", p, "ATTN_OK")
    if f8:
        assert A.lib.attn_paged_fp8_workspace_size(ctypes.byref(p)) == 0
    _run(A, "attn_paged_fp8" if f8 else "attn_paged_tree", _attend(A, True, f8, mask=0, mask_stride=stride), "ATTN_ERR_INVALID")
