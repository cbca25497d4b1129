"""Rotary positions on the GPU against the fp64 oracle (oracle/serving.py).

Tolerance: an output is rounded once, off by at most half a step (2^-9 of it in bf16, 2^-12 in fp16, 2^-25 in fp32; the
bounds below use eps / 2), after y = a c - b s in fp32: cosine and sine are each within 2^-22 (2 steps of a value in [1/2, 1],
and 2^-30 for the angle), the products and their sum are within 3 * 2^-24 of |a| + |b|. 2^-21 (|a| + |b|) * magnitude covers
both. fp16 outputs below 2^-14 step by 2^-24.
"""
import numpy as np
import pytest
import torch

from oracle import serving
from parity_util import to64

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import attn_fwd_03_gb300 as m
    assert m.attn_status() == m.ATTN_OK
    return m


def _rand(shape, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def _check(got, x, positions, freq, interleaved, magnitude=1.0, backward=False):
    """x, got [..., N, d]."""
    want = serving.rotate(to64(x), positions, freq.tolist(), interleaved, magnitude, backward)
    half, m = len(freq), 2 * len(freq)
    a = np.abs(to64(x))
    pair = np.zeros_like(a)
    if interleaved:
        pair[..., 0:m:2] = pair[..., 1:m:2] = a[..., 0:m:2] + a[..., 1:m:2]
    else:
        pair[..., :half] = pair[..., half:m] = a[..., :half] + a[..., half:m]
    bound = torch.finfo(got.dtype).eps / 2 * np.abs(want) + 2.0 ** -21 * magnitude * pair
    if got.dtype == torch.float16:
        bound = bound + 2.0 ** -25
    off = np.abs(to64(got) - want)
    assert np.all(off <= bound), f"off by {np.max(off - bound):.3e} beyond the bound"
    assert np.array_equal(to64(got)[..., m:], to64(x)[..., m:])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("d,turned", [(64, 64), (128, 128), (128, 32), (256, 256), (80, 48), (16, 16), (144, 16)])
def test_training_layout(A, d, turned, backward, interleaved, dtype):
    N = 37
    q, k = _rand((2, 3, N, d), 1, dtype), _rand((2, 1, N, d), 2, dtype)
    freq = A.rotary_frequencies(turned, device="cuda")
    pos = torch.arange(N, dtype=torch.int32, device="cuda") * 29
    turn = A.attn_rotary_bwd if backward else A.attn_rotary
    qo, ko = turn(q, k, pos, freq, interleaved=interleaved, magnitude=1.25)
    assert A.attn_status() == A.ATTN_OK
    for got, x in ((qo, q), (ko, k)):
        _check(got, x, pos.tolist(), freq, interleaved, 1.25, backward)


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 300])
@pytest.mark.parametrize("heads", [(1, 0), (5, 1), (32, 8)])
def test_ragged_rows_with_padding(A, rows, heads):
    q = _rand((rows, heads[0], 128), 3, torch.bfloat16)
    k = _rand((rows, heads[1], 128), 4, torch.bfloat16) if heads[1] else None
    freq = A.rotary_frequencies(64, device="cuda")
    pos = torch.randint(0, 200000, (rows,), generator=torch.Generator().manual_seed(5), dtype=torch.int32)
    pos[rows // 2:rows // 2 + 1] = -1
    qo, ko = torch.full_like(q, 7.0), None if k is None else torch.full_like(k, 7.0)
    got, got_k = A.attn_rotary(q, k, pos.cuda(), freq, q_out=qo, k_out=ko)
    assert got is qo and got_k is ko and A.attn_status() == A.ATTN_OK
    for o, x in ((qo, q), (ko, k)):
        if x is None:
            continue
        held = (pos >= 0).nonzero()[:, 0].cuda()
        assert torch.all(o[rows // 2] == 7.0)
        _check(o[held].transpose(0, 1), x[held].transpose(0, 1), pos[pos >= 0].tolist(), freq, False)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(A, interleaved):
    pos = [0, 1, 2, 131071, 1048575, 2 ** 24 + 1, 2 ** 31 - 1]
    freq = torch.tensor([1.0, 0.5, 3.1415927, 6.2831855, 1e-4, 1e-9, 0.7071068, 1e-30, 5e3, 2.5, 0.1, 0.0, -0.3, 1e-45, 0.9, 1.1],
                        device="cuda")
    x = _rand((len(pos), 2, 32), 6, torch.float32)
    got, _ = A.attn_rotary(x, None, torch.tensor(pos, dtype=torch.int32, device="cuda"), freq, interleaved=interleaved)
    _check(got.transpose(0, 1), x.transpose(0, 1), pos, freq, interleaved)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("turned", [32, 64])
def test_in_place_and_strided(A, dtype, turned):
    freq, pos = A.rotary_frequencies(turned, device="cuda"), torch.tensor([5, 0, 77, 3], dtype=torch.int32, device="cuda")
    wide = _rand((4, 6, 64), 7, dtype)  # q and k are heads 1 to 3 and 4 to 5 of one projection
    q, k, before = wide[:, 1:4], wide[:, 4:], wide.clone()
    want = A.attn_rotary(q.contiguous(), k.contiguous(), pos, freq)
    got = A.attn_rotary(q, k, pos, freq, q_out=q, k_out=k)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(wide[:, 0], before[:, 0])
    _check(q.transpose(0, 1), before[:, 1:4].transpose(0, 1), pos.tolist(), freq, False)
    # [B, N, H, d] in memory, positions of each batch entry
    x = _rand((2, 5, 3, 64), 8, dtype).transpose(1, 2)
    each = torch.randint(0, 50, (2, 5), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    out = torch.zeros(2, 3, 5, 64, dtype=dtype, device="cuda")
    A.attn_rotary(x, None, each.cuda(), freq, q_out=out)
    for b in range(2):
        _check(out[b], x[b], each[b].tolist(), freq, False)


def test_many_heads_and_rows_beyond_a_block(A):
    freq = A.rotary_frequencies(128, device="cuda")
    q = _rand((1, 2, 5000, 128), 9, torch.bfloat16)
    pos = torch.arange(5000, dtype=torch.int32, device="cuda")
    got, _ = A.attn_rotary(q, None, pos, freq)
    at = [0, 7, 8, 2047, 4999]
    _check(got[0][:, at], q[0][:, at], at, freq, False)
    # the same turn in either split of the work
    assert torch.equal(A.attn_rotary(q[:, :, 4992:], None, pos[4992:], freq)[0], got[:, :, 4992:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_backward_is_the_transpose_and_matches_differences(A, interleaved):
    freq, pos = A.rotary_frequencies(32, device="cuda"), torch.tensor([3, 1000, 12], dtype=torch.int32, device="cuda")
    x, w = _rand((3, 2, 48), 10, torch.float32), _rand((3, 2, 48), 11, torch.float32)
    f = lambda t: A.attn_rotary(t, None, pos, freq, interleaved=interleaved, magnitude=0.8)[0]  # noqa: E731
    grad = A.attn_rotary_bwd(w, None, pos, freq, interleaved=interleaved, magnitude=0.8)[0]
    # sum(w * f(x)) is linear in x: a difference over a step of 1 is the derivative up to the rounding of f, at most
    # 2^-21 (|a| + |b|) an entry, over two entries and two evaluations with values up to 6: 2^-21 * 4 * 12
    for r, h, c in ((0, 0, 0), (1, 1, 17), (2, 0, 31), (2, 1, 40)):
        step = torch.zeros_like(x)
        step[r, h, c] = 1.0
        diff = ((f(x + step).double() - f(x).double()) * w.double()).sum().item()
        assert abs(diff - grad[r, h, c].item()) <= 2.0 ** -21 * 48 * w.abs().max().item()


def test_graph_and_streams(A):
    freq, pos = A.rotary_frequencies(64, device="cuda"), torch.arange(9, dtype=torch.int32, device="cuda")
    q, out = _rand((9, 4, 64), 12, torch.float16), torch.zeros(9, 4, 64, dtype=torch.float16, device="cuda")
    want = A.attn_rotary(q, None, pos, freq)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = A.attn_rotary(q, None, pos, freq, stream=side)[0]
    side.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        A.attn_rotary(q, None, pos, freq, q_out=out)
    pos += 11
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, A.attn_rotary(q, None, pos, freq)[0]) and not torch.equal(out, want)


def test_nothing_to_turn(A):
    freq, none = A.rotary_frequencies(64, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    q, k = A.attn_rotary(torch.zeros(0, 4, 64, device="cuda"), torch.zeros(0, 2, 64, device="cuda"), none, freq)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    assert A.attn_rotary(torch.zeros(2, 0, 3, 64, device="cuda"), None, torch.zeros(3, dtype=torch.int32, device="cuda"), freq)[0].numel() == 0


def test_angles_near_half_a_turn(A):
    # fp32 holds an angle near half a turn to 2^-25 of that only, and the sine there is the distance to it: positions whose angle
    # is within 2^-9 of a turn of it, the sine read off as y0 of (0, -1) and y1 of (1, 0). Bound: the angle to 2^-32 of a turn,
    # 2^-29.3, and the sine's own rounding and the product's, 2^-22 of it together
    pos = [p for p in range(1, 40000) if abs(serving.turn_of(p, 1.0) - 0.5) < 2.0 ** -9]
    freq = torch.ones(8, device="cuda")
    x = torch.zeros(len(pos), 1, 16, device="cuda")
    x[..., :8] = 1.0
    got, _ = A.attn_rotary(x, None, torch.tensor(pos, dtype=torch.int32, device="cuda"), freq)
    want = serving.rotate(to64(x).transpose(1, 0, 2), pos, freq.tolist(), False).transpose(1, 0, 2)
    off = np.abs(to64(got) - want)[..., 8:]
    assert len(pos) > 100 and np.all(off <= 2.0 ** -29 + 2.0 ** -22 * np.abs(want[..., 8:]))
