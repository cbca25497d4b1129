"""Failure detection without a GPU fault.

The forward's load warp is told (through a test hook of the C ABI) to stop
after one key/value tile, so the MMA and softmax warps' bounded waits run
out. The kernel must record ATTN_ERR_TIMEOUT in the device error word and
return; attn_status() reports it once and clears it, and the context stays
usable: the next call computes the right answer. No trap, no bad address,
no endless loop is involved.
"""
import math

import pytest
import torch

import workloads as W
from oracle import ref
from parity_util import assert_close_bf16, assert_lse, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import attn_fwd_03_gb300 as m
    return m


def test_stalled_producer_reports_timeout_and_context_survives(A):
    B, H, N, d = 1, 2, 1024, 64
    t = {n: W.random_tensor((B, H, N, d), 950 + i, torch.bfloat16) for i, n in enumerate(("q", "k", "v"))}
    q, k, v = (t[n].cuda() for n in ("q", "k", "v"))
    assert A.attn_status() == A.ATTN_OK
    A.set_wait_timeout_ns(100_000_000)  # 0.1 s per wait
    A.debug_set_producer_stall(1)
    try:
        A.attn_fwd(q, k, v, causal=False)
        torch.cuda.synchronize()  # the kernel returns on its own
        assert A.attn_status() == A.ATTN_ERR_TIMEOUT
        assert "wait" in A.last_error()
        assert A.attn_status() == A.ATTN_OK  # reported once, then cleared
    finally:
        A.debug_set_producer_stall(0)
        A.set_wait_timeout_ns(2_000_000_000)
    o, lse = A.attn_fwd(q, k, v, causal=False)
    torch.cuda.synchronize()
    assert A.attn_status() == A.ATTN_OK
    O, L = ref.attention_forward(to64(t["q"]), to64(t["k"]), to64(t["v"]), 1 / math.sqrt(d), False)
    assert_close_bf16("O", o, O)
    assert_lse(lse, L)


# a batch whose CTAs all have several key tiles, for each form of the paged kernel: (rows, keys) of a sequence,
# how many of them, head dim, page size
PAGED = {
    "one-tile units, two CTAs an SM": (1, 16000, 4, 64, 128),
    "one-tile units": (1, 12000, 4, 128, 64),
    "one-tile units, V by a warp of its own": (1, 12000, 4, 128, 16),
    "short table": (1, 384, 320, 128, 64),
    "two-tile units, an issuer each": (300, 9000, 2, 64, 32),
    "two-tile units, one issuer": (300, 9000, 2, 128, 64),
}


@pytest.mark.parametrize("form", list(PAGED))
def test_stalled_paged_producers_report_timeout_and_the_workspace_survives(A, form):
    from test_paged import Case
    n, kv, seqs, d, page = PAGED[form]
    c = Case([n] * seqs, [kv] * seqs, 2, 2, d, page, torch.bfloat16, 960)
    args = c.device()
    ws = torch.zeros(A.paged_workspace_size(*args, max_q=n), dtype=torch.uint8, device="cuda")
    assert A.attn_status() == A.ATTN_OK
    A.set_wait_timeout_ns(100_000_000)
    A.debug_set_producer_stall(1)
    try:
        A.attn_paged(*args, causal=True, max_q=n, workspace=ws)
        torch.cuda.synchronize()
        assert A.attn_status() == A.ATTN_ERR_TIMEOUT and "wait" in A.last_error()
        assert A.attn_status() == A.ATTN_OK
    finally:
        A.debug_set_producer_stall(0)
        A.set_wait_timeout_ns(2_000_000_000)
    o, lse = A.attn_paged(*args, causal=True, max_q=n, workspace=ws)
    torch.cuda.synchronize()
    assert A.attn_status() == A.ATTN_OK
    c.check(o, lse, True)
