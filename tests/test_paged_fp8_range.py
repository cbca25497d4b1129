"""The 8-bit paged cache at the ends of its range on the GPU: what attn_paged promises holds for every value that the cache may
stand for, in units of every kind (up to 32 rows, up to 128, two tiles).

Bounds are those of test_paged_fp8.py unless a test derives its own.
"""
import math

import numpy as np
import pytest
import torch

from oracle import paged, serving
from parity_util import assert_close_bf16, assert_lse, assert_masked_rows_zero, to64
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


