"""Exact tiled attention for GB300 (sm_103a): a C-ABI CUDA library and its
thin Python binding.

    from attn_fwd_03_gb300 import attn_fwd, attn_bwd
    o, lse = attn_fwd(q, k, v, causal=True)            # q, k, v: [B, H, N, d] on cuda
    dq, dk, dv = attn_bwd(q, k, v, o, lse, do, causal=True)
    o1, lse1 = attn_decode(q1, k_cache, v_cache, causal=True)  # q1: [B, H, nq <= 128, d]
    cu_q, kv_len, slots, pos, left = attn_pages_plan(q_len, cached, table, free, count, 64, rows)  # paged cache
    attn_pages_write(k, v, slots, k_cache, v_cache)
    o2, lse2 = attn_paged(q2, k_cache, v_cache, table, cu_q, kv_len, causal=True)  # q2: [rows, Hq, d]
    qr, kr = attn_rotary(q2, k, pos, rotary_frequencies(128))        # rotary positions; attn_rotary_bwd: their gradients
    attn_pages_write_fp8(kr, v, slots, k8_cache, v8_cache, k_scale, v_scale)  # the same cache in 8 bits
    o3, lse3 = attn_paged_fp8(qr, k8_cache, v8_cache, k_scale, v_scale, table, cu_q, kv_len, causal=True)
    tree, pos = attn_tree_plan(parents, cu_q, kv_len, 64)            # trees of drafted tokens
    o4, lse4 = attn_paged_tree(q2, k_cache, v_cache, table, cu_q, kv_len, tree)
    o8, lse8 = attn_fwd_fp8(q8, k8, v8, q_descale, k_descale, v_descale)  # E4M3 inputs, d = 128

The kernels live in csrc/ (built in-tree by build.py); the public C header is
include/attn.h at the repository root.
"""
from ._binding import (  # noqa: F401
    ATTN_BF16, ATTN_E4M3, ATTN_ERR_ALIGN, ATTN_ERR_CUDA, ATTN_ERR_INVALID, ATTN_ERR_TIMEOUT, ATTN_ERR_UNSUPPORTED,
    ATTN_ERR_WORKSPACE, ATTN_F16, ATTN_F32, ATTN_OK, EXPORTED, LIB_PATH, AttnError, BwdParams, DecodeParams,
    Fp8Params, FwdParams, attn_bwd, attn_bwd_deterministic, attn_bwd_noalloc, attn_decode, attn_fwd, attn_fwd_fp8,
    attn_status, bwd_workspace_size, debug_set_bwd_events, debug_set_producer_stall, decode_workspace_size,
    last_error, launch_count, launch_names, lib, set_wait_timeout_ns, version,
)
from ._paged import (  # noqa: F401
    PagedParams, PagesPlanParams, PagesReleaseParams, PagesWriteParams, attn_paged, attn_pages_plan,
    attn_pages_release, attn_pages_write, paged_workspace_size,
)
from ._paged8 import (  # noqa: F401
    PagedFp8Params, PagedTreeParams, PagesFp8Params, TreePlanParams, attn_paged_fp8, attn_paged_tree, attn_pages_read_fp8,
    attn_pages_write_fp8, attn_tree_plan, paged_fp8_workspace_size,
)
from ._rotary import RotaryParams, attn_rotary, attn_rotary_bwd, rotary_frequencies  # noqa: F401
