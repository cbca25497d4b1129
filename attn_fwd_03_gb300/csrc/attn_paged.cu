// attn_paged.cu — attention of a ragged batch of new tokens over a paged cache.
//
// One warp to a (query row, head): it walks the row's keys with the online softmax's
// running max, sum and accumulator in fp32 registers.
#include <cmath>
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr unsigned kFull = 0xffffffffu;

struct PagedArgs {
    attn_paged_params p;
    int shift;
    int* err;
};

template <int D, bool F16>
__global__ void __launch_bounds__(256) paged_simple_kernel(const PagedArgs a) {
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    constexpr int PER = D / 32;
    const attn_paged_params& p = a.p;
    const int lane = threadIdx.x & 31, h = blockIdx.y;
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t >= p.total_q || t >= p.cu_q[p.num_seqs]) return;
    int lo = 0, hi = p.num_seqs;  // the last sequence that starts at or before t
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (p.cu_q[mid] <= t) lo = mid; else hi = mid;
    }
    const int start = p.cu_q[lo], n = p.cu_q[lo + 1] - start;
    long long len = p.kv_len[lo];
    const long long most = (long long)p.max_pages << a.shift;
    bool bad = len < 0 || len > most;
    len = len < 0 ? 0 : len > most ? most : len;
    const long long end = p.causal ? min(len, len - n + (t - start) + 1) : len;
    const int hk = h / (p.num_q_heads / p.num_kv_heads);
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + t * p.q_stride[0] + h * p.q_stride[1] + lane * PER;
    float qv[PER], o[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        qv[e] = ptx::h16_to_float<F16>(q[e]) * p.scale * kLog2e;
        o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (long long j = 0; j < end; ++j) {
        const int page = p.block_table[lo * p.table_stride + (j >> a.shift)];
        if (page < 0 || page >= p.num_pages) {
            bad = true;
            continue;
        }
        const long long slot = j & (p.page_size - 1);
        const uint16_t* k = static_cast<const uint16_t*>(p.k_cache) + page * p.k_stride[0] + hk * p.k_stride[1] + slot * p.k_stride[2] + lane * PER;
        const uint16_t* v = static_cast<const uint16_t*>(p.v_cache) + page * p.v_stride[0] + hk * p.v_stride[1] + slot * p.v_stride[2] + lane * PER;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < PER; ++e) s = fmaf(qv[e], ptx::h16_to_float<F16>(k[e]), s);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(kFull, s, off);
        const float mn = fmaxf(m, s), alpha = ptx::ex2(m - mn), w = ptx::ex2(s - mn);
        l = l * alpha + w;
#pragma unroll
        for (int e = 0; e < PER; ++e) o[e] = fmaf(w, ptx::h16_to_float<F16>(v[e]), o[e] * alpha);
        m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + t * p.o_stride[0] + h * p.o_stride[1] + lane * PER);
#pragma unroll
    for (int e = 0; e < PER / 2; ++e) out[e] = ptx::pack_h16<F16>(o[2 * e] * inv, o[2 * e + 1] * inv);
    if (lane == 0) p.lse[(long long)h * p.total_q + t] = l > 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;
    if (bad) atomicCAS(a.err, 0, ATTN_ERR_INVALID);
}

}  // namespace

size_t paged_workspace_bytes(const attn_paged_params&, int) { return 256; }

cudaError_t launch_paged(const attn_paged_params& p, const LaunchCommon& lc, cudaStream_t s) {
    PagedArgs a{};
    a.p = p;
    while ((1 << a.shift) < p.page_size) ++a.shift;
    a.err = lc.err;
    const bool f16 = p.dtype == ATTN_F16;
    const dim3 grid((p.total_q + 7) / 8, p.num_q_heads);
    auto k = p.d == 64 ? (f16 ? paged_simple_kernel<64, true> : paged_simple_kernel<64, false>)
                       : (f16 ? paged_simple_kernel<128, true> : paged_simple_kernel<128, false>);
    return launch_pdl(k, grid, dim3(256), 0, s, a);
}

}  // namespace attn
