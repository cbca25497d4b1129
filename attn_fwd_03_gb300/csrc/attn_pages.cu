// attn_pages.cu — the paged key/value cache's tables and writes: a step's pages,
// slots and positions from its lengths (plan), the pages of ended sequences given
// back (release), and new keys and values stored in their slots (write).
//
// The two table kernels are bound by latency: a step has a few hundred lengths and
// at most some ten thousand tokens, so each is one launch whose blocks all scan the
// lengths for themselves (a block-wide prefix sum of 256 at a time) instead of
// waiting for a scan kernel before them.
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kScan = 256;  // threads of a table block; lengths scanned at a time

__device__ __forceinline__ void note_bad(int* err) { atomicCAS(err, 0, ATTN_ERR_INVALID); }

__device__ __forceinline__ int pages_of(int tokens, int shift) { return (int)(((long long)tokens + (1 << shift) - 1) >> shift); }

// ---------------------------------------------------------------- plan
struct PlanArgs {
    attn_pages_plan_params p;
    int shift;       // log2(page_size)
    int per_block;   // tokens a block writes
    int* err;
};

// Block i writes slots and positions of tokens [i * per_block, (i + 1) * per_block) and the
// table entries that those tokens open; block 0 writes the per-sequence outputs too. Sums are
// 64-bit, so that no length a caller may leave in the arrays can wrap one into range.
__global__ void __launch_bounds__(kScan) pages_plan_kernel(const PlanArgs a) {
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const attn_pages_plan_params& p = a.p;
    __shared__ long long s_tok[kScan + 1], s_page[kScan + 1];  // exclusive sums of this chunk
    __shared__ int s_old[kScan];
    __shared__ long long s_warp[2][kScan / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long t0 = (long long)blockIdx.x * a.per_block;
    const long long t1 = min((long long)p.total_q, t0 + a.per_block);
    const int mask = p.page_size - 1;
    const int count = p.free_count[0];
    long long tok = 0, taken = 0;  // sums over the chunks before
    bool bad = false;
    if (blockIdx.x == 0 && tid == 0) p.cu_q[0] = 0;
    for (int b0 = 0; b0 < p.num_seqs; b0 += kScan) {
        if (blockIdx.x != 0 && tok >= t1) break;  // only block 0 needs every sequence
        const int b = b0 + tid;
        int n = 0, old = 0;
        if (b < p.num_seqs) {
            n = p.q_len[b];
            old = p.kv_len[b];
            bad |= n < 0 || old < 0 || (long long)old + n > (long long)p.max_pages << a.shift;
            n = max(n, 0);
            old = max(old, 0);
        }
        const long long fresh = (((long long)old + n + mask) >> a.shift) - pages_of(old, a.shift);
        long long x = n, y = fresh;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long ux = __shfl_up_sync(kFull, x, o), uy = __shfl_up_sync(kFull, y, o);
            if (lane >= o) {
                x += ux;
                y += uy;
            }
        }
        if (lane == 31) {
            s_warp[0][warp] = x;
            s_warp[1][warp] = y;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kScan / 32; ++w)
            if (w < warp) {
                x += s_warp[0][w];
                y += s_warp[1][w];
            }
        s_tok[tid + 1] = tok + x;
        s_page[tid + 1] = taken + y;
        s_old[tid] = old;
        if (tid == 0) {
            s_tok[0] = tok;
            s_page[0] = taken;
        }
        if (blockIdx.x == 0 && b < p.num_seqs) {
            const long long end = tok + x;
            bad |= end > p.total_q;
            p.cu_q[b + 1] = (int)min(end, (long long)p.total_q);
            p.new_len[b] = (int)min((long long)old + n, (long long)INT32_MAX);
        }
        __syncthreads();
        const long long lo = max(t0, s_tok[0]), hi = min(t1, s_tok[kScan]);
        for (long long t = lo + tid; t < hi; t += kScan) {
            int i = 0;  // the last sequence of the chunk that starts at or before t
#pragma unroll
            for (int step = kScan / 2; step > 0; step >>= 1)
                if (s_tok[i + step] <= t) i += step;
            const long long pos = s_old[i] + (t - s_tok[i]);
            const long long col = pos >> a.shift;
            int page = -1;
            if (col < p.max_pages) {
                int32_t* entry = p.block_table + (b0 + i) * p.table_stride + col;
                const int had = pages_of(s_old[i], a.shift);
                if (col < had) {
                    page = *entry;
                    bad |= page < 0;
                } else {
                    const long long k = count - 1 - (s_page[i] + col - had);
                    if (k >= 0) {
                        if (k < p.free_capacity) page = max(p.free_pages[k], -1);
                        bad |= page < 0;
                    }
                    if ((pos & mask) == 0) *entry = page;  // the token that opens the page
                }
            }
            const long long slot = ((long long)page << a.shift) + (pos & mask);
            const bool none = page < 0 || slot > INT32_MAX;
            bad |= page >= 0 && none;
            p.slots[t] = none ? -1 : (int)slot;
            p.positions[t] = (int)min(pos, (long long)INT32_MAX);
        }
        tok = s_tok[kScan];
        taken = s_page[kScan];
        __syncthreads();  // the next chunk overwrites the sums
    }
    for (long long t = max(t0, tok) + tid; t < t1; t += kScan) p.slots[t] = p.positions[t] = -1;
    if (blockIdx.x == 0 && tid == 0)
        p.free_left[0] = (int)max((long long)INT32_MIN, (long long)count - taken);
    if (bad) note_bad(a.err);
}

// ---------------------------------------------------------------- release
struct ReleaseArgs {
    attn_pages_release_params p;
    int shift;
    int per_block;  // sequences a block gives back
    int* err;
};

// Block i handles sequences [i * per_block, (i + 1) * per_block): it adds up the pages that the
// sequences before them give back, places its own 256 at a time by a prefix sum, and copies their table
// rows one after another.
__global__ void __launch_bounds__(kScan) pages_release_kernel(const ReleaseArgs a) {
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const attn_pages_release_params& p = a.p;
    __shared__ long long s_warp[kScan / 32], s_base[kScan];  // s_base: where a sequence's first page goes
    __shared__ int s_pages[kScan];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long b0 = (long long)blockIdx.x * a.per_block;
    const int b_end = (int)min((long long)p.num_seqs, b0 + a.per_block);
    bool bad = false;
    auto pages = [&](int gone, int len) -> int {  // pages that a sequence gives back
        return gone != 0 ? min(pages_of(max(len, 0), a.shift), p.max_pages) : 0;
    };
    long long sum = 0;
#pragma unroll 4
    for (int b = tid; b < b0; b += kScan) sum += pages(p.done[b], p.kv_len[b]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if (lane == 0) s_warp[warp] = sum;
    const int count = p.free_count[0];
    __syncthreads();
    long long base = count;
#pragma unroll
    for (int w = 0; w < kScan / 32; ++w) base += s_warp[w];
    for (int c0 = (int)b0; c0 < b_end; c0 += kScan) {
        const int b = c0 + tid;
        int m = 0;
        if (b < b_end) {
            const int gone = p.done[b], len = p.kv_len[b];
            bad |= len < 0 || len > (long long)p.max_pages << a.shift;
            m = pages(gone, len);
            p.new_len[b] = gone != 0 ? 0 : len;
        }
        long long x = m;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(kFull, x, o);
            if (lane >= o) x += u;
        }
        __syncthreads();  // the last use of the sums and places
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        x += base;
#pragma unroll
        for (int w = 0; w < kScan / 32; ++w) {
            if (w < warp) x += s_warp[w];
            base += s_warp[w];
        }
        s_base[tid] = x - m;
        s_pages[tid] = m;
        __syncthreads();
        for (int k = 0; k < min(kScan, b_end - c0); ++k) {
            const int32_t* row = p.block_table + (c0 + k) * p.table_stride;
            const long long first = s_base[k];
            const int n = s_pages[k];
#pragma unroll 4
            for (int i = tid; i < n; i += kScan) {
                const long long to = first + i;
                const int page = row[i];
                bad |= page < 0;  // a sequence that was never given all its pages
                if (to >= 0 && to < p.free_capacity)
                    p.free_pages[to] = page;
                else
                    bad = true;
            }
        }
    }
    if (b_end == p.num_seqs && tid == 0) p.free_left[0] = (int)min(base, (long long)INT32_MAX);
    if (bad) note_bad(a.err);
}

// ---------------------------------------------------------------- write
struct WriteArgs {
    attn_pages_write_params p;
    int shift;
    int pieces;  // 16-byte pieces of a row of k (all heads)
    int lanes;   // lanes that share a row: a power of two up to 32
    int* err;
};

template <int D>
__global__ void __launch_bounds__(256) pages_write_kernel(const WriteArgs a) {
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    constexpr int kPieces = D / 8;  // 16-byte pieces of one head
    const attn_pages_write_params& p = a.p;
    const int rows_per_block = 256 / a.lanes;
    const long long row = (long long)blockIdx.x * rows_per_block + threadIdx.x / a.lanes;
    if (row >= p.rows) return;
    const int slot = p.slots[row];
    if (slot < 0) return;
    const int page = slot >> a.shift;
    if (page >= p.num_pages) {
        note_bad(a.err);
        return;
    }
    const int off = slot & (p.page_size - 1);
    for (int i = threadIdx.x % a.lanes; i < a.pieces; i += a.lanes) {
        const long long h = i / kPieces, c = (i % kPieces) * 8;
        const uint16_t* k = static_cast<const uint16_t*>(p.k) + row * p.k_row_stride[0] + h * p.k_row_stride[1] + c;
        const uint16_t* v = static_cast<const uint16_t*>(p.v) + row * p.v_row_stride[0] + h * p.v_row_stride[1] + c;
        uint16_t* kc = static_cast<uint16_t*>(p.k_cache) + page * p.k_stride[0] + h * p.k_stride[1] + off * p.k_stride[2] + c;
        uint16_t* vc = static_cast<uint16_t*>(p.v_cache) + page * p.v_stride[0] + h * p.v_stride[1] + off * p.v_stride[2] + c;
        const uint4 kk = *reinterpret_cast<const uint4*>(k), vv = *reinterpret_cast<const uint4*>(v);
        *reinterpret_cast<uint4*>(kc) = kk;
        *reinterpret_cast<uint4*>(vc) = vv;
    }
}

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

}  // namespace

cudaError_t launch_pages_plan(const attn_pages_plan_params& p, const LaunchCommon& lc, cudaStream_t s) {
    PlanArgs a{};
    a.p = p;
    a.shift = log2_of(p.page_size);
    a.per_block = 2 * kScan;  // 5.0 us for 65.6k tokens of 500 sequences, 6.2 with 4 kScan, 5.2 with kScan
    a.err = lc.err;
    const int grid = p.total_q > 0 ? (int)(((long long)p.total_q + a.per_block - 1) / a.per_block) : 1;
    return launch_pdl(pages_plan_kernel, dim3(grid), dim3(kScan), 0, s, a);
}

cudaError_t launch_pages_release(const attn_pages_release_params& p, const LaunchCommon& lc, cudaStream_t s) {
    ReleaseArgs a{};
    a.p = p;
    a.shift = log2_of(p.page_size);
    // one sequence to a block, more only when that would make more than four blocks an SM (each
    // block reads the lengths before its own)
    const int blocks = 4 * lc.num_sms;
    const int even = (int)(((long long)p.num_seqs + blocks - 1) / blocks);
    a.per_block = even > 1 ? even : 1;
    a.err = lc.err;
    const int grid = p.num_seqs > 0 ? (int)(((long long)p.num_seqs + a.per_block - 1) / a.per_block) : 1;
    return launch_pdl(pages_release_kernel, dim3(grid), dim3(kScan), 0, s, a);
}

cudaError_t launch_pages_write(const attn_pages_write_params& p, const LaunchCommon& lc, cudaStream_t s) {
    WriteArgs a{};
    a.p = p;
    a.shift = log2_of(p.page_size);
    a.pieces = p.num_kv_heads * (p.d / 8);
    a.lanes = a.pieces >= 32 ? 32 : 1 << log2_of(a.pieces);
    a.err = lc.err;
    const long long per_block = 256 / a.lanes;
    const dim3 grid((unsigned)((p.rows + per_block - 1) / per_block));
    return p.d == 64 ? launch_pdl(pages_write_kernel<64>, grid, dim3(256), 0, s, a)
                     : launch_pdl(pages_write_kernel<128>, grid, dim3(256), 0, s, a);
}

}  // namespace attn
