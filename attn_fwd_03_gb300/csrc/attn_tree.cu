// attn_tree.cu — who sees whom in trees of drafted tokens, and their positions.
//
// A node's ancestors are found by following parents, each below its child, so a walk visits a row's bits
// from the highest down and ends after as many steps as the node is deep. A block takes a sequence (its
// parents in shared memory, a thread per node); the block behind the last sequence takes the padding rows.
// Bound by latency: a step's launch, two reads that depend on each other, and the deepest node's walk (one tree of 26
// nodes 1.8 us, 300 trees of up to 64 nodes 3.6 us, device time in a captured graph). Walks grow with a tree's depth, and a
// thread has up to 8 of them: a chain of 64 nodes takes 8 us, of 256 53 us, of 1024 663 us.
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxNodes = 1024;

struct TreeArgs {
    attn_tree_plan_params p;
    int* err;
};

__global__ void __launch_bounds__(kThreads) tree_plan_kernel(const TreeArgs a) {
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const attn_tree_plan_params& p = a.p;
    __shared__ int s_parent[kMaxNodes];
    const int b = blockIdx.x, tid = threadIdx.x;
    const int c0 = p.cu_q[b];
    const bool pad = b == p.num_seqs;
    const int c1 = pad ? p.total_q : p.cu_q[b + 1], len = pad ? 0 : p.kv_len[b];
    const int row0 = min(max(c0, 0), p.total_q), n = min(max(c1, row0), p.total_q) - row0;
    bool bad = c0 < 0 || c1 < c0 || c1 > p.total_q || (b == 0 && c0 != 0) || (!pad && len < n);
    const bool tree = !pad && n <= 32 * p.words;
    const long long base = (long long)len - n;
    if (tree) {
        for (int i = tid; i < n; i += kThreads) {
            int up = p.parents[row0 + i];
            if (up >= i || up < -1) {
                bad = true;
                up = -1;
            }
            s_parent[i] = up;
        }
        __syncthreads();
    }
    for (int i = tid; i < n; i += kThreads) {
        int32_t* row = p.mask + (row0 + i) * p.mask_stride;
        long long depth = i;
        if (tree) {
            depth = -1;
            int word = p.words - 1;
            uint32_t bits = 0;
            for (int at = i; at >= 0; at = s_parent[at]) {
                for (; word > at >> 5; --word) {
                    row[word] = (int32_t)bits;
                    bits = 0;
                }
                bits |= 1u << (at & 31);
                ++depth;
            }
            for (; word >= 0; --word) {
                row[word] = (int32_t)bits;
                bits = 0;
            }
        } else {
            for (int w = 0; w < p.words; ++w) row[w] = 0;
        }
        p.positions[row0 + i] = pad ? -1 : (int)max(-1ll, base + depth);
    }
    if (bad) atomicCAS(a.err, 0, ATTN_ERR_INVALID);
}

}  // namespace

cudaError_t launch_tree_plan(const attn_tree_plan_params& p, const LaunchCommon& lc, cudaStream_t s) {
    return launch_pdl(tree_plan_kernel, dim3((unsigned)p.num_seqs + 1), dim3(kThreads), 0, s, TreeArgs{p, lc.err});
}

}  // namespace attn
