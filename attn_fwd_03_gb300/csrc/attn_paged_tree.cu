// attn_paged_tree.cu — attention of trees of drafted tokens over a 16-bit paged cache (attn_paged.cuh).
#include "attn_paged.cuh"

namespace attn {

attn_status_t launch_paged_tree(const attn_paged_tree_params& p, const LaunchCommon& lc, cudaStream_t s) {
    Extra x;
    x.mask = p.mask;
    x.mask_stride = p.mask_stride;
    x.words = p.words;
    return launch_variant<kTree>(p.f, x, lc, s);
}

}  // namespace attn
