// attn_paged_fp8.cu — attention of runs and trees of tokens over an 8-bit paged cache (attn_paged.cuh).
#include "attn_paged.cuh"

namespace attn {

attn_status_t launch_paged_fp8(const attn_paged_fp8_params& p, const LaunchCommon& lc, cudaStream_t s) {
    Extra x;
    x.mask = p.t.mask;
    x.mask_stride = p.t.mask_stride;
    x.words = p.t.words;
    x.k_scale = p.k_scale;
    x.v_scale = p.v_scale;
    for (int i = 0; i < 2; ++i) {
        x.k_scale_stride[i] = p.k_scale_stride[i];
        x.v_scale_stride[i] = p.v_scale_stride[i];
    }
    return launch_variant<kBytes>(p.t.f, x, lc, s);
}

}  // namespace attn
