// attn_paged.cu — attention of runs of tokens over a 16-bit paged cache (attn_paged.cuh).
#include "attn_paged.cuh"

namespace attn {

std::mutex& paged_launch_mutex() {
    static std::mutex mu;
    return mu;
}

size_t paged_workspace_bytes(const attn_paged_params& p, int num_sms) { return plan_of(p, num_sms, kRun).bytes; }

attn_status_t launch_paged(const attn_paged_params& p, const LaunchCommon& lc, cudaStream_t s) {
    return launch_variant<kRun>(p, Extra{}, lc, s);
}

}  // namespace attn
