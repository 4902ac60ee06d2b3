// attn_scored_bf16.cu -- scored attention forward: uncapped instances and the
// choice among all (the kernel is in attn_scored_bf16.cuh).
#include "attn_scored_bf16.cuh"

namespace mha {

cudaError_t launch_attn_scored_capped(const ScoredMaps &maps, int bias, const ScoredFwdParams &p, cudaStream_t stream);

cudaError_t launch_attn_scored(const ScoredMaps &maps, bool capped, int bias, const ScoredFwdParams &p,
                               cudaStream_t stream) {
    if (capped) return launch_attn_scored_capped(maps, bias, p, stream);
    if (bias == kBiasSlopes) return scored::launch_form<false, kBiasSlopes>(maps, p, stream);
    if (bias == kBiasBuckets) return scored::launch_form<false, kBiasBuckets>(maps, p, stream);
    return scored::launch_form<false, kBiasNone>(maps, p, stream);
}

}  // namespace mha
