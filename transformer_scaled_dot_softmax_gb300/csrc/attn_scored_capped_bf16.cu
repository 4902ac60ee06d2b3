// attn_scored_capped_bf16.cu -- scored attention forward: capped instances
// (apart from the others so that the two compile in parallel).
#include "attn_scored_bf16.cuh"

namespace mha {

cudaError_t launch_attn_scored_capped(const ScoredMaps &maps, int bias, const ScoredFwdParams &p, cudaStream_t stream) {
    if (bias == kBiasSlopes) return scored::launch_form<true, kBiasSlopes>(maps, p, stream);
    if (bias == kBiasBuckets) return scored::launch_form<true, kBiasBuckets>(maps, p, stream);
    return scored::launch_form<true, kBiasNone>(maps, p, stream);
}

}  // namespace mha
