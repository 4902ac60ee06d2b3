// attn_scored_capped_bf16.cu -- scored attention forward: capped instances
// (apart from the others so that they compile in parallel).
#include "attn_scored_bf16.cuh"

namespace mha {

cudaError_t launch_attn_scored_capped(const ScoredMaps &maps, int bias, const ScoredFwdParams &p, cudaStream_t stream) {
    return scored::launch_any<true, false>(maps, bias, p, stream);
}

}  // namespace mha
