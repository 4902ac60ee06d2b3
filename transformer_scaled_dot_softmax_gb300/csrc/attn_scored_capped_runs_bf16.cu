// attn_scored_capped_runs_bf16.cu -- scored attention forward: capped instances for keys that are
// summed in runs
// (apart from the others so that they compile in parallel).
#include "attn_scored_bf16.cuh"

namespace mha {

cudaError_t launch_attn_scored_capped_runs(const ScoredMaps &maps, int bias, const ScoredFwdParams &p, cudaStream_t stream) {
    return scored::launch_any<true, true>(maps, bias, p, stream);
}

}  // namespace mha
