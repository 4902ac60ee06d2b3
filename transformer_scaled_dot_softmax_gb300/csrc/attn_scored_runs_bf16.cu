// attn_scored_runs_bf16.cu -- scored attention forward: uncapped instances for keys that are
// summed in runs
// (apart from the others so that they compile in parallel).
#include "attn_scored_bf16.cuh"

namespace mha {

cudaError_t launch_attn_scored_runs(const ScoredMaps &maps, int bias, const ScoredFwdParams &p, cudaStream_t stream) {
    return scored::launch_any<false, true>(maps, bias, p, stream);
}

}  // namespace mha
