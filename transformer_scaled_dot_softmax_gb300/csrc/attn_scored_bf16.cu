// attn_scored_bf16.cu -- scored attention forward: uncapped instances and the
// choice among all (the kernel is in attn_scored_bf16.cuh).
#include "attn_scored_bf16.cuh"

namespace mha {

cudaError_t launch_attn_scored_capped(const ScoredMaps &maps, int bias, const ScoredFwdParams &p, cudaStream_t stream);
cudaError_t launch_attn_scored_runs(const ScoredMaps &maps, int bias, const ScoredFwdParams &p, cudaStream_t stream);
cudaError_t launch_attn_scored_capped_runs(const ScoredMaps &maps, int bias, const ScoredFwdParams &p, cudaStream_t stream);

cudaError_t launch_attn_scored(const ScoredMaps &maps, bool capped, int bias, const ScoredFwdParams &p,
                               cudaStream_t stream) {
    const bool runs = needs_runs(p.part_o && p.cache_cap > p.Tk ? p.cache_cap : p.Tk);
    if (runs) return capped ? launch_attn_scored_capped_runs(maps, bias, p, stream) : launch_attn_scored_runs(maps, bias, p, stream);
    return capped ? launch_attn_scored_capped(maps, bias, p, stream) : scored::launch_any<false, false>(maps, bias, p, stream);
}

}  // namespace mha
