// paged_scored_bias.cu -- scored attention's tensor-core kernels, biased by distance.
#include "paged_scored.cuh"

namespace wf {

template <>
cudaError_t launch_scored_tc<kRuleBias>(const ScoredParams& p, const wf_pool_desc& pool, void* prep, int ctas,
                                 cudaStream_t stream) {
    return p.rows == 32 ? launch_tc<ScoredView<kRuleBias, true>>(p, pool, prep, ctas, stream)
                        : launch_tc<ScoredView<kRuleBias>>(p, pool, prep, ctas, stream);
}

}  // namespace wf
