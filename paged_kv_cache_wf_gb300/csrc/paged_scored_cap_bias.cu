// paged_scored_cap_bias.cu -- scored attention's tensor-core kernels, capped, then biased by distance.
#include "paged_scored.cuh"

namespace wf {

template <>
cudaError_t launch_scored_tc<kRuleCapBias>(const ScoredParams& p, const wf_pool_desc& pool, void* prep, int ctas,
                                 cudaStream_t stream) {
    return p.rows == 32 ? launch_tc<ScoredView<kRuleCapBias, true>>(p, pool, prep, ctas, stream)
                        : launch_tc<ScoredView<kRuleCapBias>>(p, pool, prep, ctas, stream);
}

}  // namespace wf
