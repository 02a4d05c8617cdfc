// paged_scored_cap_wide_bias.cu -- scored attention's tensor-core kernels, capped by more than kWideCap, then biased by
// distance.
#include "paged_scored.cuh"

namespace wf {

template <>
cudaError_t launch_scored_tc<kRuleWideBias>(const ScoredParams& p, const wf_pool_desc& pool, void* prep, int ctas,
                                 cudaStream_t stream) {
    return p.rows == 32 ? launch_tc<ScoredView<kRuleWideBias, true>>(p, pool, prep, ctas, stream)
                        : launch_tc<ScoredView<kRuleWideBias>>(p, pool, prep, ctas, stream);
}

}  // namespace wf
