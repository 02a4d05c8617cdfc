// paged_scored_cap_wide.cu -- scored attention's tensor-core kernels, capped by more than kWideCap.
#include "paged_scored.cuh"

namespace wf {

template <>
cudaError_t launch_scored_tc<kRuleWide>(const ScoredParams& p, const wf_pool_desc& pool, void* prep, int ctas,
                                 cudaStream_t stream) {
    return p.rows == 32 ? launch_tc<ScoredView<kRuleWide, true>>(p, pool, prep, ctas, stream)
                        : launch_tc<ScoredView<kRuleWide>>(p, pool, prep, ctas, stream);
}

}  // namespace wf
