// paged_scored_cap.cu -- scored attention's tensor-core kernels, capped.
#include "paged_scored.cuh"

namespace wf {

template <>
cudaError_t launch_scored_tc<kRuleCap>(const ScoredParams& p, const wf_pool_desc& pool, void* prep, int ctas,
                                 cudaStream_t stream) {
    return p.rows == 32 ? launch_tc<ScoredView<kRuleCap, true>>(p, pool, prep, ctas, stream)
                        : launch_tc<ScoredView<kRuleCap>>(p, pool, prep, ctas, stream);
}

}  // namespace wf
