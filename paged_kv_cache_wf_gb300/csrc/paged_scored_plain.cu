// paged_scored_plain.cu -- scored attention's tensor-core kernels, no cap, no bias.
#include "paged_scored.cuh"

namespace wf {

template <>
cudaError_t launch_scored_tc<kRulePlain>(const ScoredParams& p, const wf_pool_desc& pool, void* prep, int ctas,
                                 cudaStream_t stream) {
    return p.rows == 32 ? launch_tc<ScoredView<kRulePlain, true>>(p, pool, prep, ctas, stream)
                        : launch_tc<ScoredView<kRulePlain>>(p, pool, prep, ctas, stream);
}

}  // namespace wf
