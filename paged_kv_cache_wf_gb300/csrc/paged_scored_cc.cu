// paged_scored_cc.cu -- scored attention's CUDA-core kernels.
#include "paged_scored.cuh"
#include "paged_tree_cc.cuh"

namespace wf {

template <>
cudaError_t launch_scored_cc<kRulePlain>(const ScoredParams& p, const wf_pool_desc& pool, int ctas, cudaStream_t stream) {
    return launch_cc_pool<ScoredView<kRulePlain>>(p, pool, ctas, stream);
}
template <>
cudaError_t launch_scored_cc<kRuleBias>(const ScoredParams& p, const wf_pool_desc& pool, int ctas, cudaStream_t stream) {
    return launch_cc_pool<ScoredView<kRuleBias>>(p, pool, ctas, stream);
}
template <>
cudaError_t launch_scored_cc<kRuleCapBias>(const ScoredParams& p, const wf_pool_desc& pool, int ctas, cudaStream_t stream) {
    return launch_cc_pool<ScoredView<kRuleCapBias>>(p, pool, ctas, stream);
}
template <>
cudaError_t launch_scored_cc<kRuleCap>(const ScoredParams& p, const wf_pool_desc& pool, int ctas, cudaStream_t stream) {
    return launch_cc_pool<ScoredView<kRuleCap>>(p, pool, ctas, stream);
}

}  // namespace wf
