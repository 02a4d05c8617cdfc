// paged_scored.cuh -- what the units of scored attention share (paged_scored.cu).  The kernels are
// compiled a rule at a time, in parallel.
#pragma once

#include "paged_tree_tc.cuh"

namespace wf {

// Spread: blocks of at most 32 rows (p.rows == 32).
template <int RULE>
cudaError_t launch_scored_tc(const ScoredParams& p, const wf_pool_desc& pool, void* prep, int ctas, cudaStream_t stream);
template <int RULE>
cudaError_t launch_scored_cc(const ScoredParams& p, const wf_pool_desc& pool, int ctas, cudaStream_t stream);

}  // namespace wf
