// paged_tree_tc.cu -- tree attention on the tensor cores: which shapes, and the launch (the kernel
// and its design notes are in paged_tree_tc.cuh).
#include "paged_tree_tc.cuh"

namespace wf {

bool tree_tc_supported(const wf_pool_desc& pool, int32_t num_q_heads) {
    if (pool.dtype == WF_DTYPE_F32 || pool.block_size % 16 != 0) return false;
    // slots are TMA coordinates
    return (int64_t)pool.num_blocks * pool.block_size <= INT32_MAX && num_q_heads / pool.num_kv_heads <= 8;
}

// Units of at most 128 rows: two streams over the same rows (32 requests of up to 64 rows 34.2 us,
// with two query tiles 38.4); else two query tiles (118 of up to 244 rows 277 us, with row
// blocks of 128, each of which reads K and V, 397).  The choice is the batch's, by max_q_len: in a
// batch with two query tiles a request of at most 128 rows runs on one of the two streams (118
// requests of 4-244 rows 267 us, 184 at the copy peak).  fp8 pools stay with row blocks of 128,
// each of which reads K and V and widens V again (118 of up to 244 rows 409 us).  A second query
// tile would leave room for two K slots instead of four; that form has not been built.
TreeShape tree_tc_shape(int G, int max_q_len, bool codes) {
    const int tok = TM / G;
    const int qt = codes || max_q_len <= tok ? 1 : 2;
    // a unit's start and end in tiles: 2 measured best (1, 2, 3, 4 at a batch of 32: 40.9, 35.1, 34.9,
    // 35.7 us; 118 wide trees: 336, 337, 347, 352 us); the CUDA cores' smaller tiles: 1
    return TreeShape{qt * TM, qt * tok, TN, 1, 2};
}

// fp8 pools: the q parts and the rows' factors.
size_t tree_tc_prep_bytes(int32_t B, int32_t num_q_heads, int32_t max_q_len, const wf_pool_desc& pool) {
    const uint64_t rows = (uint64_t)B * (uint64_t)max_q_len;
    if (rows > (uint64_t)INT32_MAX / 2) return SIZE_MAX;   // a draft's row is a TMA coordinate
    return (size_t)(rows * num_q_heads) * (2 * pool.head_dim + 4);
}

cudaError_t launch_tree_tc(const TreeParams& p, const wf_pool_desc& pool, void* prep, int ctas, cudaStream_t stream) {
    return launch_tc<TreeView>(p, pool, prep, ctas, stream);
}

}  // namespace wf
