// paged_tree.cu -- attention of trees of drafted tokens over the paged cache: shapes, workspace
// and dispatch (the kernels are in paged_tree_cc.cuh and paged_tree_tc.cuh).
#include "paged_tree_cc.cuh"

namespace wf {

bool tree_shape(const wf_pool_desc& pool, int32_t num_q_heads, int32_t max_q_len, TreeShape* s) {
    if (num_q_heads % pool.num_kv_heads != 0) return false;
    const int G = num_q_heads / pool.num_kv_heads;
    if (G < 1 || G > 8) return false;
    if (tree_tc_supported(pool, num_q_heads)) {
        *s = tree_tc_shape(G, max_q_len, pool.dtype == WF_DTYPE_FP8_E4M3);
    } else {
        const int rpw = cc_rows_per_warp((int64_t)max_q_len * G), bytes = pool.dtype == WF_DTYPE_F32 ? 4 : 2;
        *s = TreeShape{kCcWarps * rpw, kCcWarps * rpw / G, kCcTile, cc_ctas_per_sm(bytes, pool.head_dim, rpw), 1};
    }
    return true;
}

// CTAs the launch may use: no more than there can be tiles.
int64_t tree_ctas(const TreeShape& s, int32_t B, int32_t H_kv, int32_t max_q_len, int32_t max_seq_len) {
    const int64_t cap = (int64_t)s.ctas_per_sm * kTreeMaxSms;
    int64_t all = 1;
    for (const int64_t f : {(int64_t)B, (int64_t)H_kv, ((int64_t)max_q_len + s.tokb - 1) / s.tokb,
                            ((int64_t)max_seq_len + s.tile - 1) / s.tile}) {
        if (f == 0) return 1;
        all = f >= cap ? cap : all * f;
        if (all > cap) all = cap;
    }
    return all;
}

cudaError_t tree_join(const TreeParams& p, const wf_pool_desc& pool, int ctas, cudaStream_t stream) {
    return pool.head_dim == 128 ? launch_join<BF16, 128>(p, ctas, stream) : launch_join<BF16, 64>(p, ctas, stream);
}

int tree_kernel_kind(const wf_pool_desc& pool, int32_t num_q_heads) {
    TreeShape s;
    if (!tree_shape(pool, num_q_heads, 1, &s)) return WF_KERNEL_NONE;
    return tree_tc_supported(pool, num_q_heads) ? WF_KERNEL_TENSOR_CORES : WF_KERNEL_CUDA_CORES;
}

size_t tree_workspace_bytes(int32_t B, int32_t num_q_heads, int32_t max_q_len, int32_t max_seq_len,
                            const wf_pool_desc& pool) {
    TreeShape s;
    if (B < 0 || max_q_len < 0 || max_seq_len < 0 || !tree_shape(pool, num_q_heads, max_q_len, &s)) return 0;
    const int64_t ctas = tree_ctas(s, B, pool.num_kv_heads, max_q_len, max_seq_len);
    const int64_t rows = 2 * ctas * s.rows;
    const size_t bytes = (size_t)(256 + kTreeRecs * (int64_t)sizeof(int4) + rows * 8 + rows * pool.head_dim * 4);
    if (pool.dtype != WF_DTYPE_FP8_E4M3 || !tree_tc_supported(pool, num_q_heads)) return bytes;
    const size_t prep = tree_tc_prep_bytes(B, num_q_heads, max_q_len, pool);
    return prep == SIZE_MAX ? 0 : bytes + prep;
}

cudaError_t launch_paged_tree(const TreeArgs& a, const wf_pool_desc& pool, uint32_t* dev_status,
                              cudaStream_t stream) {
    TreeShape s;
    if (!tree_shape(pool, a.num_q_heads, a.max_q_len, &s)) return cudaErrorNotSupported;
    const int64_t cap = tree_ctas(s, a.B, pool.num_kv_heads, a.max_q_len, a.max_seq_len);
    const int64_t fit = (int64_t)s.ctas_per_sm * num_sms();
    const int ctas = (int)(cap < fit ? cap : fit);
    const int64_t rows = 2 * cap * s.rows;
    TreeParams p;
    p.out = a.out;
    p.q = a.q;
    p.k_pool = a.k_pool;
    p.v_pool = a.v_pool;
    p.block_tables = a.block_tables;
    p.seq_lens = a.seq_lens;
    p.cu_q_lens = a.cu_q_lens;
    p.mask = a.tree_mask;
    p.dev_status = dev_status;
    p.ws_o = static_cast<float*>(a.workspace);
    p.ws_ml = reinterpret_cast<float2*>(p.ws_o + rows * pool.head_dim);
    p.ws_rec = reinterpret_cast<int4*>(p.ws_ml + rows);
    p.M = a.max_blocks_per_seq;
    p.B = a.B;
    p.total_q = a.total_q;
    p.max_q_len = a.max_q_len;
    p.max_seq_len = a.max_seq_len;
    p.H_q = a.num_q_heads;
    p.H_kv = pool.num_kv_heads;
    p.G = a.num_q_heads / pool.num_kv_heads;
    p.N = pool.num_blocks;
    p.P = pool.block_size;
    p.W = a.mask_words;
    p.rows = s.rows;
    p.tokb = s.tokb;
    p.ucost = s.ucost;
    p.q_inv = nullptr;
    p.scale_log2 = tree_factor(a.scale * 1.4426950408889634f);
    if (tree_tc_supported(pool, a.num_q_heads)) {
        void* prep = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(p.ws_rec + kTreeRecs) + 127) & ~(uintptr_t)127);
        const cudaError_t e = launch_tree_tc(p, pool, prep, ctas, stream);
        if (e != cudaSuccess || ctas == 1) return e;
        return tree_join(p, pool, ctas, stream);
    }
    return launch_cc_pool<TreeView>(p, pool, ctas, stream);
}

}  // namespace wf
