// paged_scored.cu -- attention over the paged cache whose scores are capped and biased and whose
// rows see a range of positions: the list of row blocks, the workspace and the dispatch.
//
// Row (token t at position p_t of request b, query head g) sees the positions
//     [max(begin_t, p_t - window + 1), min(end_t, len_b)),   begin_t = 0, end_t = p_t + 1 unless given,
// with scores  x = scale q K_p;  x = cap tanh(x / cap);  x = x - slope_g |p_t - p|,
// and o = softmax(x) V over them, 0 where it sees nothing.
//
// The kernels are the tree attention's (paged_tree_tc.cuh on the tensor cores, paged_tree_cc.cuh on
// the CUDA cores; paged_tree.cuh has the division of the work) over another list of units: a
// row block reads only the tiles that some of its rows see.  What those are depends on the lengths, the
// window and the ranges, so one small grid before the attention makes the list; for fp8 pools it
// also splits q into its e4m3 parts.  The attention grid is its programmatic dependent and sets
// itself up meanwhile.
#include <cooperative_groups.h>

#include "paged_scored.cuh"

namespace wf {

namespace {

namespace cg = cooperative_groups;

constexpr int kListThreads = 512, kListWarps = kListThreads / 32;
constexpr int kListCluster = 8;        // CTAs that look at the rows' ranges together
constexpr int kListShared = 2048;      // requests whose first blocks stand in shared memory

struct ListParams {
    ScoredParams s;
    int32_t* first;        // [B + 1] for batches that shared memory does not hold
    ScoredBlock* blocks;
    int32_t* before;
    int32_t* num_blocks;
    int32_t capacity;      // blocks that there is room for
    int32_t tile;
    unsigned char* parts;  // fp8: [2][total_q][H_q][D]
    float* q_inv;          // [total_q][H_q]
};

// Exclusive sum over the CTA's threads; `total` is everybody's.
__device__ __forceinline__ int64_t list_sum(int64_t mine, int64_t* warps, int64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = incl;
    __syncthreads();
    int64_t w = lane < kListWarps ? warps[lane] : 0;
    const int64_t own = w;
#pragma unroll
    for (int o = 1; o < kListWarps; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, kListWarps - 1);
    return __shfl_sync(0xffffffffu, w - own, warp) + incl - mine;
}

// The list of row blocks, by the CTAs of one cluster.
__device__ __forceinline__ void make_list(const ListParams& p, int rank, int ctas, int32_t* s_first, int64_t* s_warps) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const ScoredParams& s = p.s;
    // every CTA has all requests' first blocks
    int32_t* first = s.B <= kListShared ? s_first : p.first;
    const int per = (s.B + kListThreads - 1) / kListThreads;
    const int b0 = min(tid * per, s.B), b1 = min(b0 + per, s.B);
    const auto blocks_of = [&](const TreeReq& r) { return r.n / s.tokb + (r.n % s.tokb != 0); };
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += blocks_of(tree_request(s, b, rank == 0));
    int64_t total;
    int64_t at = list_sum(mine, s_warps, total);
    // offsets that are not in order may name rows twice
    if (total > p.capacity) {
        if (rank == 0 && tid == 0) report(s.dev_status, WF_DEV_BAD_SEQLEN);
        total = 0;
    }
    const int nb = (int)total;
    for (int b = b0; b < b1; ++b) {
        first[b] = (int32_t)min(at, (int64_t)INT32_MAX);     // (more than one CTA writes the same)
        at += blocks_of(tree_request(s, b, false));
    }
    if (tid == 0) first[s.B] = nb;
    __syncthreads();
    const bool by_warp = s.ranges != nullptr;
    const int step = ctas * (by_warp ? kListWarps : kListThreads);
    for (int x = by_warp ? rank * kListWarps + warp : rank * kListThreads + tid; x < nb; x += step) {
        int lo_b = 0, hi_b = s.B;
        while (hi_b - lo_b > 1) {
            const int mid = (lo_b + hi_b) >> 1;
            if (first[mid] <= x)
                lo_b = mid;
            else
                hi_b = mid;
        }
        const TreeReq r = tree_request(s, lo_b, false);
        const int i0 = (x - first[lo_b]) * s.tokb;
        ScoredBlock k = scored_block(s, lo_b, r, i0, p.tile);
        if (by_warp) {
            int lo = INT32_MAX, hi = 0, full_lo = 0, full_hi = INT32_MAX;
            for (int i = lane; i < k.rows_tok; i += 32) {
                const int2 see = scored_range(s, k.q_row + i, k.at + i, k.len);
                if (see.x < see.y) {
                    lo = min(lo, see.x);
                    hi = max(hi, see.y);
                }
                full_lo = max(full_lo, see.x);
                full_hi = min(full_hi, see.y);
            }
            k.lo = __reduce_min_sync(0xffffffffu, lo);
            k.hi = __reduce_max_sync(0xffffffffu, hi);
            k.full_lo = __reduce_max_sync(0xffffffffu, full_lo);
            k.full_hi = __reduce_min_sync(0xffffffffu, full_hi);
            if (k.hi == 0) k.lo = 0;
            k.tile0 = k.lo / p.tile;
            k.nt = max(1, (k.hi + p.tile - 1) / p.tile - k.tile0);
        }
        if (!by_warp || lane == 0) {
            p.blocks[x] = k;
            p.before[x] = k.nt + s.ucost;
        }
    }
    if (ctas > 1)
        cg::this_cluster().sync();
    else
        __syncthreads();
    if (rank != 0) return;
    // costs before each block
    int64_t done = 0;
    for (int x0 = 0; x0 < nb; x0 += kListThreads) {
        const int x = x0 + tid;
        const int64_t w = x < nb ? __ldcg(p.before + x) : 0;
        int64_t sum;
        const int64_t before = done + list_sum(w, s_warps, sum);
        if (x < nb) p.before[x] = (int32_t)min(before, (int64_t)INT32_MAX);
        done += sum;
    }
    if (tid == 0) {
        // cost positions are 32-bit: 2^31 tiles, which no memory holds but shared blocks could make
        const bool much = done * s.H_kv > INT32_MAX;
        if (much) report(s.dev_status, WF_DEV_BAD_SEQLEN);
        *p.num_blocks = much ? 0 : nb;
        p.before[nb] = much ? 0 : (int32_t)done;
    }
}

// CTAs 0 .. ctas - 1 make the list, the others (fp8 pools) the parts of q.
template <int D>
__global__ void __launch_bounds__(kListThreads) scored_list_kernel(const ListParams p, int ctas) {
    __shared__ int32_t s_first[kListShared + 1];
    __shared__ int64_t s_warps[kListWarps];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if ((int)blockIdx.x < ctas) {
        make_list(p, blockIdx.x, ctas, s_first, s_warps);
        return;
    }
    constexpr int kLanes = D / 8, kStep = kListThreads / kLanes;
    const int l = threadIdx.x % kLanes;
    const int64_t all = (int64_t)p.s.total_q * p.s.H_q;
    const int64_t r0 = (int64_t)(blockIdx.x - ctas) * (kStep * kPartPer) + threadIdx.x / kLanes;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.s.q);
    uint4 raw[kPartPer];
#pragma unroll
    for (int k = 0; k < kPartPer; ++k) {
        const int64_t r = r0 + k * kStep;
        raw[k] = r < all ? __ldg(reinterpret_cast<const uint4*>(q + r * D) + l) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < kPartPer; ++k) {
        const int64_t r = r0 + k * kStep;
        uint2 hi, lo;
        const float inv = split_q_row<D>(raw[k], hi, lo);
        if (r >= all) continue;
        *reinterpret_cast<uint2*>(p.parts + r * D + 8 * l) = hi;
        *reinterpret_cast<uint2*>(p.parts + (all + r) * D + 8 * l) = lo;
        if (l == 0) p.q_inv[r] = inv;
    }
}

// Blocks of at most 32 rows (tensor cores): a row stands in all four quarters of the query tile, each of
// which takes a quarter of a tile's positions, so that all eight softmax warps work on it.  (Of one token of 4
// query heads the other way has 4 lanes of one warp a stream, which was the bound: 231 capped decodes 393 us.)
bool scored_shape(const wf_pool_desc& pool, int32_t num_q_heads, int32_t max_q_len, TreeShape* s) {
    if (!tree_shape(pool, num_q_heads, max_q_len, s)) return false;
    const int G = num_q_heads / pool.num_kv_heads;
    if (tree_tc_supported(pool, num_q_heads) && max_q_len <= 32 / G) {
        s->rows = 32;
        s->tokb = 32 / G;
    }
    return true;
}

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Blocks that a batch can have.  Counted with the fewest rows that any kernel's block holds, so that
// a longer max_q_len, which may go over to larger blocks, never needs less room.
int64_t list_capacity(const wf_pool_desc& pool, int32_t num_q_heads, int32_t B, int32_t total_q, int32_t max_q_len) {
    TreeShape s;
    if (!scored_shape(pool, num_q_heads, 1, &s)) return 0;
    const int64_t by_rows = (int64_t)total_q / s.tokb + B, by_request = ((int64_t)max_q_len + s.tokb - 1) / s.tokb;
    const int64_t all = by_request == 0 ? 0 : B > by_rows / by_request ? by_rows : (int64_t)B * by_request;
    return all < by_rows ? all : by_rows;
}

struct Layout {
    int64_t rows, list, parts, q_inv, bytes;   // rows of the pieces; byte offsets behind them
    int64_t blocks, before, first, count;
};

bool scored_layout(const wf_pool_desc& pool, int32_t num_q_heads, int32_t B, int32_t total_q, int32_t max_q_len,
                   int32_t max_seq_len, TreeShape* s, int64_t* ctas, Layout* l) {
    if (B < 0 || total_q < 0 || max_q_len < 0 || max_seq_len < 0 || !scored_shape(pool, num_q_heads, max_q_len, s)) return false;
    *ctas = tree_ctas(*s, B, pool.num_kv_heads, max_q_len, max_seq_len);
    l->rows = 2 * *ctas * s->rows;
    const int64_t cap = list_capacity(pool, num_q_heads, B, total_q, max_q_len);
    // o, (m, l) and records as for tree attention, then the list and the parts of q
    l->blocks = round_up(l->rows * (pool.head_dim * 4 + 8) + kTreeRecs * (int64_t)sizeof(int4), 128);
    l->before = l->blocks + cap * (int64_t)sizeof(ScoredBlock);
    l->first = l->before + (cap + 1) * 4;
    l->count = l->first + ((int64_t)B + 1) * 4;
    l->parts = round_up(l->count + 4, 128);
    l->bytes = l->parts;
    l->q_inv = 0;
    if (pool.dtype == WF_DTYPE_FP8_E4M3 && tree_tc_supported(pool, num_q_heads)) {
        if (total_q > INT32_MAX / 2) return false;    // a token's row is a TMA coordinate
        const int64_t q = (int64_t)total_q * num_q_heads;
        l->q_inv = round_up(l->parts + 2 * q * pool.head_dim, 16);
        l->bytes = l->q_inv + 4 * q;
    }
    return true;
}

cudaError_t launch_list(const ListParams& p, bool d128, cudaStream_t stream) {
    // one CTA, or a cluster where rows' ranges have to be looked at: at one row a lane and round, four rounds
    const int ctas = p.s.blocks == nullptr ? 0 : p.s.ranges != nullptr && p.s.total_q > 4 * kListThreads ? kListCluster : 1;
    const int cluster = ctas > 0 ? ctas : 1;
    int64_t parts = 0;
    if (p.parts != nullptr) {
        const int64_t rows = (int64_t)p.s.total_q * p.s.H_q, per = kListThreads / (d128 ? 16 : 8) * kPartPer;
        parts = round_up((rows + per - 1) / per, cluster);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ctas + parts));
    cfg.blockDim = dim3(kListThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1;
    return d128 ? cudaLaunchKernelEx(&cfg, scored_list_kernel<128>, p, ctas)
                : cudaLaunchKernelEx(&cfg, scored_list_kernel<64>, p, ctas);
}

}  // namespace

size_t scored_workspace_bytes(int32_t B, int32_t num_q_heads, int32_t total_q, int32_t max_q_len, int32_t max_seq_len,
                              const wf_pool_desc& pool) {
    TreeShape s;
    int64_t ctas;
    Layout l;
    return scored_layout(pool, num_q_heads, B, total_q, max_q_len, max_seq_len, &s, &ctas, &l) ? (size_t)l.bytes : 0;
}

cudaError_t launch_paged_scored(const ScoredArgs& a, const wf_pool_desc& pool, uint32_t* dev_status, cudaStream_t stream) {
    TreeShape s;
    int64_t cap;
    Layout l;
    if (!scored_layout(pool, a.num_q_heads, a.B, a.total_q, a.max_q_len, a.max_seq_len, &s, &cap, &l))
        return cudaErrorNotSupported;
    const int64_t fit = (int64_t)s.ctas_per_sm * num_sms();
    const int ctas = (int)(cap < fit ? cap : fit);
    char* ws = static_cast<char*>(a.workspace);
    ScoredParams p;
    p.out = a.out;
    p.q = a.q;
    p.k_pool = a.k_pool;
    p.v_pool = a.v_pool;
    p.block_tables = a.block_tables;
    p.seq_lens = a.seq_lens;
    p.cu_q_lens = a.cu_q_lens;
    p.mask = nullptr;
    p.dev_status = dev_status;
    p.ws_o = reinterpret_cast<float*>(ws);
    p.ws_ml = reinterpret_cast<float2*>(p.ws_o + l.rows * pool.head_dim);
    p.ws_rec = reinterpret_cast<int4*>(p.ws_ml + l.rows);
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
    p.W = 0;
    p.rows = s.rows;
    p.tokb = s.tokb;
    p.ucost = s.ucost;
    constexpr float kLog2e = 1.4426950408889634f;
    p.scale_log2 = tree_factor(a.scale * kLog2e);
    p.ranges = reinterpret_cast<const int2*>(a.row_ranges);
    p.slopes = a.slopes;
    p.window = a.window;
    p.cap_in = p.cap_out = 0.f;
    if (a.cap > 0.f) {
        p.cap_in = (float)((double)a.scale / (double)a.cap);   // (may be 0: scores are masked behind the cap)
        p.cap_out = a.cap * kLog2e;
    }
    const bool tc = tree_tc_supported(pool, a.num_q_heads), codes = tc && pool.dtype == WF_DTYPE_FP8_E4M3;
    ListParams list;
    list.blocks = reinterpret_cast<ScoredBlock*>(ws + l.blocks);
    list.before = reinterpret_cast<int32_t*>(ws + l.before);
    list.first = reinterpret_cast<int32_t*>(ws + l.first);
    list.num_blocks = reinterpret_cast<int32_t*>(ws + l.count);
    list.capacity = (int32_t)((l.before - l.blocks) / (int64_t)sizeof(ScoredBlock));
    list.tile = s.tile;
    list.parts = codes ? reinterpret_cast<unsigned char*>(ws + l.parts) : nullptr;
    list.q_inv = reinterpret_cast<float*>(ws + l.q_inv);
    p.blocks = list.blocks;
    p.before = list.before;
    p.num_blocks = list.num_blocks;
    p.q_inv = codes ? list.q_inv : nullptr;
    // One block a request and no ranges: the kernel deals the requests by itself (one user 10.9 us, with a list 2 more).
    if (tc && s.rows == 32 && a.row_ranges == nullptr) p.blocks = nullptr;
    list.s = p;
    cudaError_t e = cudaSuccess;
    if (p.blocks != nullptr || codes) e = launch_list(list, pool.head_dim == 128, stream);
    if (e != cudaSuccess) return e;
    const bool capped = a.cap > 0.f, bias = a.slopes != nullptr;
    if (!tc)
        return capped ? bias ? launch_scored_cc<kRuleCapBias>(p, pool, ctas, stream)
                             : launch_scored_cc<kRuleCap>(p, pool, ctas, stream)
               : bias ? launch_scored_cc<kRuleBias>(p, pool, ctas, stream)
                      : launch_scored_cc<kRulePlain>(p, pool, ctas, stream);
    if (a.cap > kWideCap)
        e = bias ? launch_scored_tc<kRuleWideBias>(p, pool, list.parts, ctas, stream)
                 : launch_scored_tc<kRuleWide>(p, pool, list.parts, ctas, stream);
    else
        e = capped ? bias ? launch_scored_tc<kRuleCapBias>(p, pool, list.parts, ctas, stream)
                          : launch_scored_tc<kRuleCap>(p, pool, list.parts, ctas, stream)
            : bias ? launch_scored_tc<kRuleBias>(p, pool, list.parts, ctas, stream)
                   : launch_scored_tc<kRulePlain>(p, pool, list.parts, ctas, stream);
    if (e != cudaSuccess || ctas == 1) return e;
    return tree_join(p, pool, ctas, stream);
}

}  // namespace wf
