// paged_tree.cuh -- what the tree-attention kernels share: parameters, the division of
// the work among the CTAs, and the workspace.
//
// A unit is one block of a request's draft rows (row = (draft, query head of the
// group)) under one KV head: softmax over the request's cached positions and drafts,
// read tile by tile (kTile positions of the kernel).  Its cost is its tiles plus a
// constant for its start and end.  All units stand in a row, request by request
// (row block, then KV head innermost), and CTA k of n takes the stretch [s k, s (k + 1))
// of their total cost W, s = ceil(W / n): every CTA gets the same share of tiles
// whatever the lengths, and at most the first and the last unit of a stretch are cut.  A
// cut unit's pieces leave their running maximum, sum and unnormalised outputs in the
// workspace, two pieces a CTA at most, so the workspace does not grow with the context;
// the joining kernel adds them up in position order.
// Fixed spans (as the decode's) would write a row's partial every few hundred
// positions: at 64 drafts of 4 heads that is as many bytes as the K and V they read.
#pragma once

#include <cfloat>
#include <cmath>

#include "wf_internal.h"

namespace wf {

struct TreeParams {
    void* out;
    const void* q;
    const void* k_pool;
    const void* v_pool;
    const int32_t* block_tables;
    const int32_t* seq_lens;
    const int32_t* cu_q_lens;
    const uint32_t* mask;
    uint32_t* dev_status;
    float* ws_o;     // [2 * CTAs][row block] rows of D
    float2* ws_ml;   // [2 * CTAs][row block]
    // [kTreeRecs], a CTA each: the cut unit that starts in this CTA: {its first draft's row of q, KV head, last CTA
    // with a piece of it, rows (0: there is no such unit)}
    int4* ws_rec;
    int32_t M, B, total_q, max_q_len, max_seq_len, H_q, H_kv, G, N, P, W;
    int32_t rows;    // rows of a row block in the workspace
    int32_t tokb;    // drafts of a row block
    int32_t ucost;   // a unit's start and end, in tiles
    float scale_log2;
    const float* q_inv;   // fp8 pools on the tensor cores: factors of the prepared q rows
};

// A factor of the scores, held at fp32's smallest normal number or above (its sign kept): a
// masked score is -inf before it is scaled, and -inf * 0 is NaN.  At that factor every finite score
// has a weight of 2^0, as it has at 0.
__host__ __device__ __forceinline__ float tree_factor(float f) { return copysignf(fmaxf(fabsf(f), FLT_MIN), f); }

// Rows of a row block, drafts in it, tile and CTAs an SM of the kernel that runs a call.
struct TreeShape {
    int rows, tokb, tile, ctas_per_sm, ucost;
};

// The tensor-core kernel (paged_tree_tc.cu).
bool tree_tc_supported(const wf_pool_desc& pool, int32_t num_q_heads);
TreeShape tree_tc_shape(int G, int max_q_len, bool codes);
size_t tree_tc_prep_bytes(int32_t B, int32_t num_q_heads, int32_t max_q_len, const wf_pool_desc& pool);
cudaError_t launch_tree_tc(const TreeParams& p, const wf_pool_desc& pool, void* prep, int ctas, cudaStream_t stream);

namespace {

constexpr int kTreeMaxSms = 160;    // SMs a launch may use (the workspace holds their CTAs' pieces)
// Records in the workspace: of the most CTAs any kernel uses, not of this call's, so that more
// drafts never need less (beyond 16 rows the fp32 kernel has half the CTAs, each with twice the rows).
constexpr int kTreeRecs = 2 * kTreeMaxSms;

// A request's drafts and length, n = 0 for one that fails the checks.
struct TreeReq {
    int q_begin, n, len;
};

__device__ __forceinline__ TreeReq tree_request(const TreeParams& p, int b, bool tell) {
    TreeReq r;
    r.q_begin = __ldg(p.cu_q_lens + b);
    const int q_end = __ldg(p.cu_q_lens + b + 1);
    r.len = __ldg(p.seq_lens + b);
    r.n = q_end - r.q_begin;
    const bool bad = r.q_begin < 0 || r.n < 0 || q_end > p.total_q || r.n > p.max_q_len || r.len < r.n ||
                     r.len > p.max_seq_len || (int64_t)r.len > (int64_t)p.M * p.P;
    if (bad) {
        if (tell) report(p.dev_status, WF_DEV_BAD_SEQLEN);
        r.n = 0;
    }
    return r;
}

__device__ __forceinline__ int64_t tree_cost(const TreeParams& p, const TreeReq& r, int tile) {
    if (r.n == 0) return 0;
    return (int64_t)((r.n + p.tokb - 1) / p.tokb) * p.H_kv * ((r.len + tile - 1) / tile + p.ucost);
}

// Where a CTA's stretch begins.  In shared memory, filled by tree_begin.
struct alignas(16) TreeStart {   // 64-bit scratch follows it in shared memory
    int share;   // s
    int left;    // cost of this CTA's stretch
    int pos;     // its first cost position
    int off;     // that position within request b
    int b;
    TreeReq r;   // request b
};

// All threads of the CTA; `scratch` holds blockDim.x / 32 values.  Ends with a barrier.
// Cost positions are 32-bit from here on: a batch of 2^31 tiles, which no memory holds but
// shared blocks could make, is reported and not worked on.
__device__ __forceinline__ void tree_begin(const TreeParams& p, int tile, int cta, int ncta, TreeStart* st,
                                           int64_t* scratch) {
    const int tid = threadIdx.x, nthr = blockDim.x, lane = tid & 31, warp = tid >> 5, nwarp = nthr >> 5;
    const int per = (p.B + nthr - 1) / nthr;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    int64_t mine = 0;
    // rolled: this runs once, and what it takes of the instruction cache is missed later
#pragma unroll 1
    for (int b = b0; b < b1; ++b) mine += tree_cost(p, tree_request(p, b, cta == 0), tile);
    int64_t incl = mine;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    // sums over the warps, in two parts of 20 bits and more (2^40 stands for all that is too much)
    const int64_t v = lane < nwarp ? min(scratch[lane], (int64_t)1 << 40) : 0;
    const uint32_t lo = (uint32_t)v & 0xfffffu, hi = (uint32_t)(v >> 20);
    const auto sum = [](uint32_t h, uint32_t l) {
        return ((int64_t)__reduce_add_sync(0xffffffffu, h) << 20) + __reduce_add_sync(0xffffffffu, l);
    };
    int64_t total = sum(hi, lo);
    const int64_t before = sum(lane < warp ? hi : 0u, lane < warp ? lo : 0u);
    if (total > INT32_MAX) {
        if (cta == 0 && tid == 0) report(p.dev_status, WF_DEV_BAD_SEQLEN);
        total = mine = 0;
    }
    const uint32_t share = ((uint32_t)total + ncta - 1) / (uint32_t)ncta;
    const int s = (int)min((int64_t)share * cta, total), e = (int)min((int64_t)s + share, total);
    const int first = (int)(before + incl - mine);   // cost position of request b0
    if (tid == 0) {
        st->share = (int)share;
        st->left = e - s;
        st->pos = s;
    }
    if (s < e && first <= s && s < first + (int)mine) {
        int at = first;
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            const TreeReq r = tree_request(p, b, false);
            const int c = (int)tree_cost(p, r, tile);
            if (s < at + c) {
                st->b = b;
                st->r = r;
                st->off = s - at;
                break;
            }
            at += c;
        }
    }
    __syncthreads();
}

// One piece of work: tiles [j0, j1) of a unit of `nt`.
struct TreePiece {
    int b, h, qb;
    int q_begin, n, c;   // first row of q, drafts, cached positions
    int rows_tok;        // drafts of this row block
    int kend;            // positions of the request
    int j0, j1, nt;
    int end;             // cost position of the unit's end
};

// Walks a CTA's pieces in order.  All lanes of a warp together; every warp that walks
// sees the same pieces.
struct TreeWalk {
    int pos, left, off;
    int b, ready;        // ready: `r` holds request b
    TreeReq r;

    __device__ __forceinline__ TreeWalk(const TreeStart& st)
        : pos(st.pos), left(st.left), off(st.off), b(st.b), ready(1), r(st.r) {}

    __device__ __forceinline__ bool next(const TreeParams& p, int tile, TreePiece& it) {
        const int lane = threadIdx.x & 31;
        while (left > 0) {
            if (!ready) {
                r = tree_request(p, b, false);
                ready = 1;
            }
            const int w = (r.len + tile - 1) / tile + p.ucost;
            const int units = r.n > 0 ? (r.n + p.tokb - 1) / p.tokb * p.H_kv : 0;
            if (off >= units * w) {
                // the next request that has drafts: 32 looked at a round
                off = 0;
                ready = 0;
                for (++b; b < p.B; b += 32) {
                    const bool has = b + lane < p.B && tree_request(p, b + lane, false).n > 0;
                    const unsigned m = __ballot_sync(0xffffffffu, has);
                    if (m != 0) {
                        b += __ffs(m) - 1;
                        break;
                    }
                }
                if (b >= p.B) return false;   // not reached: the stretches end at W
                continue;
            }
            const int unit = off / w, x0 = off - unit * w;
            const int x1 = left < w - x0 ? x0 + left : w;
            it.end = pos - x0 + w;
            off += x1 - x0;
            pos += x1 - x0;
            left -= x1 - x0;
            // the unit's fixed cost stands before its tiles
            it.j0 = max(0, x0 - p.ucost);
            it.j1 = max(0, x1 - p.ucost);
            if (it.j0 >= it.j1) continue;
            it.nt = w - p.ucost;
            it.b = b;
            it.qb = unit / p.H_kv;
            it.h = unit - it.qb * p.H_kv;
            it.q_begin = r.q_begin;
            it.n = r.n;
            it.c = r.len - r.n;
            it.rows_tok = min(p.tokb, r.n - it.qb * p.tokb);
            it.kend = r.len;
            return true;
        }
        return false;
    }
};

// Workspace piece of a cut unit: its first piece in the second place of its CTA, every
// later one in the first place of its own.
__device__ __forceinline__ int tree_piece_slot(int cta, int j0) { return 2 * cta + (j0 == 0 ? 1 : 0); }

// The last CTA that holds a piece of the unit whose first piece `it` is.
__device__ __forceinline__ int tree_last(const TreeStart& st, const TreePiece& it, int cta) {
    int last = cta;
#pragma unroll 1
    for (int64_t next = (int64_t)st.share * (cta + 1); next < it.end; next += st.share) ++last;
    return last;
}

// Whether draft row i of a request sees its draft j.
__device__ __forceinline__ bool tree_bit(const TreeParams& p, int row, int j) {
    return (__ldg(p.mask + (int64_t)row * p.W + (j >> 5)) >> (j & 31)) & 1u;
}

}  // namespace

}  // namespace wf
