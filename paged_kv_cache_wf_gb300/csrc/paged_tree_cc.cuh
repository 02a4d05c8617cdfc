// paged_tree_cc.cuh -- attention of trees of drafted tokens, and scored attention, over the paged
// cache on the CUDA cores (fp32 pools, block sizes that are not multiples of 16), and the kernels
// that join the pieces of cut units, the tensor cores' too.
//
// Row i (draft i of request b, query head g of a group) sees the cached positions
// 0 .. c_b - 1 (ember, "The core idea": position p lives in block table[p / P] at
// p % P) and the drafts c_b + j that its mask names; o = softmax(scale q K^T) V over
// them, with the running maximum and sum of an online softmax in fp32 (exp2 domain).
// A scored call's row sees a range of positions, and its scores are capped and biased first.
#pragma once

#include <type_traits>

#include "paged_tree.cuh"

namespace wf {

namespace {

// ---------------------------------------------------------------------------
// CUDA cores
// ---------------------------------------------------------------------------
// A CTA takes 8 RPW rows against 64 positions at a time, a warp RPW of the rows, so that S,
// the softmax and P V of a row never leave its warp: lane l has positions l and l + 32 of S and
// columns l D / 32 .. of O.  K and V rows of the next tile are on their way in registers
// meanwhile; they are widened to fp32 into shared memory once for all warps.  With 4 rows a
// warp it runs at half the FMA pipe's rate (8 requests of up to 61 drafts, 128-wide fp32: 181 us,
// 92 of FMAs); packed FMAs (177 us) and tiles of 2 x 4 a lane, which read half as much shared
// memory (184 us), leave it there.  With 1, for
// chains and small trees, it is the start and the join: 8 requests of up to 7 drafts of 64-wide
// fp32 heads 13.6 us, 2.0 at the copy peak; blocks of 7, 8 requests of up to 16 drafts of
// 128-wide bf16 heads 63 us.
constexpr int kCcTile = 64;
constexpr int kCcWarps = 8;
constexpr int kCcThreads = 32 * kCcWarps;

template <int D, int RPW>
struct CcLayout {
    static constexpr int rows = kCcWarps * RPW;
    static constexpr int KS = D + 4;            // row stride of K in floats: eight rows meet in one conflict-free read
    static constexpr int q = 0;
    static constexpr int k = q + rows * D * 4;
    static constexpr int v = k + kCcTile * KS * 4;
    static constexpr int p = v + kCcTile * D * 4;
    static constexpr int slot = p + rows * kCcTile * 4;       // 3 x [tile] int64 slot, -1: not there
    static constexpr int start = slot + 3 * kCcTile * 8;
    static constexpr int scratch = start + (int)sizeof(TreeStart);
    static constexpr int total = scratch + 8 * kCcWarps;
    static_assert(slot % 8 == 0 && start % 16 == 0 && scratch % 8 == 0, "misaligned shared memory");
};

// 16 bytes of a pool row in fp32.
template <typename E>
__device__ __forceinline__ void cc_widen(const uint4& c, float (&f)[16 / E::kBytes]) {
    if constexpr (E::kBytes == 1) {
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = e4m3x2_to_float2(w[i]), b = e4m3x2_to_float2(w[i] >> 16);
            f[4 * i] = a.x;
            f[4 * i + 1] = a.y;
            f[4 * i + 2] = b.x;
            f[4 * i + 3] = b.y;
        }
    } else {
        widen_chunk<E>(c, f);
    }
}

template <int VPL>
__device__ __forceinline__ void cc_row(float (&f)[VPL], const float* from) {
    if constexpr (VPL == 4) {
        const float4 x = *reinterpret_cast<const float4*>(from);
        f[0] = x.x;
        f[1] = x.y;
        f[2] = x.z;
        f[3] = x.w;
    } else {
        const float2 x = *reinterpret_cast<const float2*>(from);
        f[0] = x.x;
        f[1] = x.y;
    }
}

// CTAs an SM: as many as the registers that the next tile and the rows take leave room for.
constexpr int cc_ctas_per_sm(int bytes, int D, int rpw) { return bytes == 4 && D == 128 && rpw == 4 ? 1 : 2; }
static_assert(cc_ctas_per_sm(2, 64, 1) * kTreeMaxSms <= kTreeRecs, "records for every CTA");

// Rows of a warp: the fewest that hold all rows of a request's drafts under a KV head, 4 at most
// (64-wide fp32 heads: 8 rows 13.6 us with 1, 14.9 with 2; 14 rows 53 us with 2, 73 with 4).
// max_q_len decides for the whole batch: 8 chains of up to 7 drafts take 14.8 us with a max_q_len of
// 16, 18.4 with 64.
constexpr int cc_rows_per_warp(int64_t rows) { return rows <= kCcWarps ? 1 : rows <= 2 * kCcWarps ? 2 : 4; }

// E: pool elements, A: q and out elements.
template <typename V, typename E, typename A, int D, int RPW>
__global__ void __launch_bounds__(kCcThreads, cc_ctas_per_sm(E::kBytes, D, RPW))
    paged_tree_kernel(const typename V::Params p, const HeadScales sc) {
    using L = CcLayout<D, RPW>;
    extern __shared__ __align__(16) unsigned char smem[];
    float* sq = reinterpret_cast<float*>(smem + L::q);
    float* sk = reinterpret_cast<float*>(smem + L::k);
    float* sv = reinterpret_cast<float*>(smem + L::v);
    float* sp = reinterpret_cast<float*>(smem + L::p);
    int64_t* sslot = reinterpret_cast<int64_t*>(smem + L::slot);
    using Start = typename std::conditional<V::kScored, ScoredStart, TreeStart>::type;
    Start* st = reinterpret_cast<Start*>(smem + L::start);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cta = blockIdx.x;
    constexpr int VPL = D / 32;                     // outputs of a lane in a row
    constexpr int kPC = 16 / E::kBytes;             // elements of a 16-byte chunk
    constexpr int kChunks = D / kPC;                // chunks of a K or V row
    constexpr int kStep = kCcThreads / kChunks;     // rows that the threads load at once
    constexpr int kPer = kCcTile / kStep;           // chunks of a thread in a tile, of K and of V
    const int lrow = tid / kChunks, lch = tid % kChunks;
    if constexpr (V::kScored)
        scored_begin(p, cta, gridDim.x, st);
    else
        tree_begin(p, kCcTile, cta, gridDim.x, st, reinterpret_cast<int64_t*>(smem + L::scratch));
    int4 rec = make_int4(0, 0, 0, 0);
    typename std::conditional<V::kScored, ScoredWalk<false>, TreeWalk>::type walk(*st);
    typename std::conditional<V::kScored, ScoredPiece, TreePiece>::type it;
#pragma unroll 1
    while (walk.next(p, kCcTile, it)) {
        // first row of q, rows, first position of tile 0, positions that any row and that every row sees
        int q_row, R, at0 = 0, lo = 0, hi, full0 = 0, full1, b;
        if constexpr (V::kScored) {
            q_row = it.k.q_row;
            R = it.k.rows_tok * p.G;
            at0 = it.k.tile0 * kCcTile;
            lo = it.k.lo;
            hi = it.k.hi;
            full0 = it.k.full_lo;
            full1 = it.k.full_hi;
            b = it.k.b;
        } else {
            q_row = it.q_begin + it.qb * p.tokb;
            R = it.rows_tok * p.G;
            hi = it.kend;
            full1 = it.c;
            b = it.b;
        }
        float factor = p.scale_log2;
        constexpr bool kCap = V::kCap, kBias = V::kBias;
        if constexpr (kCap) factor = p.cap_in;
        const float qscale = E::kBytes == 1 ? factor * sc.k[min(it.h, kMaxScaleHeads - 1)] : factor;
        const float vscale = E::kBytes == 1 ? sc.v[min(it.h, kMaxScaleHeads - 1)] : 1.f;
        const int32_t* trow = p.block_tables + (int64_t)b * p.M;
        const auto look_up = [&](int j) {   // slots of tile j, threads 0 .. 63
            const int pos = at0 + j * kCcTile + tid;
            int64_t slot = -1;
            if (pos < hi && pos >= lo) {
                const int blk = __ldg(trow + pos / p.P);
                if ((unsigned)blk < (unsigned)p.N)
                    slot = (int64_t)blk * p.P + pos % p.P;
                else
                    report(p.dev_status, WF_DEV_BAD_BLOCK);
            }
            sslot[j % 3 * kCcTile + tid] = slot;
        };
        uint4 kr[kPer], vr[kPer];
        const auto load = [&](int j) {      // this thread's chunks of tile j
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int64_t slot = sslot[j % 3 * kCcTile + lrow + i * kStep];
                kr[i] = vr[i] = make_uint4(0, 0, 0, 0);
                if (slot >= 0) {
                    const int64_t at = ((slot * p.H_kv + it.h) * D + lch * kPC) * E::kBytes;
                    kr[i] = ld_global_stream(static_cast<const char*>(p.k_pool) + at);
                    vr[i] = ld_global_stream(static_cast<const char*>(p.v_pool) + at);
                }
            }
        };
        __syncthreads();   // the last piece's slots and q rows are read
        if (tid < kCcTile) {
            look_up(it.j0);
            if (it.j0 + 1 < it.j1) look_up(it.j0 + 1);
        }
        // row r: draft r / G of the block, query head h G + r % G
        for (int x = tid; x < L::rows * (D / A::kPerChunk); x += kCcThreads) {
            const int r = x / (D / A::kPerChunk), ch = x % (D / A::kPerChunk);
            float f[A::kPerChunk] = {};
            if (r < R) {
                const int64_t row = (int64_t)(q_row + r / p.G) * p.H_q + it.h * p.G + r % p.G;
                widen_chunk<A>(__ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(p.q) +
                                                                    row * D * A::kBytes) + ch), f);
            }
#pragma unroll
            for (int e = 0; e < A::kPerChunk; ++e) sq[r * D + ch * A::kPerChunk + e] = f[e];
        }
        __syncthreads();
        load(it.j0);
        // rows warp + 8 a; the maximum is the same in all lanes, the sum a lane's own positions'
        float o[RPW][VPL] = {}, m_run[RPW], l_run[RPW] = {};
#pragma unroll
        for (int a = 0; a < RPW; ++a) m_run[a] = -INFINITY;
        int2 sees_of[RPW];                   // scored: what a row sees, and its bias, slope |p - ref|
        float slope[RPW];
        int ref[RPW];
        if constexpr (V::kScored) {
#pragma unroll
            for (int a = 0; a < RPW; ++a) {
                const int r = warp + kCcWarps * a, at = it.k.at + r / p.G;
                sees_of[a] = r < R ? scored_range(p, q_row + r / p.G, at, it.k.len) : make_int2(0, 0);
                slope[a] = kBias && r < R ? -1.4426950408889634f * __ldg(p.slopes + it.h * p.G + r % p.G) : 0.f;
                ref[a] = min(at, sees_of[a].y - 1);
            }
        }
#pragma unroll 1
        for (int j = it.j0; j < it.j1; ++j) {
            const int k0 = at0 + j * kCcTile;
            if (j != it.j0) __syncthreads();   // the last tile is consumed
            bool wild = false;   // a draft's V row holds an infinity or NaN
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int r = lrow + i * kStep;
                float f[kPC];
                cc_widen<E>(kr[i], f);
#pragma unroll
                for (int e = 0; e < kPC; e += 4)
                    *reinterpret_cast<float4*>(sk + r * L::KS + lch * kPC + e) =
                        make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
                cc_widen<E>(vr[i], f);
#pragma unroll
                for (int e = 0; e < kPC; e += 4)
                    *reinterpret_cast<float4*>(sv + r * D + lch * kPC + e) =
                        make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
                if (k0 + r >= full1 || k0 + r < full0) {
#pragma unroll
                    for (int e = 0; e < kPC; ++e) wild |= !(fabsf(f[e]) < INFINITY);
                }
            }
            wild = __syncthreads_or(wild) != 0;
            if (j + 1 < it.j1) load(j + 1);
            if (j + 2 < it.j1 && tid < kCcTile) look_up(j + 2);
            if (warp < R) {
                // ---- S = Q K^T ----
                float s[RPW][2] = {};
#pragma unroll 4
                for (int d = 0; d < D; d += 4) {
                    const float4 x = *reinterpret_cast<const float4*>(sk + lane * L::KS + d);
                    const float4 y = *reinterpret_cast<const float4*>(sk + (lane + 32) * L::KS + d);
#pragma unroll
                    for (int a = 0; a < RPW; ++a) {
                        const float4 q = *reinterpret_cast<const float4*>(sq + (warp + kCcWarps * a) * D + d);
                        s[a][0] = fmaf(q.x, x.x, s[a][0]);
                        s[a][1] = fmaf(q.x, y.x, s[a][1]);
                        s[a][0] = fmaf(q.y, x.y, s[a][0]);
                        s[a][1] = fmaf(q.y, y.y, s[a][1]);
                        s[a][0] = fmaf(q.z, x.z, s[a][0]);
                        s[a][1] = fmaf(q.z, y.z, s[a][1]);
                        s[a][0] = fmaf(q.w, x.w, s[a][0]);
                        s[a][1] = fmaf(q.w, y.w, s[a][1]);
                    }
                }
                // ---- online softmax ----
                uint32_t sees[RPW][2];
#pragma unroll
                for (int a = 0; a < RPW; ++a) {
                    const int r = warp + kCcWarps * a;
                    float mx = -INFINITY;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int pos = k0 + lane + 32 * u;
                        bool there = r < R && sslot[j % 3 * kCcTile + lane + 32 * u] >= 0;
                        if constexpr (V::kScored)
                            there = there && pos >= sees_of[a].x && pos < sees_of[a].y;
                        else
                            there = there && (pos < it.c || tree_bit(p, q_row + r / p.G, pos - it.c));
                        sees[a][u] = __ballot_sync(0xffffffffu, there);
                        float y = s[a][u] * qscale;
                        if constexpr (V::kScored) {
                            // (here the cap is tanhf's, whose error is a few last bits)
                            if constexpr (kCap) y = p.cap_out * tanhf(y);
                            if constexpr (kBias) y = fmaf(slope[a], fabsf((float)(pos - ref[a])), y);
                        }
                        s[a][u] = there ? y : -INFINITY;
                        mx = fmaxf(mx, s[a][u]);
                    }
#pragma unroll
                    for (int w = 16; w >= 1; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
                    const float mn = fmaxf(m_run[a], mx);
                    const float mu = mn == -INFINITY ? 0.f : mn;
                    const float al = m_run[a] == -INFINITY ? 0.f : exp2f(m_run[a] - mu);
                    l_run[a] *= al;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float e = (sees[a][u] >> lane) & 1u ? exp2f(s[a][u] - mu) : 0.f;
                        l_run[a] += e;
                        sp[r * kCcTile + lane + 32 * u] = e;
                    }
#pragma unroll
                    for (int d = 0; d < VPL; ++d) o[a][d] *= al;
                    m_run[a] = mn;
                }
                __syncwarp();
                // ---- O = O alpha + P V ----
                if (!wild) {
#pragma unroll 4
                    for (int x = 0; x < kCcTile; x += 4) {
                        float4 w[RPW];
#pragma unroll
                        for (int a = 0; a < RPW; ++a)
                            w[a] = *reinterpret_cast<const float4*>(sp + (warp + kCcWarps * a) * kCcTile + x);
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            float vf[VPL];
                            cc_row<VPL>(vf, sv + (x + u) * D + lane * VPL);
#pragma unroll
                            for (int a = 0; a < RPW; ++a) {
                                const float wu = u == 0 ? w[a].x : u == 1 ? w[a].y : u == 2 ? w[a].z : w[a].w;
#pragma unroll
                                for (int e = 0; e < VPL; ++e) o[a][e] = fmaf(wu, vf[e], o[a][e]);
                            }
                        }
                    }
                } else {   // 0 * NaN must not reach a row that does not see the draft
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll 1
                        for (int x = 0; x < 32; ++x)
#pragma unroll
                            for (int a = 0; a < RPW; ++a) {
                                if (!((sees[a][u] >> x) & 1u)) continue;
                                const float w = sp[(warp + kCcWarps * a) * kCcTile + 32 * u + x];
#pragma unroll
                                for (int e = 0; e < VPL; ++e)
                                    o[a][e] = fmaf(w, sv[(32 * u + x) * D + lane * VPL + e], o[a][e]);
                            }
                }
            }
        }
        // ---- the rows, or this piece of them ----
        const bool whole = it.j0 == 0 && it.j1 == it.nt;
        const int piece = tree_piece_slot(cta, it.j0);
        if (!whole && it.j0 == 0) rec = make_int4(q_row, it.h, tree_last(*st, it, cta), R);
#pragma unroll
        for (int a = 0; a < RPW; ++a) {
            const int r = warp + kCcWarps * a;
            if (r >= R) continue;
            float l = l_run[a];
#pragma unroll
            for (int w = 16; w >= 1; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
            const float f = whole ? (l == 0.f ? 0.f : vscale / l) : vscale;
#pragma unroll
            for (int e = 0; e < VPL; ++e) o[a][e] = l == 0.f ? 0.f : o[a][e] * f;
            if (whole) {
                const int64_t row = (int64_t)(q_row + r / p.G) * p.H_q + it.h * p.G + r % p.G;
                store_out<A, VPL>(static_cast<char*>(p.out) + (row * D + lane * VPL) * A::kBytes, o[a]);
            } else {
                const int64_t row = (int64_t)piece * p.rows + r;
                store_out<F32, VPL>(p.ws_o + row * D + lane * VPL, o[a]);
                if (lane == 0) p.ws_ml[row] = make_float2(m_run[a], l);
            }
        }
    }
    if (tid == 0) p.ws_rec[cta] = rec;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---------------------------------------------------------------------------
// joining the pieces of cut units
// ---------------------------------------------------------------------------
// CTA (k, y): the unit cut at the end of CTA k's stretch, rows 8 y .. 8 y + 7, a warp a
// row: o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i over its pieces i in position
// order.  Latency is all of it, so the first two pieces, which every cut unit has and whose
// places do not depend on the record, are read beside it, and the others kChunk at a time.
// Launched as a programmatic dependent of the kernel before it.
template <typename A, int D>
__global__ void __launch_bounds__(256) paged_tree_join_kernel(const TreeParams p) {
    constexpr int VPL = D / 32;
    constexpr int kChunk = 8;
    using Vec = typename std::conditional<VPL == 4, float4, float2>::type;
    const int lane = threadIdx.x & 31;
    const int r = blockIdx.y * 8 + (threadIdx.x >> 5);   // below p.rows, a multiple of 8
    const int first = blockIdx.x;
    Vec x[kChunk];
    float2 ml[kChunk];
    const auto load = [&](int u, int cta, int i) {   // piece i of the unit, in `cta`
        const int64_t at = (int64_t)tree_piece_slot(cta, i) * p.rows + r;
        ml[u] = __ldcg(p.ws_ml + at);
        x[u] = __ldcg(reinterpret_cast<const Vec*>(p.ws_o + at * D) + lane);
    };
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 rec = __ldcg(p.ws_rec + first);
    load(0, first, 0);
    load(1, min(first + 1, (int)gridDim.x - 1), 1);
    if (r >= rec.w) return;
    const int cnt = rec.z - first + 1;
    float M = -INFINITY, den = 0.f;
    float o[VPL] = {};
#pragma unroll 1
    for (int u0 = 0; u0 < cnt;) {
        const int take = u0 == 0 ? 2 : min(kChunk, cnt - u0);
        if (u0 > 0) {
#pragma unroll
            for (int u = 0; u < kChunk; ++u)
                if (u < take) load(u, first + u0 + u, u0 + u);
        }
        float mn = M;
#pragma unroll
        for (int u = 0; u < kChunk; ++u)
            if (u < take) mn = fmaxf(mn, ml[u].x);
        // a piece (or all before it) without a maximum has a sum of 0, or of NaN, which has to stay
        const float a = M == -INFINITY ? 1.f : exp2f(M - mn);
        den *= a;
#pragma unroll
        for (int e = 0; e < VPL; ++e) o[e] *= a;
#pragma unroll
        for (int u = 0; u < kChunk; ++u) {
            if (u >= take || ml[u].y == 0.f) continue;
            const float w = ml[u].x == -INFINITY ? 1.f : exp2f(ml[u].x - mn);
            den += w * ml[u].y;
            o[0] += w * x[u].x;
            o[1] += w * x[u].y;
            if constexpr (VPL == 4) {
                o[2] += w * x[u].z;
                o[3] += w * x[u].w;
            }
        }
        M = mn;
        u0 += take;
    }
#pragma unroll
    for (int e = 0; e < VPL; ++e) o[e] = den == 0.f ? 0.f : o[e] / den;
    const int64_t row = (int64_t)(rec.x + r / p.G) * p.H_q + rec.y * p.G + r % p.G;
    store_out<A, VPL>(static_cast<char*>(p.out) + (row * D + lane * VPL) * A::kBytes, o);
}

// The same for row blocks of many rows, in one wave: a warp takes every 8 gridDim.y-th row,
// kManyRows at once and two pieces of each at a time (nearly all units of a large batch
// have two).  Of the kernel above, 4864 CTAs (152 units of 256 rows) are four waves of three
// dependent loads each: 281 us for the whole call against 275 with this one.  Its code is longer
// and, cold at every call, costs more than it saves on smaller blocks: 152 units of 128 rows
// take 35.4 us with it and 34.7 without.
constexpr int kManyRows = 2, kManyCtasPerSm = 4;

template <typename A, int D>
__global__ void __launch_bounds__(256, kManyCtasPerSm) paged_tree_join_many_kernel(const TreeParams p) {
    constexpr int VPL = D / 32;
    using Vec = typename std::conditional<VPL == 4, float4, float2>::type;
    const int lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 rec = __ldcg(p.ws_rec + blockIdx.x);
    if (rec.w == 0) return;
    const int rows = rec.w;
    const int first = blockIdx.x, cnt = rec.z - first + 1, step = 8 * gridDim.y;
#pragma unroll 1
    for (int r = blockIdx.y * 8 + (threadIdx.x >> 5); r < rows; r += kManyRows * step) {
        float M[kManyRows], den[kManyRows] = {}, o[kManyRows][VPL] = {};
#pragma unroll
        for (int k = 0; k < kManyRows; ++k) M[k] = -INFINITY;
#pragma unroll 1
        for (int u0 = 0; u0 < cnt; u0 += 2) {
            Vec x[kManyRows][2];
            float2 ml[kManyRows][2];
#pragma unroll
            for (int k = 0; k < kManyRows; ++k)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    // a row or piece past the last reads the last one
                    const int i = min(u0 + u, cnt - 1);
                    const int64_t at = (int64_t)tree_piece_slot(first + i, i) * p.rows + min(r + k * step, rows - 1);
                    ml[k][u] = __ldcg(p.ws_ml + at);
                    x[k][u] = __ldcg(reinterpret_cast<const Vec*>(p.ws_o + at * D) + lane);
                }
#pragma unroll
            for (int k = 0; k < kManyRows; ++k) {
                if (u0 + 1 == cnt) ml[k][1] = make_float2(-INFINITY, 0.f);
                const float mn = fmaxf(M[k], fmaxf(ml[k][0].x, ml[k][1].x));
                // as above: without a maximum a sum is 0, or NaN, which has to stay
                const float a = M[k] == -INFINITY ? 1.f : exp2f(M[k] - mn);
                den[k] *= a;
#pragma unroll
                for (int e = 0; e < VPL; ++e) o[k][e] *= a;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (ml[k][u].y == 0.f) continue;
                    const float w = ml[k][u].x == -INFINITY ? 1.f : exp2f(ml[k][u].x - mn);
                    den[k] += w * ml[k][u].y;
                    o[k][0] += w * x[k][u].x;
                    o[k][1] += w * x[k][u].y;
                    if constexpr (VPL == 4) {
                        o[k][2] += w * x[k][u].z;
                        o[k][3] += w * x[k][u].w;
                    }
                }
                M[k] = mn;
            }
        }
#pragma unroll
        for (int k = 0; k < kManyRows; ++k) {
            const int rk = r + k * step;
            if (rk >= rows) break;
#pragma unroll
            for (int e = 0; e < VPL; ++e) o[k][e] = den[k] == 0.f ? 0.f : o[k][e] / den[k];
            const int64_t row = (int64_t)(rec.x + rk / p.G) * p.H_q + rec.y * p.G + rk % p.G;
            store_out<A, VPL>(static_cast<char*>(p.out) + (row * D + lane * VPL) * A::kBytes, o[k]);
        }
    }
}

template <typename A, int D>
cudaError_t launch_join(const TreeParams& p, int ctas, cudaStream_t stream) {
    // rows a row block can have: all of them, or those of max_q_len drafts
    const int y = ((p.max_q_len < p.tokb ? p.max_q_len : p.tokb) * p.G + 7) / 8;
    const int64_t all = (int64_t)p.B * p.H_kv * ((p.max_q_len + p.tokb - 1) / p.tokb);   // units at most
    const bool many = y * (all < ctas ? all : ctas) > 16 * (int64_t)num_sms();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, many ? kManyCtasPerSm * num_sms() / ctas : y);   // `ctas` is at most two an SM
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return many ? cudaLaunchKernelEx(&cfg, paged_tree_join_many_kernel<A, D>, p)
                : cudaLaunchKernelEx(&cfg, paged_tree_join_kernel<A, D>, p);
}

template <typename V, typename E, typename A, int D, int RPW>
cudaError_t launch_cc_rows(const typename V::Params& p, const HeadScales& sc, int ctas, cudaStream_t stream) {
    auto kern = paged_tree_kernel<V, E, A, D, RPW>;
    const int smem = CcLayout<D, RPW>::total;
    cudaError_t err = allow_dynamic_smem((const void*)kern, smem);
    if (err != cudaSuccess) return err;
    kern<<<ctas, kCcThreads, smem, stream>>>(p, sc);
    err = cudaGetLastError();
    if (err != cudaSuccess || ctas == 1) return err;
    return launch_join<A, D>(p, ctas, stream);
}

template <typename V, typename E, typename A, int D>
cudaError_t launch_cc(const typename V::Params& p, const HeadScales& sc, int ctas, cudaStream_t stream) {
    switch (p.rows / kCcWarps) {
        case 1: return launch_cc_rows<V, E, A, D, 1>(p, sc, ctas, stream);
        case 2: return launch_cc_rows<V, E, A, D, 2>(p, sc, ctas, stream);
        default: return launch_cc_rows<V, E, A, D, 4>(p, sc, ctas, stream);
    }
}

template <typename V>
cudaError_t launch_cc_pool(const typename V::Params& p, const wf_pool_desc& pool, int ctas, cudaStream_t stream) {
    const bool d128 = pool.head_dim == 128;
    const HeadScales sc = head_scales(pool);
    switch (pool.dtype) {
        case WF_DTYPE_F32:
            return d128 ? launch_cc<V, F32, F32, 128>(p, sc, ctas, stream) : launch_cc<V, F32, F32, 64>(p, sc, ctas, stream);
        case WF_DTYPE_BF16:
            return d128 ? launch_cc<V, BF16, BF16, 128>(p, sc, ctas, stream)
                        : launch_cc<V, BF16, BF16, 64>(p, sc, ctas, stream);
        default:
            return d128 ? launch_cc<V, FP8, BF16, 128>(p, sc, ctas, stream)
                        : launch_cc<V, FP8, BF16, 64>(p, sc, ctas, stream);
    }
}

}  // namespace

}  // namespace wf
