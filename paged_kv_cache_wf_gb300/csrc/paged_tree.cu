// paged_tree.cu -- attention of trees of drafted tokens over the paged cache: the
// CUDA-core kernel (fp32 pools, block sizes that are not multiples of 16), the kernel
// that joins the pieces of cut units, and the dispatch.
//
// Row i (draft i of request b, query head g of a group) sees the cached positions
// 0 .. c_b - 1 (ember, "The core idea": position p lives in block table[p / P] at
// p % P) and the drafts c_b + j that its mask names; o = softmax(scale q K^T) V over
// them, with the running maximum and sum of an online softmax in fp32 (exp2 domain).
#include <cfloat>
#include <cmath>

#include "paged_tree.cuh"

namespace wf {

namespace {

// ---------------------------------------------------------------------------
// CUDA cores
// ---------------------------------------------------------------------------
// A CTA takes 32 rows against 64 positions at a time: K and V rows are widened to fp32
// in shared memory (each element once), S = Q K^T is a 2 x 4 register tile a thread,
// O += P V a 2 x (D / 16) one, both fed by 16-byte shared-memory reads.  The FMA pipe is
// the bound: 2 * 32 * D FMAs a position and head against 2 * D elements read.
constexpr int kCcRows = 32;
constexpr int kCcTile = 64;
constexpr int kCcThreads = 256;

template <int D>
struct CcLayout {
    static constexpr int KS = D + 4;            // row stride of K in floats: 16 rows meet in two conflict-free reads
    static constexpr int SS = kCcTile + 4;      // row stride of S
    static constexpr int q = 0;
    static constexpr int k = q + kCcRows * D * 4;
    static constexpr int v = k + kCcTile * KS * 4;
    static constexpr int s = v + kCcTile * D * 4;
    static constexpr int vis = s + kCcRows * SS * 4;          // [rows][2] words: positions of the tile a row sees
    static constexpr int slot = vis + kCcRows * 8;            // [tile] int64 slot, -1: not there
    static constexpr int alpha = slot + kCcTile * 8;          // [rows]
    static constexpr int start = alpha + kCcRows * 4;
    static constexpr int scratch = start + (int)sizeof(TreeStart);
    static constexpr int total = scratch + 8 * (kCcThreads / 32);
    static_assert(slot % 8 == 0 && start % 16 == 0 && scratch % 8 == 0, "misaligned shared memory");
};

template <typename E, int D>
__device__ __forceinline__ void cc_load_row(float* dst, const char* pool, int64_t elem, int chunk) {
    const uint4 c = ld_global_stream(pool + elem * E::kBytes + chunk * 16);
    if constexpr (E::kBytes == 1) {
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = e4m3x2_to_float2(w[i]), b = e4m3x2_to_float2(w[i] >> 16);
            *reinterpret_cast<float4*>(dst + chunk * 16 + i * 4) = make_float4(a.x, a.y, b.x, b.y);
        }
    } else {
        float f[E::kPerChunk];
        widen_chunk<E>(c, f);
#pragma unroll
        for (int i = 0; i < E::kPerChunk; i += 4)
            *reinterpret_cast<float4*>(dst + chunk * E::kPerChunk + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    }
}

// E: pool elements, A: q and out elements.
template <typename E, typename A, int D>
__global__ void __launch_bounds__(kCcThreads, 2) paged_tree_kernel(const TreeParams p, const HeadScales sc) {
    using L = CcLayout<D>;
    extern __shared__ __align__(16) unsigned char smem[];
    float* sq = reinterpret_cast<float*>(smem + L::q);
    float* sk = reinterpret_cast<float*>(smem + L::k);
    float* sv = reinterpret_cast<float*>(smem + L::v);
    float* ss = reinterpret_cast<float*>(smem + L::s);
    uint32_t* svis = reinterpret_cast<uint32_t*>(smem + L::vis);
    int64_t* sslot = reinterpret_cast<int64_t*>(smem + L::slot);
    float* salpha = reinterpret_cast<float*>(smem + L::alpha);
    TreeStart* st = reinterpret_cast<TreeStart*>(smem + L::start);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tx = tid & 15, ty = tid >> 4;
    const int cta = blockIdx.x;
    constexpr int kChunks = D * E::kBytes / 16;     // 16-byte chunks of a K or V row
    constexpr int kDt = D / 16;                     // outputs of a thread in a row
    tree_begin(p, kCcTile, cta, gridDim.x, st, reinterpret_cast<int64_t*>(smem + L::scratch));
    int4 rec = make_int4(0, 0, 0, 0);
    TreeWalk walk(*st);
    TreePiece it;
    while (walk.next(p, kCcTile, it)) {
        const int i0 = it.qb * p.tokb;
        const int R = it.rows_tok * p.G;
        const float qscale = E::kBytes == 1 ? p.scale_log2 * sc.k[min(it.h, kMaxScaleHeads - 1)] : p.scale_log2;
        const float vscale = E::kBytes == 1 ? sc.v[min(it.h, kMaxScaleHeads - 1)] : 1.f;
        // row r: draft i0 + r / G, query head h G + r % G
        for (int x = tid; x < kCcRows * (D / A::kPerChunk); x += kCcThreads) {
            const int r = x / (D / A::kPerChunk), ch = x % (D / A::kPerChunk);
            float f[A::kPerChunk];
#pragma unroll
            for (int e = 0; e < A::kPerChunk; ++e) f[e] = 0.f;
            if (r < R) {
                const int64_t row = (int64_t)(it.q_begin + i0 + r / p.G) * p.H_q + it.h * p.G + r % p.G;
                widen_chunk<A>(__ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(p.q) +
                                                                    row * D * A::kBytes) + ch), f);
            }
#pragma unroll
            for (int e = 0; e < A::kPerChunk; ++e) sq[r * D + ch * A::kPerChunk + e] = f[e];
        }
        float o[2][kDt];
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int d = 0; d < kDt; ++d) o[a][d] = 0.f;
        // the softmax state of rows 4 * warp .. 4 * warp + 3, the same in all lanes
        float m_run[4], l_run[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            m_run[a] = -INFINITY;
            l_run[a] = 0.f;
        }
        const int32_t* trow = p.block_tables + (int64_t)it.b * p.M;
        for (int j = it.j0; j < it.j1; ++j) {
            const int k0 = j * kCcTile;
            __syncthreads();   // the last tile is consumed
            if (tid < kCcTile) {
                const int pos = k0 + tid;
                int64_t slot = -1;
                if (pos < it.kend) {
                    const int blk = __ldg(trow + pos / p.P);
                    if ((unsigned)blk < (unsigned)p.N)
                        slot = (int64_t)blk * p.P + pos % p.P;
                    else
                        report(p.dev_status, WF_DEV_BAD_BLOCK);
                }
                sslot[tid] = slot;
            }
            __syncthreads();
            bool wild = false;   // a draft's V row holds an infinity or NaN
            for (int x = tid; x < kCcTile * kChunks; x += kCcThreads) {
                const int r = x / kChunks, ch = x % kChunks;
                const int64_t slot = sslot[r];
                float* kd = sk + r * L::KS;
                float* vd = sv + r * D;
                if (slot >= 0) {
                    const int64_t elem = (slot * p.H_kv + it.h) * D;
                    cc_load_row<E, D>(kd, static_cast<const char*>(p.k_pool), elem, ch);
                    cc_load_row<E, D>(vd, static_cast<const char*>(p.v_pool), elem, ch);
                    if (k0 + r >= it.c) {
#pragma unroll
                        for (int e = 0; e < 16 / E::kBytes; ++e) wild |= !(fabsf(vd[ch * (16 / E::kBytes) + e]) < INFINITY);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16 / E::kBytes; ++e) {
                        kd[ch * (16 / E::kBytes) + e] = 0.f;
                        vd[ch * (16 / E::kBytes) + e] = 0.f;
                    }
                }
            }
            if (tid < 2 * kCcRows) {   // positions k0 + 32 * half .. of the tile that row r sees
                const int r = tid >> 1, half = tid & 1;
                uint32_t w = 0;
                if (r < R) {
                    const int row = it.q_begin + i0 + r / p.G;
                    for (int x = 0; x < 32; ++x) {
                        const int pos = k0 + half * 32 + x;
                        if (sslot[half * 32 + x] < 0) continue;
                        if (pos < it.c || tree_bit(p, row, pos - it.c)) w |= 1u << x;
                    }
                }
                svis[tid] = w;
            }
            wild = __syncthreads_or(wild) != 0;
            // ---- S = Q K^T: rows 2 ty + {0, 1}, positions tx + 16 {0 .. 3} ----
            float acc[2][4];
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[a][c] = 0.f;
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                float4 qa[2], kb[4];
#pragma unroll
                for (int a = 0; a < 2; ++a) qa[a] = *reinterpret_cast<const float4*>(sq + (2 * ty + a) * D + d);
#pragma unroll
                for (int c = 0; c < 4; ++c) kb[c] = *reinterpret_cast<const float4*>(sk + (tx + 16 * c) * L::KS + d);
#pragma unroll
                for (int a = 0; a < 2; ++a)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        acc[a][c] = fmaf(qa[a].x, kb[c].x, acc[a][c]);
                        acc[a][c] = fmaf(qa[a].y, kb[c].y, acc[a][c]);
                        acc[a][c] = fmaf(qa[a].z, kb[c].z, acc[a][c]);
                        acc[a][c] = fmaf(qa[a].w, kb[c].w, acc[a][c]);
                    }
            }
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int c = 0; c < 4; ++c) ss[(2 * ty + a) * L::SS + tx + 16 * c] = acc[a][c] * qscale;
            __syncthreads();
            // ---- online softmax: warp w has rows 4 w .. 4 w + 3, lane l positions l and l + 32 ----
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const int r = 4 * warp + a;
                const bool v0 = (svis[2 * r] >> lane) & 1u, v1 = (svis[2 * r + 1] >> lane) & 1u;
                const float s0 = v0 ? ss[r * L::SS + lane] : -INFINITY;
                const float s1 = v1 ? ss[r * L::SS + lane + 32] : -INFINITY;
                float mx = fmaxf(s0, s1);
#pragma unroll
                for (int w = 16; w >= 1; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
                const float mn = fmaxf(m_run[a], mx);
                const float mu = mn == -INFINITY ? 0.f : mn;
                const float al = m_run[a] == -INFINITY ? 0.f : exp2f(m_run[a] - mu);
                const float e0 = v0 ? exp2f(s0 - mu) : 0.f, e1 = v1 ? exp2f(s1 - mu) : 0.f;
                float sum = e0 + e1;
#pragma unroll
                for (int w = 16; w >= 1; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
                l_run[a] = l_run[a] * al + sum;
                m_run[a] = mn;
                ss[r * L::SS + lane] = e0;
                ss[r * L::SS + lane + 32] = e1;
                if (lane == 0) salpha[r] = al;
            }
            __syncthreads();
            // ---- O = O alpha + P V: rows 2 ty + {0, 1}, columns 4 (tx + 16 i) .. ----
            const float a0 = salpha[2 * ty], a1 = salpha[2 * ty + 1];
#pragma unroll
            for (int d = 0; d < kDt; ++d) {
                o[0][d] *= a0;
                o[1][d] *= a1;
            }
            if (!wild) {
#pragma unroll 2
                for (int x = 0; x < kCcTile; x += 4) {
                    const float4 p0 = *reinterpret_cast<const float4*>(ss + 2 * ty * L::SS + x);
                    const float4 p1 = *reinterpret_cast<const float4*>(ss + (2 * ty + 1) * L::SS + x);
                    const float w0[4] = {p0.x, p0.y, p0.z, p0.w}, w1[4] = {p1.x, p1.y, p1.z, p1.w};
#pragma unroll
                    for (int u = 0; u < 4; ++u)
#pragma unroll
                        for (int c = 0; c < kDt / 4; ++c) {
                            const float4 vv = *reinterpret_cast<const float4*>(sv + (x + u) * D + 4 * (tx + 16 * c));
                            const float vf[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                o[0][4 * c + e] = fmaf(w0[u], vf[e], o[0][4 * c + e]);
                                o[1][4 * c + e] = fmaf(w1[u], vf[e], o[1][4 * c + e]);
                            }
                        }
                }
            } else {   // 0 * NaN must not reach a row that does not see the draft
                for (int x = 0; x < kCcTile; ++x)
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        if (!((svis[2 * (2 * ty + a) + (x >> 5)] >> (x & 31)) & 1u)) continue;
                        const float w = ss[(2 * ty + a) * L::SS + x];
#pragma unroll
                        for (int c = 0; c < kDt / 4; ++c)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                o[a][4 * c + e] = fmaf(w, sv[x * D + 4 * (tx + 16 * c) + e], o[a][4 * c + e]);
                    }
            }
        }
        // ---- the rows, or this piece of them ----
        __syncthreads();
        if (lane < 4) salpha[4 * warp + lane] = lane == 0 ? l_run[0] : lane == 1 ? l_run[1] : lane == 2 ? l_run[2] : l_run[3];
        const bool whole = it.j0 == 0 && it.j1 == it.nt;
        const int piece = tree_piece_slot(cta, it.j0);
        if (!whole) {
            if (lane < 4) {
                const float m = lane == 0 ? m_run[0] : lane == 1 ? m_run[1] : lane == 2 ? m_run[2] : m_run[3];
                p.ws_ml[(int64_t)piece * p.rows + 4 * warp + lane] = make_float2(m, salpha[4 * warp + lane]);
            }
            if (it.j0 == 0) rec = tree_record(p, *st, it, cta);
        }
        __syncthreads();
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const int r = 2 * ty + a;
            if (r >= R) continue;
            const float l = salpha[r];
            const float f = whole ? (l == 0.f ? 0.f : vscale / l) : vscale;
            const int64_t row = (int64_t)(it.q_begin + i0 + r / p.G) * p.H_q + it.h * p.G + r % p.G;
#pragma unroll
            for (int c = 0; c < kDt / 4; ++c) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = l == 0.f ? 0.f : o[a][4 * c + e] * f;
                const int col = 4 * (tx + 16 * c);
                if (whole)
                    store_out<A, 4>(static_cast<char*>(p.out) + (row * D + col) * A::kBytes, y);
                else
                    store_out<F32, 4>(p.ws_o + ((int64_t)piece * p.rows + r) * D + col, y);
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
// order.  Pieces are read kChunk at a time, all loads before the first use.  Launched as
// a programmatic dependent of the kernel before it.
template <typename A, int D>
__global__ void __launch_bounds__(256) paged_tree_join_kernel(const TreeParams p) {
    constexpr int VPL = D / 32;
    constexpr int kChunk = 8;
    using Vec = typename std::conditional<VPL == 4, float4, float2>::type;
    const int lane = threadIdx.x & 31;
    const int r = blockIdx.y * 8 + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 rec = __ldcg(p.ws_rec + blockIdx.x);
    if (rec.w == 0) return;
    const int q_begin = __ldg(p.cu_q_lens + rec.x), n = __ldg(p.cu_q_lens + rec.x + 1) - q_begin;
    const int qb = rec.y / p.H_kv, h = rec.y - qb * p.H_kv;
    const int i0 = qb * p.tokb;
    if (r >= min(p.tokb, n - i0) * p.G) return;
    const int first = blockIdx.x, cnt = rec.z - first + 1;
    float M = -INFINITY, den = 0.f;
    float o[VPL];
#pragma unroll
    for (int e = 0; e < VPL; ++e) o[e] = 0.f;
    for (int u0 = 0; u0 < cnt; u0 += kChunk) {
        Vec x[kChunk];
        float2 ml[kChunk];
#pragma unroll
        for (int u = 0; u < kChunk; ++u) {
            ml[u] = make_float2(-INFINITY, 0.f);
            if (u0 + u < cnt) {
                const int64_t at = (int64_t)tree_piece_slot(first + u0 + u, u0 + u) * p.rows + r;
                ml[u] = __ldcg(p.ws_ml + at);
                x[u] = __ldcg(reinterpret_cast<const Vec*>(p.ws_o + at * D) + lane);
            }
        }
        float mn = M;
#pragma unroll
        for (int u = 0; u < kChunk; ++u) mn = fmaxf(mn, ml[u].x);
        // a piece (or all before it) without a maximum has a sum of 0, or of NaN, which has to stay
        const float a = M == -INFINITY ? 1.f : exp2f(M - mn);
        den *= a;
#pragma unroll
        for (int e = 0; e < VPL; ++e) o[e] *= a;
#pragma unroll
        for (int u = 0; u < kChunk; ++u) {
            if (u0 + u >= cnt || ml[u].y == 0.f) continue;
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
    }
#pragma unroll
    for (int e = 0; e < VPL; ++e) o[e] = den == 0.f ? 0.f : o[e] / den;
    const int64_t row = (int64_t)(q_begin + i0 + r / p.G) * p.H_q + h * p.G + r % p.G;
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
    const int q_begin = __ldg(p.cu_q_lens + rec.x), n = __ldg(p.cu_q_lens + rec.x + 1) - q_begin;
    const int qb = rec.y / p.H_kv, h = rec.y - qb * p.H_kv;
    const int i0 = qb * p.tokb;
    const int rows = min(p.tokb, n - i0) * p.G;
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
            const int64_t row = (int64_t)(q_begin + i0 + rk / p.G) * p.H_q + h * p.G + rk % p.G;
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

template <typename E, typename A, int D>
cudaError_t launch_cc(const TreeParams& p, const HeadScales& sc, int ctas, cudaStream_t stream) {
    auto kern = paged_tree_kernel<E, A, D>;
    const int smem = CcLayout<D>::total;
    cudaError_t err = allow_dynamic_smem((const void*)kern, smem);
    if (err != cudaSuccess) return err;
    kern<<<ctas, kCcThreads, smem, stream>>>(p, sc);
    err = cudaGetLastError();
    if (err != cudaSuccess || ctas == 1) return err;
    return launch_join<A, D>(p, ctas, stream);
}

}  // namespace

static bool tree_shape(const wf_pool_desc& pool, int32_t num_q_heads, int32_t max_q_len, TreeShape* s) {
    if (num_q_heads % pool.num_kv_heads != 0) return false;
    const int G = num_q_heads / pool.num_kv_heads;
    if (G < 1 || G > 8) return false;
    *s = tree_tc_supported(pool, num_q_heads) ? tree_tc_shape(G, max_q_len, pool.dtype == WF_DTYPE_FP8_E4M3)
                                              : TreeShape{kCcRows, kCcRows / G, kCcTile, 2, 1};
    return true;
}

// CTAs the launch may use: no more than there can be tiles.
static int64_t tree_ctas(const TreeShape& s, int32_t B, int32_t H_kv, int32_t max_q_len, int32_t max_seq_len) {
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
    const size_t bytes = (size_t)(256 + ctas * (int64_t)sizeof(int4) + rows * 8 + rows * pool.head_dim * 4);
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
    p.scale_log2 = a.scale * 1.4426950408889634f;
    // a masked score is -inf before it is scaled: a scale of 0 (equal weights) stands as the
    // smallest normal number, which leaves every finite score a weight of 2^0
    if (fabsf(p.scale_log2) < FLT_MIN) p.scale_log2 = copysignf(FLT_MIN, p.scale_log2);
    const bool d128 = pool.head_dim == 128;
    if (tree_tc_supported(pool, a.num_q_heads)) {
        void* prep = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(p.ws_rec + cap) + 127) & ~(uintptr_t)127);
        const cudaError_t e = launch_tree_tc(p, pool, prep, ctas, stream);
        if (e != cudaSuccess || ctas == 1) return e;
        return d128 ? launch_join<BF16, 128>(p, ctas, stream) : launch_join<BF16, 64>(p, ctas, stream);
    }
    const HeadScales sc = head_scales(pool);
    switch (pool.dtype) {
        case WF_DTYPE_F32:
            return d128 ? launch_cc<F32, F32, 128>(p, sc, ctas, stream) : launch_cc<F32, F32, 64>(p, sc, ctas, stream);
        case WF_DTYPE_BF16:
            return d128 ? launch_cc<BF16, BF16, 128>(p, sc, ctas, stream)
                        : launch_cc<BF16, BF16, 64>(p, sc, ctas, stream);
        default:
            return d128 ? launch_cc<FP8, BF16, 128>(p, sc, ctas, stream)
                        : launch_cc<FP8, BF16, 64>(p, sc, ctas, stream);
    }
}

}  // namespace wf
