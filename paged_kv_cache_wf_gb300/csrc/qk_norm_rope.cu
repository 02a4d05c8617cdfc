// qk_norm_rope.cu -- per-head RMS norm and position rotation of this step's q and k,
// and the scatter of the new K and V rows into the block pool, in one pass.
//
// tiny-vllm-py, "KV Cache": the cache holds RoPE-rotated K and plain V; weft, "Cache
// layouts": write = scatter via slot_mapping.  Per head row x of D elements:
//   y_e  = x_e * w_e / sqrt(mean(x^2) + eps)                     (rows with a weight)
//   z_a  = y_a cos_i - y_b sin_i,  z_b = y_b cos_i + y_a sin_i   (pairs a, b below
//                                                                 rotary_dim)
// q rows go to q_out, k rows to the pool, v rows to the pool as they are; fp8 pools
// store e4m3(value * (1 / scale)).
//
// HBM-bound: every byte of q, k, v is read once and every result written once; doing
// it in one pass saves the second read and write of q and k that separate norm,
// rotation and scatter passes make.  What has to be watched is the instruction count:
// with one 16-byte chunk a lane, pairs exchanged by shuffle, 8193 tokens of Llama-3-8B
// heads into fp8 pools, whose bytes take 28 us, took 41 us (51 us before the rows of a
// warp were of one kind).  So a lane has two chunks of a head row, both halves of its
// pairs, and no element passes from lane to lane; a warp's rows are of one kind (each
// kind's rows are padded to whole warps), which keeps the choice of q, k or v a branch
// of the warp; arithmetic is on pairs (two fp32 operations an instruction); an instance
// without weights has no norm in it.  The sum of squares is a shuffle reduction over the
// row's lanes.  A lane reads its cos and sin once for IT rows.
// With norm weights the same 8193 tokens take 33.5 us (fp8 pools; without 30.5) and 34.5 us (bf16
// pools, whose bytes take 30.3).  Rotation widths that are no multiple of 16 read each pair's other
// half, cos and sin element by element: 75.7 us at a width of 120 for the 30.5.
#include "wf_internal.h"

namespace wf {

namespace {

struct RopeParams {
    RopeArgs a;
    int64_t num_slots;
    int H_kv;
    uint32_t* dev_status;
};

struct InvScales {
    float k[kMaxScaleHeads];
    float v[kMaxScaleHeads];
};

// One element of a row, widened.
template <typename E>
__device__ __forceinline__ float widen_one(const void* row, int e);
template <>
__device__ __forceinline__ float widen_one<F32>(const void* row, int e) {
    return __ldg(static_cast<const float*>(row) + e);
}
template <>
__device__ __forceinline__ float widen_one<BF16>(const void* row, int e) {
    return __uint_as_float((uint32_t)__ldg(static_cast<const unsigned short*>(row) + e) << 16);
}

// A 16-byte chunk as pairs of floats, and back.
template <typename E>
__device__ __forceinline__ void to_pairs(const uint4& c, float2* f);
template <>
__device__ __forceinline__ void to_pairs<F32>(const uint4& c, float2* f) {
    f[0] = make_float2(__uint_as_float(c.x), __uint_as_float(c.y));
    f[1] = make_float2(__uint_as_float(c.z), __uint_as_float(c.w));
}
template <>
__device__ __forceinline__ void to_pairs<BF16>(const uint4& c, float2* f) {
    f[0] = bf16x2_to_float2(c.x);
    f[1] = bf16x2_to_float2(c.y);
    f[2] = bf16x2_to_float2(c.z);
    f[3] = bf16x2_to_float2(c.w);
}
template <typename E>
__device__ __forceinline__ uint4 from_pairs(const float2* f);
template <>
__device__ __forceinline__ uint4 from_pairs<F32>(const float2* f) {
    return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                      __float_as_uint(f[1].y));
}
template <>
__device__ __forceinline__ uint4 from_pairs<BF16>(const float2* f) {
    return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                      pack_bf16x2(f[3].x, f[3].y));
}

// Four values -> their e4m3 codes.
__device__ __forceinline__ uint32_t codes4(const float2& a, const float2& b, const float2& inv) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(__fmul2_rn(a, inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(__fmul2_rn(b, inv), __NV_SATFINITE, __NV_E4M3);
    return (lo & 0xffffu) | (hi << 16);
}

// A chunk's codes.
template <int NP>
__device__ __forceinline__ void store_codes(char* out, const float2* y, float inv) {
    const float2 f = make_float2(inv, inv);
    static_assert(NP == 4 || NP == 2, "a chunk is 8 or 4 elements");
    if constexpr (NP == 4)
        *reinterpret_cast<uint2*>(out) = make_uint2(codes4(y[0], y[1], f), codes4(y[2], y[3], f));
    else
        *reinterpret_cast<uint32_t*>(out) = codes4(y[0], y[1], f);
}

constexpr int kThreads = 128;

// Rows of one kind, in whole warps.
template <typename E, int D>
__host__ __device__ constexpr int padded_rows(int n) {
    constexpr int RPW = 32 * 2 * E::kPerChunk / D;
    return (n + RPW - 1) / RPW * RPW;
}

// WIDE: rotary_dim is a multiple of 16, so the other halves of a chunk's elements are one
// chunk, at the same places, and the table is read in 16-byte pieces.  Otherwise each
// element fetches its pair's other half, its cos and its sin by itself.
// CTA (t, y): token t, row places y RPB IT .. ; a place is q's rows, then k's, then v's.
template <typename E, bool CODES, int D, int IT, bool WIDE, bool NORM>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeParams p, const InvScales inv) {
    constexpr int VEC = E::kPerChunk, NP = VEC / 2, LG = D / VEC / 2, RPB = kThreads / LG;
    const int l = threadIdx.x % LG;
    const int place0 = blockIdx.y * (RPB * IT) + threadIdx.x / LG;
    const int H_q = p.a.num_q_heads;
    const int q_end = padded_rows<E, D>(H_q), k_end = q_end + padded_rows<E, D>(p.H_kv);
    const int rot = p.a.rotary_dim, half = rot >> 1;
    const bool inter = p.a.interleaved != 0;
    // the lane's chunks start at elements ea and eb: the halves of its pairs, or (interleaved,
    // not WIDE, past rotary_dim) neighbours
    const int hc = half / VEC;
    const bool halves = WIDE && !inter && l < hc;
    const int ea = (halves ? l : 2 * l) * VEC;
    const int eb = halves ? ea + half : ea + VEC;
    const bool turned = halves || (inter && ea < rot) || (!WIDE && ea < rot);
    const int64_t t = blockIdx.x;
    const int64_t slot = __ldg(p.a.slot_mapping + t);
    const int pos = rot > 0 ? __ldg(p.a.positions + t) : 0;
    uint4 xa[IT], xb[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int place = place0 + i * RPB;
        const int kind = place < q_end ? 0 : place < k_end ? 1 : 2;
        const int h = place - (kind == 0 ? 0 : kind == 1 ? q_end : k_end);
        const char* base = static_cast<const char*>(kind == 0 ? p.a.q : kind == 1 ? p.a.k : p.a.v);
        const int64_t stride = kind == 0 ? p.a.q_stride : kind == 1 ? p.a.k_stride : p.a.v_stride;
        xa[i] = xb[i] = make_uint4(0u, 0u, 0u, 0u);
        if (h < (kind == 0 ? H_q : p.H_kv)) {
            const char* row = base + (t * stride + h * D) * E::kBytes;
            xa[i] = ld_global_stream(row + ea * E::kBytes);
            xb[i] = ld_global_stream(row + eb * E::kBytes);
        }
    }
    if (slot < 0) return;   // padding token
    if (slot >= p.num_slots || (unsigned)pos >= (unsigned)(rot > 0 ? p.a.max_position : 1)) {
        if (threadIdx.x == 0 && blockIdx.y == 0)
            report(p.dev_status, slot >= p.num_slots ? WF_DEV_BAD_SLOT : WF_DEV_BAD_POSITION);
        return;
    }
    // halves: cos and sin of the NP * 2 pairs.  Interleaved: of the VEC pairs of both chunks, NP
    // of each: c[0 .. NP / 2) two pairs' cos of chunk a each, the rest of chunk b
    const float* table = p.a.cos_sin + (int64_t)pos * rot;
    float2 c[NP], s[NP];
    if (WIDE && turned) {
        const float* tc = table + (inter ? ea / 2 : ea);
#pragma unroll
        for (int e = 0; e < NP; e += 2) {
            const float4 cc = __ldg(reinterpret_cast<const float4*>(tc + 2 * e));
            const float4 ss = __ldg(reinterpret_cast<const float4*>(tc + half + 2 * e));
            c[e] = make_float2(cc.x, cc.y);
            c[e + 1] = make_float2(cc.z, cc.w);
            s[e] = make_float2(ss.x, ss.y);
            s[e + 1] = make_float2(ss.z, ss.w);
        }
    }
    const int64_t slot_row = slot * p.H_kv * D, token_row = t * H_q * D;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int place = place0 + i * RPB;
        float2 a[NP], b[NP];
        if (place >= k_end) {                       // V: as it is
            const int h = place - k_end;
            if (h >= p.H_kv) continue;
            char* out = static_cast<char*>(p.a.v_pool) + (slot_row + h * D) * (CODES ? 1 : E::kBytes);
            if constexpr (CODES) {
                const float f = inv.v[min(h, kMaxScaleHeads - 1)];
                to_pairs<E>(xa[i], a);
                to_pairs<E>(xb[i], b);
                store_codes<NP>(out + ea, a, f);
                store_codes<NP>(out + eb, b, f);
            } else {
                st_global_v4(out + ea * E::kBytes, xa[i]);
                st_global_v4(out + eb * E::kBytes, xb[i]);
            }
            continue;
        }
        const bool is_q = place < q_end;
        const int h = is_q ? place : place - q_end;
        const bool live = h < (is_q ? H_q : p.H_kv);
        const void* w = is_q ? p.a.q_weight : p.a.k_weight;
        to_pairs<E>(xa[i], a);
        to_pairs<E>(xb[i], b);
        float rs = 1.f;
        if (NORM && w != nullptr) {
            float2 sq = __fmul2_rn(a[0], a[0]);
#pragma unroll
            for (int e = 1; e < NP; ++e) sq = __ffma2_rn(a[e], a[e], sq);
#pragma unroll
            for (int e = 0; e < NP; ++e) sq = __ffma2_rn(b[e], b[e], sq);
            float ss = sq.x + sq.y;
#pragma unroll
            for (int o = LG / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            rs = rsqrtf(ss * (1.f / D) + p.a.eps);
            const float2 r2 = make_float2(rs, rs);
            float2 f[NP];
            to_pairs<E>(__ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(w) + ea * E::kBytes)), f);
#pragma unroll
            for (int e = 0; e < NP; ++e) a[e] = __fmul2_rn(__fmul2_rn(a[e], r2), f[e]);
            to_pairs<E>(__ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(w) + eb * E::kBytes)), f);
#pragma unroll
            for (int e = 0; e < NP; ++e) b[e] = __fmul2_rn(__fmul2_rn(b[e], r2), f[e]);
        }
        if (!live) continue;
        if (WIDE && turned) {
            if (!inter) {          // (a, b) -> (a cos - b sin, b cos + a sin)
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    const float2 y = __fmul2_rn(a[e], c[e]), z = __fmul2_rn(b[e], c[e]);
                    const float2 n = make_float2(-s[e].x, -s[e].y), a0 = a[e];
                    a[e] = __ffma2_rn(b[e], n, y);
                    b[e] = __ffma2_rn(a0, s[e], z);
                }
            } else {               // the same within each pair of neighbours
                auto turn = [](float2& x, float cs, float sn) {
                    x = __ffma2_rn(make_float2(x.y, x.x), make_float2(-sn, sn), __fmul2_rn(x, make_float2(cs, cs)));
                };
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    const float2 ca = c[e / 2], sa = s[e / 2], cb = c[(NP + e) / 2], sb = s[(NP + e) / 2];
                    turn(a[e], (e & 1) ? ca.y : ca.x, (e & 1) ? sa.y : sa.x);
                    turn(b[e], (e & 1) ? cb.y : cb.x, (e & 1) ? sb.y : sb.x);
                }
            }
        } else if (!WIDE && turned) {
            const char* row = static_cast<const char*>(is_q ? p.a.q : p.a.k) +
                              (t * (is_q ? p.a.q_stride : p.a.k_stride) + h * D) * E::kBytes;
            auto one = [&](float x, int g) -> float {      // element g, normed, turned with its pair's other half
                if (g >= rot) return x;
                const bool first = inter ? (g & 1) == 0 : g < half;
                const int pair = inter ? g >> 1 : first ? g : g - half;
                const int o = inter ? g ^ 1 : first ? g + half : g - half;
                float y = widen_one<E>(row, o);
                if (NORM && w != nullptr) y = y * rs * widen_one<E>(w, o);
                const float sn = __ldg(table + half + pair);
                return fmaf(y, first ? -sn : sn, x * __ldg(table + pair));
            };
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                a[e] = make_float2(one(a[e].x, ea + 2 * e), one(a[e].y, ea + 2 * e + 1));
                b[e] = make_float2(one(b[e].x, eb + 2 * e), one(b[e].y, eb + 2 * e + 1));
            }
        }
        if (CODES && !is_q) {
            const float f = inv.k[min(h, kMaxScaleHeads - 1)];
            char* out = static_cast<char*>(p.a.k_pool) + slot_row + h * D;
            store_codes<NP>(out + ea, a, f);
            store_codes<NP>(out + eb, b, f);
        } else {
            char* out = is_q ? static_cast<char*>(p.a.q_out) + (token_row + h * D) * E::kBytes
                             : static_cast<char*>(p.a.k_pool) + (slot_row + h * D) * E::kBytes;
            st_global_v4(out + ea * E::kBytes, from_pairs<E>(a));
            st_global_v4(out + eb * E::kBytes, from_pairs<E>(b));
        }
    }
}

template <typename E, bool CODES, int D, int IT>
cudaError_t launch_rows(const RopeParams& p, const InvScales& inv, int places, cudaStream_t stream) {
    constexpr int RPB = kThreads / (D / E::kPerChunk / 2);
    const dim3 grid((unsigned)p.a.num_tokens, (unsigned)((places + RPB * IT - 1) / (RPB * IT)));
    const bool norm = p.a.q_weight != nullptr || p.a.k_weight != nullptr;
    if (p.a.rotary_dim % 16 != 0)
        qk_norm_rope_kernel<E, CODES, D, IT, false, true><<<grid, kThreads, 0, stream>>>(p, inv);
    else if (norm)
        qk_norm_rope_kernel<E, CODES, D, IT, true, true><<<grid, kThreads, 0, stream>>>(p, inv);
    else
        qk_norm_rope_kernel<E, CODES, D, IT, true, false><<<grid, kThreads, 0, stream>>>(p, inv);
    return cudaGetLastError();
}

template <typename E, bool CODES, int D>
cudaError_t launch_width(const RopeParams& p, const InvScales& inv, cudaStream_t stream) {
    constexpr int RPB = kThreads / (D / E::kPerChunk / 2);
    const int places = padded_rows<E, D>(p.a.num_q_heads) + 2 * padded_rows<E, D>(p.H_kv);
    const int64_t one = (int64_t)p.a.num_tokens * ((places + RPB - 1) / RPB);
    // few tokens: a CTA for every kThreads / LG rows; many: one that reads its table row for three
    // times as many (bf16, 32 + 8 + 8 heads of 128: 400 tokens 3.07 against 3.18 us, 800 tokens
    // 4.75 against 4.28 us)
    if (one <= 8 * (int64_t)num_sms()) return launch_rows<E, CODES, D, 1>(p, inv, places, stream);
    return launch_rows<E, CODES, D, 3>(p, inv, places, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, const wf_pool_desc& pool, uint32_t* dev_status,
                                cudaStream_t stream) {
    RopeParams p;
    p.a = a;
    p.num_slots = (int64_t)pool.num_blocks * pool.block_size;
    p.H_kv = pool.num_kv_heads;
    p.dev_status = dev_status;
    InvScales inv;
    const bool codes = pool.dtype == WF_DTYPE_FP8_E4M3;
    if (codes) {
        const HeadScales sc = head_scales(pool);
        for (int h = 0; h < kMaxScaleHeads; ++h) {
            inv.k[h] = 1.0f / sc.k[h];
            inv.v[h] = 1.0f / sc.v[h];
        }
    }
    const bool wide = pool.head_dim == 128;
    if (pool.dtype == WF_DTYPE_F32)
        return wide ? launch_width<F32, false, 128>(p, inv, stream) : launch_width<F32, false, 64>(p, inv, stream);
    if (codes)
        return wide ? launch_width<BF16, true, 128>(p, inv, stream) : launch_width<BF16, true, 64>(p, inv, stream);
    return wide ? launch_width<BF16, false, 128>(p, inv, stream) : launch_width<BF16, false, 64>(p, inv, stream);
}

}  // namespace wf
