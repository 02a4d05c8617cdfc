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
// a form of 166 instructions a warp and row pair took 51 us for 8193 tokens of
// Llama-3-8B heads into fp8 pools, whose bytes take 28.  So a head row is D / VEC lanes
// of one 16-byte chunk each and a warp's rows are of one kind (each kind's rows are
// padded to whole warps), which keeps the choice of q, k or v a branch of the warp;
// arithmetic is on pairs (two fp32 operations an instruction); and an instance without
// weights has no norm in it.  The sum of squares is a shuffle reduction over the row's
// lanes, and a rotated pair's other half comes from the lane that holds it (one shuffle
// a 32-bit word, of the raw chunk: both halves share the row's norm factor).  A lane
// reads its cos and sin once for IT rows.
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

// A 16-byte chunk of weights.
template <typename E>
__device__ __forceinline__ void weight_pairs(const void* w, int chunk, float2* f) {
    to_pairs<E>(__ldg(static_cast<const uint4*>(w) + chunk), f);
}

// Rows of one kind, in whole warps.
template <typename E, int D>
__host__ __device__ constexpr int padded_rows(int n) {
    constexpr int RPW = 32 * E::kPerChunk / D > 0 ? 32 * E::kPerChunk / D : 1;
    return (n + RPW - 1) / RPW * RPW;
}

// WIDE: rotary_dim is a multiple of 16, so a chunk's other halves lie in one chunk, at
// the same places, and the table is read in 16-byte pieces.  Otherwise each element
// fetches its pair's other half, its cos and its sin by itself.
// CTA (t, y): token t, row places y RPB IT .. ; a place is q's rows, then k's, then v's.
template <typename E, bool CODES, int D, int IT, bool WIDE, bool NORM>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const RopeParams p, const InvScales inv) {
    constexpr int VEC = E::kPerChunk, NP = VEC / 2, LG = D / VEC, RPB = 256 / LG;
    const int lg = threadIdx.x % LG, lane = threadIdx.x & 31;
    const int place0 = blockIdx.y * (RPB * IT) + threadIdx.x / LG;
    const int e0 = lg * VEC;
    const int H_q = p.a.num_q_heads;
    const int q_end = padded_rows<E, D>(H_q), k_end = q_end + padded_rows<E, D>(p.H_kv);
    const int rot = p.a.rotary_dim, half = rot >> 1;
    const bool turned = e0 < rot, inter = p.a.interleaved != 0, low = e0 < half;
    const int64_t t = blockIdx.x;
    const int64_t slot = __ldg(p.a.slot_mapping + t);
    const int pos = rot > 0 ? __ldg(p.a.positions + t) : 0;
    uint4 x[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int place = place0 + i * RPB;
        const int kind = place < q_end ? 0 : place < k_end ? 1 : 2;
        const int h = place - (kind == 0 ? 0 : kind == 1 ? q_end : k_end);
        const char* base = static_cast<const char*>(kind == 0 ? p.a.q : kind == 1 ? p.a.k : p.a.v);
        const int64_t stride = kind == 0 ? p.a.q_stride : kind == 1 ? p.a.k_stride : p.a.v_stride;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (h < (kind == 0 ? H_q : p.H_kv)) x[i] = ld_global_stream(base + (t * stride + h * D + e0) * E::kBytes);
    }
    if (slot < 0) return;   // padding token
    if (slot >= p.num_slots || (unsigned)pos >= (unsigned)(rot > 0 ? p.a.max_position : 1)) {
        if (threadIdx.x == 0 && blockIdx.y == 0)
            report(p.dev_status, slot >= p.num_slots ? WF_DEV_BAD_SLOT : WF_DEV_BAD_POSITION);
        return;
    }
    // cos and (signed) sin of this lane's elements, and the lane that holds their other halves
    const float* table = p.a.cos_sin + (int64_t)pos * rot;
    float2 c[NP], s[NP];
    int mate = lane;
    if (turned) {
        if constexpr (WIDE) {
            if (inter) {
#pragma unroll
                for (int e = 0; e < NP; e += 2) {
                    const float2 cc = __ldg(reinterpret_cast<const float2*>(table + e0 / 2 + e));
                    const float2 ss = __ldg(reinterpret_cast<const float2*>(table + half + e0 / 2 + e));
                    c[e] = make_float2(cc.x, cc.x);
                    c[e + 1] = make_float2(cc.y, cc.y);
                    s[e] = make_float2(-ss.x, ss.x);
                    s[e + 1] = make_float2(-ss.y, ss.y);
                }
            } else {
                const float* tc = table + (low ? e0 : e0 - half);
                const float sign = low ? -1.f : 1.f;
                mate = low ? lane + half / VEC : lane - half / VEC;
#pragma unroll
                for (int e = 0; e < NP; e += 2) {
                    const float4 cc = __ldg(reinterpret_cast<const float4*>(tc + 2 * e));
                    const float4 ss = __ldg(reinterpret_cast<const float4*>(tc + half + 2 * e));
                    c[e] = make_float2(cc.x, cc.y);
                    c[e + 1] = make_float2(cc.z, cc.w);
                    s[e] = __fmul2_rn(make_float2(ss.x, ss.y), make_float2(sign, sign));
                    s[e + 1] = __fmul2_rn(make_float2(ss.z, ss.w), make_float2(sign, sign));
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int g = e0 + e;
                const bool first = inter ? (g & 1) == 0 : g < half;
                const int i = inter ? g >> 1 : first ? g : g - half;
                const float cs = g < rot ? __ldg(table + i) : 1.f;
                float sn = g < rot ? __ldg(table + half + i) : 0.f;
                if (first) sn = -sn;
                if (e & 1) {
                    c[e / 2].y = cs;
                    s[e / 2].y = sn;
                } else {
                    c[e / 2].x = cs;
                    s[e / 2].x = sn;
                }
            }
        }
    }
    const int64_t slot_row = slot * p.H_kv * D + e0, token_row = t * H_q * D + e0;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int place = place0 + i * RPB;
        if (place >= k_end) {                       // V: as it is
            const int h = place - k_end;
            if (h >= p.H_kv) continue;
            char* out = static_cast<char*>(p.a.v_pool) + (slot_row + h * D) * (CODES ? 1 : E::kBytes);
            if constexpr (CODES) {
                const float f = inv.v[min(h, kMaxScaleHeads - 1)];
                float2 y[NP];
                to_pairs<E>(x[i], y);
                *reinterpret_cast<uint2*>(out) = make_uint2(codes4(y[0], y[1], make_float2(f, f)),
                                                            codes4(y[NP - 2], y[NP - 1], make_float2(f, f)));
            } else {
                st_global_v4(out, x[i]);
            }
            continue;
        }
        const bool is_q = place < q_end;
        const int h = is_q ? place : place - q_end;
        const bool live = h < (is_q ? H_q : p.H_kv);
        const void* w = is_q ? p.a.q_weight : p.a.k_weight;
        float2 y[NP], z[NP];
        to_pairs<E>(x[i], y);
        if (WIDE && rot > 0 && !inter) {
            uint4 m;
            m.x = __shfl_sync(0xffffffffu, x[i].x, mate);
            m.y = __shfl_sync(0xffffffffu, x[i].y, mate);
            m.z = __shfl_sync(0xffffffffu, x[i].z, mate);
            m.w = __shfl_sync(0xffffffffu, x[i].w, mate);
            to_pairs<E>(m, z);
        }
        float rs = 1.f;
        if (NORM && w != nullptr) {
            float2 sq = __fmul2_rn(y[0], y[0]);
#pragma unroll
            for (int e = 1; e < NP; ++e) sq = __ffma2_rn(y[e], y[e], sq);
            float ss = sq.x + sq.y;
#pragma unroll
            for (int o = LG / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            rs = rsqrtf(ss * (1.f / D) + p.a.eps);
            const float2 r2 = make_float2(rs, rs);
            float2 f[NP];
            weight_pairs<E>(w, lg, f);
#pragma unroll
            for (int e = 0; e < NP; ++e) y[e] = __fmul2_rn(__fmul2_rn(y[e], r2), f[e]);
            if (WIDE && !inter && turned) {
                weight_pairs<E>(w, lg + mate - lane, f);
#pragma unroll
                for (int e = 0; e < NP; ++e) z[e] = __fmul2_rn(__fmul2_rn(z[e], r2), f[e]);
            }
        }
        if (!live) continue;
        if (turned) {
            if (inter) {   // pairs lie side by side in the chunk, normed already
#pragma unroll
                for (int e = 0; e < NP; ++e) z[e] = make_float2(y[e].y, y[e].x);
            } else if constexpr (!WIDE) {
                const char* row = static_cast<const char*>(is_q ? p.a.q : p.a.k) +
                                  (t * (is_q ? p.a.q_stride : p.a.k_stride) + h * D) * E::kBytes;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int g = e0 + e;
                    const int o = g < half ? g + half : g - half;
                    float b = 0.f;
                    if (g < rot) {
                        b = widen_one<E>(row, o);
                        if (NORM && w != nullptr) b = b * rs * widen_one<E>(w, o);
                    }
                    if (e & 1) z[e / 2].y = b;
                    else z[e / 2].x = b;
                }
            }
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                const float2 r2 = __ffma2_rn(z[e], s[e], __fmul2_rn(y[e], c[e]));
                if (WIDE || e0 + 2 * e + 1 < rot) y[e] = r2;   // rotary_dim is even: a pair is in or out
            }
        }
        if (is_q) {
            st_global_v4(static_cast<char*>(p.a.q_out) + (token_row + h * D) * E::kBytes, from_pairs<E>(y));
        } else if constexpr (CODES) {
            const float f = inv.k[min(h, kMaxScaleHeads - 1)];
            *reinterpret_cast<uint2*>(static_cast<char*>(p.a.k_pool) + slot_row + h * D) =
                make_uint2(codes4(y[0], y[1], make_float2(f, f)), codes4(y[NP - 2], y[NP - 1], make_float2(f, f)));
        } else {
            st_global_v4(static_cast<char*>(p.a.k_pool) + (slot_row + h * D) * E::kBytes, from_pairs<E>(y));
        }
    }
}

template <typename E, bool CODES, int D, int IT>
cudaError_t launch_rows(const RopeParams& p, const InvScales& inv, int places, cudaStream_t stream) {
    constexpr int RPB = 256 / (D / E::kPerChunk);
    const dim3 grid((unsigned)p.a.num_tokens, (unsigned)((places + RPB * IT - 1) / (RPB * IT)));
    const bool norm = p.a.q_weight != nullptr || p.a.k_weight != nullptr;
    if (p.a.rotary_dim % 16 != 0)
        qk_norm_rope_kernel<E, CODES, D, IT, false, true><<<grid, 256, 0, stream>>>(p, inv);
    else if (norm)
        qk_norm_rope_kernel<E, CODES, D, IT, true, true><<<grid, 256, 0, stream>>>(p, inv);
    else
        qk_norm_rope_kernel<E, CODES, D, IT, true, false><<<grid, 256, 0, stream>>>(p, inv);
    return cudaGetLastError();
}

template <typename E, bool CODES, int D>
cudaError_t launch_width(const RopeParams& p, const InvScales& inv, cudaStream_t stream) {
    constexpr int RPB = 256 / (D / E::kPerChunk);
    const int places = padded_rows<E, D>(p.a.num_q_heads) + 2 * padded_rows<E, D>(p.H_kv);
    const int64_t one = (int64_t)p.a.num_tokens * ((places + RPB - 1) / RPB);
    if (one <= 4 * (int64_t)num_sms()) return launch_rows<E, CODES, D, 1>(p, inv, places, stream);
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
