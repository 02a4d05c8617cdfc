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
// rotation and scatter passes make.  A head row is D / VEC lanes of one 16-byte chunk
// each, so a warp holds one, two or four rows; the sum of squares is a shuffle
// reduction over the row's lanes, and a rotated pair's other half comes from the lane
// that holds it (one shuffle a 32-bit word, of the raw chunk: both halves share the
// row's norm factor).  A CTA works on IT rows a lane group of one token, so a lane
// reads its cos and sin once for IT rows.
#include "wf_internal.h"

namespace wf {

namespace {

struct RopeParams {
    RopeArgs a;
    int64_t num_slots;
    int rows;          // H_q + 2 H_kv
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

template <typename E>
__device__ __forceinline__ uint4 narrow_chunk(const float* f);
template <>
__device__ __forceinline__ uint4 narrow_chunk<F32>(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <>
__device__ __forceinline__ uint4 narrow_chunk<BF16>(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ uint32_t codes4(const float* f, float inv) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[0] * inv, f[1] * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[2] * inv, f[3] * inv), __NV_SATFINITE, __NV_E4M3);
    return (lo & 0xffffu) | (hi << 16);
}

// WIDE: rotary_dim is a multiple of 16, so no pair's halves cross a chunk border at
// different places and the table is read in 16-byte chunks.  Otherwise each element
// fetches its pair's other half, its cos and its sin by itself.
template <typename E, bool CODES, int D, int IT, bool WIDE>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const RopeParams p, const InvScales inv) {
    constexpr int VEC = E::kPerChunk, LG = D / VEC, RPB = 256 / LG, WORDS = 4;
    const int64_t t = blockIdx.x;
    const int lg = threadIdx.x % LG;
    const int row0 = blockIdx.y * (RPB * IT) + threadIdx.x / LG;
    const int e0 = lg * VEC;
    const int H_q = p.a.num_q_heads;
    const int64_t slot = __ldg(p.a.slot_mapping + t);
    const int rot = p.a.rotary_dim, half = rot >> 1;
    const int pos = rot > 0 ? __ldg(p.a.positions + t) : 0;
    auto row_ptr = [&](int r) -> const char* {
        const int64_t off = r < H_q            ? t * p.a.q_stride + (int64_t)r * D
                            : r < H_q + p.H_kv ? t * p.a.k_stride + (int64_t)(r - H_q) * D
                                               : t * p.a.v_stride + (int64_t)(r - H_q - p.H_kv) * D;
        const void* base = r < H_q ? p.a.q : r < H_q + p.H_kv ? p.a.k : p.a.v;
        return static_cast<const char*>(base) + off * E::kBytes;
    };
    uint4 x[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int r = row0 + i * RPB;
        x[i] = r < p.rows ? ld_global_stream(row_ptr(r) + lg * 16) : make_uint4(0u, 0u, 0u, 0u);
    }
    if (slot < 0) return;   // padding token
    if (slot >= p.num_slots || (unsigned)pos >= (unsigned)(rot > 0 ? p.a.max_position : 1)) {
        if (threadIdx.x == 0 && blockIdx.y == 0)
            report(p.dev_status, slot >= p.num_slots ? WF_DEV_BAD_SLOT : WF_DEV_BAD_POSITION);
        return;
    }
    // cos and (signed) sin of this lane's elements, and the lane that holds their pairs
    const bool turned = e0 < rot, inter = p.a.interleaved != 0;
    const float* table = p.a.cos_sin + (int64_t)pos * rot;
    float c[VEC], s[VEC];
    int mate = threadIdx.x & 31;
    if (turned) {
        if constexpr (WIDE) {
            if (inter) {
                const float* tc = table + e0 / 2;
                const float* ts = tc + half;
#pragma unroll
                for (int e = 0; e < VEC; e += 4) {
                    const float2 cc = __ldg(reinterpret_cast<const float2*>(tc + e / 2));
                    const float2 ss = __ldg(reinterpret_cast<const float2*>(ts + e / 2));
                    c[e] = c[e + 1] = cc.x;
                    c[e + 2] = c[e + 3] = cc.y;
                    s[e] = -ss.x; s[e + 1] = ss.x;
                    s[e + 2] = -ss.y; s[e + 3] = ss.y;
                }
            } else {
                const bool low = e0 < half;
                const float* tc = table + (low ? e0 : e0 - half);
                const float* ts = tc + half;
                mate += low ? half / VEC : -(half / VEC);
#pragma unroll
                for (int e = 0; e < VEC; e += 4) {
                    const float4 cc = __ldg(reinterpret_cast<const float4*>(tc + e));
                    const float4 ss = __ldg(reinterpret_cast<const float4*>(ts + e));
                    c[e] = cc.x; c[e + 1] = cc.y; c[e + 2] = cc.z; c[e + 3] = cc.w;
                    s[e] = low ? -ss.x : ss.x; s[e + 1] = low ? -ss.y : ss.y;
                    s[e + 2] = low ? -ss.z : ss.z; s[e + 3] = low ? -ss.w : ss.w;
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int g = e0 + e;
                const bool first = inter ? (g & 1) == 0 : g < half;
                const int i = inter ? g >> 1 : first ? g : g - half;
                c[e] = g < rot ? __ldg(table + i) : 1.f;
                const float sn = g < rot ? __ldg(table + half + i) : 0.f;
                s[e] = first ? -sn : sn;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int r = row0 + i * RPB;
        const bool live = r < p.rows;
        const bool is_q = r < H_q, is_k = !is_q && r < H_q + p.H_kv;
        const int h = is_q ? r : is_k ? r - H_q : r - H_q - p.H_kv;
        float y[VEC];
        widen_chunk<E>(x[i], y);
        const void* w = is_q ? p.a.q_weight : is_k ? p.a.k_weight : nullptr;
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss += y[e] * y[e];
#pragma unroll
        for (int o = LG / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float rs = w != nullptr ? rsqrtf(ss * (1.f / D) + p.a.eps) : 1.f;
        // the other halves, raw: from the lane that holds them
        float z[VEC];
        if constexpr (WIDE) {
            uint32_t m[WORDS] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int k = 0; k < WORDS; ++k) m[k] = __shfl_sync(0xffffffffu, m[k], mate);
            widen_chunk<E>(make_uint4(m[0], m[1], m[2], m[3]), z);
        }
        if (!live) continue;
        if (w != nullptr) {
            float f[VEC];
            widen_chunk<E>(__ldg(reinterpret_cast<const uint4*>(w) + lg), f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) y[e] = y[e] * rs * f[e];
        }
        if (turned && (is_q || is_k)) {
            if (inter) {   // pairs lie side by side in the chunk, normed already
#pragma unroll
                for (int e = 0; e < VEC; e += 2) {
                    z[e] = y[e + 1];
                    z[e + 1] = y[e];
                }
            } else if constexpr (WIDE) {
                if (w != nullptr) {
                    float f[VEC];
                    widen_chunk<E>(__ldg(reinterpret_cast<const uint4*>(w) + (lg + mate - (int)(threadIdx.x & 31))), f);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) z[e] = z[e] * rs * f[e];
                }
            } else {
                const char* src = row_ptr(r);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int g = e0 + e;
                    const int o = g < half ? g + half : g - half;
                    float b = 0.f;
                    if (g < rot) {
                        b = widen_one<E>(src, o);
                        if (w != nullptr) b = b * rs * widen_one<E>(w, o);
                    }
                    z[e] = b;
                }
            }
            if constexpr (WIDE) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) y[e] = y[e] * c[e] + z[e] * s[e];
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (e0 + e < rot) y[e] = y[e] * c[e] + z[e] * s[e];
            }
        }
        if (is_q) {
            st_global_v4(static_cast<char*>(p.a.q_out) + ((t * H_q + h) * D + e0) * E::kBytes, narrow_chunk<E>(y));
        } else {
            char* pool = static_cast<char*>(is_k ? p.a.k_pool : p.a.v_pool);
            const int64_t at = (slot * p.H_kv + h) * D + e0;
            if constexpr (CODES) {
                const int hs = min(h, kMaxScaleHeads - 1);
                const float iv = is_k ? inv.k[hs] : inv.v[hs];
                *reinterpret_cast<uint2*>(pool + at) = make_uint2(codes4(y, iv), codes4(y + 4, iv));
            } else {
                st_global_v4(pool + at * E::kBytes, narrow_chunk<E>(y));
            }
        }
    }
}

template <typename E, bool CODES, int D, int IT>
cudaError_t launch_rows(const RopeParams& p, const InvScales& inv, cudaStream_t stream) {
    constexpr int RPB = 256 / (D / E::kPerChunk);
    const dim3 grid((unsigned)p.a.num_tokens, (unsigned)((p.rows + RPB * IT - 1) / (RPB * IT)));
    if (p.a.rotary_dim % 16 == 0)
        qk_norm_rope_kernel<E, CODES, D, IT, true><<<grid, 256, 0, stream>>>(p, inv);
    else
        qk_norm_rope_kernel<E, CODES, D, IT, false><<<grid, 256, 0, stream>>>(p, inv);
    return cudaGetLastError();
}

template <typename E, bool CODES, int D>
cudaError_t launch_width(const RopeParams& p, const InvScales& inv, cudaStream_t stream) {
    constexpr int RPB = 256 / (D / E::kPerChunk);
    const int64_t one = (int64_t)p.a.num_tokens * ((p.rows + RPB - 1) / RPB);
    if (one <= 4 * (int64_t)num_sms()) return launch_rows<E, CODES, D, 1>(p, inv, stream);
    return launch_rows<E, CODES, D, 3>(p, inv, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, const wf_pool_desc& pool, uint32_t* dev_status,
                                cudaStream_t stream) {
    RopeParams p;
    p.a = a;
    p.num_slots = (int64_t)pool.num_blocks * pool.block_size;
    p.H_kv = pool.num_kv_heads;
    p.rows = a.num_q_heads + 2 * pool.num_kv_heads;
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
