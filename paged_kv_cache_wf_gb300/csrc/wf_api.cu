// wf_api.cu -- the extern "C" boundary of libwf: argument validation (before any
// launch), status mapping, and dispatch to the kernels' launchers.
#include <cudaTypedefs.h>

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <unordered_map>
#include <utility>

#include "wf_internal.h"

namespace wf {

int num_sms() {
    static std::mutex mu;
    static std::unordered_map<int, int> cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    std::lock_guard<std::mutex> lock(mu);
    auto it = cache.find(dev);
    if (it != cache.end()) return it->second;
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) n = 148;
    cache[dev] = n;
    return n;
}

cudaError_t allow_dynamic_smem(const void* kernel, int bytes) {
    static std::mutex mu;
    static std::unordered_map<uint64_t, int> done;  // (device, kernel) -> bytes granted
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t key = (reinterpret_cast<uint64_t>(kernel) << 8) ^ (uint64_t)dev;
    std::lock_guard<std::mutex> lock(mu);
    auto it = done.find(key);
    if (it != done.end() && it->second >= bytes) return cudaSuccess;
    if (bytes > 48 * 1024) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (err != cudaSuccess) return err;
    }
    done[key] = bytes;
    return cudaSuccess;
}

cudaError_t allow_large_cluster(const void* kernel) {
    static std::mutex mu;
    static std::unordered_map<uint64_t, bool> done;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t key = (reinterpret_cast<uint64_t>(kernel) << 8) ^ (uint64_t)dev;
    std::lock_guard<std::mutex> lock(mu);
    if (done.count(key)) return cudaSuccess;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (err == cudaSuccess) done[key] = true;
    return err;
}

cudaError_t encode_tiled_bf16(CUtensorMap* map, void* base, int rank, const uint64_t* dims,
                              const uint64_t* strides, const uint32_t* box, CUtensorMapL2promotion promotion) {
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, rank, dims, strides, box,
                        CU_TENSOR_MAP_SWIZZLE_128B, promotion);
}

cudaError_t encode_tiled(CUtensorMap* map, CUtensorMapDataType type, void* base, int rank, const uint64_t* dims,
                         const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle swizzle,
                         CUtensorMapL2promotion promotion) {
    static std::mutex mu;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (fn == nullptr) {
            void* f = nullptr;
            cudaDriverEntryPointQueryResult q;
            cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
            if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || f == nullptr) return cudaErrorNotSupported;
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
        }
    }
    cuuint64_t d[5];
    cuuint64_t s[4];
    cuuint32_t bx[5], es[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        bx[i] = box[i];
        es[i] = 1;
        if (i + 1 < rank) s[i] = strides[i];
    }
    const CUresult r = fn(map, type, (cuuint32_t)rank, base, d, s, bx, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                          promotion, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace wf

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}

wf_status check_pool(const wf_pool_desc& pool) {
    if (pool.num_blocks < 1 || pool.block_size < 1 || pool.block_size > 1024 ||
        pool.num_kv_heads < 1)
        return WF_ERR_INVALID_ARG;
    if (pool.dtype != WF_DTYPE_F32 && pool.dtype != WF_DTYPE_BF16 && pool.dtype != WF_DTYPE_FP8_E4M3)
        return WF_ERR_UNSUPPORTED;
    if (pool.dtype == WF_DTYPE_FP8_E4M3) {
        auto ok = [](float x) { return x > 0.f && x <= 3.0e38f; };   // finite and positive (NaN fails)
        if (pool.k_head_scales == nullptr && !ok(pool.k_scale)) return WF_ERR_INVALID_ARG;
        if (pool.v_head_scales == nullptr && !ok(pool.v_scale)) return WF_ERR_INVALID_ARG;
        if ((pool.k_head_scales || pool.v_head_scales) && pool.num_kv_heads > wf::kMaxScaleHeads)
            return WF_ERR_UNSUPPORTED;
        for (int h = 0; h < pool.num_kv_heads; ++h) {
            if (pool.k_head_scales && !ok(pool.k_head_scales[h])) return WF_ERR_INVALID_ARG;
            if (pool.v_head_scales && !ok(pool.v_head_scales[h])) return WF_ERR_INVALID_ARG;
        }
    }
    if (pool.head_dim != 64 && pool.head_dim != 128) return WF_ERR_UNSUPPORTED;
    const int64_t slots = (int64_t)pool.num_blocks * pool.block_size;
    if (slots > (int64_t)INT32_MAX * 64) return WF_ERR_INVALID_ARG;
    return WF_OK;
}

wf_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return WF_OK;
    if (e == cudaErrorNotSupported) return WF_ERR_UNSUPPORTED;
    return WF_ERR_CUDA;
}

}  // namespace

extern "C" {

int wf_abi_version(void) { return 104; }

const char* wf_status_string(wf_status s) {
    switch (s) {
        case WF_OK: return "ok";
        case WF_ERR_INVALID_ARG: return "invalid argument";
        case WF_ERR_UNSUPPORTED: return "unsupported configuration";
        case WF_ERR_WORKSPACE: return "workspace missing or too small";
        case WF_ERR_CUDA: return "CUDA error";
        case WF_ERR_NO_BLOCKS: return "not enough free blocks";
    }
    return "unknown status";
}

wf_status wf_reshape_and_cache(const void* k, const void* v, void* k_pool, void* v_pool,
                               const int64_t* slot_mapping, int32_t num_tokens,
                               wf_pool_desc pool, uint32_t* dev_status, cudaStream_t stream) {
    wf_status s = check_pool(pool);
    if (s != WF_OK) return s;
    if (num_tokens < 0) return WF_ERR_INVALID_ARG;
    if (num_tokens == 0) return WF_OK;
    if (!k || !v || !k_pool || !v_pool || !slot_mapping) return WF_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_pool) || !aligned16(v_pool) ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
        return WF_ERR_INVALID_ARG;
    return from_cuda(wf::launch_reshape_and_cache(k, v, k_pool, v_pool, slot_mapping, num_tokens,
                                                  pool, dev_status, stream));
}

wf_status wf_qk_norm_rope_and_cache(void* q_out, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                    const void* v, int64_t v_stride, const void* q_weight, const void* k_weight,
                                    float eps, const float* cos_sin, int32_t max_position, int32_t rotary_dim,
                                    int32_t interleaved, const int32_t* positions, void* k_pool, void* v_pool,
                                    const int64_t* slot_mapping, int32_t num_tokens, int32_t num_q_heads,
                                    wf_pool_desc pool, uint32_t* dev_status, cudaStream_t stream) {
    wf_status s = check_pool(pool);
    if (s != WF_OK) return s;
    if (num_tokens < 0 || num_q_heads < 1 || num_q_heads % pool.num_kv_heads != 0) return WF_ERR_INVALID_ARG;
    if (rotary_dim < 0 || rotary_dim > pool.head_dim || rotary_dim % 2 != 0) return WF_ERR_INVALID_ARG;
    if (rotary_dim > 0 && max_position < 1) return WF_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.f) return WF_ERR_INVALID_ARG;
    if (num_tokens == 0) return WF_OK;
    if (!q_out || !q || !k || !v || !k_pool || !v_pool || !slot_mapping) return WF_ERR_INVALID_ARG;
    if (rotary_dim > 0 && (!cos_sin || !positions || !aligned16(cos_sin) ||
                           (reinterpret_cast<uintptr_t>(positions) & 3u)))
        return WF_ERR_INVALID_ARG;
    if (!aligned16(q_out) || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(k_pool) ||
        !aligned16(v_pool) || (q_weight && !aligned16(q_weight)) || (k_weight && !aligned16(k_weight)) ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
        return WF_ERR_INVALID_ARG;
    const int64_t act = pool.dtype == WF_DTYPE_F32 ? 4 : 2;
    const int64_t qrow = (int64_t)num_q_heads * pool.head_dim, krow = (int64_t)pool.num_kv_heads * pool.head_dim;
    if (num_tokens > 1) {
        if (q_stride < qrow || k_stride < krow || v_stride < krow) return WF_ERR_INVALID_ARG;
        if (q_stride * act % 16 != 0 || k_stride * act % 16 != 0 || v_stride * act % 16 != 0)
            return WF_ERR_INVALID_ARG;
        // beyond any device's memory: keeps every byte offset within 63 bits
        const int64_t cap = (int64_t)1 << 40;
        if (q_stride > cap || k_stride > cap || v_stride > cap) return WF_ERR_INVALID_ARG;
    } else {
        q_stride = qrow;
        k_stride = v_stride = krow;
    }
    // a row is read by several threads while others write q_out
    const int64_t out_bytes = num_tokens * qrow * act, last = num_tokens - 1;
    if (overlap(q_out, out_bytes, q, (last * q_stride + qrow) * act) ||
        overlap(q_out, out_bytes, k, (last * k_stride + krow) * act) ||
        overlap(q_out, out_bytes, v, (last * v_stride + krow) * act))
        return WF_ERR_INVALID_ARG;
    const wf::RopeArgs a{q_out, q, k, v, q_stride, k_stride, v_stride, q_weight, k_weight, eps, cos_sin, max_position,
                         rotary_dim, interleaved, positions, k_pool, v_pool, slot_mapping, num_tokens, num_q_heads};
    return from_cuda(wf::launch_qk_norm_rope(a, pool, dev_status, stream));
}

wf_status wf_keep_accepted(void* k_pool, void* v_pool, const int32_t* block_tables, int32_t max_blocks_per_seq,
                           const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* accepted,
                           int32_t max_accepted, const int32_t* num_accepted, int32_t* new_seq_lens, int32_t B,
                           wf_pool_desc pool, uint32_t* dev_status, cudaStream_t stream) {
    wf_status s = check_pool(pool);
    if (s != WF_OK) return s;
    if (B < 0 || max_accepted < 0 || max_blocks_per_seq < 1) return WF_ERR_INVALID_ARG;
    if (B == 0) return WF_OK;
    if (!k_pool || !v_pool || !block_tables || !seq_lens || !cu_q_lens || !num_accepted ||
        (max_accepted > 0 && !accepted))
        return WF_ERR_INVALID_ARG;
    if (!aligned16(k_pool) || !aligned16(v_pool)) return WF_ERR_INVALID_ARG;
    for (const void* p : {(const void*)block_tables, (const void*)seq_lens, (const void*)cu_q_lens,
                          (const void*)accepted, (const void*)num_accepted, (const void*)new_seq_lens})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return WF_ERR_INVALID_ARG;
    if (new_seq_lens == seq_lens || new_seq_lens == num_accepted) return WF_ERR_INVALID_ARG;
    return from_cuda(wf::launch_keep_accepted(k_pool, v_pool, block_tables, max_blocks_per_seq, seq_lens, cu_q_lens,
                                              accepted, max_accepted, num_accepted, new_seq_lens, B, pool, dev_status,
                                              stream));
}

wf_status wf_verify_drafts(int32_t* accepted, int32_t max_accepted, int32_t* num_accepted, int32_t* next_tokens,
                           const void* target, int64_t target_stride, const void* draft, int64_t draft_stride,
                           int32_t vocab, int32_t probs_dtype, const int32_t* tokens, const int32_t* parents,
                           const int32_t* cu_q_lens, const float* coins, const float* picks, int32_t B, int32_t total_q,
                           int32_t max_q_len, uint32_t* dev_status, cudaStream_t stream) {
    if (B < 0 || total_q < 0 || max_q_len < 0 || max_accepted < 1 || vocab < 1) return WF_ERR_INVALID_ARG;
    if (probs_dtype != WF_DTYPE_F32 && probs_dtype != WF_DTYPE_BF16) return WF_ERR_UNSUPPORTED;
    if (max_q_len > wf::kMaxVerifyNodes || vocab > wf::kMaxVocab || B > (1 << 24)) return WF_ERR_UNSUPPORTED;
    if (B == 0) return WF_OK;
    if (!accepted || !num_accepted || !next_tokens || !cu_q_lens || !picks) return WF_ERR_INVALID_ARG;
    const int64_t elt = probs_dtype == WF_DTYPE_F32 ? 4 : 2, cap = (int64_t)1 << 40;
    if (total_q > 0) {
        if (!target || !tokens || !coins) return WF_ERR_INVALID_ARG;
        if (target_stride < vocab || target_stride > cap) return WF_ERR_INVALID_ARG;
        if (draft && (draft_stride < vocab || draft_stride > cap)) return WF_ERR_INVALID_ARG;
    }
    if ((reinterpret_cast<uintptr_t>(target) | reinterpret_cast<uintptr_t>(draft)) & (uintptr_t)(elt - 1))
        return WF_ERR_INVALID_ARG;
    for (const void* p : {(const void*)accepted, (const void*)num_accepted, (const void*)next_tokens,
                          (const void*)tokens, (const void*)parents, (const void*)cu_q_lens, (const void*)coins,
                          (const void*)picks})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return WF_ERR_INVALID_ARG;
    // written while other requests' inputs are read
    const int64_t reqs = 4 * (int64_t)B, nodes = 4 * (int64_t)total_q;
    const auto rows = [&](int64_t stride) { return total_q > 0 ? ((int64_t)(total_q - 1) * stride + vocab) * elt : 0; };
    const struct {
        const void* p;
        int64_t bytes;
    } in[] = {{target, rows(target_stride)}, {draft, draft ? rows(draft_stride) : 0}, {tokens, nodes},
              {parents, parents ? nodes : 0}, {coins, nodes}, {cu_q_lens, reqs + 4}, {picks, reqs}},
      out[] = {{accepted, reqs * max_accepted}, {num_accepted, reqs}, {next_tokens, reqs}};
    for (int o = 0; o < 3; ++o) {
        for (const auto& i : in)
            if (i.bytes > 0 && overlap(out[o].p, out[o].bytes, i.p, i.bytes)) return WF_ERR_INVALID_ARG;
        for (int x = o + 1; x < 3; ++x)
            if (overlap(out[o].p, out[o].bytes, out[x].p, out[x].bytes)) return WF_ERR_INVALID_ARG;
    }
    const wf::VerifyArgs a{accepted, num_accepted, next_tokens, max_accepted, target, draft, target_stride, draft_stride,
                           vocab, probs_dtype, tokens, parents, cu_q_lens, coins, picks, B, total_q, max_q_len};
    return from_cuda(wf::launch_verify_drafts(a, dev_status, stream));
}

wf_status wf_build_step(int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                        const int32_t* new_lens, const int32_t* free_blocks, const int32_t* num_free,
                        const int32_t* depths, int32_t* new_seq_lens, int32_t* new_num_free, int32_t* cu_q_lens,
                        int64_t* slot_mapping, int32_t* positions, int32_t B, int32_t max_tokens, int32_t num_blocks,
                        int32_t block_size, uint32_t* dev_status, cudaStream_t stream) {
    if (B < 0 || max_tokens < 0 || max_blocks_per_seq < 1 || num_blocks < 1 || block_size < 1 || block_size > 1024)
        return WF_ERR_INVALID_ARG;
    if (B > wf::kMaxStepRequests) return WF_ERR_UNSUPPORTED;
    if (!free_blocks || !num_free || !new_num_free || !cu_q_lens) return WF_ERR_INVALID_ARG;
    if (B > 0 && (!block_tables || !seq_lens || !new_lens || !new_seq_lens)) return WF_ERR_INVALID_ARG;
    if (max_tokens > 0 && (!slot_mapping || !positions)) return WF_ERR_INVALID_ARG;
    for (const void* p : {(const void*)block_tables, (const void*)seq_lens, (const void*)new_lens,
                          (const void*)free_blocks, (const void*)num_free, (const void*)depths,
                          (const void*)new_seq_lens, (const void*)new_num_free, (const void*)cu_q_lens,
                          (const void*)positions})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return WF_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) return WF_ERR_INVALID_ARG;
    // written while others are read; seq_lens and num_free may be updated in place, from their first element on
    const int64_t lens = 4 * (int64_t)B, rows = 4 * (int64_t)max_tokens;
    const struct {
        const void* p;
        int64_t bytes;
    } in[] = {{seq_lens, lens}, {new_lens, lens}, {free_blocks, 4 * (int64_t)num_blocks}, {num_free, 4}, {depths, depths ? rows : 0}},
      out[] = {{block_tables, 4 * (int64_t)B * max_blocks_per_seq}, {new_seq_lens, lens}, {new_num_free, 4},
               {cu_q_lens, lens + 4}, {slot_mapping, 2 * rows}, {positions, rows}};
    constexpr int kOut = sizeof(out) / sizeof(out[0]);
    for (int o = 0; o < kOut; ++o) {
        if (out[o].bytes == 0) continue;
        for (const auto& i : in) {
            const bool in_place = (out[o].p == new_seq_lens && i.p == seq_lens && new_seq_lens == seq_lens) ||
                                  (out[o].p == new_num_free && i.p == num_free && new_num_free == num_free);
            if (i.bytes > 0 && !in_place && overlap(out[o].p, out[o].bytes, i.p, i.bytes)) return WF_ERR_INVALID_ARG;
        }
        for (int x = o + 1; x < kOut; ++x)
            if (out[x].bytes > 0 && overlap(out[o].p, out[o].bytes, out[x].p, out[x].bytes)) return WF_ERR_INVALID_ARG;
    }
    const wf::BuildArgs a{block_tables, max_blocks_per_seq, seq_lens, new_lens, free_blocks, num_free, depths,
                          new_seq_lens, new_num_free, cu_q_lens, slot_mapping, positions, B, max_tokens, num_blocks,
                          block_size};
    return from_cuda(wf::launch_build_step(a, dev_status, stream));
}

wf_status wf_trim_blocks(const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                         const int32_t* kept_lens, int32_t* free_blocks, const int32_t* num_free, int32_t* new_num_free,
                         int32_t B, int32_t num_blocks, int32_t block_size, uint32_t* dev_status, cudaStream_t stream) {
    if (B < 0 || max_blocks_per_seq < 1 || num_blocks < 1 || block_size < 1 || block_size > 1024)
        return WF_ERR_INVALID_ARG;
    if (B > wf::kMaxStepRequests) return WF_ERR_UNSUPPORTED;
    if (!free_blocks || !num_free || !new_num_free) return WF_ERR_INVALID_ARG;
    if (B > 0 && (!block_tables || !seq_lens || !kept_lens)) return WF_ERR_INVALID_ARG;
    for (const void* p : {(const void*)block_tables, (const void*)seq_lens, (const void*)kept_lens,
                          (const void*)free_blocks, (const void*)num_free, (const void*)new_num_free})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return WF_ERR_INVALID_ARG;
    const int64_t lens = 4 * (int64_t)B, list = 4 * (int64_t)num_blocks, table = lens * max_blocks_per_seq;
    if (overlap(free_blocks, list, num_free, 4) || overlap(free_blocks, list, new_num_free, 4)) return WF_ERR_INVALID_ARG;
    if (B > 0)
        for (const auto& [p, bytes] : {std::pair<const void*, int64_t>{block_tables, table}, {seq_lens, lens}, {kept_lens, lens}})
            if (overlap(free_blocks, list, p, bytes) || overlap(new_num_free, 4, p, bytes)) return WF_ERR_INVALID_ARG;
    const wf::TrimArgs a{block_tables, max_blocks_per_seq, seq_lens, kept_lens, free_blocks, num_free, new_num_free, B,
                         num_blocks, block_size};
    return from_cuda(wf::launch_trim_blocks(a, dev_status, stream));
}

wf_status wf_copy_blocks(void* k_pool, void* v_pool, const int32_t* block_pairs, int32_t num_pairs,
                         wf_pool_desc pool, uint32_t* dev_status, cudaStream_t stream) {
    wf_status s = check_pool(pool);
    if (s != WF_OK) return s;
    if (num_pairs < 0) return WF_ERR_INVALID_ARG;
    if (num_pairs == 0) return WF_OK;
    if (!k_pool || !v_pool || !block_pairs) return WF_ERR_INVALID_ARG;
    if (!aligned16(k_pool) || !aligned16(v_pool) || (reinterpret_cast<uintptr_t>(block_pairs) & 3u))
        return WF_ERR_INVALID_ARG;
    return from_cuda(wf::launch_copy_blocks(k_pool, v_pool, block_pairs, num_pairs, pool, dev_status, stream));
}

size_t wf_paged_decode_workspace_size(int32_t B, int32_t num_q_heads, int32_t max_seq_len,
                                      wf_pool_desc pool) {
    if (check_pool(pool) != WF_OK || num_q_heads < 1) return 0;
    return wf::decode_workspace_bytes(B, num_q_heads, max_seq_len, pool);
}

}  // extern "C"

namespace {

// wf_paged_decode's argument rules (WF_OK also for an empty batch, which launches
// nothing).
wf_status decode_args(void* out, const void* q, const void* k_pool, const void* v_pool, const int32_t* block_tables,
                      int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t B, int32_t max_seq_len,
                      int32_t num_q_heads, float scale, const wf_pool_desc& pool, void* workspace,
                      size_t workspace_bytes) {
    wf_status s = check_pool(pool);
    if (s != WF_OK) return s;
    if (B < 0 || num_q_heads < 1 || max_blocks_per_seq < 1 || max_seq_len < 1) return WF_ERR_INVALID_ARG;
    if (num_q_heads % pool.num_kv_heads != 0) return WF_ERR_INVALID_ARG;
    if (num_q_heads / pool.num_kv_heads > 8) return WF_ERR_UNSUPPORTED;
    if ((int64_t)max_seq_len > (int64_t)max_blocks_per_seq * pool.block_size) return WF_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return WF_ERR_INVALID_ARG;
    if (B == 0) return WF_OK;
    if (!out || !q || !k_pool || !v_pool || !block_tables || !seq_lens) return WF_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) ||
        (reinterpret_cast<uintptr_t>(block_tables) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
        return WF_ERR_INVALID_ARG;
    const size_t need = wf::decode_workspace_bytes(B, num_q_heads, max_seq_len, pool);
    if (need == 0) return WF_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return WF_ERR_WORKSPACE;
    return WF_OK;
}

}  // namespace

extern "C" {

wf_status wf_paged_decode(void* out, const void* q, const void* k_pool, const void* v_pool,
                          const int32_t* block_tables, int32_t max_blocks_per_seq,
                          const int32_t* seq_lens, int32_t B, int32_t max_seq_len,
                          int32_t num_q_heads, float scale, wf_pool_desc pool,
                          void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                          cudaStream_t stream) {
    const wf_status s = decode_args(out, q, k_pool, v_pool, block_tables, max_blocks_per_seq, seq_lens, B,
                                    max_seq_len, num_q_heads, scale, pool, workspace, workspace_bytes);
    if (s != WF_OK || B == 0) return s;
    return from_cuda(wf::launch_paged_decode(out, q, k_pool, v_pool, block_tables, max_blocks_per_seq,
                                             seq_lens, B, max_seq_len, num_q_heads, scale, pool,
                                             workspace, dev_status, stream));
}

}  // extern "C"

namespace {

// wf_paged_prefill's argument rules (WF_OK also for calls that launch nothing).
wf_status prefill_args(void* out, const void* q, const void* k_pool, const void* v_pool,
                       const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                       const int32_t* cu_q_lens, int32_t B, int32_t total_q, int32_t max_q_len, int32_t max_seq_len,
                       int32_t num_q_heads, float scale, const wf_pool_desc& pool) {
    wf_status s = check_pool(pool);
    if (s != WF_OK) return s;
    if (pool.dtype != WF_DTYPE_BF16) return WF_ERR_UNSUPPORTED;
    if (B < 0 || total_q < 0 || max_q_len < 0 || num_q_heads < 1 || max_blocks_per_seq < 1 ||
        max_seq_len < 0)
        return WF_ERR_INVALID_ARG;
    if (num_q_heads % pool.num_kv_heads != 0) return WF_ERR_INVALID_ARG;
    if ((int64_t)max_seq_len > (int64_t)max_blocks_per_seq * pool.block_size) return WF_ERR_INVALID_ARG;
    if (max_q_len > max_seq_len) return WF_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return WF_ERR_INVALID_ARG;
    if (B == 0 || total_q == 0 || max_q_len == 0) return WF_OK;
    if (!out || !q || !k_pool || !v_pool || !block_tables || !seq_lens || !cu_q_lens)
        return WF_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) ||
        (reinterpret_cast<uintptr_t>(block_tables) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u) ||
        (reinterpret_cast<uintptr_t>(cu_q_lens) & 3u))
        return WF_ERR_INVALID_ARG;
    return WF_OK;
}

bool prefill_launches(int32_t B, int32_t total_q, int32_t max_q_len) { return B > 0 && total_q > 0 && max_q_len > 0; }

}  // namespace

extern "C" {

wf_status wf_paged_prefill(void* out, const void* q, const void* k_pool, const void* v_pool,
                           const int32_t* block_tables, int32_t max_blocks_per_seq,
                           const int32_t* seq_lens, const int32_t* cu_q_lens, int32_t B,
                           int32_t total_q, int32_t max_q_len, int32_t max_seq_len,
                           int32_t num_q_heads, float scale, wf_pool_desc pool,
                           uint32_t* dev_status, cudaStream_t stream) {
    const wf_status s = prefill_args(out, q, k_pool, v_pool, block_tables, max_blocks_per_seq, seq_lens, cu_q_lens,
                                     B, total_q, max_q_len, max_seq_len, num_q_heads, scale, pool);
    if (s != WF_OK || !prefill_launches(B, total_q, max_q_len)) return s;
    return from_cuda(wf::launch_paged_prefill(out, q, k_pool, v_pool, block_tables, max_blocks_per_seq,
                                              seq_lens, cu_q_lens, B, total_q, max_q_len, max_seq_len,
                                              num_q_heads, scale, pool, dev_status, stream));
}

wf_status wf_paged_prefill_decode(void* pf_out, const void* pf_q, const int32_t* pf_block_tables,
                                  int32_t pf_max_blocks_per_seq, const int32_t* pf_seq_lens,
                                  const int32_t* cu_q_lens, int32_t pf_B, int32_t total_q, int32_t max_q_len,
                                  int32_t pf_max_seq_len, void* dec_out, const void* dec_q,
                                  const int32_t* dec_block_tables, int32_t dec_max_blocks_per_seq,
                                  const int32_t* dec_seq_lens, int32_t dec_B, int32_t dec_max_seq_len,
                                  const void* k_pool, const void* v_pool, int32_t num_q_heads, float scale,
                                  wf_pool_desc pool, void* workspace, size_t workspace_bytes,
                                  uint32_t* dev_status, cudaStream_t stream) {
    wf_status s = prefill_args(pf_out, pf_q, k_pool, v_pool, pf_block_tables, pf_max_blocks_per_seq, pf_seq_lens,
                               cu_q_lens, pf_B, total_q, max_q_len, pf_max_seq_len, num_q_heads, scale, pool);
    if (s != WF_OK) return s;
    s = decode_args(dec_out, dec_q, k_pool, v_pool, dec_block_tables, dec_max_blocks_per_seq, dec_seq_lens, dec_B,
                    dec_max_seq_len, num_q_heads, scale, pool, workspace, workspace_bytes);
    if (s != WF_OK) return s;
    const bool pf = prefill_launches(pf_B, total_q, max_q_len);
    if (!pf && dec_B == 0) return WF_OK;
    return from_cuda(wf::launch_paged_prefill_decode(
        pf_out, pf_q, pf_block_tables, pf_max_blocks_per_seq, pf_seq_lens, cu_q_lens, pf ? pf_B : 0, total_q,
        max_q_len, pf_max_seq_len, dec_out, dec_q, dec_block_tables, dec_max_blocks_per_seq, dec_seq_lens, dec_B,
        dec_max_seq_len, k_pool, v_pool, num_q_heads, scale, pool, workspace, dev_status, stream));
}

size_t wf_paged_tree_decode_workspace_size(int32_t B, int32_t num_q_heads, int32_t max_q_len, int32_t max_seq_len,
                                           wf_pool_desc pool) {
    if (check_pool(pool) != WF_OK || num_q_heads < 1) return 0;
    return wf::tree_workspace_bytes(B, num_q_heads, max_q_len, max_seq_len, pool);
}

wf_status wf_paged_tree_decode(void* out, const void* q, const void* k_pool, const void* v_pool,
                               const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                               const int32_t* cu_q_lens, const uint32_t* tree_mask, int32_t mask_words, int32_t B,
                               int32_t total_q, int32_t max_q_len, int32_t max_seq_len, int32_t num_q_heads,
                               float scale, wf_pool_desc pool, void* workspace, size_t workspace_bytes,
                               uint32_t* dev_status, cudaStream_t stream) {
    wf_status s = check_pool(pool);
    if (s != WF_OK) return s;
    if (B < 0 || total_q < 0 || max_q_len < 0 || max_seq_len < 0 || num_q_heads < 1 || max_blocks_per_seq < 1)
        return WF_ERR_INVALID_ARG;
    if (num_q_heads % pool.num_kv_heads != 0) return WF_ERR_INVALID_ARG;
    if (num_q_heads / pool.num_kv_heads > 8) return WF_ERR_UNSUPPORTED;
    if ((int64_t)max_seq_len > (int64_t)max_blocks_per_seq * pool.block_size || max_q_len > max_seq_len)
        return WF_ERR_INVALID_ARG;
    // positions are 32-bit and looked at a tile past the end
    if (max_seq_len >= INT32_MAX - 1023) return WF_ERR_INVALID_ARG;
    if (mask_words < 0 || (int64_t)mask_words * 32 < max_q_len) return WF_ERR_INVALID_ARG;
    // the kernels take scores to powers of two: an infinite factor would make a score of 0 NaN
    if (!std::isfinite(scale * 1.4426950408889634f)) return WF_ERR_INVALID_ARG;
    if (B == 0 || total_q == 0 || max_q_len == 0) return WF_OK;
    if (!out || !q || !k_pool || !v_pool || !block_tables || !seq_lens || !cu_q_lens || !tree_mask)
        return WF_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool)) return WF_ERR_INVALID_ARG;
    for (const void* p : {(const void*)block_tables, (const void*)seq_lens, (const void*)cu_q_lens,
                          (const void*)tree_mask})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return WF_ERR_INVALID_ARG;
    const size_t need = wf::tree_workspace_bytes(B, num_q_heads, max_q_len, max_seq_len, pool);
    if (need == 0) return WF_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return WF_ERR_WORKSPACE;
    const int64_t rows_bytes = (int64_t)total_q * num_q_heads * pool.head_dim * (pool.dtype == WF_DTYPE_F32 ? 4 : 2);
    if (overlap(out, rows_bytes, q, rows_bytes)) return WF_ERR_INVALID_ARG;
    const wf::TreeArgs a{out, q, k_pool, v_pool, block_tables, max_blocks_per_seq, seq_lens, cu_q_lens, tree_mask,
                         mask_words, B, total_q, max_q_len, max_seq_len, num_q_heads, scale, workspace};
    return from_cuda(wf::launch_paged_tree(a, pool, dev_status, stream));
}

size_t wf_paged_scored_attention_workspace_size(int32_t B, int32_t num_q_heads, int32_t total_q, int32_t max_q_len,
                                                int32_t max_seq_len, wf_pool_desc pool) {
    if (check_pool(pool) != WF_OK || num_q_heads < 1) return 0;
    return wf::scored_workspace_bytes(B, num_q_heads, total_q, max_q_len, max_seq_len, pool);
}

wf_status wf_paged_scored_attention(void* out, const void* q, const void* k_pool, const void* v_pool,
                                    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                    const int32_t* cu_q_lens, int32_t B, int32_t total_q, int32_t max_q_len,
                                    int32_t max_seq_len, int32_t num_q_heads, float scale, float cap, int32_t window,
                                    const float* slopes, const int32_t* row_ranges, wf_pool_desc pool, void* workspace,
                                    size_t workspace_bytes, uint32_t* dev_status, cudaStream_t stream) {
    wf_status s = check_pool(pool);
    if (s != WF_OK) return s;
    if (B < 0 || total_q < 0 || max_q_len < 0 || max_seq_len < 0 || num_q_heads < 1 || max_blocks_per_seq < 1 || window < 0)
        return WF_ERR_INVALID_ARG;
    if (num_q_heads % pool.num_kv_heads != 0) return WF_ERR_INVALID_ARG;
    if (num_q_heads / pool.num_kv_heads > 8) return WF_ERR_UNSUPPORTED;
    if ((int64_t)max_seq_len > (int64_t)max_blocks_per_seq * pool.block_size || max_q_len > max_seq_len)
        return WF_ERR_INVALID_ARG;
    // positions are 32-bit and looked at a tile past the end
    if (max_seq_len >= INT32_MAX - 1023) return WF_ERR_INVALID_ARG;
    // the kernels take scores to powers of two: an infinite factor would make a score of 0 NaN
    constexpr float kLog2e = 1.4426950408889634f;
    if (!std::isfinite(scale * kLog2e) || !(cap >= 0.f) || !std::isfinite(cap * kLog2e)) return WF_ERR_INVALID_ARG;
    if (cap > 0.f) {
        const double in = std::fabs((double)scale / (double)cap);
        if (!std::isfinite((float)(2.0 * kLog2e * in))) return WF_ERR_INVALID_ARG;
        // what is left of a score above this, or of its factor below that, is too little to tell scores apart by
        if (cap > 0x1p100f || (in > 0.0 && in < (double)FLT_MIN)) return WF_ERR_INVALID_ARG;
    }
    if (B == 0 || total_q == 0 || max_q_len == 0) return WF_OK;
    if (!out || !q || !k_pool || !v_pool || !block_tables || !seq_lens || !cu_q_lens) return WF_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool)) return WF_ERR_INVALID_ARG;
    for (const void* p : {(const void*)block_tables, (const void*)seq_lens, (const void*)cu_q_lens, (const void*)slopes})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return WF_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(row_ranges) & 7u) return WF_ERR_INVALID_ARG;
    const size_t need = wf::scored_workspace_bytes(B, num_q_heads, total_q, max_q_len, max_seq_len, pool);
    if (need == 0) return WF_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return WF_ERR_WORKSPACE;
    const int64_t rows_bytes = (int64_t)total_q * num_q_heads * pool.head_dim * (pool.dtype == WF_DTYPE_F32 ? 4 : 2);
    if (overlap(out, rows_bytes, q, rows_bytes)) return WF_ERR_INVALID_ARG;
    const wf::ScoredArgs a{out, q, k_pool, v_pool, block_tables, max_blocks_per_seq, seq_lens, cu_q_lens, row_ranges, slopes,
                           cap, window, B, total_q, max_q_len, max_seq_len, num_q_heads, scale, workspace};
    return from_cuda(wf::launch_paged_scored(a, pool, dev_status, stream));
}

wf_status wf_decode_worker(void* out, const void* q, int32_t num_rows, const void* k_pool, const void* v_pool,
                           const int32_t* block_tables, int32_t num_table_rows, int32_t max_blocks_per_seq,
                           int32_t num_q_heads, float scale, wf_pool_desc pool, const wf_decode_task* tasks,
                           int32_t task_capacity, wf_worker_mailbox* mailbox, int32_t num_workers,
                           uint64_t idle_timeout_ns, uint32_t* dev_status, cudaStream_t stream) {
    wf_status s = check_pool(pool);
    if (s != WF_OK) return s;
    if (pool.dtype == WF_DTYPE_FP8_E4M3) return WF_ERR_UNSUPPORTED;
    if (num_rows < 0 || num_table_rows < 0 || max_blocks_per_seq < 1 || num_q_heads < 1 || task_capacity < 0)
        return WF_ERR_INVALID_ARG;
    if (num_q_heads % pool.num_kv_heads != 0) return WF_ERR_INVALID_ARG;
    if (num_q_heads / pool.num_kv_heads > 8) return WF_ERR_UNSUPPORTED;
    if (num_workers < 1 || num_workers > 4096 || idle_timeout_ns == 0) return WF_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return WF_ERR_INVALID_ARG;
    if (!mailbox || (reinterpret_cast<uintptr_t>(mailbox) & 15u)) return WF_ERR_INVALID_ARG;
    if (task_capacity > 0 && (!tasks || (reinterpret_cast<uintptr_t>(tasks) & 15u))) return WF_ERR_INVALID_ARG;
    if (num_rows > 0 && (!out || !q || !aligned16(out) || !aligned16(q))) return WF_ERR_INVALID_ARG;
    if (!k_pool || !v_pool || !aligned16(k_pool) || !aligned16(v_pool)) return WF_ERR_INVALID_ARG;
    if (num_table_rows > 0 && (!block_tables || (reinterpret_cast<uintptr_t>(block_tables) & 3u)))
        return WF_ERR_INVALID_ARG;
    return from_cuda(wf::launch_decode_worker(out, q, num_rows, k_pool, v_pool, block_tables, num_table_rows,
                                              max_blocks_per_seq, num_q_heads, scale, pool, tasks, task_capacity,
                                              mailbox, num_workers, idle_timeout_ns, dev_status, stream));
}

int wf_paged_prefill_decode_fused(wf_pool_desc pool, int32_t num_q_heads) {
    if (check_pool(pool) != WF_OK || num_q_heads < 1) return 0;
    return wf::mixed_tc_supported(pool, num_q_heads) ? 1 : 0;
}

int wf_paged_decode_kernel(wf_pool_desc pool, int32_t num_q_heads) {
    if (check_pool(pool) != WF_OK || num_q_heads < 1) return WF_KERNEL_NONE;
    return wf::decode_kernel_kind(pool, num_q_heads);
}

int wf_paged_prefill_kernel(wf_pool_desc pool, int32_t num_q_heads) {
    if (check_pool(pool) != WF_OK || num_q_heads < 1) return WF_KERNEL_NONE;
    return wf::prefill_kernel_kind(pool, num_q_heads);
}

int wf_paged_tree_decode_kernel(wf_pool_desc pool, int32_t num_q_heads) {
    if (check_pool(pool) != WF_OK || num_q_heads < 1) return WF_KERNEL_NONE;
    return wf::tree_kernel_kind(pool, num_q_heads);
}

int wf_paged_prefill_persistent(wf_pool_desc pool, int32_t num_q_heads, int32_t B, int32_t max_q_len) {
    if (check_pool(pool) != WF_OK || num_q_heads < 1) return 0;
    if (wf::prefill_kernel_kind(pool, num_q_heads) != WF_KERNEL_TENSOR_CORES) return 0;
    return wf::prefill_tc_persistent(pool, num_q_heads, B, max_q_len) ? 1 : 0;
}

wf_status wf_device_status_fetch(uint32_t* dev_status, uint32_t* host_status, int clear,
                                 cudaStream_t stream) {
    if (!dev_status || !host_status) return WF_ERR_INVALID_ARG;
    cudaError_t e = cudaMemcpyAsync(host_status, dev_status, sizeof(uint32_t), cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess && clear) {
        e = cudaMemsetAsync(dev_status, 0, sizeof(uint32_t), stream);
        if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    }
    return from_cuda(e);
}

}  // extern "C"
