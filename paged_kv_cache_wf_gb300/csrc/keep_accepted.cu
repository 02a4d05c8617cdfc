// keep_accepted.cu -- the accepted path's K and V rows move to the front of each
// request's drafts, in both pools.
//
// Row of draft a_j (a strictly increasing) goes to position c + j.  Because a is
// increasing, a_j >= j: a thread that owns one 16-byte column of the rows and goes
// through j in order never overwrites a source it still has to read (targets 0 .. j
// lie below every later source a_j' > a_j >= j), so the move needs no second buffer.
// It reads kBatch rows before it writes them, to have that many loads in flight.
//
// Bound: latency (the path, a table entry and one row round trip, each dependent on the
// one before); the bytes are two rows read and written per kept draft.  One CTA per request:
// its threads first resolve the path to slots in shared memory, then own the columns of
// both pools' rows.  One request 2.7 us, of which a launch alone is about 2; 231 requests
// with up to 9 accepted of 61 drafts (128-wide bf16, 8 heads) 4.4 us, their 9.3 MB 1.4 us
// at the copy peak.
#include "wf_internal.h"

namespace wf {

namespace {

constexpr int kPathChunk = 64;   // path entries resolved at a time
constexpr int kBatch = 8;

__global__ void __launch_bounds__(256) keep_accepted_kernel(
    uint4* k_pool, uint4* v_pool, const int32_t* __restrict__ block_tables, int32_t M,
    const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ cu_q_lens, const int32_t* __restrict__ accepted,
    int32_t A, const int32_t* __restrict__ num_accepted, int32_t* new_seq_lens, int32_t N, int32_t P, int row_chunks,
    uint32_t* dev_status) {
    __shared__ int64_t s_src[kPathChunk], s_dst[kPathChunk];
    const int b = blockIdx.x;
    const int q0 = __ldg(cu_q_lens + b), n = __ldg(cu_q_lens + b + 1) - q0;
    const int len = __ldg(seq_lens + b);
    const int num = __ldg(num_accepted + b);
    if (q0 < 0 || n < 0 || len < n || (int64_t)len > (int64_t)M * P) {
        if (threadIdx.x == 0) report(dev_status, WF_DEV_BAD_SEQLEN);
        return;
    }
    const int c = len - n;
    const int32_t* path = accepted + (int64_t)b * A;
    bool bad = num < 0 || num > n || num > A;
    if (!bad) {
        for (int j = threadIdx.x; j < num; j += blockDim.x) {
            const int a = __ldg(path + j);
            const int before = j > 0 ? __ldg(path + j - 1) : -1;
            bad |= a <= before || a >= n;
        }
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) report(dev_status, WF_DEV_BAD_NODE);
        return;
    }
    if (threadIdx.x == 0 && new_seq_lens != nullptr) new_seq_lens[b] = c + num;
    const int32_t* table = block_tables + (int64_t)b * M;
    for (int j0 = 0; j0 < num; j0 += kPathChunk) {
        const int cnt = min(kPathChunk, num - j0);
        if (j0 > 0) __syncthreads();
        if (threadIdx.x < cnt) {
            const int j = j0 + threadIdx.x;
            const int from = c + __ldg(path + j), to = c + j;
            const int fb = __ldg(table + from / P), tb = __ldg(table + to / P);
            const bool in = (unsigned)fb < (unsigned)N && (unsigned)tb < (unsigned)N;
            if (!in) report(dev_status, WF_DEV_BAD_BLOCK);
            // a row that is in place already, or not in the pool, does not move
            s_src[threadIdx.x] = in && from != to ? (int64_t)fb * P + from % P : -1;
            s_dst[threadIdx.x] = (int64_t)tb * P + to % P;
        }
        __syncthreads();
        for (int col = threadIdx.x; col < 2 * row_chunks; col += blockDim.x) {
            uint4* pool = col < row_chunks ? k_pool + col : v_pool + (col - row_chunks);
            for (int u0 = 0; u0 < cnt; u0 += kBatch) {
                uint4 r[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    if (u0 + u < cnt && s_src[u0 + u] >= 0) r[u] = __ldcg(pool + s_src[u0 + u] * row_chunks);
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    if (u0 + u < cnt && s_src[u0 + u] >= 0) st_global_v4(pool + s_dst[u0 + u] * row_chunks, r[u]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_keep_accepted(void* k_pool, void* v_pool, const int32_t* block_tables, int32_t max_blocks_per_seq,
                                 const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* accepted,
                                 int32_t max_accepted, const int32_t* num_accepted, int32_t* new_seq_lens, int32_t B,
                                 const wf_pool_desc& pool, uint32_t* dev_status, cudaStream_t stream) {
    const int row_chunks = (int)((int64_t)pool.num_kv_heads * pool.head_dim * dtype_bytes(pool.dtype) / 16);
    keep_accepted_kernel<<<B, 256, 0, stream>>>((uint4*)k_pool, (uint4*)v_pool, block_tables, max_blocks_per_seq,
                                                seq_lens, cu_q_lens, accepted, max_accepted, num_accepted,
                                                new_seq_lens, pool.num_blocks, pool.block_size, row_chunks,
                                                dev_status);
    return cudaGetLastError();
}

}  // namespace wf
