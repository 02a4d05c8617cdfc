// step_tables.cu -- a step's block tables, slots, positions and offsets from the requests'
// lengths (wf_build_step), and the blocks of shortened requests back to the free list
// (wf_trim_blocks), without the host.
//
// Request b holds len_b tokens in h_b = ceil(len_b / P) blocks and gets n_b more, for which
// it needs r_b = ceil((len_b + n_b) / P) - h_b blocks.  With the exclusive sums
// t_b = sum_{i<b} n_i and s_b = sum_{i<b} r_i its i-th new token is row t_b + i of the step at
// position p = len_b + i, and its k-th new block is free[F - 1 - (s_b + k)] of F free ones: the
// list is a stack, taken request by request, as the host's block manager does.
// The trim puts the blocks behind ceil(kept_b / P) back so that the next step takes them in the
// same order.
//
// Bound: latency.  The bytes are 12 a token and a few a request; what the call takes is a launch
// and three dependent rounds of loads (lengths; tail block or free list; the same again for a
// token): a step of 231 decodes 4.4 us, one of 8 prompts and 120 others (8300 rows) 6.7, a trim of one
// request 2.6, of 231 (14 of them whole) 4.6.  One cluster does all of it: every CTA sums over all requests by itself (that takes
// less than handing the sums on), and a cluster barrier stands between the last read of the
// lengths and counts and the first write, so that both may be updated in place.
#include <cooperative_groups.h>

#include "wf_internal.h"

namespace wf {

namespace {

namespace cg = cooperative_groups;

constexpr int kStepThreads = 512, kStepWarps = kStepThreads / 32;
constexpr int kStepCluster = 8;        // CTAs at most: the portable size of a cluster
// Entries (rows of the step, or blocks to look at) that a CTA of its own pays for: with less for
// each the barrier and the sums repeated cost more than the entries.
constexpr int64_t kStepPerCta = 1024;

// Exclusive sums of two counts over the requests, this thread's requests being [b0, b1).
// `totals` in shared memory receives both sums.
struct TwoSums {
    int64_t a, b;
};

__device__ __forceinline__ TwoSums exclusive(TwoSums mine, TwoSums* warps, TwoSums* totals) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    TwoSums incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl.a, o), y = __shfl_up_sync(0xffffffffu, incl.b, o);
        if (lane >= o) {
            incl.a += x;
            incl.b += y;
        }
    }
    if (lane == 31) warps[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        TwoSums w = lane < kStepWarps ? warps[lane] : TwoSums{0, 0};
        const TwoSums own = w;
#pragma unroll
        for (int o = 1; o < kStepWarps; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, w.a, o), y = __shfl_up_sync(0xffffffffu, w.b, o);
            if (lane >= o) {
                w.a += x;
                w.b += y;
            }
        }
        if (lane < kStepWarps) warps[lane] = TwoSums{w.a - own.a, w.b - own.b};
        if (lane == kStepWarps - 1) *totals = w;
    }
    __syncthreads();
    return TwoSums{warps[warp].a + incl.a - mine.a, warps[warp].b + incl.b - mine.b};
}

// The last request whose sum is at most x: sums[0 .. B] do not decrease, sums[0] = 0 <= x < sums[B].
__device__ __forceinline__ int request_of(const int32_t* sums, int B, int x) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

struct BuildParams {
    int32_t* block_tables;
    const int32_t *seq_lens, *new_lens, *free_blocks, *num_free, *depths;
    int32_t *new_seq_lens, *new_num_free, *cu_q_lens, *positions;
    int64_t* slot_mapping;
    uint32_t* dev_status;
    int32_t M, B, max_tokens, N, P;
};

__device__ __forceinline__ int blocks_of(int tokens, int P) { return tokens / P + (tokens % P != 0); }

__global__ void __launch_bounds__(kStepThreads) build_step_kernel(const BuildParams p) {
    extern __shared__ int32_t sums[];      // [B + 1] rows before a request, [B + 1] blocks before it, [B] lengths
    __shared__ TwoSums warps[kStepWarps], totals;
    __shared__ uint32_t s_bad;
    int32_t *rows = sums, *taken = rows + p.B + 1, *lens = taken + p.B + 1;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int tid = threadIdx.x;
    if (tid == 0) s_bad = 0;
    const int F = __ldcg(p.num_free);
    const int per = (p.B + kStepThreads - 1) / kStepThreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    const int64_t room = min((int64_t)p.M * p.P, (int64_t)INT32_MAX);
    uint32_t bad = F < 0 || F > p.N ? WF_DEV_BAD_BLOCK : 0u;
    TwoSums mine{0, 0};
    for (int b = b0; b < b1; ++b) {
        const int len = __ldcg(p.seq_lens + b), n = __ldcg(p.new_lens + b);
        lens[b] = len;
        if (len < 0 || n < 0 || (int64_t)len + n > room) {
            bad |= WF_DEV_BAD_SEQLEN;
            rows[b] = taken[b] = 0;
            continue;
        }
        const int held = blocks_of(len, p.P), more = blocks_of(len + n, p.P) - held;
        // a partly filled block takes the first new tokens
        if (n > 0 && len % p.P != 0 && (unsigned)p.block_tables[(int64_t)b * p.M + held - 1] >= (unsigned)p.N)
            bad |= WF_DEV_BAD_BLOCK;
        rows[b] = n;
        taken[b] = more;
        mine.a += n;
        mine.b += more;
    }
    TwoSums at = exclusive(mine, warps, &totals);
    const int64_t T = totals.a, R = totals.b;
    if (T > p.max_tokens) bad |= WF_DEV_BAD_SEQLEN;
    if (R > F) bad |= WF_DEV_NO_BLOCKS;
    for (int b = b0; b < b1; ++b) {
        const int n = rows[b], more = taken[b];
        rows[b] = (int32_t)at.a;           // wraps only in a step that is refused
        taken[b] = (int32_t)at.b;
        at.a += n;
        at.b += more;
    }
    // the blocks that are taken, a part of them by each CTA
    if (R <= F && F <= p.N)
        for (int64_t j = rank * kStepThreads + tid; j < R; j += (int64_t)ctas * kStepThreads)
            if ((unsigned)__ldcg(p.free_blocks + F - 1 - j) >= (unsigned)p.N) bad |= WF_DEV_BAD_BLOCK;
    bad = __reduce_or_sync(0xffffffffu, bad);
    if (bad && (tid & 31) == 0) atomicOr(&s_bad, bad);
    if (tid == 0) {
        rows[p.B] = (int32_t)min(T, (int64_t)INT32_MAX);
        taken[p.B] = (int32_t)min(R, (int64_t)INT32_MAX);
    }
    // all lengths and counts are read, and every CTA's findings are there
    if (ctas > 1)
        cluster.sync();
    else
        __syncthreads();
    bad = 0;
    for (int c = 0; c < ctas; ++c) bad |= *(volatile uint32_t*)cluster.map_shared_rank(&s_bad, c);
    const bool good = bad == 0;
    if (rank == 0) {
        if (tid == 0) {
            if (!good) report(p.dev_status, bad);
            *p.new_num_free = good ? F - (int)R : F;
            p.cu_q_lens[p.B] = good ? (int)T : 0;
        }
        for (int b = tid; b < p.B; b += kStepThreads) {
            p.cu_q_lens[b] = good ? rows[b] : 0;
            p.new_seq_lens[b] = good ? lens[b] + (rows[b + 1] - rows[b]) : lens[b];
        }
    }
    const int first = rank * kStepThreads + tid, step = ctas * kStepThreads;
    if (good) {
        for (int j = first; j < (int)R; j += step) {
            const int b = request_of(taken, p.B, j);
            p.block_tables[(int64_t)b * p.M + blocks_of(lens[b], p.P) + j - taken[b]] = __ldcg(p.free_blocks + F - 1 - j);
        }
    }
    for (int64_t row = first; row < p.max_tokens; row += step) {
        int64_t slot = -1;
        int position = 0;
        if (good && row < T) {
            const int b = request_of(rows, p.B, (int)row);
            const int at_b = lens[b] + (int)row - rows[b];
            const int k = at_b / p.P, held = blocks_of(lens[b], p.P);
            const int id = k < held ? p.block_tables[(int64_t)b * p.M + k]
                                    : __ldcg(p.free_blocks + F - 1 - (taken[b] + k - held));
            slot = (int64_t)id * p.P + (at_b - k * p.P);
            position = p.depths != nullptr ? lens[b] + __ldg(p.depths + row) : at_b;
        }
        p.slot_mapping[row] = slot;
        p.positions[row] = position;
    }
    if (ctas > 1) cluster.sync();          // no CTA's shared memory goes while another reads its findings
}

struct TrimParams {
    const int32_t *block_tables, *seq_lens, *kept_lens, *num_free;
    int32_t *free_blocks, *new_num_free;
    uint32_t* dev_status;
    int32_t M, B, N, P;
};

__global__ void __launch_bounds__(kStepThreads) trim_blocks_kernel(const TrimParams p) {
    extern __shared__ int32_t sums[];      // [B + 1] blocks before a request, [B] its first block that goes
    __shared__ TwoSums warps[kStepWarps], totals;
    __shared__ uint32_t s_bad;
    int32_t *back = sums, *from = back + p.B + 1;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int tid = threadIdx.x;
    if (tid == 0) s_bad = 0;
    const int F = __ldcg(p.num_free);
    const int per = (p.B + kStepThreads - 1) / kStepThreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    const int64_t room = min((int64_t)p.M * p.P, (int64_t)INT32_MAX);
    uint32_t bad = F < 0 || F > p.N ? WF_DEV_BAD_BLOCK : 0u;
    TwoSums mine{0, 0};
    for (int b = b0; b < b1; ++b) {
        const int len = __ldcg(p.seq_lens + b), kept = __ldcg(p.kept_lens + b);
        back[b] = from[b] = 0;
        if (kept < 0 || kept > len || len > room) {
            bad |= WF_DEV_BAD_SEQLEN;
            continue;
        }
        from[b] = blocks_of(kept, p.P);
        back[b] = blocks_of(len, p.P) - from[b];
        mine.a += back[b];
    }
    TwoSums at = exclusive(mine, warps, &totals);
    const int64_t R = totals.a;
    if (F + R > p.N) bad |= WF_DEV_BAD_BLOCK;   // more than there are: some are held twice
    for (int b = b0; b < b1; ++b) {
        const int n = back[b];
        back[b] = (int32_t)at.a;
        at.a += n;
    }
    if (tid == 0) back[p.B] = (int32_t)min(R, (int64_t)INT32_MAX);
    __syncthreads();
    const auto block = [&](int j) {
        const int b = request_of(back, p.B, j);
        return __ldg(p.block_tables + (int64_t)b * p.M + from[b] + j - back[b]);
    };
    const int first = rank * kStepThreads + tid, step = ctas * kStepThreads;
    if (F >= 0 && F + R <= p.N)
        for (int j = first; j < (int)R; j += step)
            if ((unsigned)block(j) >= (unsigned)p.N) bad |= WF_DEV_BAD_BLOCK;
    bad = __reduce_or_sync(0xffffffffu, bad);
    if (bad && (tid & 31) == 0) atomicOr(&s_bad, bad);
    if (ctas > 1)
        cluster.sync();
    else
        __syncthreads();
    bad = 0;
    for (int c = 0; c < ctas; ++c) bad |= *(volatile uint32_t*)cluster.map_shared_rank(&s_bad, c);
    if (bad == 0)
        for (int j = first; j < (int)R; j += step) p.free_blocks[F + (int)R - 1 - j] = block(j);
    if (rank == 0 && tid == 0) {
        if (bad) report(p.dev_status, bad);
        *p.new_num_free = bad ? F : F + (int)R;
    }
    if (ctas > 1) cluster.sync();
}

template <typename Params>
cudaError_t launch_step(void (*kern)(const Params), const Params& p, int64_t entries, int smem, cudaStream_t stream) {
    cudaError_t err = allow_dynamic_smem((const void*)kern, smem);
    if (err != cudaSuccess) return err;
    int ctas = 1;
    while (ctas < kStepCluster && ctas * kStepPerCta < entries) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kStepThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_build_step(const BuildArgs& a, uint32_t* dev_status, cudaStream_t stream) {
    const BuildParams p{a.block_tables, a.seq_lens,     a.new_lens,  a.free_blocks, a.num_free,
                        a.depths,       a.new_seq_lens, a.new_num_free, a.cu_q_lens, a.positions,
                        a.slot_mapping, dev_status,     a.max_blocks_per_seq, a.B, a.max_tokens,
                        a.num_blocks,   a.block_size};
    return launch_step(build_step_kernel, p, (int64_t)a.max_tokens, (3 * a.B + 2) * (int)sizeof(int32_t), stream);
}

cudaError_t launch_trim_blocks(const TrimArgs& a, uint32_t* dev_status, cudaStream_t stream) {
    const TrimParams p{a.block_tables, a.seq_lens, a.kept_lens, a.num_free,   a.free_blocks,
                       a.new_num_free, dev_status, a.max_blocks_per_seq, a.B, a.num_blocks, a.block_size};
    // What goes back is known on the device only: taken as 16 blocks a request (finished ones among them).
    return launch_step(trim_blocks_kernel, p, 16 * (int64_t)a.B, (2 * a.B + 1) * (int)sizeof(int32_t), stream);
}

}  // namespace wf
