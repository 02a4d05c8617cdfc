// verify_drafts.cu -- which drafted tokens are kept, and the token after them, from the
// target's probabilities and given random numbers.
//
// A request's nodes form a tree with its newest token as node 0; row u of `target` is the
// target's distribution p_u of the token after node u, row u of `draft` the distribution q_u
// that u's children were drawn from.  From the root on, the children of the path's last node u
// are tried in order.  With k rejected, what is left of p_u is, up to its sum,
//     drawn children:  w_k(x) = max(p_u(x) - c_k q_u(x), 0),  c_0 = 0, c_{k+1} = c_k + N_k,
//                      N_0 = 1, N_k = sum_x w_k(x)
// (the usual step p' = max(p' / N' - q, 0) with its divisions taken out: each turns into a
// factor of both sides), and child i with token x is kept when
//     coin_i q_u(x) N_k < w_k(x).
// Fixed candidates (no `draft`) are kept when coin_i N_k < w_k(x), where w_k is p_u without the
// rejected tokens and N_k = 1 - their probabilities.  When no child is kept (or the path is
// full) the next token is the first x whose running sum of w passes pick_b times the whole sum.
//
// Numbers are compared with borders that they may lie next to, so sums are exact to about 2^-46:
// w is formed as a pair of fp32 numbers (products and differences with their rounding errors), a
// lane adds pairs with their errors, and lanes' sums are added in fp64.  (fp64 throughout would be
// the bound: this GPU has a 64th of its fp32 rate for it.)
//
// Bound: HBM, one or two rows of the vocabulary a request.  A cluster of 8 CTAs takes a request;
// every CTA walks the tree by itself on the gathered p_u(x), q_u(x) of all nodes and reads an
// eighth of a row where a sum is needed, which is once for a chain: the sums that a rejection's
// remainder needs are the running sums of the next token too, up to the 512 or so tokens of the
// one warp that holds it, which looks at them again.
#include <cooperative_groups.h>

#include "wf_internal.h"

namespace wf {

namespace {

namespace cg = cooperative_groups;

constexpr int kVerifyThreads = 512, kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyCtas = 8;                              // of a cluster
constexpr int kSlices = kVerifyCtas * kVerifyWarps;         // a row's parts, a warp each
constexpr int kStep = 128;                                  // tokens a warp reads at once
constexpr int kAhead = 4;                                   // such reads in flight

struct VerifyParams {
    int32_t *accepted, *num_accepted, *next_tokens;
    const void *target, *draft;
    int64_t target_stride, draft_stride;
    const int32_t *tokens, *parents, *cu_q_lens;
    const float *coins, *picks;
    uint32_t* dev_status;
    int32_t vocab, max_accepted, total, max_q_len;
    int32_t slice;      // tokens of a warp: a multiple of kStep
};

// x + y as a rounded sum and its error.
__device__ __forceinline__ void two_sum(float x, float y, float& s, float& e) {
    s = __fadd_rn(x, y);
    const float b = __fsub_rn(s, x);
    e = __fadd_rn(__fsub_rn(x, __fsub_rn(s, b)), __fsub_rn(y, b));
}

// max(p - (ch + cl) q, 0) as hi + lo; NaN and what is below 0 count as 0.
template <bool DRAWN>
__device__ __forceinline__ void weight(float p, float q, float ch, float cl, float& hi, float& lo) {
    if constexpr (DRAWN) {
        q = fmaxf(q, 0.f);
        const float t = __fmul_rn(ch, q);
        const float te = __fmaf_rn(ch, q, -t);
        float d, e;
        two_sum(p, -t, d, e);
        const float r = __fsub_rn(__fsub_rn(e, te), __fmul_rn(cl, q));
        two_sum(d, r, hi, lo);
    } else {
        hi = p;
        lo = 0.f;
    }
    if (!(hi > 0.f)) hi = lo = 0.f;
}

template <typename E>
__device__ __forceinline__ float element(const void* row, int64_t i) {
    if constexpr (E::kBytes == 4)
        return __ldg(static_cast<const float*>(row) + i);
    else
        return __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(row) + i));
}

// Four tokens from `i` on (those past the vocabulary 0).
template <typename E, bool VEC>
__device__ __forceinline__ void four(const void* row, int i, int vocab, float (&f)[4]) {
    if (VEC && i + 4 <= vocab) {
        if constexpr (E::kBytes == 4) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(row) + i));
            f[0] = x.x;
            f[1] = x.y;
            f[2] = x.z;
            f[3] = x.w;
        } else {
            const uint2 x = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(row) + i));
            const float2 a = bf16x2_to_float2(x.x), b = bf16x2_to_float2(x.y);
            f[0] = a.x;
            f[1] = a.y;
            f[2] = b.x;
            f[3] = b.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = i + e < vocab ? element<E>(row, i + e) : 0.f;
    }
}

struct Gone {        // tokens whose weight is 0: rejected fixed candidates
    const int32_t* token;
    int n;
    __device__ __forceinline__ bool has(int x) const {
        for (int k = 0; k < n; ++k)
            if (token[k] == x) return true;
        return false;
    }
};

// This lane's part of the sum of w over a warp's slice.
template <typename E, bool DRAWN, bool VEC>
__device__ __forceinline__ double slice_sum(const void* p, const void* q, int first, int last, int vocab, float ch,
                                            float cl, const Gone& gone) {
    const int lane = threadIdx.x & 31;
    float sh = 0.f, sl = 0.f;
    const auto add = [&](float hi, float lo) {
        float s, e;
        two_sum(sh, hi, s, e);
        sh = s;
        sl += e + lo;
    };
#pragma unroll 1
    for (int i0 = first; i0 < last; i0 += kAhead * kStep) {
        float a[kAhead][4], b[kAhead][4];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            // without vectors a warp's read is 32 tokens side by side: any order will do for a sum
            const int i = i0 + u * kStep;
            if constexpr (VEC) {
                const int at = i < last ? i + 4 * lane : vocab;
                four<E, VEC>(p, at, vocab, a[u]);
                if constexpr (DRAWN) four<E, VEC>(q, at, vocab, b[u]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int at = i + 32 * e + lane;
                    const bool in = i < last && at < vocab;
                    a[u][e] = in ? element<E>(p, at) : 0.f;
                    if constexpr (DRAWN) b[u][e] = in ? element<E>(q, at) : 0.f;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float hi, lo;
                weight<DRAWN>(a[u][e], DRAWN ? b[u][e] : 0.f, ch, cl, hi, lo);
                if (!DRAWN && gone.n > 0 && gone.has(VEC ? i0 + u * kStep + 4 * lane + e : i0 + u * kStep + 32 * e + lane))
                    hi = lo = 0.f;
                add(hi, lo);
            }
    }
    return (double)sh + (double)sl;
}

template <typename E, bool DRAWN>
__global__ void __launch_bounds__(kVerifyThreads) verify_drafts_kernel(const VerifyParams p) {
    extern __shared__ unsigned char smem[];
    __shared__ double s_part[kVerifyWarps];     // this CTA's slices, read by the whole cluster
    __shared__ double s_all[kSlices];           // all slices of the row
    __shared__ int s_walk[4], s_owner;
    __shared__ double s_c, s_total, s_before;
    float* pv = reinterpret_cast<float*>(smem);            // p_parent(token) of each node
    float* qv = pv + p.max_q_len;
    float* coin = qv + p.max_q_len;
    int32_t* token = reinterpret_cast<int32_t*>(coin + p.max_q_len);
    int32_t* parent = token + p.max_q_len;
    int32_t* gone_list = parent + p.max_q_len;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank();
    const int b = blockIdx.x / kVerifyCtas;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int q0 = __ldg(p.cu_q_lens + b), n = __ldg(p.cu_q_lens + b + 1) - q0;
    const float pick = __ldg(p.picks + b);
    int32_t* path = p.accepted + (int64_t)b * p.max_accepted;
    // all CTAs of a cluster come to the same of this and of the next check, so they leave together
    if (q0 < 0 || n < 0 || n > p.max_q_len || (int64_t)q0 + n > p.total) {
        if (rank == 0 && tid == 0) report(p.dev_status, WF_DEV_BAD_SEQLEN);
        return;
    }
    const size_t tstep = (size_t)p.target_stride * E::kBytes, dstep = (size_t)p.draft_stride * E::kBytes;
    const char* target = static_cast<const char*>(p.target) + q0 * tstep;
    const char* draft = DRAWN ? static_cast<const char*>(p.draft) + q0 * dstep : nullptr;
    if (!(pick >= 0.f && pick < 1.f)) {
        if (rank == 0 && tid == 0) report(p.dev_status, WF_DEV_BAD_PROBS);
        return;
    }
    bool bad = false;
    for (int i = tid; i < n; i += kVerifyThreads) {
        const int up = i == 0 ? -1 : p.parents != nullptr ? __ldg(p.parents + q0 + i) : i - 1;
        const int x = __ldg(p.tokens + q0 + i);
        parent[i] = up;
        token[i] = x;
        coin[i] = __ldg(p.coins + q0 + i);
        if (i > 0) {
            const bool ok = up >= 0 && up < i && (unsigned)x < (unsigned)p.vocab;
            bad |= !ok;
            pv[i] = ok ? fmaxf(element<E>(target + up * tstep, x), 0.f) : 0.f;
            if constexpr (DRAWN) qv[i] = ok ? fmaxf(element<E>(draft + up * dstep, x), 0.f) : 0.f;
        }
    }
    if (__syncthreads_or(bad)) {
        if (rank == 0 && tid == 0) report(p.dev_status, WF_DEV_BAD_NODE);
        return;
    }
    const auto fill = [&](int from) {           // the rest of the path's row
        if (rank == 0)
            for (int j = from + tid; j < p.max_accepted; j += kVerifyThreads) path[j] = -1;
    };
    if (n == 0) {
        fill(0);
        if (rank == 0 && tid == 0) {
            p.num_accepted[b] = 0;
            p.next_tokens[b] = -1;
        }
        return;
    }
    // Warp 0 walks; what it hands over: 0 a sum to form (N_k) and more children to try, 1 the end
    // of the path.  here, depth, the last child tried, c and N live in its registers.
    int here = 0, depth = 1, tried = 0, ngone = 0;
    double c = 0.0, whole = 1.0;
    if (rank == 0 && tid == 0) path[0] = 0;
    for (;;) {
        if (warp == 0) {
            int mode = 1;
            const bool full = depth >= p.max_accepted;
            for (int i = tried + 1; !full; ) {
                // the next child of `here` from node i on
                int child = -1;
                for (int i0 = i; i0 < n && child < 0; i0 += 32) {
                    const unsigned m = __ballot_sync(0xffffffffu, i0 + lane < n && parent[i0 + lane] == here);
                    if (m != 0) child = i0 + __ffs(m) - 1;
                }
                if (child < 0) break;
                if constexpr (DRAWN) {
                    if (c > 0.0 && whole < 0.0) {        // N_k is not there yet
                        tried = child - 1;
                        mode = 0;
                        break;
                    }
                }
                bool keep;
                if constexpr (DRAWN) {
                    const double w = (double)pv[child] - c * (double)qv[child];
                    keep = (double)coin[child] * (double)qv[child] * whole < (w > 0.0 ? w : 0.0);
                } else {
                    bool again = false;                  // its token was rejected before
                    for (int k = lane; k < ngone; k += 32) again |= gone_list[k] == token[child];
                    again = __any_sync(0xffffffffu, again);
                    keep = !again && (double)coin[child] * whole < (double)pv[child];
                    if (!keep && !again) {
                        whole -= (double)pv[child];
                        if (lane == 0) gone_list[ngone] = token[child];
                        ++ngone;
                        __syncwarp();
                    }
                }
                if (keep) {
                    if (rank == 0 && lane == 0) path[depth] = child;
                    here = child;
                    ++depth;
                    c = 0.0;
                    whole = 1.0;
                    ngone = 0;
                    if (depth >= p.max_accepted) break;
                } else if constexpr (DRAWN) {
                    c += whole;
                    whole = -1.0;
                }
                tried = child;
                i = child + 1;
            }
            if (lane == 0) {
                s_walk[0] = mode;
                s_walk[1] = here;
                s_walk[2] = depth;
                s_walk[3] = ngone;
                s_c = c;
            }
        }
        __syncthreads();
        const int mode = s_walk[0], at = s_walk[1];
        double taken = s_c;
        const char* prow = target + at * tstep;
        const char* qrow = DRAWN ? draft + at * dstep : nullptr;
        Gone gone{gone_list, DRAWN ? 0 : s_walk[3]};
        const int first = (rank * kVerifyWarps + warp) * p.slice;
        const int last = min(first + p.slice, p.vocab);
        const bool vec = ((reinterpret_cast<uintptr_t>(prow) | (DRAWN ? reinterpret_cast<uintptr_t>(qrow) : 0)) &
                          (4 * E::kBytes - 1)) == 0;
        double total;
        bool whole_row = false;    // nothing was left of the row: the row itself
        for (;;) {
            const float ch = (float)taken, cl = (float)(taken - (double)ch);
            double sum = 0.0;
            if (first < p.vocab) {
                // what is not taken off need not be read
                if (DRAWN && taken > 0.0)
                    sum = vec ? slice_sum<E, DRAWN, true>(prow, qrow, first, last, p.vocab, ch, cl, gone)
                              : slice_sum<E, DRAWN, false>(prow, qrow, first, last, p.vocab, ch, cl, gone);
                else
                    sum = vec ? slice_sum<E, false, true>(prow, nullptr, first, last, p.vocab, 0.f, 0.f, gone)
                              : slice_sum<E, false, false>(prow, nullptr, first, last, p.vocab, 0.f, 0.f, gone);
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            }
            if (lane == 0) s_part[warp] = sum;
            cluster.sync();
            if (tid < kSlices) s_all[tid] = *cluster.map_shared_rank(&s_part[tid % kVerifyWarps], tid / kVerifyWarps);
            cluster.sync();        // everyone's parts are read: they may change, and CTAs may leave
            __syncthreads();
            if (warp == 0) {
                // running sums, four slices a lane
                double part[4], s = 0.0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    part[k] = s_all[4 * lane + k];
                    s += part[k];
                }
                double incl = s;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
                const double all = __shfl_sync(0xffffffffu, incl, 31);
                // the slice with the next token: the first with a weight whose running sum passes the threshold
                double run = incl - s, before = 0.0;
                int owner = INT32_MAX;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (owner == INT32_MAX && part[k] > 0.0 && run + part[k] > (double)pick * all) {
                        owner = 4 * lane + k;
                        before = run;
                    }
                    run += part[k];
                }
                const int first_owner = __reduce_min_sync(0xffffffffu, owner);
                if (owner == first_owner) {          // of all lanes where there is none: it is not used then
                    s_owner = first_owner;
                    s_before = before;
                }
                if (lane == 0) s_total = all;
            }
            __syncthreads();
            total = s_total;
            if (mode == 0 || total > 0.0 || whole_row || !(taken > 0.0 || gone.n > 0)) break;
            whole_row = true;
            taken = 0.0;
            gone.n = 0;
        }
        if (mode == 0) {
            whole = total;
            continue;
        }
        const int found = s_walk[2];
        fill(found);
        const bool fine = total > 0.0 && total < INFINITY;
        if (rank == 0 && tid == 0) {
            p.num_accepted[b] = found;
            if (!fine) {
                p.next_tokens[b] = -1;
                report(p.dev_status, WF_DEV_BAD_PROBS);
            }
        }
        if (!fine) return;
        // the warp whose slice the sum passes the threshold in looks for the token
        const double threshold = (double)pick * total;
        if (rank * kVerifyWarps + warp != s_owner) return;
        const float ch = (float)taken, cl = (float)(taken - (double)ch);
        double base = s_before;
        int answer = -1, positive = -1;
        for (int i0 = first; i0 < last && answer < 0; i0 += kStep) {
            float a[4], q[4] = {};
            const int i = i0 + 4 * lane;
            four<E, false>(prow, i, p.vocab, a);
            if (DRAWN && taken > 0.0) four<E, false>(qrow, i, p.vocab, q);
            double run[4], s = 0.0;
            int some = -1;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float hi, lo;
                weight<DRAWN>(a[e], q[e], ch, cl, hi, lo);
                if (!DRAWN && gone.n > 0 && gone.has(i + e)) hi = lo = 0.f;
                if (hi > 0.f) some = i + e;
                s += (double)hi + (double)lo;
                run[e] = s;
            }
            double incl = s;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            int hit = INT32_MAX;
#pragma unroll
            for (int e = 3; e >= 0; --e)
                if (base + (incl - s) + run[e] > threshold) hit = i + e;
            hit = __reduce_min_sync(0xffffffffu, hit);
            positive = max(positive, __reduce_max_sync(0xffffffffu, some));
            if (hit != INT32_MAX) answer = hit;
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
        // the two ways to add up differ in the last bits: past the slice's end it is its last token
        if (lane == 0) p.next_tokens[b] = answer >= 0 ? answer : positive;
        return;
    }
}

template <typename E>
cudaError_t launch_verify(const VerifyParams& p, int B, bool drawn, cudaStream_t stream) {
    auto kern = drawn ? verify_drafts_kernel<E, true> : verify_drafts_kernel<E, false>;
    const int smem = 6 * 4 * p.max_q_len;
    cudaError_t err = allow_dynamic_smem((const void*)kern, smem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)B * kVerifyCtas);
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kVerifyCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyArgs& a, uint32_t* dev_status, cudaStream_t stream) {
    const int per = (a.vocab + kSlices - 1) / kSlices;
    const VerifyParams p{a.accepted, a.num_accepted, a.next_tokens, a.target, a.draft, a.target_stride, a.draft_stride,
                         a.tokens,   a.parents,      a.cu_q_lens,   a.coins,  a.picks, dev_status,      a.vocab,
                         a.max_accepted, a.total, a.max_q_len, (per + kStep - 1) / kStep * kStep};
    return a.probs_dtype == WF_DTYPE_F32 ? launch_verify<F32>(p, a.B, a.draft != nullptr, stream)
                                         : launch_verify<BF16>(p, a.B, a.draft != nullptr, stream);
}

}  // namespace wf
