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
// Numbers are compared with borders that they may lie next to, so sums are kept in pairs of fp32 numbers: products
// and differences with their rounding errors, and sums with theirs.  Eight additions of a thread
// lose 2^-42 of its sum at worst, so n of them n 2^-46 (their sum grows meanwhile): 2^-39 for 2^18 tokens in
// clusters of 4, 2^-27 for 2^28 in one CTA.  The errors have both signs, and what is left is rather the square root
// of that count: 2^-44 and 2^-38.
// (In fp64, which this GPU has a 64th of its fp32 rate for, the sums over a warp's lanes alone took
// longer than reading the rows: 64 trees 19 us instead of 12; now 10.9.)
//
// Bound: HBM, one or two rows of the vocabulary a request.  A cluster takes a request; every CTA
// walks the tree by itself on the gathered p_u(x), q_u(x) of all nodes and reads its part of a row
// where a sum is needed, which is once for a chain: the sums that a rejection's remainder needs are
// the running sums of the next token too, up to the slice of the one warp that holds it, which looks
// at it again.  231 chains of up to 4 drafts over 128000 fp32 tokens 46.6 us, 172 MB that are 25.4 at the copy peak:
// a request is about 6 us of dependent rounds around its 6-16 us of loads, and a second row for a rejected draft with
// a sibling comes on top.  Slices' sums are written to every CTA of the cluster, so a row takes one barrier.
#include <cooperative_groups.h>

#include "wf_internal.h"

namespace wf {

namespace {

namespace cg = cooperative_groups;

constexpr int kVerifyThreads = 256, kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyCtas = 16;                             // of a cluster at most (more than 8 by opt-in)
constexpr int kVerifyPerSm = 4;                             // CTAs an SM holds
constexpr int kSlices = kVerifyCtas * kVerifyWarps;         // a row's parts at most, a warp each
constexpr int kStep = 128;                                  // tokens a warp reads at once
constexpr int kSliceStep = 4 * 32 * kVerifyWarps;           // a slice is a multiple of what a CTA looks at in fours

struct VerifyParams {
    int32_t *accepted, *num_accepted, *next_tokens;
    const void *target, *draft;
    int64_t target_stride, draft_stride;
    const int32_t *tokens, *parents, *cu_q_lens;
    const float *coins, *picks;
    uint32_t* dev_status;
    int32_t vocab, max_accepted, total, max_q_len;
    int32_t slice;      // tokens of a warp: a multiple of kSliceStep
};

// A number as the sum of two, h the rounded one.
struct Pair {
    float h, l;
};
// a + b with the larger number first.
__device__ __forceinline__ Pair ordered_sum(float a, float b) {
    const float h = __fadd_rn(a, b);
    return Pair{h, __fsub_rn(b, __fsub_rn(h, a))};
}
__device__ __forceinline__ Pair any_sum(float a, float b) {
    const float h = __fadd_rn(a, b), x = __fsub_rn(h, a);
    return Pair{h, __fadd_rn(__fsub_rn(a, __fsub_rn(h, x)), __fsub_rn(b, x))};
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
    const Pair s = any_sum(a.h, b.h);
    return ordered_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Pair operator-(Pair a, Pair b) { return a + Pair{-b.h, -b.l}; }
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
    const float t = __fmul_rn(a.h, b.h);
    const float e = __fmaf_rn(a.h, b.h, -t);
    return ordered_sum(t, __fmaf_rn(a.h, b.l, __fmaf_rn(a.l, b.h, e)));
}
__device__ __forceinline__ bool operator<(Pair a, Pair b) { return a.h < b.h || (a.h == b.h && a.l < b.l); }
__device__ __forceinline__ Pair shfl_up(Pair a, int o) {
    return Pair{__shfl_up_sync(0xffffffffu, a.h, o), __shfl_up_sync(0xffffffffu, a.l, o)};
}
// Running sums over the lanes.
__device__ __forceinline__ Pair lane_sums(Pair a) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Pair y = shfl_up(a, o);
        if (lane >= o) a = a + y;
    }
    return a;
}

// max(p - (ch + cl) q, 0) of two tokens as hi + lo; NaN and what is below 0 count as 0.  Where the
// result counts p is above the product, so that the error of the difference is (p - d) - t.
template <bool DRAWN>
__device__ __forceinline__ void weight(float2 p, float2 q, float ch, float cl, float2& hi, float2& lo) {
    if constexpr (DRAWN) {
        q = make_float2(fmaxf(q.x, 0.f), fmaxf(q.y, 0.f));
        const float2 c2 = make_float2(ch, ch), minus = make_float2(-1.f, -1.f);
        const float2 t = __fmul2_rn(c2, q);
        const float2 nt = make_float2(-t.x, -t.y);
        const float2 te = __ffma2_rn(c2, q, nt);
        hi = __fadd2_rn(p, nt);
        const float2 e = __fadd2_rn(__ffma2_rn(hi, minus, p), nt);
        lo = __ffma2_rn(q, make_float2(-cl, -cl), __ffma2_rn(te, minus, e));
        const float2 w = __fadd2_rn(hi, lo);
        // (an infinite p stays: its lo is NaN, and so becomes the sum)
        if (!(w.x > 0.f) && !(hi.x == INFINITY)) hi.x = lo.x = 0.f;
        if (!(w.y > 0.f) && !(hi.y == INFINITY)) hi.y = lo.y = 0.f;
    } else {
        hi = make_float2(fmaxf(p.x, 0.f), fmaxf(p.y, 0.f));
        lo = make_float2(0.f, 0.f);
    }
}

// A sum of pairs: the rounded sum and its errors.
struct PairSum {
    float2 s = make_float2(0.f, 0.f), e = make_float2(0.f, 0.f);
    __device__ __forceinline__ void add(float2 hi, float2 lo) {
        const float2 minus = make_float2(-1.f, -1.f);
        const float2 t = __fadd2_rn(s, hi);
        const float2 b = __ffma2_rn(s, minus, t);                            // what came of hi
        const float2 x = __ffma2_rn(__ffma2_rn(b, minus, t), minus, s);      // what s lost
        const float2 y = __ffma2_rn(b, minus, hi);                           // what hi lost
        s = t;
        e = __fadd2_rn(e, __fadd2_rn(__fadd2_rn(x, y), lo));
    }
    // The errors into the sum, so that their own sum stays small beside it: left alone it grows with the tokens, and with it
    // its rounding (2^17 equal tokens of one thread: off by 2^-22 of their sum).
    __device__ __forceinline__ void fold() {
        const float2 minus = make_float2(-1.f, -1.f);
        const float2 t = __fadd2_rn(s, e);
        e = __ffma2_rn(__ffma2_rn(s, minus, t), minus, e);
        s = t;
    }
    __device__ __forceinline__ Pair value() const {
        return any_sum(s.x, s.y) + any_sum(e.x, e.y);
    }
};

template <typename E>
__device__ __forceinline__ float element(const void* row, int64_t i) {
    if constexpr (E::kBytes == 4)
        return __ldg(static_cast<const float*>(row) + i);
    else
        return __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(row) + i));
}

// A row (of the target, the draft or both) as places: token x is place x + lo, lo < 4, where place 0
// lies on a boundary of four elements, so that an odd row is read in fours too, all but its first and last.
// `vec`: both rows lie on the same boundary; else lo is 0 and they are read element by element.
struct Row {
    const char *p, *q;
    int lo, hi;          // places [lo, hi) are there
    bool vec;
};

template <typename E, bool DRAWN>
__device__ __forceinline__ Row row_places(const char* p, const char* q, int vocab) {
    constexpr int kMask = 4 * E::kBytes - 1;
    const int a = (int)(reinterpret_cast<uintptr_t>(p) & kMask), b = DRAWN ? (int)(reinterpret_cast<uintptr_t>(q) & kMask) : a;
    Row r{p, q, 0, vocab, a == b};
    if (r.vec) {
        r.lo = a / E::kBytes;
        r.hi += r.lo;
        r.p -= a;
        if (DRAWN) r.q -= a;
    }
    return r;
}

// Four places from `i`, a multiple of four, on (0 for those that are not there).
template <typename E>
__device__ __forceinline__ void four(const char* row, int i, const Row& r, float (&f)[4]) {
    if (r.vec && i >= r.lo && i + 4 <= r.hi) {
        if constexpr (E::kBytes == 4) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(row) + i));
            f[0] = x.x;
            f[1] = x.y;
            f[2] = x.z;
            f[3] = x.w;
        } else {
            const uint2 x = __ldg(reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(row) + i));
            const float2 a = bf16x2_to_float2(x.x), b = bf16x2_to_float2(x.y);
            f[0] = a.x;
            f[1] = a.y;
            f[2] = b.x;
            f[3] = b.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = i + e >= r.lo && i + e < r.hi ? element<E>(row, i + e) : 0.f;
    }
}

// Tokens whose weight is 0, rejected fixed candidates.
struct Gone {
    const int32_t* token;
    int n;
    // Calls f(place) in all lanes for each of them in places [first, last).
    template <typename F>
    __device__ __forceinline__ void each(int first, int last, int lo, F f) const {
        for (int k0 = 0; k0 < n; k0 += 32) {
            const int k = k0 + (int)(threadIdx.x & 31);
            const int x = k < n ? token[k] + lo : -1;
            for (unsigned m = __ballot_sync(0xffffffffu, x >= first && x < last); m != 0; m &= m - 1)
                f(__shfl_sync(0xffffffffu, x, __ffs(m) - 1));
        }
    }
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// This lane's part of the sum of w over places [first, last), last - first a multiple of kStep.
template <typename E, bool DRAWN>
__device__ __forceinline__ Pair slice_sum(const Row& r, int first, int last, float ch, float cl, const Gone& gone) {
    constexpr int kAhead = 4;        // reads of a row in flight (8 of a row alone: 12.0 us instead of 10.5 for 64 trees)
    const int lane = threadIdx.x & 31;
    PairSum sum;
#pragma unroll 1
    for (int i0 = first; i0 < last; i0 += kAhead * kStep) {
        float a[kAhead][4], b[DRAWN ? kAhead : 1][4];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u * kStep < last ? i0 + u * kStep + 4 * lane : r.hi;
            four<E>(r.p, i, r, a[u]);
            if constexpr (DRAWN) four<E>(r.q, i, r, b[u]);
        }
        if constexpr (!DRAWN)
            gone.each(i0, i0 + kAhead * kStep, r.lo, [&](int x) {
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (x == i0 + u * kStep + 4 * lane + e) a[u][e] = 0.f;
            });
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                float2 hi, lo, b2 = make_float2(0.f, 0.f);
                if constexpr (DRAWN) b2 = make_float2(b[u][e], b[u][e + 1]);
                weight<DRAWN>(make_float2(a[u][e], a[u][e + 1]), b2, ch, cl, hi, lo);
                sum.add(hi, lo);
            }
        sum.fold();
    }
    return sum.value();
}

template <typename E, bool DRAWN>
__global__ void __launch_bounds__(kVerifyThreads, kVerifyPerSm) verify_drafts_kernel(const VerifyParams p) {
    extern __shared__ unsigned char smem[];
    __shared__ Pair s_sums[2][kSlices];       // a row's slices, written by the whole cluster; two rows in turn
    __shared__ int s_walk[4], s_owner;
    __shared__ Pair s_c, s_total, s_before, s_part[kVerifyWarps];
    float* pv = reinterpret_cast<float*>(smem);            // p_parent(token) of each node
    float* qv = pv + p.max_q_len;
    float* coin = qv + p.max_q_len;
    int32_t* token = reinterpret_cast<int32_t*>(coin + p.max_q_len);
    int32_t* parent = token + p.max_q_len;
    int32_t* gone_list = parent + p.max_q_len;
    int32_t* mark = gone_list + p.max_q_len;               // kKeep, kAgain
    constexpr int kKeep = 1, kAgain = 2;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int b = blockIdx.x / ctas;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int q0 = __ldg(p.cu_q_lens + b), n = __ldg(p.cu_q_lens + b + 1) - q0;
    const float pick = __ldg(p.picks + b);
    int32_t* path = p.accepted + (int64_t)b * p.max_accepted;
    cluster_arrive();      // waited for before the first write to another CTA's shared memory
    for (int i = tid; i < kSlices; i += kVerifyThreads)
        if (i >= ctas * kVerifyWarps) s_sums[0][i] = s_sums[1][i] = Pair{0.f, 0.f};
    // all CTAs of a cluster come to the same of this and of the next checks, so they leave together
    if (q0 < 0 || n < 0 || n > p.max_q_len || (int64_t)q0 + n > p.total) {
        if (rank == 0 && tid == 0) report(p.dev_status, WF_DEV_BAD_SEQLEN);
        cluster_wait();
        return;
    }
    const size_t tstep = (size_t)p.target_stride * E::kBytes, dstep = (size_t)p.draft_stride * E::kBytes;
    const char* target = static_cast<const char*>(p.target) + q0 * tstep;
    const char* draft = DRAWN ? static_cast<const char*>(p.draft) + q0 * dstep : nullptr;
    if (!(pick >= 0.f && pick < 1.f)) {
        if (rank == 0 && tid == 0) report(p.dev_status, WF_DEV_BAD_PROBS);
        cluster_wait();
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
        cluster_wait();
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
        cluster_wait();
        return;
    }
    // What becomes of a node if it is tried: of a fixed candidate all of it, its earlier siblings
    // being rejected then; of a drawn one if it is the first (the others need a row's sum).
    if constexpr (!DRAWN) {
        for (int i = tid; i < n; i += kVerifyThreads) {
            bool again = false;        // a sibling before it has its token
            for (int j = parent[i] + 1; j < i; ++j) again |= parent[j] == parent[i] && token[j] == token[i];
            mark[i] = again ? kAgain : 0;
        }
        __syncthreads();
    }
    for (int i = tid; i < n; i += kVerifyThreads) {
        if constexpr (DRAWN) {
            mark[i] = Pair{coin[i], 0.f} * Pair{qv[i], 0.f} < Pair{pv[i], 0.f} ? kKeep : 0;
        } else if (!(mark[i] & kAgain)) {
            Pair whole{1.f, 0.f};
            for (int j = parent[i] + 1; j < i; ++j)
                if (parent[j] == parent[i] && !(mark[j] & kAgain)) whole = whole - Pair{pv[j], 0.f};
            if (Pair{coin[i], 0.f} * whole < Pair{pv[i], 0.f}) atomicOr(&mark[i], kKeep);   // (others read its kAgain)
        }
    }
    __syncthreads();
    // Warp 0 walks; what it hands over: 0 a sum to form (N_k) and more children to try, 1 the end
    // of the path.  here, depth, the last child tried, c and N live in its registers.
    int here = 0, depth = 1, tried = 0, row = 0;
    Pair c{0.f, 0.f}, whole{1.f, 0.f};
    if (rank == 0 && tid == 0) path[0] = 0;
    for (;;) {
        if (warp == 0) {
            int mode = 1, ngone = 0;
            // the first node from i on that hangs on `here` and has all bits of `want`
            const auto next = [&](int i, int want) {
                for (int i0 = i; i0 < n; i0 += 32) {
                    const int x = i0 + lane;
                    const unsigned m = __ballot_sync(0xffffffffu, x < n && parent[x] == here && (mark[x] & want) == want);
                    if (m != 0) return i0 + __ffs(m) - 1;
                }
                return -1;
            };
            while (depth < p.max_accepted) {
                const int child = next(tried + 1, DRAWN ? 0 : kKeep);
                if (child < 0) break;
                if constexpr (DRAWN) {
                    if (whole.h < 0.f) {      // N_k is not there yet
                        mode = 0;
                        break;
                    }
                    bool keep = c.h == 0.f && (mark[child] & kKeep);
                    if (c.h > 0.f) {
                        const Pair q{qv[child], 0.f}, w = Pair{pv[child], 0.f} - c * q;
                        keep = Pair{coin[child], 0.f} * q * whole < (w.h > 0.f ? w : Pair{0.f, 0.f});
                    }
                    if (!keep) {
                        c = c + whole;
                        whole = Pair{-1.f, 0.f};
                        tried = child;
                        continue;
                    }
                }
                if (rank == 0 && lane == 0) path[depth] = child;
                here = tried = child;
                ++depth;
                c = Pair{0.f, 0.f};
                whole = Pair{1.f, 0.f};
            }
            if (!DRAWN && depth < p.max_accepted) {
                // its children were all rejected
                for (int i0 = here + 1; i0 < n; i0 += 32) {
                    const int x = i0 + lane;
                    const bool gone = x < n && parent[x] == here && !(mark[x] & kAgain);
                    const unsigned m = __ballot_sync(0xffffffffu, gone);
                    if (gone) gone_list[ngone + __popc(m & ((1u << lane) - 1u))] = token[x];
                    ngone += __popc(m);
                }
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
        Pair taken = s_c;
        const char* prow = target + at * tstep;
        const char* qrow = DRAWN ? draft + at * dstep : nullptr;
        const Row r = row_places<E, DRAWN>(prow, qrow, p.vocab);
        const int first = (rank * kVerifyWarps + warp) * p.slice;
        Gone gone{gone_list, DRAWN ? 0 : s_walk[3]};
        Pair total;
        bool whole_row = false;    // nothing was left of the row: the row itself
        for (;;) {
            Pair sum{0.f, 0.f};
            if (first < r.hi) {
                // what is not taken off need not be read
                if (DRAWN && taken.h > 0.f)
                    sum = slice_sum<E, DRAWN>(r, first, first + p.slice, taken.h, taken.l, gone);
                else
                    sum = slice_sum<E, false>(r, first, first + p.slice, 0.f, 0.f, gone);
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1)
                    sum = sum + Pair{__shfl_xor_sync(0xffffffffu, sum.h, o), __shfl_xor_sync(0xffffffffu, sum.l, o)};
            }
            Pair* all_sums = s_sums[row & 1];
            if (row++ == 0) cluster_wait();
            if (lane < ctas) *cluster.map_shared_rank(&all_sums[rank * kVerifyWarps + warp], lane) = sum;
            __syncwarp();
            cluster_arrive();
            cluster_wait();
            if (warp == 0) {
                // running sums, kSlices / 32 of them a lane
                Pair part[kSlices / 32], s{0.f, 0.f};
#pragma unroll
                for (int k = 0; k < kSlices / 32; ++k) {
                    part[k] = all_sums[kSlices / 32 * lane + k];
                    s = s + part[k];
                }
                const Pair incl = lane_sums(s);
                const Pair all{__shfl_sync(0xffffffffu, incl.h, 31), __shfl_sync(0xffffffffu, incl.l, 31)};
                const Pair threshold = Pair{pick, 0.f} * all;
                // the slice with the next token: the first with a weight whose running sum passes the threshold
                Pair run = shfl_up(incl, 1), before{0.f, 0.f};
                if (lane == 0) run = Pair{0.f, 0.f};
                int owner = INT32_MAX, some = -1;
                Pair some_before{0.f, 0.f};
#pragma unroll
                for (int k = 0; k < kSlices / 32; ++k) {
                    const Pair up = run + part[k];
                    if (part[k].h > 0.f) {
                        some = kSlices / 32 * lane + k;
                        some_before = run;
                    }
                    if (owner == INT32_MAX && part[k].h > 0.f && threshold < up) {
                        owner = kSlices / 32 * lane + k;
                        before = run;
                    }
                    run = up;
                }
                int first_owner = __reduce_min_sync(0xffffffffu, owner);
                if (first_owner == INT32_MAX) {      // a sum so small that the threshold rounds up to it: the last one
                    first_owner = __reduce_max_sync(0xffffffffu, some);
                    owner = some;
                    before = some_before;
                }
                if (owner == first_owner) {          // (of all lanes where there is none: it is not used then)
                    s_owner = first_owner;
                    s_before = before;
                }
                if (lane == 0) s_total = all;
            }
            __syncthreads();
            total = s_total;
            if (mode == 0 || total.h > 0.f || whole_row || !(taken.h > 0.f || gone.n > 0)) break;
            whole_row = true;
            taken = Pair{0.f, 0.f};
            gone.n = 0;
        }
        if (mode == 0) {
            whole = total;
            continue;
        }
        const int found = s_walk[2];
        fill(found);
        const bool fine = total.h > 0.f && total.h < INFINITY;
        if (rank == 0 && tid == 0) {
            p.num_accepted[b] = found;
            if (!fine) {
                p.next_tokens[b] = -1;
                report(p.dev_status, WF_DEV_BAD_PROBS);
            }
        }
        if (!fine) return;
        // The CTA whose slice the running sum passes the threshold in looks for the token: each warp takes a
        // part of the slice and each lane p.slice / 256 places of it side by side.
        const Pair threshold = Pair{pick, 0.f} * total;
        if (rank != s_owner / kVerifyWarps) return;
        const int per = p.slice / (32 * kVerifyWarps);
        const int start = s_owner * p.slice + warp * (p.slice / kVerifyWarps);
        const auto weights = [&](int i, float2 (&hi)[2], float2 (&lo)[2]) {     // of four places
            float a[4], q[4] = {};
            four<E>(r.p, i, r, a);
            if (DRAWN && taken.h > 0.f) four<E>(r.q, i, r, q);
            for (int k = 0; k < gone.n; ++k) {
                const int x = gone.token[k] + r.lo - i;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (x == e) a[e] = 0.f;
            }
            weight<DRAWN>(make_float2(a[0], a[1]), make_float2(q[0], q[1]), taken.h, taken.l, hi[0], lo[0]);
            weight<DRAWN>(make_float2(a[2], a[3]), make_float2(q[2], q[3]), taken.h, taken.l, hi[1], lo[1]);
        };
        PairSum part;
#pragma unroll 2
        for (int k = 0; k < per; k += 4) {
            float2 hi[2], lo[2];
            weights(start + lane * per + k, hi, lo);
            part.add(hi[0], lo[0]);
            part.add(hi[1], lo[1]);
            part.fold();
        }
        const Pair sum = part.value(), incl = lane_sums(sum);
        if (lane == 31) s_part[warp] = incl;
        __syncthreads();
        // The first warp, lane and place whose running sum passes the threshold.  Sums that are added up in
        // another way differ in their last bits: where none passes, it is the last with a weight.
        Pair base = s_before, at_warp{0.f, 0.f}, last_base{0.f, 0.f};
        int its = -1, last = -1;
        for (int w = 0; w < kVerifyWarps && its < 0; ++w) {
            const Pair up = base + s_part[w];
            if (s_part[w].h > 0.f) {
                last = w;
                last_base = base;
                if (threshold < up) {
                    its = w;
                    at_warp = base;
                }
            }
            base = up;
        }
        if (its < 0) {
            its = last;
            at_warp = last_base;
        }
        if (warp != its) return;
        const unsigned some = __ballot_sync(0xffffffffu, sum.h > 0.f);
        const unsigned over = __ballot_sync(0xffffffffu, sum.h > 0.f && threshold < at_warp + incl);
        const int owner = over != 0 ? __ffs(over) - 1 : 31 - __clz(some);
        Pair run = shfl_up(incl, 1);
        if (lane != owner) return;
        run = lane == 0 ? at_warp : at_warp + run;
        // For the same reason the sum before this lane may pass the threshold already, though no place before it was
        // found to: then it is the lane's first with a weight.
        int answer = -1;
        for (int k = 0; k < per; k += 4) {
            float2 hi[2], lo[2];
            const int i = start + lane * per + k;
            weights(i, hi, lo);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 h = hi[e >> 1], l = lo[e >> 1];
                const Pair w{(e & 1) ? h.y : h.x, (e & 1) ? l.y : l.x};
                // (w.h is 0, or below it, where the rounded difference is and the rest is not)
                if (w.h + w.l > 0.f && (answer < 0 || !(threshold < run))) {
                    answer = i + e;
                    run = run + w;
                }
            }
            if (answer >= 0 && threshold < run) break;
        }
        p.next_tokens[b] = answer - r.lo;
        return;
    }
}

template <typename E>
cudaError_t launch_verify(VerifyParams p, int B, bool drawn, cudaStream_t stream) {
    auto kern = drawn ? verify_drafts_kernel<E, true> : verify_drafts_kernel<E, false>;
    const int smem = 7 * 4 * p.max_q_len;
    cudaError_t err = allow_dynamic_smem((const void*)kern, smem);
    if (err != cudaSuccess) return err;
    // More CTAs a request shorten its row, more requests at once hide what is dependent loads (about
    // 6 us a request): as many as make two rounds of the CTAs that are resident.  231 chains over 128000
    // tokens in clusters of 2, 4, 8, 16: 53, 46, 50, 71 us; 64 trees over 50257: 17, 12, 10.5, 26 us; one
    // chain: 16.8, 11.1, 8.7, 7.8 us.  16 only where the batch leaves half of the room: more of them wait for
    // one another's places.
    int ctas = 8;
    while (ctas > 1 && (int64_t)B * ctas > 2 * kVerifyPerSm * (int64_t)num_sms()) ctas /= 2;
    if ((int64_t)B * kVerifyCtas <= kVerifyPerSm / 2 * (int64_t)num_sms()) ctas = kVerifyCtas;
    const int per = (p.vocab + 3 + ctas * kVerifyWarps - 1) / (ctas * kVerifyWarps);
    p.slice = (per + kSliceStep - 1) / kSliceStep * kSliceStep;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)B * ctas);
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    if (ctas > 8) {
        err = allow_large_cluster((const void*)kern);
        if (err != cudaSuccess) return err;
    }
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyArgs& a, uint32_t* dev_status, cudaStream_t stream) {
    const VerifyParams p{a.accepted, a.num_accepted, a.next_tokens, a.target, a.draft, a.target_stride, a.draft_stride,
                         a.tokens,   a.parents,      a.cu_q_lens,   a.coins,  a.picks, dev_status,      a.vocab,
                         a.max_accepted, a.total, a.max_q_len, 0};
    return a.probs_dtype == WF_DTYPE_F32 ? launch_verify<F32>(p, a.B, a.draft != nullptr, stream)
                                         : launch_verify<BF16>(p, a.B, a.draft != nullptr, stream);
}

}  // namespace wf
