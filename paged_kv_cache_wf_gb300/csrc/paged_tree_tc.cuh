// paged_tree_tc.cuh -- tree attention and scored attention on the tensor cores (tcgen05, TMA,
// TMEM) for bf16 and fp8 pools whose block size is a multiple of 16.
//
// What is computed is paged_tree_cc.cuh's: row (draft, query head) sees its request's cached
// positions and the drafts of its mask; o = softmax(scale q K^T) V.
//
// GB300 design.  A work unit (paged_tree.cuh) is one row block of a request under one
// KV head.  Its K and V tiles (128 positions, gathered 16-position box by box through
// the block table, 128-byte swizzle) run through a K ring and a V ring without a break
// from piece to piece, and two softmax warpgroups (one thread a row, one TMEM lane a
// thread) keep the tensor core on S = Q K^T of one stream while the other's softmax
// runs.  What the two streams are is the template's choice:
//   QT = 1  (all units of the batch have at most 128 rows): both streams are the same
//           128 rows, on alternate tiles, each with its own running maximum, sum and O
//           accumulator; at a piece's end the two are joined from TMEM, each warpgroup
//           half of the columns.
//   QT = 2  (up to 256 rows a unit): one 128-row query tile each, on the same tiles, so
//           a loaded tile serves 256 rows.
// Device time of a call in a graph of many (issued one by one a call takes 1-2 us more, the widest
// 8-15), and of its bytes at the copy peak: 32 requests of 1-16 drafts 33.9
// and 18.1 us, 118 of 33-61 drafts (QT = 2) 273-280 and 190 us, 64 of 3-13 drafts of 64-wide heads
// 40.3 and 15.5 us, 64 of 8-24 drafts over fp8 94.0 and 37.0 us (64-wide 72 and 18.5 us), 118 of
// 33-61 drafts over fp8 405 and 118 us (64-wide 290 and 59 us); one request of 8 drafts 11.0 us.
// What is left: 5 us from launch to the first product (division of the work, first block ids,
// first tiles, cold code); 2-5 us around every piece's end, where its streams wait for one
// another and O is joined; 2-10 us of the join; and with long pieces the chain S -> softmax ->
// P V of a stream, 4600 clocks a 128-wide tile of which the softmax is 2700, for two streams.
// 16 warps: 0-7 softmax (stream t = warp / 4), 8 K loads, 9 V loads, 10 the walk over the
// CTA's pieces (a ring of records that the other warps read) and the query tiles, 11 and
// 12 MMA issue (a stream each), 13-15 the V tiles' finish.  The softmax warps take
// registers from the others.
// The finish of a V tile: a weight of 0 hides a position only from finite values (0 *
// NaN is NaN in P V).  Rows past the request's end or of a bad block are zeroed; an
// element of a draft's row that is not finite is zeroed too, and the epilogue adds it
// to the rows that see the draft.  Only tiles that reach the drafts are looked at (scored: tiles that
// some row does not see whole).
//
// fp8 pools (CODES; QT = 1, see tree_tc_shape).  S takes the K codes as they are (e4m3 x e4m3 ->
// fp32): a small grid before this one splits every q row, scaled by a power of two so
// that its largest magnitude lies in [128, 256), into hi = e4m3(q) and lo = e4m3(q - hi).
// hi keeps four of a bf16 value's eight significant bits and lo the rest, so their sum is
// the row up to 2^-10 (a 2^-17 part of its largest value).  The row's power of two and
// the K scale go into the exponent's factor.  V codes are widened to fp16, which is exact
// and which the hardware converts two at a time, by the finishing warps, into the ring
// that P V reads, and the weights (2^7 of them, see kCodesUp) are rounded to fp16, whose
// step is an eighth of bf16's; the V scale multiplies the outputs.  To bf16 there is no
// conversion, and shifting and scaling the codes there took the call from 94 us (V not
// widened) to 135 us, batch of 64.  Widening K too would cost twice the finishing warps'
// work, and splitting the weights into two e4m3 parts would cost the softmax warps more
// conversions than they have time for.
//
// Scored attention (ScoredView; paged_scored.cu has the formulas).  A unit's tiles are those that some
// of its rows see, from the last one down, and two things differ in the softmax:
//   - Half tiles (row blocks of more than 32 rows).  A step takes 64 positions: S of the second half runs
//     while the first is worked on, and S of the next tile's first half as soon as P V has read its
//     columns, so a stream waits for S 300 clocks a half instead of 2000 a tile.  Eight prompts of
//     128-2048 tokens: 194 us plain, 215 with a bias, 261 capped, 311 capped and biased (96 us of products at
//     the bf16 rate); a capped half step takes about 2300 clocks.
//   - Spread (at most 32 rows).  The rows stand in all four quarters of the query tile and each quarter's
//     warp takes a quarter of a tile's positions, so eight warps share what one warp a stream had: 231 capped
//     decodes 260-267 us (252 at the copy peak; 393 before).  The quarters' sums and outputs are joined at a piece's end.
// Row blocks of fp8 pools stay at 128 rows or 32.  What is left: packed documents (200 us, 31 of products) spend half
// of their time on their pieces' ends, 1.8 tiles a piece and stream; one user (10.9 us) is the start, one tile and the join.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "paged_tree.cuh"

namespace wf {

namespace {

constexpr int TM = 128;           // rows of a query tile (TMEM lanes)
constexpr int TN = 128;           // positions of a tile
constexpr float kLazyMax = 8.f;   // rescale O only when a row's maximum grows by more than 2^8
// fp16 weights (fp8 pools) carry a factor of 2^7, which the sum has too: up to 2^15 of fp16's
// 2^16.  A weight below 2^-21 of the row's largest loses bits, one below 2^-32 is 0 (without the
// factor 2^-14 and 2^-25, which a long tail of small weights would feel).
constexpr float kCodesUp = 7.f;
static_assert(kLazyMax + kCodesUp <= 15.f, "fp16 weights overflow");
// Scored calls over bf16 pools: bf16 weights and fp32 sums have the range for more (values of V up to 2^90 or so),
// and then hardly any tile after a row's first rescales (with 8 some row of a warp did every few tiles, a sixth of
// the time).
constexpr float kLazyFar = 24.f;
constexpr int kSoftW = 8, kKW = 8, kVW = 9, kWalkW = 10, kMmaW = 11, kFinW = 13, kFin = 3;
constexpr int kTcThreads = (kFinW + kFin) * 32;
constexpr int kSoftRegs = 192, kOtherRegs = 64;
static_assert(kTcThreads / 2 * (kSoftRegs + kOtherRegs) <= 65536, "register split exceeds the block's registers");

template <int N>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A piece as the warps read it; nt = 0 ends the list.
struct PieceRec {
    int b, h, q_row, n;      // request, KV head, first row of q of the row block, drafts of the request
    int tok0, rows_tok;      // first draft of the row block, drafts in it
    int c, kend;             // cached positions, all positions
    int j0, j1, nt, last;    // tiles [j0, j1) of nt; last CTA with a piece of the unit
};

// The same of a scored call.
struct ScoredRec {
    int j0, j1, nt, last;
    ScoredBlock k;           // and the unit's KV head in it
};

template <typename V>
using RecOf = typename std::conditional<V::kScored, ScoredRec, PieceRec>::type;
template <typename V>
using StartOf = typename std::conditional<V::kScored, ScoredStart, TreeStart>::type;

template <typename V, int D, int QT, bool CODES>
struct TtLayout {
    static_assert(QT == 1 || !CODES, "fp8 pools have one query tile");
    static constexpr int kRing = V::kScored ? 4 : 8;     // records (a scored one is larger)
    static constexpr int NC = D / 64;                    // 64-wide column blocks of D
    static constexpr int QTILE = TM * D * 2;             // bf16, or the two e4m3 parts
    static constexpr int KTILE = TN * D * (CODES ? 1 : 2);
    static constexpr int VTILE = TN * D * 2;
    static constexpr int RAW = CODES ? TN * D : 0;       // V codes before they are widened
    static constexpr int ATOM = NC == 2 ? 2048 : 1024;   // bf16: stride between 8-position atoms
    static constexpr int HALF_OFF = 1024;                // bf16: offset of the second 64-wide half
    static constexpr int BOX = 16 * D * (CODES ? 1 : 2); // one 16-position box
    // slots of the K ring, the V ring and (CODES) the ring of V codes
    static constexpr int KS = D == 128 ? (CODES ? 4 : 2) : QT == 1 ? 6 : 5;
    static constexpr int VS = D == 128 ? 2 : QT == 1 ? 4 : 5;
    static constexpr int RS = CODES ? (D == 128 ? 2 : 4) : 0;
    // QT = 1: a slot belongs to one stream, which so sees every phase of its barriers (see ring_tiles)
    static_assert(QT == 2 || (KS % 2 == 0 && VS % 2 == 0), "two streams share a ring of an odd number of slots");
    static constexpr int NSLOT = KS + VS;
    static constexpr int q = 0;
    static constexpr int k = q + QT * QTILE;
    static constexpr int v = k + KS * KTILE;
    static constexpr int raw = v + VS * VTILE;
    static constexpr int stage = raw + RS * RAW;         // a 32 x 32 fp32 block a softmax warp, for whole-line stores
    static constexpr int ml = stage + kSoftW * 4096;     // QT = 1: (m, l) of both streams' rows
    static constexpr int bars = ml + (QT == 1 ? 2 * TM * 8 : 0);
    // q_full[QT], q_empty[QT], k_full[KS], k_empty[KS], v_full[VS] (CODES: not used), v_empty[VS], v_ready[VS],
    // raw_full[RS], raw_empty[RS], per stream s_full, p_full, pv_done, then x_ready, x_done and
    // piece_full[kRing], piece_empty[kRing], per stream mma_end
    // and (spread) a meeting per stream, or (half tiles) s_full, p_full and pv_done of each stream's second half
    static constexpr bool kHalf = V::kScored && !V::kSpread;
    static constexpr int nbars = 2 * QT + 2 * NSLOT + VS + 2 * RS + 6 + 2 + 2 * kRing + 2 + (V::kSpread ? 2 : kHalf ? 6 : 0);
    static_assert(!V::kSpread || QT == 1, "spread rows have one query tile");
    static constexpr int ring = bars + nbars * 8;        // [kRing] records of pieces
    static constexpr int start = (ring + kRing * (int)sizeof(RecOf<V>) + 15) / 16 * 16;
    static constexpr int scratch = start + (int)sizeof(StartOf<V>);
    static constexpr int misc = scratch + 16 * 8;        // [0] TMEM address, [1] abort
    static constexpr int wild = misc + 16;               // [kRing]: a byte a finishing warp
    static constexpr int okm = wild + kRing * 4;         // [K, V][16 tiles]: boxes with a good block id
    static constexpr int total = okm + 32;
    static constexpr int SCOL = 128, OCOL = 256, TMEM_COLS = 512;
    static_assert(total <= 232448, "tree CTA exceeds shared memory");
    static_assert(bars % 8 == 0 && ring % 8 == 0 && start % 16 == 0 && scratch % 8 == 0 && misc % 8 == 0 && wild % 4 == 0,
                  "misaligned shared memory");
};

__device__ __forceinline__ void scale32(float (&o)[32], float w) {
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        const float2 y = __fmul2_rn(make_float2(o[e], o[e + 1]), make_float2(w, w));
        o[e] = y.x;
        o[e + 1] = y.y;
    }
}

// 32 drafts' bits of a mask row from draft `first` on (which may lie before 0 or past the
// row): bit x is draft first + x, set for positions before the drafts, clear past n.
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* row, int words, int first, int n) {
    if (first + 31 < 0) return 0xffffffffu;
    if (first >= n) return 0u;
    const int w = first >> 5;
    const uint32_t lo = w >= 0 && w < words ? __ldg(row + w) : 0u;
    const uint32_t hi = w + 1 < words ? __ldg(row + w + 1) : 0u;
    uint32_t r = __funnelshift_r(lo, hi, first & 31);
    if (first < 0) r |= (1u << -first) - 1u;
    if (n - first < 32) r &= (1u << (n - first)) - 1u;
    return r;
}

// Bits x of 32 positions from `first` on with lo <= first + x < hi.
__device__ __forceinline__ uint32_t range_bits(int lo, int hi, int first) {
    const int a = min(max(lo - first, 0), 32), b = min(max(hi - first, 0), 32);
    const uint32_t upto = b == 32 ? 0xffffffffu : (1u << b) - 1u;
    return a == 32 ? 0u : upto & (0xffffffffu << a);
}

// Zeroes the halves of w that are infinite or NaN; true when there were any.
__device__ __forceinline__ bool tame(uint32_t& w) {
    const uint32_t e = w & 0x7f807f80u;
    uint32_t m = 0;
    if ((e & 0xffffu) == 0x7f80u) m |= 0xffffu;
    if ((e & 0xffff0000u) == 0x7f800000u) m |= 0xffff0000u;
    w &= ~m;
    return m != 0;
}

// tcgen05.mma with operand descriptors in halves: within a CTA only the low word, which
// holds the address, changes, and adding to it is one instruction.  KIND 0: f16, A in
// shared memory; 1: f16, A in tensor memory; 2: f8f6f4.
template <int KIND>
__device__ __forceinline__ void mma(uint32_t d_tmem, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi, uint32_t idesc,
                                    uint32_t accumulate) {
    if constexpr (KIND == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t"
            "setp.ne.b32 p, %5, 0;\n\t"
            "mov.b64 y, {%2, %3};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d_tmem),
            "r"(a), "r"(b), "r"(b_hi), "r"(idesc), "r"(accumulate)
            : "memory");
    else if constexpr (KIND == 0)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "mov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t}" ::"r"(d_tmem),
            "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "mov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %5, p;\n\t}" ::"r"(d_tmem),
            "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "r"(accumulate)
            : "memory");
}

__device__ __forceinline__ void st_16words(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Not 0 when one of 16 codes is NaN (S.1111.111).
__device__ __forceinline__ uint32_t nan_codes(const uint4& c) {
    auto n = [](uint32_t w) { return (w & 0x7f7f7f7fu) + 0x01010101u; };
    return (n(c.x) | n(c.y) | n(c.z) | n(c.w)) & 0x80808080u;
}

struct NoScales {};

// The factors of a capped score (of a view that has them).
template <typename P>
__device__ __forceinline__ float cap_in_of(const P& p) {
    if constexpr (std::is_same<P, ScoredParams>::value) return p.cap_in;
    else return 0.f;
}
template <typename P>
__device__ __forceinline__ float cap_out_of(const P& p) {
    if constexpr (std::is_same<P, ScoredParams>::value) return p.cap_out;
    else return 0.f;
}

// ---- scored calls: the scores of 32 positions of a row ----

// tanh(t) of |t| <= kTanhNear as t (1 + c1 t^2 + c2 t^4), fitted here for the least largest error relative to tanh, 2^-17.2, that
// is below 2^-19.1 in itself.  The leading 1 keeps a score's error a part of the score however large its cap.
// Most scores lie well inside their cap, and then a tile needs no other special function than its weights'
// exponentials (eight prompts: 303 us with two more coefficients and a limit of 0.75, 343 with tanh =
// 1 - 2 / (1 + 2^z) for all scores, and a reciprocal shared by four of them was slower still).
constexpr float kTanhNear = 0.38f;

// cap_out tanh(k s) + add of two scores.
struct Cap {
    float k, z, out, c1, c2;                     // z = 2 log2(e) k
    __device__ __forceinline__ Cap(float k_, float out_)
        : k(k_), z(2.f * 1.4426950408889634f * k_), out(out_), c1(out_ * -0.33284658f), c2(out_ * 0.12280992f) {}
    __device__ __forceinline__ float2 near(float2 s, float2 add) const {
        const float2 t = __fmul2_rn(s, make_float2(k, k)), w = __fmul2_rn(t, t);
        float2 y = __ffma2_rn(make_float2(c2, c2), w, make_float2(c1, c1));
        y = __ffma2_rn(y, w, make_float2(out, out));
        return __ffma2_rn(t, y, add);
    }
    // Off by 2^-20 of the cap or so: the exponential by 2^-22, the sum by 2^-24, the reciprocal by 2^-23, times 2.
    __device__ __forceinline__ float2 far(float2 s) const {
        const float2 e = __fmul2_rn(s, make_float2(z, z));
        const float2 u = __fadd2_rn(make_float2(ex2(e.x), ex2(e.y)), make_float2(1.f, 1.f));
        const float2 v = make_float2(rcp_approx(u.x), rcp_approx(u.y));
        return __ffma2_rn(v, make_float2(-2.f * out, -2.f * out), make_float2(out, out));
    }
    // Each score in the form that is exact to a part of itself: 2^-20 of the cap is below 2^-18 of a score beyond kTanhNear.
    __device__ __forceinline__ float2 either(float2 s) const {
        const float2 a = near(s, make_float2(0.f, 0.f)), b = far(s), t = __fmul2_rn(s, make_float2(k, k));
        return make_float2(fabsf(t.x) <= kTanhNear ? a.x : b.x, fabsf(t.y) <= kTanhNear ? a.y : b.y);
    }
};

// The largest and (WIDE) the smallest of 32 scores.
template <bool WIDE>
__device__ __forceinline__ void extremes(const float (&s)[32], float& top, float& low) {
    float a[4], b[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        a[x] = fmaxf(s[x], s[x + 4]);
        if constexpr (WIDE) b[x] = fminf(s[x], s[x + 4]);
    }
#pragma unroll
    for (int e = 8; e < 32; e += 8)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            a[x] = fmax3(a[x], s[e + x], s[e + x + 4]);
            if constexpr (WIDE) b[x] = fmin3(b[x], s[e + x], s[e + x + 4]);
        }
    top = fmaxf(top, fmax3(a[0], a[1], fmaxf(a[2], a[3])));
    if constexpr (WIDE) low = fminf(low, fmin3(b[0], b[1], fminf(b[2], b[3])));
}

// scale s + slope |p - ref| of positions first .. first + 31, d = first - ref: up to ref it is a line, of which
// eight positions' steps are kept (`step`, -slope times 0 .. 7).
__device__ __forceinline__ void bias_word(float (&s)[32], float scale, float slope, const float2 (&step)[4], float d,
                                          bool ahead) {
    if (!ahead) {
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            const float base = -slope * (d + (float)(e & ~7));
            const float2 b = __fadd2_rn(make_float2(base, base), step[(e & 7) >> 1]);
            const float2 y = __ffma2_rn(make_float2(s[e], s[e + 1]), make_float2(scale, scale), b);
            s[e] = y.x;
            s[e + 1] = y.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) s[e] = fmaf(slope, fabsf(d + (float)e), s[e] * scale);
    }
}

// What infinities and NaN in 32 columns of V from `v` on (those of the pool's first row) add to a row that sees positions
// [lo, hi) of a request: a bit a column where it is +infinity, one where it is -infinity, both for NaN.  All lanes of a
// warp together, a row each; a lane looks at every 32nd position of all of them, and only where some element is not
// finite do the rows look at the position.  (Each row by itself, an element at a time, took 32 loads a position, and a
// context of some 10000 of them longer than the other warps' waits last.)
// Written to be short: the loops around it share the instruction cache.
template <bool CODES>
__device__ __forceinline__ uint2 wild_columns(const unsigned char* v, int64_t row, const int32_t* table, int P, int N, int lo,
                                              int hi) {
    constexpr int kWords = CODES ? 8 : 16;               // of 32 columns
    const int lane = threadIdx.x & 31;
    const int last = __reduce_max_sync(0xffffffffu, lo < hi ? hi : 0);
    uint2 got = make_uint2(0u, 0u);
#pragma unroll 1
    for (int base = __reduce_min_sync(0xffffffffu, lo < hi ? lo : INT32_MAX); base < last; base += 32) {
        uint32_t up = 0, down = 0;
        const int at = base + lane;
        const int blk = at < last ? __ldg(table + at / P) : -1;
        if ((unsigned)blk < (unsigned)N) {
            const uint32_t* from = reinterpret_cast<const uint32_t*>(v + ((int64_t)blk * P + at % P) * row);
            uint32_t m = 0;
#pragma unroll 1
            for (int w = 0; w < kWords; w += 4) {
                const uint4 x = __ldg(reinterpret_cast<const uint4*>(from + w));
                if constexpr (CODES) {
                    m |= nan_codes(x);
                } else {
                    const auto full = [](uint32_t y) { return (y & 0x7f807f80u) + 0x00800080u; };
                    m |= (full(x.x) | full(x.y) | full(x.z) | full(x.w)) & 0x80008000u;
                }
            }
            if (m != 0) {
#pragma unroll 1
                for (int e = 0; e < 32; ++e) {
                    const uint32_t bit = 1u << e;
                    if constexpr (CODES) {
                        if ((reinterpret_cast<const unsigned char*>(from)[e] & 0x7f) == 0x7f) up |= bit;
                    } else {
                        const float x = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(from)[e]);
                        if (!(x < INFINITY)) up |= bit;
                        if (!(x > -INFINITY)) down |= bit;
                    }
                }
                if constexpr (CODES) down = up;
            }
        }
#pragma unroll 1
        for (unsigned m = __ballot_sync(0xffffffffu, (up | down) != 0); m != 0; m &= m - 1) {
            const int j = __ffs(m) - 1;
            const uint32_t u = __shfl_sync(0xffffffffu, up, j), d = __shfl_sync(0xffffffffu, down, j);
            if (base + j >= lo && base + j < hi) {
                got.x |= u;
                got.y |= d;
            }
        }
    }
    return got;
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

// x, the same in all lanes, as a value that the compiler knows to be.
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }

template <typename V, int D, int QT, bool CODES>
__global__ void __launch_bounds__(kTcThreads, 1)
    paged_tree_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const typename V::Params p, const int box_tok,
                         const typename std::conditional<CODES, HeadScales, NoScales>::type sc) {
    using L = TtLayout<V, D, QT, CODES>;
    using Rec = RecOf<V>;
    constexpr int kRing = L::kRing;
    extern __shared__ __align__(1024) unsigned char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::bars);
    uint64_t* q_full = bars;
    uint64_t* q_empty = q_full + QT;
    uint64_t* k_full = q_empty + QT;
    uint64_t* k_empty = k_full + L::KS;
    uint64_t* v_full = k_empty + L::KS;
    uint64_t* v_empty = v_full + L::VS;
    uint64_t* v_ready = v_empty + L::VS;
    uint64_t* raw_full = v_ready + L::VS;
    uint64_t* raw_empty = raw_full + L::RS;
    uint64_t* tb = raw_empty + L::RS;
    auto s_full = [&](int t) { return tb + t * 3; };
    auto p_full = [&](int t) { return tb + t * 3 + 1; };
    auto pv_done = [&](int t) { return tb + t * 3 + 2; };
    uint64_t* x_ready = tb + 6;
    uint64_t* x_done = x_ready + 1;
    uint64_t* piece_full = x_done + 1;
    uint64_t* piece_empty = piece_full + kRing;
    uint64_t* mma_end = piece_empty + kRing;
    uint64_t* meet = mma_end + 2;                        // spread: the warps of a stream
    // A scored call's softmax takes a tile in halves of 64 positions, a half's S product being issued while
    // the other's softmax runs: its columns of S are free once P V of the tile before has them read.
    constexpr bool kHalf = L::kHalf;
    // Each half has barriers of its own: a wait tells no phase from the one two before it, and both halves'
    // products may be under way.
    auto s_full_of = [&](int t, int h) { return h == 0 ? s_full(t) : meet + 3 * t; };
    auto p_full_of = [&](int t, int h) { return h == 0 ? p_full(t) : meet + 3 * t + 1; };
    auto pv_done_of = [&](int t, int h) { return h == 0 ? pv_done(t) : meet + 3 * t + 2; };
    Rec* ring = reinterpret_cast<Rec*>(smem + L::ring);
    StartOf<V>* st = reinterpret_cast<StartOf<V>*>(smem + L::start);
    volatile int* misc = reinterpret_cast<volatile int*>(smem + L::misc);
    auto fail = [&]() { misc[1] = 1; };   // reported at the end

    if (warp == kMmaW) {
        tc::alloc(reinterpret_cast<uint32_t*>(smem + L::misc), L::TMEM_COLS);
        tc::relinquish();
    }
    if (threadIdx.x == 0) {
        for (int t = 0; t < QT; ++t) {
            mbar_init(&q_full[t], 1);
            mbar_init(&q_empty[t], QT == 1 ? 2 : 1);
        }
        for (int i = 0; i < L::KS; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], QT);   // QT = 1: a tile belongs to one stream
        }
        for (int i = 0; i < L::VS; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], QT);
            mbar_init(&v_ready[i], kFin);
        }
        for (int i = 0; i < L::RS; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], kFin);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full(t), 1);
            mbar_init(p_full(t), 4);
            mbar_init(pv_done(t), 1);
            mbar_init(&mma_end[t], 1);
            if constexpr (V::kSpread) mbar_init(&meet[t], 4);
            if constexpr (kHalf) {
                mbar_init(s_full_of(t, 1), 1);
                mbar_init(p_full_of(t, 1), 4);
                mbar_init(pv_done_of(t, 1), 1);
            }
        }
        mbar_init(x_ready, kSoftW);
        mbar_init(x_done, kSoftW);
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&piece_full[i], 1);
            mbar_init(&piece_empty[i], kTcThreads / 32 - 1);   // all warps but the walk's
        }
        fence_mbar_init();
        for (const CUtensorMap* m : {&tm_q, &tm_k, &tm_v})
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
        misc[1] = 0;
        for (int i = 0; i < kRing * 4; ++i) smem[L::wild + i] = 0;
    }
    tc::fence_before_sync();
    if constexpr (V::kScored) {
        if (V::kSpread && p.blocks == nullptr)
            scored_begin_here(p, TN, cta, gridDim.x, st, reinterpret_cast<int64_t*>(smem + L::scratch));
        else
            scored_begin(p, cta, gridDim.x, st);
    } else
        tree_begin(p, TN, cta, gridDim.x, st, reinterpret_cast<int64_t*>(smem + L::scratch));
    tc::fence_after_sync();
    const uint32_t tmem = (uint32_t)misc[0];
    const int tok_tile = (V::kSpread ? 32 : TM) / p.G;   // drafts of a query tile
    auto rows_tok_of = [](const Rec& it) {
        if constexpr (V::kScored) return it.k.rows_tok;
        else return it.rows_tok;
    };
    // request, first tile's position, first row of q, and the end of a piece's positions
    auto b_of = [](const Rec& it) {
        if constexpr (V::kScored) return it.k.b;
        else return it.b;
    };
    auto h_of = [](const Rec& it) {
        if constexpr (V::kScored) return it.k.h;
        else return it.h;
    };
    auto at_of = [](const Rec& it) {
        if constexpr (V::kScored) return it.k.tile0 * TN;
        else return 0;
    };
    auto q_row_of = [](const Rec& it) {
        if constexpr (V::kScored) return it.k.q_row;
        else return it.q_row;
    };
    auto end_of = [](const Rec& it) {
        if constexpr (V::kScored) return it.k.hi;
        else return it.kend;
    };
    auto begin_of = [](const Rec& it) {
        if constexpr (V::kScored) return it.k.lo;
        else return 0;
    };
    // steps of stream t over a piece of nt tiles (QT = 2: t's query tile may be empty),
    // and the tile of its step u
    auto steps = [&](const Rec& it, int t) {
        const int nt = it.j1 - it.j0;
        if constexpr (QT == 1) return (nt + 1 - t) >> 1;
        return t == 0 || rows_tok_of(it) > tok_tile ? nt : 0;
    };
    // Tiles of a piece in the rings.  QT = 1: an odd piece is followed by an empty tile, so
    // that stream t's tiles always lie in slots of t's parity.  A parity wait tells a phase
    // from the one two before it only for a waiter that is at most one phase ahead: a stream
    // that met a slot after the other stream's tile in it could take the phase before that
    // tile's for its own.
    auto ring_tiles = [&](int nt) { return QT == 1 ? (nt + 1) & ~1 : nt; };
    auto tile_at = [&](int t, int u) { return QT == 1 ? 2 * u + t : u; };
    auto full_of = [](const Rec& it) {
        if constexpr (V::kScored) return make_int2(it.k.full_lo, it.k.full_hi);
        else return make_int2(0, it.c);
    };
    volatile unsigned char* wild_of = smem + L::wild;
    volatile unsigned char* okm_of = smem + L::okm;
    // the record of piece i, when it is there: false ends a warp's loop
    auto piece = [&](int i) -> bool {
        if (__any_sync(0xffffffffu, misc[1] != 0)) return false;
        if (!mbar_wait_warp(&piece_full[i % kRing], (i / kRing) & 1)) {
            if (lane == 0) fail();
            return false;
        }
        return ring[i % kRing].nt != 0;
    };
    auto piece_done = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&piece_empty[i % kRing]);
    };
    if (warp >= kSoftW) {
        regs_down<kOtherRegs>();
        if (warp == kKW || warp == kVW) {
            // ============================= K and V loads =================================
            // one 16-position box a lane; block ids are read one tile ahead
            const bool isv = warp == kVW;
            const CUtensorMap* tm = isv ? &tm_v : &tm_k;
            const int nslots = !isv ? L::KS : CODES ? L::RS : L::VS;
            const int slot_bytes = !isv ? L::KTILE : CODES ? L::RAW : L::VTILE;
            unsigned char* slots = smem + (!isv ? L::k : CODES ? L::raw : L::v);
            uint64_t* full = !isv ? k_full : CODES ? raw_full : v_full;
            uint64_t* empty = !isv ? k_empty : CODES ? raw_empty : v_empty;
            int x = 0, g = 0;       // slot and number of the next tile
            uint32_t par = 1;       // parity of the slot's last release: 1 passes before the first
            bool ok = true;
            for (int i = 0; ok && piece(i); ++i) {
                const Rec& it = ring[i % kRing];
                const int32_t* trow = p.block_tables + (int64_t)b_of(it) * p.M;
                const int h = h_of(it), kend = end_of(it);
                const int kbegin = V::kScored ? begin_of(it) - 15 : 0;   // of a box that a row sees some of
                // a scored piece's tiles from the last one down (see the softmax)
                constexpr int kOn = V::kScored ? -TN : TN;
                int pos = at_of(it) + (V::kScored ? it.j1 - 1 : it.j0) * TN + lane * 16;
                int real = it.j1 - it.j0;        // what is left of the piece, and of its tiles in the ring
                int left = ring_tiles(real);
                int blk_next = lane < 8 && pos < kend && pos >= kbegin ? __ldg(trow + pos / p.P) : 0;
#pragma unroll 1
                for (; left > 0; --left, --real, pos += kOn, ++g) {
                    const int blk = blk_next;
                    const bool in = lane < 8 && real > 0 && pos < kend && pos >= kbegin;
                    if (real > 1 && lane < 8 && pos + kOn < kend && pos + kOn >= kbegin) blk_next = __ldg(trow + (pos + kOn) / p.P);
                    if (!mbar_wait_warp(&empty[x], par)) {
                        if (lane == 0) fail();
                        ok = false;
                        break;
                    }
                    const bool okb = in && (unsigned)blk < (unsigned)p.N;
                    if (in && !okb && !isv) report(p.dev_status, WF_DEV_BAD_BLOCK);
                    const unsigned okm = __ballot_sync(0xffffffffu, okb);
                    if (lane == 0) {
                        // 16 tiles on, the tile's readers are past it
                        okm_of[(isv ? 16 : 0) + (g & 15)] = (unsigned char)okm;
                        mbar_arrive_expect_tx(&full[x], (uint32_t)__popc(okm) * (uint32_t)L::BOX);
                    }
                    __syncwarp();
                    if (okb) {
                        const int slot = blk * p.P + pos % p.P;   // a multiple of 16
                        unsigned char* dst = slots + x * slot_bytes + lane * L::BOX;
                        if constexpr (L::NC == 2 && !CODES)
                            tma_load_5d(dst, tm, 0, 0, 0, slot >> 3, h, &full[x]);
                        else
                            tma_load_3d_nohint(dst, tm, 0, slot, h, &full[x]);
                    }
                    if (++x == nslots) {
                        x = 0;
                        par ^= 1;
                    }
                }
                piece_done(i);
            }
            if (!mbar_drain_ring(full, nslots, g) && lane == 0) fail();   // see the end of the kernel
        } else if (warp == kWalkW) {
            // ============================= walk, query tiles =============================
            // publishes records as far ahead as the ring allows and loads each piece's query
            // tiles once the products that read the tiles before are done
            typename std::conditional<V::kScored, ScoredWalk<V::kSpread>, TreeWalk>::type walk(*st);
            typename std::conditional<V::kScored, ScoredPiece, TreePiece>::type it;
            bool more = true;
            int made = 0, asked = 0, second = 0;   // records, pieces whose tiles are asked for, second tiles
            int t = 0;
            uint32_t idle = 0;
            while ((more || asked < made) && !__any_sync(0xffffffffu, misc[1] != 0)) {
                bool did = false;
                if (more && (made < kRing || __shfl_sync(0xffffffffu, (int)mbar_test(&piece_empty[made % kRing],
                                                                                      (made / kRing - 1) & 1), 0))) {
                    more = walk.next(p, TN, it);
                    if (lane == 0) {
                        Rec& e = ring[made % kRing];
                        e.nt = more ? it.nt : 0;
                        if constexpr (V::kScored) {
                            if (more) {
                                e.k = it.k;
                                e.k.h = it.h;
                                e.j0 = it.j0;
                                e.j1 = it.j1;
                                e.last = it.j0 == 0 && it.j1 < it.nt ? tree_last(*st, it, cta) : 0;
                            }
                        } else if (more) {
                            e.b = it.b;
                            e.h = it.h;
                            e.tok0 = it.qb * p.tokb;
                            e.q_row = it.q_begin + e.tok0;
                            e.n = it.n;
                            e.rows_tok = it.rows_tok;
                            e.c = it.c;
                            e.kend = it.kend;
                            e.j0 = it.j0;
                            e.j1 = it.j1;
                            e.last = it.j0 == 0 && it.j1 < it.nt ? tree_last(*st, it, cta) : 0;
                        }
                        mbar_arrive(&piece_full[made % kRing]);
                    }
                    __syncwarp();
                    if (more) ++made;
                    did = true;
                }
                if (asked < made) {
                    const Rec& e = ring[asked % kRing];
                    if (CODES && asked == 0) asm volatile("griddepcontrol.wait;" ::: "memory");   // the q parts
                    const int prev = t == 0 ? asked : second;
                    if (prev == 0 || __shfl_sync(0xffffffffu, (int)mbar_test(&q_empty[t], (prev - 1) & 1), 0)) {
                        if (lane == 0) {
                            constexpr int kCopies = V::kSpread ? 4 : 1;   // spread: in every quarter of the tile's rows
                            mbar_arrive_expect_tx(&q_full[t], (uint32_t)(kCopies * 2 * D * box_tok * p.G));
#pragma unroll
                            for (int x = 0; x < kCopies; ++x)
                            if constexpr (CODES) {
#pragma unroll
                                for (int part = 0; part < 2; ++part) {   // hi rows, then lo rows
                                    int row;
                                    if constexpr (V::kScored)
                                        row = part * p.total_q + e.k.q_row;
                                    else
                                        row = (part * p.B + e.b) * p.max_q_len + e.tok0;
                                    tma_load_3d_nohint(smem + L::q + part * (TM * D) + x * 32 * D, &tm_q, 0, h_of(e) * p.G, row, &q_full[t]);
                                }
                            } else {
#pragma unroll
                                for (int cb = 0; cb < L::NC; ++cb)
                                    tma_load_3d_nohint(smem + L::q + t * L::QTILE + cb * (TM * 128) + x * 32 * 128, &tm_q, cb * 64,
                                                       h_of(e) * p.G, q_row_of(e) + t * tok_tile, &q_full[t]);
                            }
                        }
                        __syncwarp();
                        if (QT == 2 && t == 0 && rows_tok_of(e) > tok_tile) {
                            t = 1;
                        } else {
                            second += t;
                            t = 0;
                            ++asked;
                        }
                        did = true;
                    }
                }
                if (did) {
                    idle = 0;
                } else {
                    if (++idle > (1u << 24)) {
                        if (lane == 0) fail();
                        break;
                    }
                    __nanosleep(64);
                }
            }
            bool landed = mbar_drain_warp(&q_full[0], asked + t);
            if constexpr (QT == 2) landed &= mbar_drain_warp(&q_full[1], second);
            if (!landed && lane == 0) fail();
        } else if (warp >= kFinW) {
            // ============================= V finish ======================================
            // a third of a tile's rows each, dealt in turn
            const int fw = warp - kFinW;
            int x = 0, rx = 0, g = 0;       // slots of the V ring and of the ring of codes; tile
            uint32_t par = 0, rpar = 0;
            bool ok = true;
            for (int i = 0; ok && piece(i); ++i) {
                const Rec& it = ring[i % kRing];
                bool wild = false;
                const int j1 = it.j1, kend = end_of(it);
                // positions that every row sees: nothing to look for there
                const int full0 = V::kScored ? full_of(it).x : 0, c0 = full_of(it).y;
                const int kbegin = begin_of(it), at0 = at_of(it);
#pragma unroll 1
                for (int j = it.j0, end = j + ring_tiles(j1 - j); j < end; ++j) {
                    const int k0 = at0 + (V::kScored ? it.j0 + j1 - 1 - j : j) * TN;
                    if (CODES ? !mbar_wait_warp(&raw_full[rx], rpar) || !mbar_wait_warp(&v_empty[x], par ^ 1)
                              : !mbar_wait_warp(&v_full[x], par)) {
                        if (lane == 0) fail();
                        ok = false;
                        break;
                    }
                    const unsigned okm = okm_of[16 + (g & 15)];
                    ++g;
                    unsigned char* base = smem + L::v + x * L::VTILE;
                    const int r0 = min(TN, max(0, c0 - k0)), r1 = min(TN, kend - k0);
                    // scored: rows below rb are nobody's, those below rf not everybody's
                    const int rb = V::kScored ? kbegin - k0 : 0, rf = V::kScored ? full0 - k0 : 0;
                    const bool whole_tile = k0 + TN <= c0 && (!V::kScored || k0 >= full0);
                    if (j >= j1) {
                        // the empty tile
                    } else if constexpr (CODES) {
                        const unsigned char* raw = smem + L::raw + rx * L::RAW;
                        constexpr int kRowChunks = D / 16;       // chunks of 16 codes
                        constexpr int kStep = 32 / kRowChunks;   // rows a warp covers in a round: 4 or 8
                        constexpr int kRounds = TN / kStep;
                        const int ch = lane % kRowChunks, rr = lane / kRowChunks;
                        const int cb = ch >> 2, cc = (ch & 3) * 2;
                        // round y: rows kStep y + rr; where two rounds make an 8-row atom (D = 128), the
                        // odd one's rows are 4 further on, which flips bit 2 of a swizzled chunk's place
                        const unsigned char* src = raw + rr * D + ch * 16;
                        unsigned char* dst = base + cb * L::HALF_OFF + rr * 128;
                        const int o0 = (cc ^ rr) << 4, o1 = ((cc + 1) ^ rr) << 4;
                        auto out_at = [&](int y, int o) {
                            return kStep == 8 ? dst + y * L::ATOM + o
                                              : dst + (y >> 1) * L::ATOM + (y & 1) * 512 + (o ^ ((y & 1) << 6));
                        };
                        auto live = [&](int y) {
                            const int row = kStep * y + rr;
                            return row < r1 && row >= rb && ((okm >> (row >> 4)) & 1u);
                        };
                        uint32_t nan = 0;
                        if (okm == 0xffu && whole_tile) {
                            // All of it cached context: nothing to look for, every place a constant from
                            // the warp's own, so a round is a load, eight conversions and two stores.  (These
                            // warps are few and run in order: with the checks of the other form in it, the
                            // call took 136 us instead of 117, batch of 64.)
                            const unsigned char* from = src + fw * kStep * D;
                            unsigned char* even[2] = {out_at(fw, o0), out_at(fw, o1)};
                            unsigned char* odd[2] = {out_at(fw + kFin, o0), out_at(fw + kFin, o1)};
                            constexpr int kMine = (kRounds + kFin - 1) / kFin;   // the last may be past the tile
                            constexpr int kPair = kStep == 8 ? 2 * kFin * L::ATOM : kFin * L::ATOM;   // two rounds on
                            constexpr int kBatch = (kMine + 1) / 2;
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                uint4 c[kBatch];
#pragma unroll
                                for (int k = 0; k < kBatch; ++k) {
                                    const int m = b * kBatch + k;
                                    if (m < kMine && (m + 1 < kMine || fw + m * kFin < kRounds))
                                        c[k] = ld_shared_v4(from + m * kFin * kStep * D);
                                }
#pragma unroll
                                for (int k = 0; k < kBatch; ++k) {
                                    const int m = b * kBatch + k;
                                    if (m < kMine && (m + 1 < kMine || fw + m * kFin < kRounds)) {
                                        uint32_t v[8];
                                        e4m3x16_to_f16(c[k], v);
                                        unsigned char* const* to = (m & 1) ? odd : even;
                                        const int at = (m >> 1) * kPair;
                                        *reinterpret_cast<uint4*>(to[0] + at) = make_uint4(v[0], v[1], v[2], v[3]);
                                        *reinterpret_cast<uint4*>(to[1] + at) = make_uint4(v[4], v[5], v[6], v[7]);
                                    }
                                }
                            }
                        } else {
                            constexpr int kBatch = 2;
#pragma unroll 1
                            for (int y0 = fw; y0 < kRounds; y0 += kFin * kBatch) {
                                uint4 c[kBatch];
#pragma unroll
                                for (int k = 0; k < kBatch; ++k) {
                                    const int y = y0 + k * kFin;
                                    c[k] = make_uint4(0u, 0u, 0u, 0u);
                                    if (y < kRounds && live(y)) c[k] = ld_shared_v4(src + y * kStep * D);
                                }
#pragma unroll
                                for (int k = 0; k < kBatch; ++k) {
                                    const int y = y0 + k * kFin;
                                    if (y >= kRounds) break;
                                    uint32_t v[8];
                                    e4m3x16_to_f16(c[k], v);
                                    if (kStep * y + rr >= r0 || kStep * y + rr < rf) nan |= nan_codes(c[k]);
                                    *reinterpret_cast<uint4*>(out_at(y, o0)) = make_uint4(v[0], v[1], v[2], v[3]);
                                    *reinterpret_cast<uint4*>(out_at(y, o1)) = make_uint4(v[4], v[5], v[6], v[7]);
                                }
                            }
                        }
                        if (__any_sync(0xffffffffu, nan != 0)) {
                            // a draft's NaN elements are set aside
#pragma unroll 1
                            for (int y = fw; y < kRounds; y += kFin) {
                                if (!live(y) || (kStep * y + rr < r0 && kStep * y + rr >= rf)) continue;
#pragma unroll 1
                                for (int e = 0; e < 16; ++e) {
                                    if ((src[y * kStep * D + e] & 0x7f) != 0x7f) continue;
                                    *reinterpret_cast<unsigned short*>(out_at(y, e < 8 ? o0 : o1) + (e & 7) * 2) = 0;
                                    wild = true;
                                }
                            }
                        }
                        tc::fence_proxy_async_smem();
                    } else if (okm != 0xffu || !whole_tile) {
                        // 16-byte chunk cc of row r (its place within the swizzle does not matter);
                        // with every block id in range, the rows before the first draft stay
                        const int first = !V::kScored && okm == (1u << ((r1 + 15) >> 4)) - 1u ? r0 : 0;
                        constexpr int kRowChunks = L::NC * 8;
                        constexpr int kStep = 32 / kRowChunks;
                        const int rr = lane / kRowChunks, cb = (lane >> 3) % L::NC, cc = lane & 7;
                        for (int r = first + fw * kStep + rr; r < TN; r += kFin * kStep) {
                            uint4* at = reinterpret_cast<uint4*>(base + (r >> 3) * L::ATOM + cb * L::HALF_OFF +
                                                                 (r & 7) * 128 + cc * 16);
                            if (r >= r1 || r < rb || !((okm >> (r >> 4)) & 1u)) {
                                *at = make_uint4(0u, 0u, 0u, 0u);
                            } else if (r >= r0 || r < rf) {
                                uint4 v = *at;
                                bool w = tame(v.x);
                                w |= tame(v.y);
                                w |= tame(v.z);
                                w |= tame(v.w);
                                if (w) *at = v;
                                wild |= w;
                            }
                        }
                        tc::fence_proxy_async_smem();
                    }
                    wild = __any_sync(0xffffffffu, wild);
                    if (lane == 0) {
                        if (j + 1 == j1) wild_of[(i % kRing) * 4 + fw] = wild ? 1 : 0;
                        mbar_arrive(&v_ready[x]);
                        if constexpr (CODES) mbar_arrive(&raw_empty[rx]);
                    }
                    if (++x == L::VS) {
                        x = 0;
                        par ^= 1;
                    }
                    if (CODES && ++rx == L::RS) {
                        rx = 0;
                        rpar ^= 1;
                    }
                }
                piece_done(i);
            }
        } else {
            // ============================= MMA issue =====================================
            // One warp a stream: its products run in order S(0), P(0) V, S(1), P(1) V, ...: S(u + 1)
            // overwrites the columns P(u) lives in, and the tensor core executes one thread's
            // products in issue order.  One issuer for both streams was the bound at 16 products a
            // tile and stream.
            constexpr int kSN = kHalf ? TN / 2 : TN;
            constexpr uint32_t idS = CODES ? tc::idesc_e4m3_f32(TM, kSN, 0, 0) : tc::idesc_bf16_f32(TM, kSN, 0, 0);
            constexpr uint32_t idO = CODES ? tc::idesc_f16_f32(TM, D, 0, 1) : tc::idesc_bf16_f32(TM, D, 0, 1);
            // An MMA takes its operands from uniform registers.  The slots and parities here are the
            // same in all lanes, and are kept so that the compiler sees it: otherwise each of a
            // product's operands is moved over, MMA by MMA, and issuing took longer than computing.
            const int t = uniform(warp) - kMmaW;
            const int tq = QT == 1 ? 0 : t;
            // K-major rows of 128 bytes, or (codes, D = 64) of 64
            auto kmajor = [](uint32_t at, uint32_t atom) {
                return CODES && D == 64 ? tc::sdesc_sw64(at, 16, 512) : tc::sdesc_sw128(at, 16, CODES ? 1024 : atom);
            };
            const uint64_t qdesc = kmajor(smem_u32(smem + L::q + tq * L::QTILE), 1024);
            const uint64_t kdesc = kmajor(smem_u32(smem + L::k), L::ATOM);
            const uint64_t vdesc = tc::sdesc_sw128(smem_u32(smem + L::v), L::HALF_OFF, L::ATOM);
            const uint32_t tm = (uint32_t)uniform((int)tmem);
            const uint32_t dS = tm + t * L::SCOL, dO = tm + L::OCOL + t * D;
            int kx = 0, vx = 0;                 // slots of the next tile
            uint32_t kpar = 0, vpar = 0;        // and their parities
            uint32_t qpar = 0, ppar = 0;
            bool ok = true;
            auto need = [&](uint64_t* bar, uint32_t par) {
                // (of all lanes: none may still be polling when one hands the barrier's slot on)
                if (ok && !mbar_wait_warp(bar, par)) {
                    if (lane == 0) fail();
                    ok = false;
                }
                return ok;
            };
            auto step = [&](int& x, uint32_t& par, int n) {
                if (++x == n) {
                    x = 0;
                    par ^= 1;
                }
            };
            auto advance = [&]() {              // to the stream's next tile
#pragma unroll
                for (int k = 0; k < (QT == 1 ? 2 : 1); ++k) {
                    step(kx, kpar, L::KS);
                    step(vx, vpar, L::VS);
                }
            };
            if (QT == 1 && t == 1) {            // the first tile is stream 0's
                step(kx, kpar, L::KS);
                step(vx, vpar, L::VS);
            }
            for (int i = 0; ok && __all_sync(0xffffffffu, piece(i)); ++i) {
                const Rec& it = ring[i % kRing];
                const int nt = uniform(steps(it, t)), all = uniform(it.j1 - it.j0);
                if (QT == 2 && nt == 0) {       // no rows: hand the tiles on as they land
                    for (int u = 0; u < all && ok; ++u) {
                        if (need(&k_full[kx], kpar) && lane == 0) mbar_arrive(&k_empty[kx]);
                        if (need(&v_ready[vx], vpar) && lane == 0) mbar_arrive(&v_empty[vx]);
                        advance();
                    }
                    piece_done(i);
                    continue;
                }
                if (!need(&q_full[tq], qpar)) break;
                qpar ^= 1;
                if (nt == 0 && lane == 0) mbar_arrive(&q_empty[tq]);
                if constexpr (kHalf) {
                    // S(0) in both halves, then P(u) V and S(u + 1) half by half
                    const auto issue_s = [&](int h, bool last) {
                        if (elect_one()) {
                            const uint32_t kd = (uint32_t)kdesc + ((kx * L::KTILE + h * (L::KTILE / 2)) >> 4), qd = (uint32_t)qdesc;
                            const uint32_t khi = (uint32_t)(kdesc >> 32), qhi = (uint32_t)(qdesc >> 32);
                            if constexpr (CODES) {       // the two parts of q, one after the other
#pragma unroll
                                for (int x = 0; x < 2 * D / 32; ++x) {
                                    const int part = x / (D / 32), kk = x % (D / 32);
                                    mma<2>(dS + h * 64, qd + ((part * TM * D + kk * 32) >> 4), qhi, kd + ((kk * 32) >> 4), khi,
                                           idS, x > 0 ? 1u : 0u);
                                }
                            } else {
#pragma unroll
                                for (int kk = 0; kk < D / 16; ++kk) {
                                    const uint32_t qoff = (kk >> 2) * (TM * 128) + (kk & 3) * 32;
                                    const uint32_t koff = (kk >> 2) * L::HALF_OFF + (kk & 3) * 32;
                                    mma<0>(dS + h * 64, qd + (qoff >> 4), qhi, kd + (koff >> 4), khi, idS, kk > 0 ? 1u : 0u);
                                }
                            }
                            tc::commit(s_full_of(t, h));
                            if (h == 1) {
                                tc::commit(&k_empty[kx]);
                                if (last) tc::commit(&q_empty[tq]);
                            }
                        }
                        __syncwarp();
                    };
                    const auto next_k = [&]() {
#pragma unroll
                        for (int k = 0; k < (QT == 1 ? 2 : 1); ++k) step(kx, kpar, L::KS);
                    };
                    if (nt > 0 && need(&k_full[kx], kpar)) {
                        tc::fence_after_sync();
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) issue_s(h, h == 1 && nt == 1);
                        next_k();
                    }
#pragma unroll 1
                    for (int u = 0; u < nt && ok; ++u) {
                        if (!need(&v_ready[vx], vpar)) break;
                        const uint32_t vd = (uint32_t)vdesc + ((vx * L::VTILE) >> 4);
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
                            if (!need(p_full_of(t, h), ppar)) break;
                            tc::fence_after_sync();
                            if (elect_one()) {
#pragma unroll
                                for (int kk = 0; kk < TN / 32; ++kk)
                                    mma<1>(dO, dS + h * 64 + kk * 8, 0u, vd + (((h * (TN / 32) + kk) * 2 * L::ATOM) >> 4),
                                           (uint32_t)(vdesc >> 32), idO, (u > 0 || h > 0 || kk > 0) ? 1u : 0u);
                                if (h == 1) tc::commit(&v_empty[vx]);
                                tc::commit(pv_done_of(t, h));
                            }
                            __syncwarp();
                            if (u + 1 < nt) {
                                if (h == 0 && !need(&k_full[kx], kpar)) break;
                                tc::fence_after_sync();
                                issue_s(h, u + 2 == nt);
                            }
                        }
                        if (!ok) break;
                        ppar ^= 1;
                        if (u + 1 < nt) next_k();
#pragma unroll
                        for (int k = 0; k < (QT == 1 ? 2 : 1); ++k) step(vx, vpar, L::VS);
                    }
                } else {
#pragma unroll 1
                    for (int u = -1; u < nt && ok; ++u) {
                        // P V of step u ...
                        if (u >= 0) {
                            if (!need(&v_ready[vx], vpar) || !need(p_full(t), ppar)) break;
                            ppar ^= 1;
                            tc::fence_after_sync();
                            const uint32_t vd = (uint32_t)vdesc + ((vx * L::VTILE) >> 4);
                            if (elect_one()) {
#pragma unroll
                                for (int kk = 0; kk < TN / 16; ++kk)
                                    mma<1>(dO, dS + kk * 8 + (kk >= 4 ? 32 : 0), 0u, vd + ((kk * 2 * L::ATOM) >> 4),
                                           (uint32_t)(vdesc >> 32), idO, (u > 0 || kk > 0) ? 1u : 0u);
                                tc::commit(&v_empty[vx]);
                                tc::commit(pv_done(t));
                            }
                            __syncwarp();
                            advance();
                        }
                        // ... then S of step u + 1
                        if (u + 1 < nt) {
                            if (!need(&k_full[kx], kpar)) break;
                            tc::fence_after_sync();
                            if (elect_one()) {
                                const uint32_t kd = (uint32_t)kdesc + ((kx * L::KTILE) >> 4), qd = (uint32_t)qdesc;
                                const uint32_t khi = (uint32_t)(kdesc >> 32), qhi = (uint32_t)(qdesc >> 32);
                                if constexpr (CODES) {       // the two parts of q, one after the other
#pragma unroll
                                    for (int x = 0; x < 2 * D / 32; ++x) {
                                        const int part = x / (D / 32), kk = x % (D / 32);
                                        mma<2>(dS, qd + ((part * TM * D + kk * 32) >> 4), qhi, kd + ((kk * 32) >> 4), khi, idS,
                                               x > 0 ? 1u : 0u);
                                    }
                                } else {
#pragma unroll
                                    for (int kk = 0; kk < D / 16; ++kk) {
                                        const uint32_t qoff = (kk >> 2) * (TM * 128) + (kk & 3) * 32;
                                        const uint32_t koff = (kk >> 2) * L::HALF_OFF + (kk & 3) * 32;
                                        mma<0>(dS, qd + (qoff >> 4), qhi, kd + (koff >> 4), khi, idS, kk > 0 ? 1u : 0u);
                                    }
                                }
                                tc::commit(s_full(t));
                                tc::commit(&k_empty[kx]);
                                if (u + 2 == nt) tc::commit(&q_empty[tq]);
                            }
                            __syncwarp();
                        }
                    }
                }
                if (QT == 1 && ok && 2 * nt + t < ring_tiles(all)) {   // stream 1's empty tile: hand it back
                    if (need(&k_full[kx], kpar) && lane == 0) mbar_arrive(&k_empty[kx]);
                    if (need(&v_ready[vx], vpar) && lane == 0) mbar_arrive(&v_empty[vx]);
                    advance();
                }
                piece_done(i);
            }
            if (elect_one()) tc::commit(&mma_end[t]);
            if (!mbar_drain_warp(&mma_end[t], 1) && lane == 0) fail();
        }
    } else {
        // ============================= softmax =======================================
        regs_up<kSoftRegs>();
        const int t = warp >> 2;
        const int quad = warp & 3;
        const int r = quad * 32 + lane;                  // TMEM lane
        const uint32_t lane_addr = (uint32_t)(quad * 32) << 16;
        const uint32_t sbase = tmem + lane_addr + t * L::SCOL;
        const uint32_t obase = tmem + lane_addr + L::OCOL + t * D;
        unsigned char* stage = smem + L::stage + warp * 4096;
        const int tr = V::kSpread ? lane : r;            // row of the query tile
        const int tok = (QT == 2 ? t * tok_tile : 0) + tr / p.G;
        const bool row_fits = tr < tok_tile * p.G;
        constexpr int kWords = V::kSpread ? 1 : kHalf ? 2 : 4;   // runs of 32 positions that a thread takes at once
        constexpr int kSteps = kHalf ? 2 : 1;            // and how often in a tile
        int hf = 0;                                      // half tiles: which
        auto word = [&](int w) { return V::kSpread ? quad : kHalf ? 2 * hf + w : w; };
        int met = 0;                                     // spread: meetings of the stream's warps
        auto meeting = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(&meet[t]);
            const bool came = mbar_wait_warp(&meet[t], met & 1);
            ++met;
            if (!came && lane == 0) fail();
            return came;
        };
        const int g_inv = (65536 + p.G - 1) / p.G;       // row / G for rows below 128
        constexpr bool kCap = V::kCap, kBias = V::kBias, kWide = V::kWide;
        float scale = kCap ? cap_in_of(p) : p.scale_log2;
        const bool negate = V::kRule == kRulePlain && p.scale_log2 < 0.f;
        int4 rec = make_int4(0, 0, 0, 0);
        const float fill = negate ? INFINITY : -INFINITY;   // of a masked score: a weight of 0
        int gs = 0, g = 0;   // steps of the stream and tiles before this piece
        bool ok = true;
        for (int i = 0; ok && piece(i); ++i) {
            const Rec& it = ring[i % kRing];
            const int nt = steps(it, t);
            const bool row_valid = row_fits && tok < rows_tok_of(it);
            const bool warp_live = __any_sync(0xffffffffu, row_valid);
            const int j0 = it.j0, at0 = at_of(it);
            const int q_row = q_row_of(it) + (row_valid ? tok : 0);   // this row's draft
            const int32_t* trow = p.block_tables + (int64_t)b_of(it) * p.M;
            int c = 0, n = 0;
            const uint32_t* mrow = nullptr;
            int2 sees = make_int2(0, 0);                              // scored: the row's positions
            float slope = 0.f;                                        // and its bias, slope |p - ref|
            int ref = 0;
            float2 step[4] = {};
            int all_lo = 0, all_hi = 0;                               // positions that all of the warp's rows see
            bool ahead = false;                                       // some row sees past its own position
            if constexpr (V::kScored) {
                const int at = it.k.at + tok;
                // (a row that is not there sees what the others do, so that it holds nobody up)
                sees = row_valid ? scored_range(p, q_row, at, it.k.len) : make_int2(0, INT32_MAX);
                if constexpr (kBias) {
                    if (row_valid) {
                        slope = -1.4426950408889634f * __ldg(p.slopes + h_of(it) * p.G + tr % p.G);
                        // distances from the nearest position that the row sees on its own side: a shift of
                        // all its scores, which keeps far rows' distances exact
                        ref = min(at, sees.y - 1);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) step[e] = make_float2(-slope * (float)(2 * e), -slope * (float)(2 * e + 1));
                    ahead = __any_sync(0xffffffffu, row_valid && sees.y > at + 1);
                }
                all_lo = __reduce_max_sync(0xffffffffu, sees.x);
                all_hi = __reduce_min_sync(0xffffffffu, sees.y);
            } else {
                c = it.c;
                n = it.n;
                mrow = p.mask + (int64_t)q_row * p.W;
            }
            float v_scale = 1.f;
            if constexpr (CODES) {
                if (i == 0) asm volatile("griddepcontrol.wait;" ::: "memory");   // the q rows' factors
                const int hs = min(h_of(it), kMaxScaleHeads - 1);
                int64_t row;
                if constexpr (V::kScored)
                    row = (int64_t)q_row * p.H_q + h_of(it) * p.G + tr % p.G;
                else
                    row = ((int64_t)it.b * p.max_q_len + it.tok0 + tok) * p.H_q + h_of(it) * p.G + tr % p.G;
                const float inv = row_valid ? __ldcg(p.q_inv + row) : 1.f;
                scale = kCap ? cap_in_of(p) * sc.k[hs] * inv : tree_factor(p.scale_log2 * sc.k[hs] * inv);
                v_scale = sc.v[hs];
            }
            float m_ref = -INFINITY, l_run = 0.f;
#pragma unroll 1
            for (int su = 0; su < nt * kSteps; ++su) {
                const int u = su / kSteps;
                hf = su % kSteps;
                // Scored: the last tile first.  Where a bias grows towards a row's own position its maximum is there, and
                // later tiles do not move it (from the first on they did almost each time: prompts with slopes 294 us).
                const int k0 = at0 + (V::kScored ? it.j1 - 1 - tile_at(t, u) : j0 + tile_at(t, u)) * TN;
                // positions of this tile that the row sees, when it is not all of them
                bool masked;
                uint32_t vis[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
                if constexpr (V::kScored) {
                    masked = all_lo > k0 + 32 * word(0) || all_hi < k0 + 32 * word(kWords - 1) + 32;
                } else {
                    masked = k0 + TN > c;
                    if (warp_live && masked) {
#pragma unroll
                        for (int w = 0; w < 4; ++w) vis[w] = row_valid ? mask_bits(mrow, p.W, k0 + 32 * w - c, n) : 0u;
                    }
                }
                // Scored: S is there more often than not, so one poll stands before the loop (packed documents 206 -> 200 us,
                // prompts with a bias 223 -> 214; of the other waits it only made the code longer: capped prompts 278 -> 303).
                uint64_t* made_s = kHalf ? s_full_of(t, hf) : s_full(t);
                if (!(V::kScored && __all_sync(0xffffffffu, mbar_try_wait(made_s, (gs + u) & 1))) &&
                    !mbar_wait_warp(made_s, (gs + u) & 1)) {
                    if (lane == 0) fail();
                    ok = false;
                    break;
                }
                if constexpr (V::kScored) {
                    if (warp_live) {
                        tc::fence_after_sync();
                        const uint32_t okm = okm_of[(g + tile_at(t, u)) & 15];
                        masked |= okm != 0xffu;
                        uint32_t seen[kWords];
                        bool idle = false;              // none of it is seen by the warp's rows
                        if (masked) {
                            uint32_t some = 0;
#pragma unroll
                            for (int w = 0; w < kWords; ++w) {
                                seen[w] = range_bits(sees.x, sees.y, k0 + 32 * word(w)) &
                                          (((okm >> (2 * word(w))) & 1u ? 0xffffu : 0u) |
                                           ((okm >> (2 * word(w) + 1)) & 1u ? 0xffff0000u : 0u));
                                some |= seen[w];
                            }
                            idle = __all_sync(0xffffffffu, some == 0);
                        }
                        if (idle) {
                            const uint32_t zeros[16] = {};
#pragma unroll
                            for (int w = 0; w < 4; ++w)
                                if (!kHalf || w / 2 == hf) st_16words(sbase + (w >> 1) * 64 + (w & 1) * 16, zeros);
                            tc::wait_st();
                            tc::fence_before_sync();
                        } else {
                            // the row's positions in registers
                            float s[kWords][32];
#pragma unroll
                            for (int w = 0; w < kWords; ++w) tc::ld_32cols(sbase + word(w) * 32, s[w]);
                            tc::wait_ld();
                            const Cap cap(scale, cap_out_of(p));
                            bool near = false;
                            float top = -INFINITY, low = INFINITY;
                            if constexpr (kCap) {
                                // Only in a tile that all rows see: what is not seen must not choose the way, which changes
                                // last bits.  (Chosen among what is seen it cost 231 decodes 271 us instead of 264.)
                                if (!masked) {
#pragma unroll
                                    for (int w = 0; w < kWords; ++w) extremes<true>(s[w], top, low);
                                    near = scale > 0.f &&
                                           __all_sync(0xffffffffu, !row_valid || fmaxf(top, -low) * scale <= kTanhNear);
                                }
                            }
                            // Scores that are final before the weights: biased ones, and capped ones of the longer way.
                            const bool made = kBias || (kCap && !near);
                            if constexpr (kCap) {
                                const auto capped = [&](auto f) {
#pragma unroll
                                    for (int w = 0; w < kWords; ++w)
#pragma unroll
                                        for (int e = 0; e < 32; e += 2) {
                                            const float2 y = f(make_float2(s[w][e], s[w][e + 1]), make_float2(0.f, 0.f));
                                            s[w][e] = y.x;
                                            s[w][e + 1] = y.y;
                                        }
                                };
                                if (!near)
                                    capped([&](float2 x, float2) { return kWide ? cap.either(x) : cap.far(x); });
                                else if (kBias)
                                    capped([&](float2 x, float2 none) { return cap.near(x, none); });
                            }
                            if constexpr (kBias) {
#pragma unroll
                                for (int w = 0; w < kWords; ++w)
                                    bias_word(s[w], kCap ? 1.f : scale, slope, step, (float)(k0 + 32 * word(w) - ref), ahead);
                            }
                            if (masked) {
#pragma unroll
                                for (int w = 0; w < kWords; ++w) {
                                    for (int e = 0; e < 32; ++e) s[w][e] = (seen[w] >> e) & 1u ? s[w][e] : fill;
                                }
                            }
                            if (!kCap || made) {
                                top = -INFINITY;
                                if (negate) {   // the largest scaled score is the smallest score's
                                    float no = 0.f;
                                    low = INFINITY;
#pragma unroll
                                    for (int w = 0; w < kWords; ++w) extremes<true>(s[w], no, low);
                                } else {
#pragma unroll
                                    for (int w = 0; w < kWords; ++w) extremes<false>(s[w], top, low);
                                }
                            }
                            float mt = V::kRule != kRulePlain ? top : negate ? low * scale : top * scale;
                            if constexpr (kCap && !kBias) {
                                // tanh keeps their order
                                if (near) mt = cap.near(make_float2(top, top), make_float2(0.f, 0.f)).x;
                            }
                            float alpha = 1.f;
                            if (m_ref == -INFINITY) {
                                m_ref = mt;
                            } else if (row_valid && mt > m_ref + (CODES ? kLazyMax : kLazyFar)) {
                                alpha = ex2(m_ref - mt);
                                m_ref = mt;
                            }
                            if (__any_sync(0xffffffffu, alpha != 1.f)) {
                                if (!mbar_wait_warp(kHalf ? pv_done_of(t, hf ^ 1) : pv_done(t),
                                                    (kHalf && hf == 1 ? gs + u : gs + u - 1) & 1))
                                    fail();
                                tc::fence_after_sync();
    #pragma unroll 1
                                for (int c = 0; c < D; c += 16) {
                                    float o[16];
                                    uint32_t w[16];
                                    tc::ld_16cols(obase + c, o);
                                    tc::wait_ld();
    #pragma unroll
                                    for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * alpha);
                                    st_16words(obase + c, w);
                                }
                                tc::wait_st();
                            }
                            l_run *= alpha;
                            const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
                            const float up = CODES ? kCodesUp - m_use : -m_use;
                            const float2 nm2 = make_float2(up, up), sc2 = make_float2(scale, scale);
                            float2 ps[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                                            make_float2(0.f, 0.f)};
                            // the weights of positions 0-63 take columns 0-31, those of 64-127 columns 64-95
                            const auto weigh = [&](auto score) {
#pragma unroll
                                for (int w = 0; w < kWords; ++w) {
                                    uint32_t pw[16];
#pragma unroll
                                    for (int v = 0; v < 16; ++v) {
                                        const float2 x = score(make_float2(s[w][2 * v], s[w][2 * v + 1]));
                                        const float2 e2 = make_float2(ex2(x.x), ex2(x.y));
                                        ps[v & 3] = __fadd2_rn(ps[v & 3], e2);
                                        pw[v] = CODES ? pack_f16x2(e2.x, e2.y) : pack_bf16x2(e2.x, e2.y);
                                    }
                                    st_16words(sbase + (word(w) >> 1) * 64 + (word(w) & 1) * 16, pw);
                                }
                            };
                            if constexpr (V::kRule == kRulePlain) {
                                weigh([&](float2 x) { return __ffma2_rn(x, sc2, nm2); });
                            } else if (kCap && !kBias && near) {
                                weigh([&](float2 x) { return cap.near(x, nm2); });
                            } else {
                                weigh([&](float2 x) { return __fadd2_rn(x, nm2); });
                            }
                            if constexpr (V::kSpread) {          // the other positions are other quarters'
                                const uint32_t zeros[16] = {};
#pragma unroll
                                for (int w = 1; w < 4; ++w) {
                                    const int x = (quad + w) & 3;
                                    st_16words(sbase + (x >> 1) * 64 + (x & 1) * 16, zeros);
                                }
                            }
                            tc::wait_st();
                            const float2 ps01 = __fadd2_rn(ps[0], ps[1]), ps23 = __fadd2_rn(ps[2], ps[3]);
                            const float2 pst = __fadd2_rn(ps01, ps23);
                            l_run += pst.x + pst.y;
                            tc::fence_before_sync();
                        }
                    }
                } else if (warp_live) {
                    tc::fence_after_sync();
                    const uint32_t okm = okm_of[(g + tile_at(t, u)) & 15];
                    if (!masked && okm != 0xffu) masked = true;
                    if (masked) {   // boxes past the request's end are not in okm either
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            vis[w] &= ((okm >> (2 * w)) & 1u ? 0xffffu : 0u) |
                                      ((okm >> (2 * w + 1)) & 1u ? 0xffff0000u : 0u);
                    }
                    // the whole row in registers: one TMEM round trip a tile
                    float s[4][32];
#pragma unroll
                    for (int w = 0; w < 4; ++w) tc::ld_32cols(sbase + w * 32, s[w]);
                    tc::wait_ld();
                    if (masked) {
#pragma unroll
                        for (int w = 0; w < 4; ++w)
#pragma unroll
                            for (int e = 0; e < 32; ++e) s[w][e] = (vis[w] >> e) & 1u ? s[w][e] : fill;
                    }
                    float m8[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) m8[e] = fmax3(s[0][e], s[0][e + 8], s[0][e + 16]);
#pragma unroll
                    for (int w = 1; w < 4; ++w)
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            m8[e] = fmax3(m8[e], s[w - 1][e + 24], s[w][e]);
                            m8[e] = fmax3(m8[e], s[w][e + 8], s[w][e + 16]);
                        }
#pragma unroll
                    for (int e = 0; e < 8; ++e) m8[e] = fmaxf(m8[e], s[4 - 1][e + 24]);
                    float top = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
                    if (negate) {   // the largest scaled score is the smallest score's
                        top = INFINITY;
#pragma unroll
                        for (int w = 0; w < 4; ++w)
#pragma unroll
                            for (int e = 0; e < 32; ++e) top = fminf(top, s[w][e]);
                    }
                    const float mt = top * scale;
                    float alpha = 1.f;
                    if (m_ref == -INFINITY) {
                        m_ref = mt;
                    } else if (row_valid && mt > m_ref + kLazyMax) {
                        alpha = ex2(m_ref - mt);
                        m_ref = mt;
                    }
                    if (__any_sync(0xffffffffu, alpha != 1.f)) {
                        if (!mbar_wait_warp(pv_done(t), (gs + u - 1) & 1)) fail();
                        tc::fence_after_sync();
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            float o[16];
                            uint32_t w[16];
                            tc::ld_16cols(obase + c, o);
                            tc::wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * alpha);
                            st_16words(obase + c, w);
                        }
                        tc::wait_st();
                    }
                    l_run *= alpha;
                    const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
                    const float2 sc2 = make_float2(scale, scale);
                    const float up = CODES ? kCodesUp - m_use : -m_use;
                    const float2 nm2 = make_float2(up, up);
                    float2 ps[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                                    make_float2(0.f, 0.f)};
                    // the weights of positions 0-63 take columns 0-31, those of 64-127 columns 64-95
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t pw[16];
#pragma unroll
                        for (int v = 0; v < 16; ++v) {
                            const float2 x = __ffma2_rn(make_float2(s[w][2 * v], s[w][2 * v + 1]), sc2, nm2);
                            const float2 e2 = make_float2(ex2(x.x), ex2(x.y));
                            ps[v & 3] = __fadd2_rn(ps[v & 3], e2);
                            pw[v] = CODES ? pack_f16x2(e2.x, e2.y) : pack_bf16x2(e2.x, e2.y);
                        }
                        st_16words(sbase + (w >> 1) * 64 + (w & 1) * 16, pw);
                    }
                    tc::wait_st();
                    const float2 ps01 = __fadd2_rn(ps[0], ps[1]), ps23 = __fadd2_rn(ps[2], ps[3]);
                    const float2 pst = __fadd2_rn(ps01, ps23);
                    l_run += pst.x + pst.y;
                    tc::fence_before_sync();
                }
                __syncwarp();
                // the first P of a piece lets P V overwrite O, which the last piece's join reads
                if (QT == 1 && su == 0 && i > 0 && !mbar_wait_warp(x_done, (i - 1) & 1)) {
                    if (lane == 0) fail();
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_arrive(kHalf ? p_full_of(t, hf) : p_full(t));
            }
            if (!ok) break;
            // ---- epilogue: the rows, or this piece of them ------------------------------
            if (nt > 0 && !mbar_wait_warp(kHalf ? pv_done_of(t, 1) : pv_done(t), (gs + nt - 1) & 1)) {
                if (lane == 0) fail();
                break;
            }
            gs += nt;
            g += ring_tiles(it.j1 - it.j0);
            const bool whole = it.j0 == 0 && it.j1 == it.nt;
            float w0 = 1.f, w1 = 0.f;                     // weights of the streams' O (QT = 1)
            const float2* ml = reinterpret_cast<const float2*>(smem + L::ml);
            if constexpr (QT == 1) {
                if (nt == 0 && i > 0 && !mbar_wait_warp(x_done, (i - 1) & 1)) {
                    if (lane == 0) fail();
                    break;
                }
                reinterpret_cast<float2*>(smem + L::ml)[t * TM + r] = make_float2(m_ref, l_run);
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(x_ready);
                if (!mbar_wait_warp(x_ready, i & 1)) {
                    if (lane == 0) fail();
                    break;
                }
                const float2 a = ml[r], b = ml[TM + r];
                float mm = fmaxf(a.x, b.x);
                if constexpr (V::kSpread) {
#pragma unroll
                    for (int x = 1; x < 4; ++x) {
                        const int at = ((quad + x) & 3) * 32 + lane;
                        mm = fmax3(mm, ml[at].x, ml[TM + at].x);
                    }
                }
                // a stream without a maximum has a sum and an O of 0, or of NaN, which has to stay
                w0 = a.x == -INFINITY ? 1.f : ex2(a.x - mm);
                w1 = b.x == -INFINITY ? 1.f : ex2(b.x - mm);
                m_ref = mm;
                l_run = w0 * a.y + w1 * b.y;
                if constexpr (V::kSpread) {              // in one order in all quarters
                    l_run = 0.f;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const float2 e = ml[y * TM + x * 32 + lane];
                            l_run += (e.x == -INFINITY ? 1.f : ex2(e.x - mm)) * e.y;
                        }
                    }
                }
            }
            tc::fence_after_sync();
            const bool both = QT == 1 && it.j1 - it.j0 > 1;    // stream 1 has an O
            const bool wild = reinterpret_cast<const volatile uint32_t*>(wild_of)[i % kRing] != 0;
            const int slot_of_piece = tree_piece_slot(cta, j0);
            // this query tile: its rows, first draft row of q, first row of the workspace
            const int t0 = QT == 2 ? t * tok_tile : 0;
            const int live_rows = min(tok_tile, rows_tok_of(it) - t0) * p.G;
            const int tile_row = q_row_of(it) + t0;
            const int64_t wbase = (int64_t)slot_of_piece * p.rows + t0 * p.G;
            if (!whole) {
                if (it.j0 == 0) rec = make_int4(q_row_of(it), h_of(it), it.last, rows_tok_of(it) * p.G);
                if (row_valid && (QT == 2 || t == 0) && (!V::kSpread || quad == 0)) p.ws_ml[wbase + tr] = make_float2(m_ref, l_run);
            }
            const float f = v_scale * (!whole ? 1.f : l_run == 0.f ? 0.f : 1.f / l_run);
            w0 *= f;
            w1 *= f;
            constexpr int kParts = QT == 1 ? D / 64 : D / 32;      // 32-column groups of this warp
            bool odd = false;                                      // spread: a sum that is not finite
            if (nt > 0 || QT == 1) {
#pragma unroll 1
                for (int part = 0; part < kParts; ++part) {
                    const int col = (QT == 1 ? t * (D / 2) : 0) + part * 32;
                    float o[32];
                    if (warp_live) {
                        if constexpr (QT == 1) {
                            tc::ld_32cols(tmem + lane_addr + L::OCOL + col, o);
                            tc::wait_ld();
                            scale32(o, w0);
                            if (both) {
                                float o1[32];
                                tc::ld_32cols(tmem + lane_addr + L::OCOL + D + col, o1);
                                tc::wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const float2 y = __ffma2_rn(make_float2(o1[e], o1[e + 1]), make_float2(w1, w1),
                                                                make_float2(o[e], o[e + 1]));
                                    o[e] = y.x;
                                    o[e + 1] = y.y;
                                }
                            }
                        } else {
                            tc::ld_32cols(obase + col, o);
                            tc::wait_ld();
                            scale32(o, w0);
                        }
                    }
                    if (!warp_live) continue;
                    // through shared memory, so that a store writes whole lines: a thread has one
                    // row, and 32 rows a store would be 32 lines of 16 bytes
#pragma unroll
                    for (int e4 = 0; e4 < 8; ++e4)
                        *reinterpret_cast<float4*>(stage + lane * 128 + ((e4 ^ (lane & 7)) << 4)) =
                            make_float4(o[e4 * 4], o[e4 * 4 + 1], o[e4 * 4 + 2], o[e4 * 4 + 3]);
                    // drafts whose V row is not finite: what was zeroed for P V, added to the rows that see them
                    if constexpr (!V::kScored) {
                        if (wild && row_valid) {
                            const int pos0 = max(c, j0 * TN), pos1 = min(c + n, it.j1 * TN);
#pragma unroll 1
                            for (int pos = pos0; pos < pos1; ++pos) {
                                const int blk = __ldg(trow + pos / p.P);
                                if ((unsigned)blk >= (unsigned)p.N) continue;
                                if (!tree_bit(p, q_row, pos - c)) continue;
                                const int64_t slot = (int64_t)blk * p.P + pos % p.P;
                                const int64_t at = (slot * p.H_kv + h_of(it)) * D + col;
#pragma unroll 1
                                for (int e = 0; e < 32; ++e) {
                                    float x;
                                    if constexpr (CODES)
                                        x = (static_cast<const unsigned char*>(p.v_pool)[at + e] & 0x7f) == 0x7f ? NAN : 0.f;
                                    else
                                        x = __bfloat162float(static_cast<const __nv_bfloat16*>(p.v_pool)[at + e]);
                                    float* y = reinterpret_cast<float*>(stage + lane * 128 +
                                                                        (((e >> 2) ^ (lane & 7)) << 4)) + (e & 3);
                                    if (!(fabsf(x) < INFINITY)) *y += x;
                                }
                            }
                        }
                    }
                    if constexpr (V::kSpread) {
                        // the quarters' parts of a row, added up: 8 rows a warp
                        if (!meeting()) {
                            ok = false;
                            break;
                        }
                        const unsigned char* from = smem + L::stage + t * 4 * 4096;
                        const auto sum_at = [&](int rr, int cc) {
                            const int at = rr * 128 + ((cc ^ (rr & 7)) << 4);
                            float4 a = ld_shared_f4(from + at);
#pragma unroll
                            for (int x = 1; x < 4; ++x) {
                                const float4 b = ld_shared_f4(from + x * 4096 + at);
                                a.x += b.x;
                                a.y += b.y;
                                a.z += b.z;
                                a.w += b.w;
                            }
                            return a;
                        };
                        const auto finite = [](const float4& y) {
                            return (y.x - y.x) + (y.y - y.y) + (y.z - y.z) + (y.w - y.w) == 0.f;
                        };
                        if (whole) {
                            const int row = quad * 8 + (lane >> 2), cc = (lane & 3) * 2;
                            const float4 a = sum_at(row, cc), b = sum_at(row, cc + 1);
                            if (row < live_rows) {
                                odd |= !finite(a) || !finite(b);
                                const int dr = (row * g_inv) >> 16;
                                const int64_t at = (int64_t)(tile_row + dr) * p.H_q + h_of(it) * p.G + row - dr * p.G;
                                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + at * D + col + cc * 4) =
                                    make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y),
                                               pack_bf16x2(b.z, b.w));
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int row = quad * 8 + k * 4 + (lane >> 3), cc = lane & 7;
                                const float4 a = sum_at(row, cc);
                                if (row < live_rows) {
                                    odd |= !finite(a);
                                    *reinterpret_cast<float4*>(p.ws_o + (wbase + row) * D + col + cc * 4) = a;
                                }
                            }
                        }
                        if (!meeting()) {
                            ok = false;
                            break;
                        }
                        continue;
                    }
                    __syncwarp();
                    // Rolled where the warps' loops and this fill the instruction cache (capped prompts 266 us instead of 277,
                    // with the first products of a piece).  Trees show the loads' and stores' latency: one request of 8 drafts
                    // 10.9 us, rolled 11.4 (over fp8 12.3 unrolled, 12.4 by fours, 12.8 rolled; 64 requests there 95.0, 94.0, 93.7).
                    constexpr int kUnrollWhole = V::kScored || CODES ? 1 : 2, kUnrollPiece = V::kScored ? 1 : CODES ? 4 : 8;
                    if (whole) {
#pragma unroll kUnrollWhole
                        for (int k = 0; k < 4; ++k) {           // 8 rows of 64 bytes a store
                            const int rr = k * 8 + (lane >> 2), cc = (lane & 3) * 2;
                            const float4 a = ld_shared_f4(stage + rr * 128 + ((cc ^ (rr & 7)) << 4));
                            const float4 b = ld_shared_f4(stage + rr * 128 + (((cc + 1) ^ (rr & 7)) << 4));
                            const int row = quad * 32 + rr;      // of the query tile
                            if (row < live_rows) {
                                const int dr = (row * g_inv) >> 16;
                                const int64_t at = (int64_t)(tile_row + dr) * p.H_q + h_of(it) * p.G + row - dr * p.G;
                                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + at * D + col + cc * 4) =
                                    make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y),
                                               pack_bf16x2(b.z, b.w));
                            }
                        }
                    } else {
#pragma unroll kUnrollPiece
                        for (int k = 0; k < 8; ++k) {           // 4 rows of 128 bytes a store
                            const int rr = k * 4 + (lane >> 3), cc = lane & 7;
                            const float4 a = ld_shared_f4(stage + rr * 128 + ((cc ^ (rr & 7)) << 4));
                            const int row = quad * 32 + rr;
                            if (row < live_rows)
                                *reinterpret_cast<float4*>(p.ws_o + (wbase + row) * D + col + cc * 4) = a;
                        }
                    }
                    __syncwarp();
                }
            }
            if (!ok) break;
            if constexpr (V::kScored) {
                // Elements of V that are not finite: what a row sees of them decides its columns, over what is stored.  (They
                // were zeroed for P V unless all rows see them, and then an infinity is NaN in the quarters that have a weight
                // of 0 for it; fp8 codes have no infinities.)  Spread: lane k < 8 has row quad * 8 + k.
                if (__any_sync(0xffffffffu, wild || (!CODES && odd)) && warp_live) {
                    const int row = V::kSpread ? quad * 8 + (lane & 7) : r;
                    int2 at = sees;
                    float l = l_run;
                    if constexpr (V::kSpread) {
                        at = make_int2(__shfl_sync(0xffffffffu, sees.x, row), __shfl_sync(0xffffffffu, sees.y, row));
                        l = __shfl_sync(0xffffffffu, l_run, row);
                    }
                    at.x = max(at.x, at0 + j0 * TN);
                    at.y = row < live_rows ? min(at.y, at0 + it.j1 * TN) : 0;
                    const int dr = (row * g_inv) >> 16;
                    const int64_t out_row = (int64_t)(tile_row + dr) * p.H_q + h_of(it) * p.G + row - dr * p.G;
                    __syncwarp();                                  // other lanes stored this row
#pragma unroll 1
                    for (int part = 0; part < kParts; ++part) {
                        const int col = (QT == 1 ? t * (D / 2) : 0) + part * 32;
                        constexpr int kElt = CODES ? 1 : 2;
                        const uint2 got = wild_columns<CODES>(
                            static_cast<const unsigned char*>(p.v_pool) + (h_of(it) * D + col) * kElt,
                            (int64_t)p.H_kv * D * kElt, trow, p.P, p.N, at.x, at.y);
                        if (!(l == l) || (V::kSpread && lane >= 8)) continue;      // (of NaN among the scores all is NaN)
#pragma unroll 1
                        for (uint32_t m = got.x | got.y; m != 0; m &= m - 1) {
                            const int e = __ffs(m) - 1;
                            const float y = !((got.y >> e) & 1u) ? INFINITY : !((got.x >> e) & 1u) ? -INFINITY : NAN;
                            if (whole)
                                static_cast<__nv_bfloat16*>(p.out)[out_row * D + col + e] = __float2bfloat16(y);
                            else
                                p.ws_o[(wbase + row) * D + col + e] = y;
                        }
                    }
                }
            }
            // O (and the streams' sums) are read: the next piece may overwrite them
            tc::fence_before_sync();
            if constexpr (QT == 1) {
                __syncwarp();
                if (lane == 0) mbar_arrive(x_done);
            }
            piece_done(i);
        }
        if (threadIdx.x == 0) p.ws_rec[cta] = rec;
    }

    // Every role has waited (within a limit) for the copies and products it issued, also where it
    // gave up on another's: none reaches this CTA's shared or tensor memory after it is gone.
    tc::fence_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && misc[1]) report(p.dev_status, WF_DEV_TIMEOUT);
    if (warp == kMmaW) {
        __syncwarp();
        tc::fence_after_sync();
        tc::dealloc(tmem, L::TMEM_COLS);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// A lane's 8 elements of a row of q, D / 8 lanes a row, as the e4m3 parts of the row times 2^e;
// returns 2^-e.
template <int D>
__device__ __forceinline__ float split_q_row(const uint4& raw, uint2& hi, uint2& lo) {
    constexpr int kLanes = D / 8;
            float x[8];
            widen_chunk<BF16>(raw, x);
            float top = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e]));
#pragma unroll
            for (int o = kLanes / 2; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            int ex = 0;
            if (top > 0.f && top < INFINITY) {
                // floor(log2 top) from the exponent bits; 2^ex and 2^-ex stay normal numbers
                const int E = max(-126, (int)((__float_as_uint(top) >> 23) & 0xffu) - 127);
                ex = min(126, max(-126, 7 - E));
            }
            const float up = __uint_as_float((uint32_t)(ex + 127) << 23);
            uint32_t h[2] = {}, w[2] = {};
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                float a = x[e] * up, c = x[e + 1] * up;
                // the format has no infinities: they count as NaN here, as q K^T of one would be
                if (!(fabsf(a) < INFINITY)) a = NAN;
                if (!(fabsf(c) < INFINITY)) c = NAN;
                const uint32_t h2 = __nv_cvt_float2_to_fp8x2(make_float2(a, c), __NV_SATFINITE, __NV_E4M3) & 0xffffu;
                const float2 back = e4m3x2_to_float2(h2);
                const uint32_t l2 = __nv_cvt_float2_to_fp8x2(make_float2(a - back.x, c - back.y), __NV_SATFINITE, __NV_E4M3) &
                                    0xffffu;
                h[e / 4] |= h2 << (8 * (e & 3));
                w[e / 4] |= l2 << (8 * (e & 3));
            }
    hi = make_uint2(h[0], h[1]);
    lo = make_uint2(w[0], w[1]);
    return __uint_as_float((uint32_t)(127 - ex) << 23);
}

// q [rows of all requests, D] bf16 -> the e4m3 parts of q 2^e_r, row r of a request b and
// draft i at ((b max_q_len + i) H_q + head): hi, then (B max_q_len H_q rows on) lo; and
// q_inv = 2^-e_r.  A request's rows lie together on both sides, so a CTA takes
// kPartRows of one request and a lane 8 elements of each of its kPartStep-th rows, whose loads
// stand before their first use: at a row a warp, 6144 CTAs came in five waves of two dependent
// loads each.
constexpr int kPartThreads = 256, kPartPer = 4;
template <int D>
constexpr int kPartStep = kPartThreads / (D / 8);
template <int D>
constexpr int kPartRows = kPartStep<D> * kPartPer;

template <int D>
__global__ void __launch_bounds__(kPartThreads) tree_q_parts_kernel(const TreeParams p, unsigned char* __restrict__ parts,
                                                                    float* __restrict__ q_inv, uint32_t chunks) {
    constexpr int kLanes = D / 8;
    // the attention grid may start its set-up now; it waits for this grid before it reads
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = (int)(blockIdx.x / chunks);
    const TreeReq req = tree_request(p, b, false);
    const int64_t live = (int64_t)req.n * p.H_q;
    const int l = threadIdx.x % kLanes;
    const int64_t r0 = (int64_t)(blockIdx.x % chunks) * kPartRows<D> + threadIdx.x / kLanes;   // row of the request
    if (r0 - threadIdx.x / kLanes >= live) return;
    const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(p.q) + (int64_t)req.q_begin * p.H_q * D;
    const int64_t all = (int64_t)p.B * p.max_q_len * p.H_q, to0 = (int64_t)b * p.max_q_len * p.H_q;
    uint4 raw[kPartPer];
#pragma unroll
    for (int k = 0; k < kPartPer; ++k) {
        const int64_t r = r0 + k * kPartStep<D>;
        raw[k] = r < live ? __ldg(reinterpret_cast<const uint4*>(from + r * D) + l) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < kPartPer; ++k) {
        const int64_t r = r0 + k * kPartStep<D>;
        uint2 hi, lo;
        const float inv = split_q_row<D>(raw[k], hi, lo);
        if (r >= live) continue;
        *reinterpret_cast<uint2*>(parts + (to0 + r) * D + 8 * l) = hi;
        *reinterpret_cast<uint2*>(parts + (all + to0 + r) * D + 8 * l) = lo;
        if (l == 0) q_inv[to0 + r] = inv;
    }
}

// A pool row of one head is 128 bytes or fewer (fp8, and 64-wide bf16): an L2 miss that fetches
// 256 brings a part of the next head, which the CTA that wants it may come for too late (303 MB
// read from memory for 251 wanted, 64 requests over fp8: 107.2 us, and 105.4 this way; 64-wide
// bf16 40.9 and 40.4 us).
constexpr CUtensorMapL2promotion kNarrowRows = CU_TENSOR_MAP_L2_PROMOTION_L2_128B;

// A programmatic dependent of the grid before it: its set-up overlaps.
template <typename Kern, typename... Args>
cudaError_t launch_after(Kern kern, int ctas, int smem, cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename V, int D, int QT>
cudaError_t launch_bf16(const typename V::Params& p, int ctas, cudaStream_t stream) {
    const int tok = (V::kSpread ? 32 : TM) / p.G;
    const int box_tok = p.max_q_len < tok ? p.max_q_len : tok;   // drafts of a query tile's box
    CUtensorMap tq, tk, tv;
    const uint64_t slots = (uint64_t)p.N * p.P;
    const uint64_t row = (uint64_t)p.H_kv * D * 2;   // bytes of one pool slot
    cudaError_t e;
    {
        const uint64_t dims[3] = {(uint64_t)D, (uint64_t)p.H_q, (uint64_t)p.total_q};
        const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)p.H_q * D * 2};
        const uint32_t box[3] = {64, (uint32_t)p.G, (uint32_t)box_tok};
        e = encode_tiled_bf16(&tq, const_cast<void*>(p.q), 3, dims, strides, box);
        if (e != cudaSuccess) return e;
    }
    if constexpr (D == 128) {
        // (d 0-63, slot % 8, d half, slot / 8, head): a 16-slot box of one head holds both
        // halves of D as [slot/8 % 2][half][slot % 8][64]
        const uint64_t dims[5] = {64, 8, 2, slots / 8, (uint64_t)p.H_kv};
        const uint64_t strides[4] = {row, 128, 8 * row, (uint64_t)D * 2};
        const uint32_t box[5] = {64, 8, 2, 2, 1};
        e = encode_tiled_bf16(&tk, const_cast<void*>(p.k_pool), 5, dims, strides, box);
        if (e == cudaSuccess) e = encode_tiled_bf16(&tv, const_cast<void*>(p.v_pool), 5, dims, strides, box);
    } else {
        const uint64_t dims[3] = {(uint64_t)D, slots, (uint64_t)p.H_kv};
        const uint64_t strides[2] = {row, (uint64_t)D * 2};
        const uint32_t box[3] = {64, 16, 1};
        e = encode_tiled_bf16(&tk, const_cast<void*>(p.k_pool), 3, dims, strides, box, kNarrowRows);
        if (e == cudaSuccess) e = encode_tiled_bf16(&tv, const_cast<void*>(p.v_pool), 3, dims, strides, box, kNarrowRows);
    }
    if (e != cudaSuccess) return e;
    auto kern = paged_tree_tc_kernel<V, D, QT, false>;
    const int smem = TtLayout<V, D, QT, false>::total;
    e = allow_dynamic_smem((const void*)kern, smem);
    if (e != cudaSuccess) return e;
    bool after = false;                      // the grid that makes a scored call's list
    if constexpr (V::kScored) after = p.blocks != nullptr;
    if (after) {
        return launch_after(kern, ctas, smem, stream, tq, tk, tv, p, box_tok, NoScales{});
    } else {
        kern<<<ctas, kTcThreads, smem, stream>>>(tq, tk, tv, p, box_tok, NoScales{});
        return cudaGetLastError();
    }
}

template <typename V, int D>
cudaError_t launch_codes(typename V::Params p, const HeadScales& sc, void* prep, int ctas, cudaStream_t stream) {
    const int tok = (V::kSpread ? 32 : TM) / p.G;
    const int box_tok = p.max_q_len < tok ? p.max_q_len : tok;
    const uint64_t drafts = V::kScored ? (uint64_t)p.total_q : (uint64_t)p.B * p.max_q_len;
    const uint64_t slots = (uint64_t)p.N * p.P, row = (uint64_t)p.H_kv * D;
    unsigned char* parts = static_cast<unsigned char*>(prep);
    float* q_inv = reinterpret_cast<float*>(parts + 2 * drafts * p.H_q * D);
    p.q_inv = q_inv;
    const CUtensorMapSwizzle swizzle = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    CUtensorMap tq, tk, tv;
    const uint64_t qdims[3] = {(uint64_t)D, (uint64_t)p.H_q, 2 * drafts};
    const uint64_t qstrides[2] = {(uint64_t)D, (uint64_t)p.H_q * D};
    const uint32_t qbox[3] = {(uint32_t)D, (uint32_t)p.G, (uint32_t)box_tok};
    const uint64_t dims[3] = {(uint64_t)D, slots, (uint64_t)p.H_kv};
    const uint64_t strides[2] = {row, (uint64_t)D};
    const uint32_t box[3] = {(uint32_t)D, 16, 1};
    cudaError_t e = encode_tiled(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT8, parts, 3, qdims, qstrides, qbox, swizzle);
    if (e == cudaSuccess)
        e = encode_tiled(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<void*>(p.k_pool), 3, dims, strides, box, swizzle,
                         kNarrowRows);
    if (e == cudaSuccess)
        e = encode_tiled(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<void*>(p.v_pool), 3, dims, strides, box,
                         CU_TENSOR_MAP_SWIZZLE_NONE, kNarrowRows);
    if (e != cudaSuccess) return e;
    auto kern = paged_tree_tc_kernel<V, D, 1, true>;
    const int smem = TtLayout<V, D, 1, true>::total;
    e = allow_dynamic_smem((const void*)kern, smem);
    if (e != cudaSuccess) return e;
    if constexpr (!V::kScored) {   // (a scored call's parts are made with its list of blocks)
        const uint32_t chunks = (uint32_t)(((uint64_t)p.max_q_len * p.H_q + kPartRows<D> - 1) / kPartRows<D>);
        tree_q_parts_kernel<D><<<p.B * chunks, kPartThreads, 0, stream>>>(p, parts, q_inv, chunks);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return launch_after(kern, ctas, smem, stream, tq, tk, tv, p, box_tok, sc);
}

template <typename V>
cudaError_t launch_tc(const typename V::Params& p, const wf_pool_desc& pool, void* prep, int ctas, cudaStream_t stream) {
    const bool d128 = pool.head_dim == 128;
    if (pool.dtype == WF_DTYPE_FP8_E4M3) {
        const HeadScales sc = head_scales(pool);
        return d128 ? launch_codes<V, 128>(p, sc, prep, ctas, stream) : launch_codes<V, 64>(p, sc, prep, ctas, stream);
    }
    if constexpr (!V::kSpread) {
        if (p.rows != TM)
            return d128 ? launch_bf16<V, 128, 2>(p, ctas, stream) : launch_bf16<V, 64, 2>(p, ctas, stream);
    }
    return d128 ? launch_bf16<V, 128, 1>(p, ctas, stream) : launch_bf16<V, 64, 1>(p, ctas, stream);
}

}  // namespace

}  // namespace wf
