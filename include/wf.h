/*
 * wf.h -- C ABI of libwf: attention over a paged KV cache on GB300 (sm_103a).
 *
 * Three calls make up one attention step of an LLM serving engine that keeps
 * its KV cache in fixed-size blocks:
 *
 *   wf_reshape_and_cache  write this step's new K/V rows into the block pool
 *   wf_paged_decode       one query per sequence over its whole cached context
 *   wf_paged_prefill      causal attention of new tokens over prefix + themselves
 *
 * A step that verifies drafted tokens (speculative decoding with a draft tree) has
 * three of its own over the same pool:
 *
 *   wf_qk_norm_rope_and_cache  per-head norms and rotation of q and k, and the scatter
 *   wf_paged_tree_decode       attention of every draft over the context and its ancestors
 *   wf_verify_drafts           the accepted path, from the target's probabilities
 *   wf_keep_accepted           the accepted path's rows moved to the front of the drafts
 *
 * Models whose scores are capped by a tanh or biased by distance, windows, packed documents and
 * prefixes seen in both directions have
 *
 *   wf_paged_scored_attention  for single tokens and prompts alike
 *
 * And a step's tables need not come from the host:
 *
 *   wf_build_step         block tables, slots, positions and offsets from the requests' lengths
 *   wf_trim_blocks        the blocks of shortened or finished requests back to the free list
 *
 * Sources (page title, section):
 *   weft, "Shapes and symbols": B, H_q, H_kv (H_q / H_kv = GQA group), D, N, P, T_total.
 *   weft, "Cache layouts": per-layer paged view [N, P, H_kv, D]; write = scatter
 *     via slot_mapping; read = gather by block_table; blocks handed out per request.
 *   ember, "The core idea, in one picture": position p of a sequence lives in
 *     block block_table[p // P] at offset p % P.
 *   tiny-vllm-py, "KV Cache": the cache holds RoPE-rotated K and plain V; at
 *     decode the new token attends to every earlier position and to itself; prefill
 *     attention is causal ("Mistakes I made in Initial Implementation").
 *
 * Conventions for every call
 *   - Every pointer argument is DEVICE memory owned by the caller, dense and
 *     row-major as documented, 16-byte aligned (the optional per-head fp8 scale
 *     arrays inside wf_pool_desc are the one exception: small host arrays).  The library allocates nothing,
 *     keeps no per-call state, and never synchronises the stream (except
 *     wf_device_status_fetch).  Calls are asynchronous and stream-ordered.
 *   - q, k, v, pools and outputs all use the pool's dtype (float32 or bfloat16);
 *     arithmetic is float32.  Outputs are rounded to nearest-even.
 *   - Argument errors are returned synchronously, before anything is launched.
 *   - Values that only the device can see (slots, block ids, sequence lengths)
 *     are bounds-checked by the kernels: a bad one is skipped (never read or
 *     written out of bounds) and a bit is OR-ed into *dev_status (a device
 *     uint32_t; may be NULL to not record).  Read it with wf_device_status_fetch.
 *   - Outputs never alias inputs.  K and V pools are separate buffers.
 */
#ifndef WF_H
#define WF_H

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum wf_status {
    WF_OK = 0,
    WF_ERR_INVALID_ARG = 1,  /* null pointer, bad size, misaligned pointer, H_q % H_kv != 0 */
    WF_ERR_UNSUPPORTED = 2,  /* dtype / head_dim / group size this build does not handle     */
    WF_ERR_WORKSPACE = 3,    /* workspace missing or smaller than the *_workspace_size value */
    WF_ERR_CUDA = 4,         /* a CUDA runtime call or kernel launch failed                  */
    WF_ERR_NO_BLOCKS = 5     /* block manager: not enough free blocks (nothing was changed)  */
} wf_status;

typedef enum wf_dtype {
    WF_DTYPE_F32 = 0,
    WF_DTYPE_BF16 = 1,
    /* fp8 e4m3 pools (OCP E4M3: 4 exponent bits, bias 7, 3 mantissa bits, largest
     * 448, no infinities).  q, new k/v rows and outputs stay bfloat16; the pools
     * hold codes that stand for k_scale * value (V: v_scale * value).
     * (ember, "Deliberately out of scope": paged KV quantization (fp8/int8)) */
    WF_DTYPE_FP8_E4M3 = 2
} wf_dtype;

/* Bits the kernels OR into *dev_status. */
#define WF_DEV_BAD_SLOT    0x1u  /* slot_mapping[t] >= N*P: token t not written              */
#define WF_DEV_BAD_BLOCK   0x2u  /* block id outside [0, N): that block's rows were skipped
                                    (fp8 pools at D = 64: the 32 positions of its tile)       */
#define WF_DEV_BAD_SEQLEN  0x4u  /* seq_lens[b] < 1, > max_seq_len, > M*P, or < q_len:
                                    sequence b was skipped and its output left unwritten    */
#define WF_DEV_TIMEOUT     0x8u  /* a wait gave up: an internal pipeline wait (should never
                                    happen), or a decode worker idle past its limit          */
#define WF_DEV_BAD_TASK    0x10u /* decode worker: a task record out of range (skipped)     */
#define WF_DEV_BAD_POSITION 0x20u /* norm + rotation: a position outside the table: token
                                    skipped                                                 */
#define WF_DEV_BAD_NODE    0x40u /* accepted path out of range or not increasing: request
                                    skipped                                                 */
#define WF_DEV_NO_BLOCKS   0x80u /* building a step: fewer free blocks than it needs        */
#define WF_DEV_BAD_PROBS   0x100u /* verification: a row whose probabilities have no positive,
                                    finite sum, or a pick outside [0, 1)                    */

/* One layer's pool geometry.  k_pool and v_pool are each [N, P, H_kv, D]. */
typedef struct wf_pool_desc {
    int32_t num_blocks;    /* N: blocks in the pool                       */
    int32_t block_size;    /* P: tokens per block, 1 .. 1024              */
    int32_t num_kv_heads;  /* H_kv                                        */
    int32_t head_dim;      /* D: 64 or 128                                */
    int32_t dtype;         /* wf_dtype of the pools; q, k, v and outputs
                              have it too, except that fp8 pools take
                              bfloat16 q, k, v and give bfloat16 outputs  */
    float k_scale;         /* fp8 pools: a K code c stands for k_scale *
                              value(c); the scatter stores
                              e4m3(float(k) * (1.0f / k_scale)), rounded
                              to nearest even and saturated at +-448.
                              Must be finite and > 0 for fp8; ignored
                              otherwise.                                  */
    float v_scale;         /* the same for V                              */
    const float* k_head_scales; /* fp8 pools, optional: NULL, or host memory
                              holding num_kv_heads scales (num_kv_heads <= 64),
                              one per KV head, read during the call and not
                              kept.  When set, codes of head h stand for
                              k_head_scales[h] * value(c) and k_scale is not
                              used.  Each must be finite and > 0.          */
    const float* v_head_scales; /* the same for V                         */
} wf_pool_desc;

/*
 * wf_reshape_and_cache -- scatter new K/V rows into the block pool.
 * (weft, "Cache layouts": "write: scatter via slot_mapping")
 *
 *   k, v          [T, H_kv, D]   rows of this step's T new tokens
 *   k_pool,v_pool [N, P, H_kv, D] updated in place
 *   slot_mapping  [T] int64: token t goes to block slot/P, offset slot%P.
 *                 A negative slot means "padding token": nothing is written.
 *                 Two tokens with the same slot: one of them wins (unspecified).
 *   num_tokens    T >= 0 (0 is a no-op)
 * Pure byte copy: pool bytes equal the input bytes exactly.  fp8 pools: k, v are
 * bfloat16 and each element of KV head h is stored as the e4m3 code of
 * float(x) * (1.0f / scale_h) (scale_h = k_head_scales[h] if given, else
 * k_scale; likewise for V), rounded to nearest even, saturated at +-448, NaN kept.
 * Slots >= N*P are skipped and flagged WF_DEV_BAD_SLOT.
 */
wf_status wf_reshape_and_cache(const void* k, const void* v, void* k_pool, void* v_pool,
                               const int64_t* slot_mapping, int32_t num_tokens,
                               wf_pool_desc pool, uint32_t* dev_status, cudaStream_t stream);

/*
 * wf_qk_norm_rope_and_cache -- what stands between a layer's q, k, v projections and
 * its attention, in one pass: the norms of queries and keys per head, their rotation
 * by position, and the write of the new rows into the block pool.
 * (tiny-vllm-py, "KV Cache": the cache holds RoPE-rotated K and plain V; weft, "Cache
 *  layouts": write = scatter via slot_mapping)
 *
 *   q_out        [T, H_q, D] dense: the normed and rotated queries (must not overlap q, k or v)
 *   q            [T, H_q, D], k and v [T, H_kv, D]: heads and elements of a token are
 *                dense; *_stride is the distance between tokens in elements (at least
 *                the token's own size when T > 1, a multiple of 16 bytes), so the three
 *                may be cut from one fused projection.
 *   q_weight     [D] weights of the RMS norm of each query head, in q's dtype:
 *                y = x / sqrt(mean(x^2) + eps) * w.  NULL: queries are not normed.
 *   k_weight     the same for keys
 *   eps          finite, >= 0
 *   cos_sin      [max_position, rotary_dim] float32: row p holds cos of the
 *                rotary_dim / 2 angles of position p, then their sin
 *   positions    [T] int32: the token's position, 0 <= positions[t] < max_position
 *   rotary_dim   even, 0 .. D: the leading elements of each head that are rotated,
 *                (a, b) -> (a cos_i - b sin_i, b cos_i + a sin_i), i < rotary_dim / 2.
 *                0: no rotation; cos_sin and positions are not read and may be NULL.
 *   interleaved  0: a, b are elements i and i + rotary_dim / 2; else 2i and 2i + 1
 *   k_pool, v_pool, slot_mapping, num_tokens: as for wf_reshape_and_cache.  Two tokens
 *                with the same slot: each 16 bytes there are one's or the other's.
 * q, k, v and q_out have the pool's dtype (bfloat16 for fp8 pools).  Norm and rotation
 * are float32 and each result is rounded once, K straight to the pool's type: an fp8
 * code is e4m3(y * (1.0f / scale_h)) of the float32 y, which is not always the code
 * that wf_reshape_and_cache stores for a y rounded to bfloat16 first.  The sum of squares
 * is float32 too: head rows whose sum leaves its range (elements of 1e18 and more, or
 * an eps of 0 beside elements of 1e-20 and less) are not normed rightly.
 * A token with a negative slot is padding: nothing is written for it, its q_out row
 * included, and its position is not looked at.  A token with a slot >= N*P
 * (WF_DEV_BAD_SLOT) or a position out of range (WF_DEV_BAD_POSITION) is skipped and
 * flagged the same way.
 * Any rotary_dim is taken; multiples of 16 read the table in 16-byte chunks.
 */
wf_status wf_qk_norm_rope_and_cache(void* q_out, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                    const void* v, int64_t v_stride, const void* q_weight, const void* k_weight,
                                    float eps, const float* cos_sin, int32_t max_position, int32_t rotary_dim,
                                    int32_t interleaved, const int32_t* positions, void* k_pool, void* v_pool,
                                    const int64_t* slot_mapping, int32_t num_tokens, int32_t num_q_heads,
                                    wf_pool_desc pool, uint32_t* dev_status, cudaStream_t stream);

/*
 * wf_copy_blocks -- copy-on-write block copy for prefix sharing.
 * (tiny-vllm-py, "Prefix Sharing": requests with a common prefix share its blocks,
 *  and a shared, partly filled block is copied before a request appends to it;
 *  ember, "Deliberately out of scope": copy-on-write block tables)
 *
 *   k_pool, v_pool  [N, P, H_kv, D], 16-byte aligned, modified in place
 *   block_pairs     [num_pairs, 2] int32 device array of (src, dst) block ids:
 *                   block dst of both pools becomes a byte copy of block src.
 *   Destinations must be distinct and no block may be both a source and a
 *   destination (the copies run in parallel); otherwise the result is undefined.
 *   Ids outside [0, N) are skipped and flagged WF_DEV_BAD_BLOCK in *dev_status.
 * num_pairs == 0 is a no-op.  Any pool dtype.
 */
wf_status wf_copy_blocks(void* k_pool, void* v_pool, const int32_t* block_pairs, int32_t num_pairs,
                         wf_pool_desc pool, uint32_t* dev_status, cudaStream_t stream);

/*
 * Bytes of caller-allocated device workspace wf_paged_decode needs for a batch
 * of at most B sequences of at most max_seq_len tokens.  Depends only on its
 * arguments; 0 if they are invalid.
 */
size_t wf_paged_decode_workspace_size(int32_t B, int32_t num_q_heads, int32_t max_seq_len,
                                      wf_pool_desc pool);

/*
 * wf_paged_decode -- one query token per sequence against its paged context.
 * (ember, "The core idea"; tiny-vllm-py, "KV Cache": decode is not causal over
 *  the cache and includes the just-written token)
 *
 *   out          [B, H_q, D]  out[b,g] = softmax_p(scale * q[b,g].K_p) V_p
 *   q            [B, H_q, D]
 *   k_pool, v_pool [N, P, H_kv, D] (already holding this step's new token)
 *   block_tables [B, max_blocks_per_seq] int32, row-major.  Only the first
 *                ceil(seq_lens[b] / P) entries of row b are read.
 *   seq_lens     [B] int32: positions 0 .. seq_lens[b]-1 of sequence b are attended.
 *                Must satisfy 1 <= seq_lens[b] <= max_seq_len <= max_blocks_per_seq*P.
 *   num_q_heads  H_q; query head g reads KV head g / (H_q / H_kv).  H_q/H_kv <= 8.
 *   scale        softmax scale (normally 1/sqrt(D))
 *   workspace    device scratch of >= wf_paged_decode_workspace_size(B, H_q,
 *                max_seq_len, pool) bytes, 16-byte aligned; contents need no
 *                initialisation and are clobbered.  Calls that overlap in time
 *                must not share a workspace.
 * Launches a split-K kernel and, when any sequence spans more than one split, a
 * combine kernel.  The split boundaries depend only on the pool geometry, so a
 * sequence's output does not depend on the rest of the batch.
 * fp8 e4m3 pools: q and out are bfloat16; K_p and V_p are k_scale_h * value and
 * v_scale_h * value of the stored codes (h the KV head; per-pool or per-head
 * scales).  Every geometry of the bf16 path is supported.  For H_kv = 8, D = 128,
 * P a multiple of 16, H_q / H_kv in {2, 4} and N*P <= 2^31 - 1 both products run
 * on the tensor cores on the codes (e4m3 x e4m3 -> fp32): q is split into two e4m3
 * parts whose sum is q exactly, and the softmax weights into two parts (about 8
 * significant bits).  Other shapes run on the CUDA cores, which widen the codes to
 * fp32 exactly and keep fp32 weights.
 */
wf_status wf_paged_decode(void* out, const void* q, const void* k_pool, const void* v_pool,
                          const int32_t* block_tables, int32_t max_blocks_per_seq,
                          const int32_t* seq_lens, int32_t B, int32_t max_seq_len,
                          int32_t num_q_heads, float scale, wf_pool_desc pool,
                          void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                          cudaStream_t stream);

/*
 * wf_paged_prefill -- causal varlen attention of new tokens over the pool.
 * (tiny-vllm-py, "KV Cache": prefill is causal; "Dense vs. Ragged batching":
 *  requests are packed back to back with per-request offsets, no padding)
 *
 *   out        [T_total, H_q, D]
 *   q          [T_total, H_q, D]: request b owns rows cu_q_lens[b] .. cu_q_lens[b+1]-1
 *   cu_q_lens  [B+1] int32, cu_q_lens[0] = 0, non-decreasing, cu_q_lens[B] = T_total
 *   seq_lens   [B] int32: tokens of request b in the pool INCLUDING its n_b new ones
 *              (already written by wf_reshape_and_cache).  With c_b = seq_lens[b] - n_b,
 *              query row i of request b attends to positions 0 .. c_b + i.
 *   max_q_len  >= every n_b (sizes the launch)
 * bfloat16 only; QK^T and PV run on the tensor cores (bf16 operands, fp32
 * accumulation in tensor memory); the softmax weights are rounded to bf16 for PV.
 * Schedule (no effect on the result: the same bytes either way): a batch of at
 * most 1024 requests and 4096 (request, query block) pairs -- a query block is
 * 256 (token, query head) rows of one KV head -- runs as one persistent grid, one
 * CTA per SM, each taking its share of the blocks longest first; a larger batch
 * runs one CTA per query block.
 */
wf_status wf_paged_prefill(void* out, const void* q, const void* k_pool, const void* v_pool,
                           const int32_t* block_tables, int32_t max_blocks_per_seq,
                           const int32_t* seq_lens, const int32_t* cu_q_lens, int32_t B,
                           int32_t total_q, int32_t max_q_len, int32_t max_seq_len,
                           int32_t num_q_heads, float scale, wf_pool_desc pool,
                           uint32_t* dev_status, cudaStream_t stream);

/*
 * wf_paged_prefill_decode -- the attention of a mixed continuous-batching step:
 * wf_paged_prefill of the step's new requests and wf_paged_decode of its running
 * sequences, over one pool, in one call.
 * (tiny-vllm-py, "Inference Server Flow": a step mixes prefill and decode work;
 *  ember, "Deliberately out of scope": a proper prefill/decode mix per step)
 *
 * The pf_* arguments are those of wf_paged_prefill, the dec_* ones those of
 * wf_paged_decode (its workspace too), and both share the pools, num_q_heads,
 * scale and pool descriptor; every rule of the two calls applies.  The outputs
 * are those of the two calls (the prefill and the decode outputs must not
 * overlap).  For bf16 pools whose prefill and decode both run on the tensor cores,
 * H_kv a multiple of 8 and GQA groups of 1, 2 or 4, both run in one grid: its first
 * CTAs are the prefill's, the rest are persistent decode CTAs that take decode
 * work from a queue as the prefill's CTAs finish, so the decode fills the SMs the
 * prefill's tail leaves idle.  Other shapes run the two calls one after the other.
 */
wf_status wf_paged_prefill_decode(void* pf_out, const void* pf_q, const int32_t* pf_block_tables,
                                  int32_t pf_max_blocks_per_seq, const int32_t* pf_seq_lens,
                                  const int32_t* cu_q_lens, int32_t pf_B, int32_t total_q, int32_t max_q_len,
                                  int32_t pf_max_seq_len, void* dec_out, const void* dec_q,
                                  const int32_t* dec_block_tables, int32_t dec_max_blocks_per_seq,
                                  const int32_t* dec_seq_lens, int32_t dec_B, int32_t dec_max_seq_len,
                                  const void* k_pool, const void* v_pool, int32_t num_q_heads, float scale,
                                  wf_pool_desc pool, void* workspace, size_t workspace_bytes,
                                  uint32_t* dev_status, cudaStream_t stream);
/* 1 when wf_paged_prefill_decode runs both in one grid for this geometry, else 0
 * (host-only, no CUDA call). */
int wf_paged_prefill_decode_fused(wf_pool_desc pool, int32_t num_q_heads);

/*
 * Bytes of caller-allocated device workspace wf_paged_tree_decode needs for at most B
 * requests of at most max_q_len drafts and max_seq_len tokens.  Depends only on its
 * arguments; 0 if they are invalid.
 */
size_t wf_paged_tree_decode_workspace_size(int32_t B, int32_t num_q_heads, int32_t max_q_len, int32_t max_seq_len,
                                           wf_pool_desc pool);

/*
 * wf_paged_tree_decode -- attention of trees of drafted tokens over the pool: every
 * draft sees its request's cached context and those drafts of its own request that its
 * mask row names (itself and its ancestors in the tree, as a rule).
 * (the decode of wf_paged_decode and the packed rows of wf_paged_prefill; the pages
 *  have no drafts)
 *
 *   out, q     [T_total, H_q, D]: request b owns rows cu_q_lens[b] .. cu_q_lens[b+1]-1,
 *              its n_b drafts.  Rows past cu_q_lens[B] are not written.  out must not
 *              overlap q.
 *   cu_q_lens  [B+1] int32, cu_q_lens[0] = 0, non-decreasing, cu_q_lens[B] <= T_total
 *   seq_lens   [B] int32: tokens of request b in the pool INCLUDING its n_b drafts,
 *              already written: with c_b = seq_lens[b] - n_b, draft j lies at cache
 *              position c_b + j whatever its depth in the tree.
 *   tree_mask  [T_total, mask_words] uint32: row i of request b attends to positions
 *              0 .. c_b - 1 and to every c_b + j, j < n_b, whose bit j % 32 of word
 *              j / 32 is set.  Bits of j >= n_b are ignored; a row's own bit is not
 *              implied.  mask_words >= ceil(max_q_len / 32).
 *   max_q_len  >= every n_b; max_seq_len >= every seq_lens[b], below 2^31 - 1024.
 *              max_q_len also decides how the rows of all requests are laid over the
 *              GPU: the result is the same to rounding, but a max_q_len far above the
 *              batch's drafts costs time (up to 16 drafts of 4 query heads a KV head:
 *              34 us with 16, 38 with 64).
 *   scale      softmax scale; scale * log2(e) must be finite in float32
 *   workspace  device scratch of >= wf_paged_tree_decode_workspace_size(B, H_q,
 *              max_q_len, max_seq_len, pool) bytes, 16-byte aligned; needs no
 *              initialisation.  Calls that overlap in time must not share one.
 * A row that sees nothing (no context and no bit set) gives zeros.  A draft that a row
 * does not see has no effect on it, whatever its K and V rows hold (NaN and infinities
 * included); the same holds for pool rows past a request's length.  Requests
 * with n_b = 0 are no-ops.  A request whose n_b or length is out of range
 * (WF_DEV_BAD_SEQLEN) is skipped and its rows are left unwritten; positions of a block
 * id out of range (WF_DEV_BAD_BLOCK) are left out of the softmax.
 * float32, bfloat16 and fp8 e4m3 pools (q and out bfloat16 for fp8), H_q / H_kv <= 8.
 * Context tiles are dealt to the CTAs in equal shares, so where a request's softmax is
 * cut and joined (in float32) depends on the whole batch: the outputs of two calls with
 * the same inputs are the same bytes, those of one request in two different batches
 * need not be.
 */
wf_status wf_paged_tree_decode(void* out, const void* q, const void* k_pool, const void* v_pool,
                               const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                               const int32_t* cu_q_lens, const uint32_t* tree_mask, int32_t mask_words, int32_t B,
                               int32_t total_q, int32_t max_q_len, int32_t max_seq_len, int32_t num_q_heads,
                               float scale, wf_pool_desc pool, void* workspace, size_t workspace_bytes,
                               uint32_t* dev_status, cudaStream_t stream);

/*
 * wf_keep_accepted -- after a tree of drafts is verified: the K and V rows of each
 * request's accepted path move to the front of its drafts, where the next step expects
 * them, in both pools.
 *
 *   block_tables, seq_lens, cu_q_lens: as for wf_paged_tree_decode (seq_lens still
 *              counts the drafts)
 *   accepted   [B, max_accepted] int32: the accepted drafts of request b (as wf_verify_drafts
 *              gives them), strictly increasing node numbers below n_b; entries past
 *              num_accepted[b] are not read
 *   num_accepted [B] int32, 0 <= num_accepted[b] <= min(max_accepted, n_b)
 *   new_seq_lens [B] int32, may be NULL: receives c_b + num_accepted[b] (must not overlap
 *              another argument)
 * Row c_b + accepted[b][j] is copied to c_b + j, byte for byte, as if all rows were read
 * before any is written; rows behind the kept ones are left as they are.  K rows carry
 * the rotation of their position in the text (context + depth), which is the position
 * they move to.  The drafts' blocks must belong to one request each.  (The block manager
 * of wf_blocks.h has no call that shortens a sequence: it goes on counting all drafts
 * that were appended.  A caller that verifies drafts keeps the lengths and the blocks of
 * its drafts itself, or on the GPU by wf_build_step and wf_trim_blocks.)
 * A request whose lengths are out of range (WF_DEV_BAD_SEQLEN) or whose path is
 * (WF_DEV_BAD_NODE) is skipped whole, its new_seq_lens entry left unwritten; a row whose
 * source or target block id is out of range (WF_DEV_BAD_BLOCK) is not moved.
 */
wf_status wf_keep_accepted(void* k_pool, void* v_pool, const int32_t* block_tables, int32_t max_blocks_per_seq,
                           const int32_t* seq_lens, const int32_t* cu_q_lens, const int32_t* accepted,
                           int32_t max_accepted, const int32_t* num_accepted, int32_t* new_seq_lens, int32_t B,
                           wf_pool_desc pool, uint32_t* dev_status, cudaStream_t stream);

/*
 * Bytes of caller-allocated device workspace wf_paged_scored_attention needs for at most B
 * requests of at most max_q_len new tokens each, total_q in all, and max_seq_len tokens.  Depends
 * only on its arguments, and larger ones never need less; 0 if they are invalid.
 */
size_t wf_paged_scored_attention_workspace_size(int32_t B, int32_t num_q_heads, int32_t total_q, int32_t max_q_len,
                                                int32_t max_seq_len, wf_pool_desc pool);

/*
 * wf_paged_scored_attention -- attention of new tokens (one a request, a few, or whole
 * prompts, mixed as they come) over the pool, with capped scores, a bias by distance, and a
 * window or a range of positions for each row.
 * (the reads of wf_paged_decode and the packed rows of wf_paged_prefill; the pages' models
 *  have plain causal scores)
 *
 *   out, q     [T_total, H_q, D]: request b owns rows cu_q_lens[b] .. cu_q_lens[b+1]-1, its n_b
 *              new tokens.  Rows past cu_q_lens[B] are not written.  out must not overlap q.
 *   cu_q_lens  [B+1] int32, cu_q_lens[0] = 0, non-decreasing, cu_q_lens[B] <= T_total
 *   seq_lens   [B] int32: tokens of request b in the pool INCLUDING its n_b new ones, already
 *              written.  Row i is the token at position t = seq_lens[b] - n_b + i.
 *   scale      softmax scale; scale * log2(e) must be finite in float32
 *   cap        > 0: a score x = scale q.K_p becomes cap tanh(x / cap); 0: it stays.  At most 2^100, and
 *              scale / cap 0 or a normal float32.  On the tensor cores a capped score is off by up to
 *              2^-17 of itself or, for caps up to 256, 2^-20 of the cap
 *   slopes     [H_q] float32 or NULL: then slopes[g] |t - p| is taken off it (any sign)
 *   window     > 0: position p is seen only if p > t - window; 0: no window
 *   row_ranges [T_total, 2] int32, 8-byte aligned, or NULL: row r sees the positions p with
 *              row_ranges[r][0] <= p < row_ranges[r][1] (cut to the request's tokens); NULL: p <= t.
 *              So a document packed with others starts its rows' ranges at its first position, a
 *              prefix seen in both directions ends them at its last one, and an empty range is a
 *              row of padding.  The window cuts a range too.
 *   max_q_len  >= every n_b; max_seq_len >= every seq_lens[b], below 2^31 - 1024;
 *              max_q_len <= max_seq_len <= max_blocks_per_seq*P.  max_q_len also decides how the rows
 *              of all requests are laid over the GPU: single tokens beside long prompts run as the
 *              prompts do, and faster in a call of their own (8 capped prompts of 128-2048 tokens and
 *              120 single tokens: 370 us in one call, 178 and 119 in two).
 *   workspace  device scratch of >= wf_paged_scored_attention_workspace_size(B, H_q, T_total,
 *              max_q_len, max_seq_len, pool) bytes, 16-byte aligned; needs no initialisation.
 *              Calls that overlap in time must not share one.
 * A row that sees nothing gives zeros.  Positions that a row does not see have no effect on it,
 * whatever their K and V rows hold (NaN and infinities included), and table entries of blocks before
 * the first position and behind the last one that any row of a request sees are not read: a window's
 * past may be given back.  An infinity in V that a row sees makes that column of it infinite, two of
 * opposite signs or a NaN make it NaN; so may an infinity whose weight is below 2^-126 of the row's
 * largest.  Requests
 * with n_b = 0 are no-ops.  A request whose n_b or length is out of range (WF_DEV_BAD_SEQLEN) is
 * skipped and its rows are left unwritten; positions of a block id out of range
 * (WF_DEV_BAD_BLOCK) are left out of the softmax.
 * float32, bfloat16 and fp8 e4m3 pools (q and out bfloat16 for fp8), H_q / H_kv <= 8.  bf16 and fp8
 * pools of block sizes that are multiples of 16 run on the tensor cores (the kernel is
 * wf_paged_tree_decode_kernel's), others on the CUDA cores.  Scores, cap, bias and softmax are
 * float32; the weights that multiply V are rounded as in wf_paged_tree_decode.  Over bf16 pools a row's
 * weights may reach 2^24 before they are divided by their sum: the sum of |V| over the positions that a
 * row sees is to stay below 2^104.
 * As there, where a request's softmax is cut and joined depends on the whole batch: two calls with the
 * same inputs give the same bytes, one request in two batches need not.
 */
wf_status wf_paged_scored_attention(void* out, const void* q, const void* k_pool, const void* v_pool,
                                    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                    const int32_t* cu_q_lens, int32_t B, int32_t total_q, int32_t max_q_len,
                                    int32_t max_seq_len, int32_t num_q_heads, float scale, float cap, int32_t window,
                                    const float* slopes, const int32_t* row_ranges, wf_pool_desc pool, void* workspace,
                                    size_t workspace_bytes, uint32_t* dev_status, cudaStream_t stream);

/*
 * wf_verify_drafts -- which drafted tokens are kept, and the token after them.
 * (the step between wf_paged_tree_decode's layers and wf_keep_accepted; the pages have no
 *  drafts)
 *
 *   target       [total_q, vocab] probabilities, row stride target_stride elements: row
 *                cu_q_lens[b] + u is the target's distribution p_u of the token after node u
 *                of request b
 *   draft        [total_q, vocab], row stride draft_stride, or NULL: the distribution q_u that
 *                the children of node u were drawn from, each by itself (with replacement).
 *                NULL: the children are fixed candidates.
 *   vocab        1 .. 2^28; probs_dtype: WF_DTYPE_F32 or WF_DTYPE_BF16, of both
 *   tokens       [total_q] int32: token of each node (node 0's is not looked at)
 *   parents      [total_q] int32: node i's parent within its request, 0 <= parents < i; node
 *                0, the request's newest token, has none (its entry is not looked at).
 *                NULL: chains, node i hangs on node i - 1.
 *   cu_q_lens    [B+1] int32: request b has the n_b rows cu_q_lens[b] .. cu_q_lens[b+1]-1
 *   max_q_len    >= every n_b, at most 4096
 *   coins        [total_q] float32 in [0, 1): a node's random number (node 0's is not used)
 *   picks        [B] float32 in [0, 1): the next token's
 *   accepted     [B, max_accepted] int32 receives the path's nodes, 0 first, each the parent
 *                of the next, then -1: what wf_keep_accepted takes
 *   num_accepted [B] int32 receives their number, 1 .. min(max_accepted, n_b)
 *   next_tokens  [B] int32 receives the token after the path
 * From node u = 0 on, u's children are tried in order: with w_0 = p_u and N_0 = 1, child i of
 * token x is kept if coins[i] q_u(x) N_k < w_k(x), and u = i; else
 * w_{k+1} = max(w_k - N_k q_u, 0) and N_{k+1} = sum w_{k+1}.  Fixed candidates: kept if
 * coins[i] N_k < w_k(x), else w_{k+1} is w_k without token x and N_{k+1} = N_k - w_k(x).  The
 * path ends where no child is kept, or at max_accepted nodes (whose last has no children
 * tried).  The next token is the first x with w(0) + .. + w(x) > picks[b] sum w (w = p_u where
 * sum w is 0).  So the tokens are distributed as the target's own if the coins and picks are
 * independent and uniform, p and q sum to 1, and drawn children come from q.  Sums carry about 46
 * bits over usual vocabularies (2^-44 of a sum up to 2^18 tokens, 2^-36 at 2^28), so a seed gives the same
 * tokens anywhere but where a number lies that close to a border: in which order a row is added up
 * depends on the size of the batch.
 * Negative probabilities and NaN count as 0.
 * A request with n_b = 0 gets num_accepted 0 and next token -1.  One whose rows
 * (WF_DEV_BAD_SEQLEN), parents or tokens (WF_DEV_BAD_NODE), or pick (WF_DEV_BAD_PROBS) are out of
 * range is skipped and its outputs are left unwritten; where p_u has no positive finite sum its
 * next token is -1 (WF_DEV_BAD_PROBS).
 * Outputs must not overlap inputs or one another.
 * Pointers are aligned to their elements; 16-byte aligned fp32 (8-byte bf16) rows are read
 * faster.  No workspace.
 */
wf_status wf_verify_drafts(int32_t* accepted, int32_t max_accepted, int32_t* num_accepted, int32_t* next_tokens,
                           const void* target, int64_t target_stride, const void* draft, int64_t draft_stride,
                           int32_t vocab, int32_t probs_dtype, const int32_t* tokens, const int32_t* parents,
                           const int32_t* cu_q_lens, const float* coins, const float* picks, int32_t B, int32_t total_q,
                           int32_t max_q_len, uint32_t* dev_status, cudaStream_t stream);

/*
 * wf_build_step -- a step's block tables, slots, positions and offsets from the requests'
 * lengths, on the GPU: what wf_blocks.h's wf_bm_append and wf_bm_tables give on the host, for
 * requests that share no blocks.
 * (tiny-vllm-py, "Mental Model": a request grows block by block; weft, "Cache layouts":
 *  blocks are handed out to requests from a shared pool)
 *
 *   block_tables  [B, max_blocks_per_seq] int32, updated in place: the entries of the blocks
 *                 that a request grows by are written, no others
 *   seq_lens      [B] int32: tokens that request b holds, in ceil(seq_lens[b] / P) blocks
 *   new_lens      [B] int32: tokens n_b >= 0 that it gets this step
 *   free_blocks   [num_blocks] int32: the ids of the free blocks, num_free[0] of them in use,
 *                 taken from the end (the last freed first), request by request
 *   num_free      [1] int32
 *   depths        [max_tokens] int32 or NULL: a row's position behind its request's tokens where
 *                 that is not its place there (drafts of a tree)
 *   new_seq_lens  [B] int32 receives seq_lens[b] + n_b; may be seq_lens itself
 *   new_num_free  [1] int32 receives what is left; may be num_free itself
 *   cu_q_lens     [B+1] int32 receives the offsets of the requests' rows
 *   slot_mapping  [max_tokens] int64 receives each row's slot; rows past the last are padding: -1
 *   positions     [max_tokens] int32 receives seq_lens[b] + i of row i of request b, or
 *                 seq_lens[b] + depths[row]; padding rows get 0
 *   B             0 .. 16384; block_size P 1 .. 1024
 * A step is built whole or not at all: lengths out of range (negative, past
 * max_blocks_per_seq * P or 2^31 - 1), more than max_tokens rows (WF_DEV_BAD_SEQLEN), too few
 * free blocks (WF_DEV_NO_BLOCKS), a free block's id or a request's partly filled block out of
 * range (WF_DEV_BAD_BLOCK) leave the tables as they are, new_seq_lens = seq_lens,
 * new_num_free = num_free, all offsets 0 and all slots -1, so that the calls that follow have
 * no rows.  Apart from the two pairs named, outputs must not overlap inputs.
 */
wf_status wf_build_step(int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                        const int32_t* new_lens, const int32_t* free_blocks, const int32_t* num_free,
                        const int32_t* depths, int32_t* new_seq_lens, int32_t* new_num_free, int32_t* cu_q_lens,
                        int64_t* slot_mapping, int32_t* positions, int32_t B, int32_t max_tokens, int32_t num_blocks,
                        int32_t block_size, uint32_t* dev_status, cudaStream_t stream);

/*
 * wf_trim_blocks -- the blocks that requests no longer need go back to the free list: those of
 * rejected drafts, or (kept_lens 0) of finished requests.
 *
 *   block_tables, seq_lens, free_blocks, num_free: as for wf_build_step; the tables are only read
 *   kept_lens     [B] int32: tokens that request b keeps, 0 <= kept_lens[b] <= seq_lens[b] (what
 *                 wf_keep_accepted gives as new_seq_lens).  Its blocks ceil(kept_lens[b] / P) ..
 *                 ceil(seq_lens[b] / P) - 1 go back.
 *   free_blocks   receives them behind the num_free[0] that are there, the last request's last
 *                 block first, so that the next wf_build_step hands them out in the order they
 *                 had
 *   new_num_free  [1] int32 receives the number of free blocks; may be num_free itself
 *   B             0 .. 16384
 * Blocks that several tables hold must not be among those that go back.  All or nothing, as for
 * wf_build_step: lengths out of range (WF_DEV_BAD_SEQLEN), block ids out of range or more blocks
 * than num_blocks (WF_DEV_BAD_BLOCK) leave the list as it is and new_num_free = num_free.
 */
wf_status wf_trim_blocks(const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                         const int32_t* kept_lens, int32_t* free_blocks, const int32_t* num_free, int32_t* new_num_free,
                         int32_t B, int32_t num_blocks, int32_t block_size, uint32_t* dev_status, cudaStream_t stream);

/*
 * Size of the fixed device array wf_paged_decode_static_scratch uses as its
 * workspace (32 MiB).  A device holds it from the first
 * wf_paged_decode_static_scratch call on that device until the process exits.
 */
#define WF_STATIC_SCRATCH_BYTES (32u * 1024u * 1024u)

/*
 * wf_paged_decode_static_scratch -- wf_paged_decode for callers that cannot
 * allocate device memory.  The pages have no counterpart: this is a library
 * convenience, not part of the method.
 *
 * Some callers cannot call cudaMalloc when they run attention: an allocator or
 * memory manager that must not re-enter itself, a plugin whose host framework
 * owns every device allocation, or a runtime that forbids allocation after
 * start-up to keep its memory use fixed.  This call takes the same arguments as
 * wf_paged_decode except the workspace: it uses a file-scope device array of
 * WF_STATIC_SCRATCH_BYTES instead, and it allocates nothing (no cudaMalloc,
 * no cudaFree, no allocating library call).
 *
 *   - Arguments are checked as wf_paged_decode checks them, first: an invalid
 *     one returns that call's status.  A valid batch that needs more than
 *     WF_STATIC_SCRATCH_BYTES (compare wf_paged_decode_workspace_size(B,
 *     num_q_heads, max_seq_len, pool)) returns WF_ERR_WORKSPACE.  Either way
 *     nothing is launched.
 *   - The first call on a device looks up the array's device address with that
 *     device current (cudaGetSymbolAddress) and caches it.  Under CUDA's default
 *     lazy module loading that lookup is also what maps the array on the device,
 *     so the device's memory use grows by WF_STATIC_SCRATCH_BYTES at that first
 *     call and not before.  Make that first call before any stream capture.
 *   - A device reset (cudaDeviceReset, or the primary context destroyed and
 *     created again) invalidates the cached address: do not call this entry
 *     point on a device after resetting it.
 *   - Every call on a device shares the one array, which keeps the last call's
 *     contents (nothing in it needs to start at zero).  Calls that overlap in
 *     time on the same device, e.g. on two streams, race on it and give wrong
 *     results: serialise them.
 */
wf_status wf_paged_decode_static_scratch(void* out, const void* q, const void* k_pool,
                                         const void* v_pool, const int32_t* block_tables,
                                         int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                         int32_t B, int32_t max_seq_len, int32_t num_q_heads,
                                         float scale, wf_pool_desc pool, uint32_t* dev_status,
                                         cudaStream_t stream);

/*
 * wf_decode_worker -- a persistent decode worker that takes tasks while it runs.
 * (Awesome System Papers wiki, WEAVER summary, "核心方法": a receiver kernel spins
 *  on a task counter, runs the attention it finds and bumps a completion counter,
 *  so no host launch sits between a request and its attention.)
 *
 * The worker grid (num_workers CTAs of 256 threads) is launched once on `stream`.
 * A feeder outside it -- typically a host thread issuing cudaMemcpyAsync on
 * another non-blocking stream, so the copy engine writes while the worker runs --
 * appends task records to `tasks` and then raises mailbox->posted.  Each CTA
 * claims the next task index (one atomic increment of mailbox->claimed), waits
 * until that task is posted, decodes it and, once its output is written,
 * increments mailbox->done.
 *
 *   tasks      device array of task_capacity records; task t lives in tasks[t].
 *              Write a record before raising `posted` past it (e.g. its copy
 *              earlier on the same stream as the copy of `posted`).
 *   mailbox    device memory (16-byte aligned):
 *                posted   feeder: tasks 0 .. posted-1 are readable (<= task_capacity)
 *                stop     feeder: nonzero = leave once every posted task is claimed;
 *                         write it after the last `posted`
 *                claimed  worker: next task to claim
 *                done     worker: tasks whose outputs are written
 *              The call zeroes `claimed` and `done` on `stream` before the worker
 *              starts; `posted` and `stop` are the feeder's (zero them before).
 *   task       {seq_len, table_row, q_row, out_row}: out[out_row] = decode of
 *              q[q_row] over positions 0 .. seq_len-1 mapped by
 *              block_tables[table_row] (the computation of wf_paged_decode for
 *              one sequence).  Records with an index out of range are skipped
 *              and flagged WF_DEV_BAD_TASK (they still count as done).
 *   out, q     [num_rows, H_q, D] of the pool dtype (float32 or bfloat16 pools)
 *   block_tables [num_table_rows, max_blocks_per_seq] int32
 *   idle_timeout_ns  longest time a CTA waits for its claimed task; past it the
 *              CTA sets WF_DEV_TIMEOUT in *dev_status and returns, leaving its
 *              task unrun.  While a CTA waits it has no copy or tensor-core
 *              operation in flight.
 * The worker holds num_workers CTAs until it stops or times out: anything that
 * waits for the whole device (cudaDeviceSynchronize, cudaMalloc/cudaFree in many
 * allocators) blocks until then, so a feeder must not call such things.
 * fp8 pools: WF_ERR_UNSUPPORTED.
 */
typedef struct wf_worker_mailbox {
    uint32_t posted;
    uint32_t stop;
    uint32_t claimed;
    uint32_t done;
} wf_worker_mailbox;

typedef struct wf_decode_task {
    int32_t seq_len;
    int32_t table_row;
    int32_t q_row;
    int32_t out_row;
} wf_decode_task;

wf_status wf_decode_worker(void* out, const void* q, int32_t num_rows, const void* k_pool, const void* v_pool,
                           const int32_t* block_tables, int32_t num_table_rows, int32_t max_blocks_per_seq,
                           int32_t num_q_heads, float scale, wf_pool_desc pool, const wf_decode_task* tasks,
                           int32_t task_capacity, wf_worker_mailbox* mailbox, int32_t num_workers,
                           uint64_t idle_timeout_ns, uint32_t* dev_status, cudaStream_t stream);

/*
 * Which kernel wf_paged_decode / wf_paged_prefill / wf_paged_tree_decode runs for a
 * pool geometry and query-head count (host-only, no CUDA call; for tests and tooling).  Returns a
 * wf_kernel value; WF_KERNEL_NONE when the geometry is invalid or unsupported.
 */
typedef enum wf_kernel {
    WF_KERNEL_NONE = 0,
    WF_KERNEL_CUDA_CORES = 1,            /* decode, tree decode: kernel on the CUDA cores      */
    WF_KERNEL_TENSOR_CORES = 2,          /* decode: split-K tcgen05 kernel (bf16, or fp8 codes);
                                            prefill, tree decode: warp-specialised pipelined
                                            tcgen05 kernel                                     */
    WF_KERNEL_TENSOR_CORES_SIMPLE = 3    /* prefill: single-stage tcgen05 kernel (any P)       */
} wf_kernel;
int wf_paged_decode_kernel(wf_pool_desc pool, int32_t num_q_heads);
int wf_paged_prefill_kernel(wf_pool_desc pool, int32_t num_q_heads);
int wf_paged_tree_decode_kernel(wf_pool_desc pool, int32_t num_q_heads);
/*
 * 1 when wf_paged_prefill runs a batch of B requests of at most max_q_len new tokens
 * as the persistent grid (WF_KERNEL_TENSOR_CORES geometries within the work list's
 * limits: B <= 1024 and B * ceil(max_q_len / query block) <= 4096), 0 when it runs one
 * CTA per query block (or the geometry is not WF_KERNEL_TENSOR_CORES).  Host-only.
 */
int wf_paged_prefill_persistent(wf_pool_desc pool, int32_t num_q_heads, int32_t B, int32_t max_q_len);

/*
 * Wait for `stream`, copy *dev_status to *host_status and, if clear != 0, reset
 * it to zero.  The only call that synchronises.
 */
wf_status wf_device_status_fetch(uint32_t* dev_status, uint32_t* host_status, int clear,
                                 cudaStream_t stream);

/* Static text for a status code. */
const char* wf_status_string(wf_status s);

/* ABI version of this header (major * 100 + minor). */
int wf_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* WF_H */
