/*
 * flint_ops.h -- C ABI of the operators that a decode step runs around the MoE layer of
 * flint_moe.h: linear layers with 4-bit weights, the paged cache's append, decode attention
 * over that cache with a shared prefix, and log probabilities of given tokens.
 *
 * The Flint model's attention (recipes.vllm.ai "RecursiveSI/flint", Overview; neoteo.com
 * specification table; qantcore.space review, section 02): 32 query and 4 key/value heads of
 * 128, per-head RMSNorm of queries and keys, learnable attention sinks, 35 sliding-window
 * layers (513 tokens, the current one included) with rotary positions and 14 full layers
 * without, a bf16 cache.  Its output layer has a 4-bit form (mrchatgpt.org explainer,
 * section 4).
 *
 * Conventions are those of flint_moe.h: device pointers, all work queued on `stream` and
 * nothing allocated or synchronised, bf16 values as uint16 bits, FLINT_* status codes with
 * the arguments checked before any HIP call, inputs never written and not aliased by
 * outputs (the exceptions are named), a batch of 0 a no-op once the rest is valid.
 * Pointers are 16-byte aligned unless stated; a row stride `ld*` counts elements and lets a
 * matrix be a slice of a wider one.  Workspaces need no initialisation and hold nothing
 * between calls; calls that share one must not overlap.  All calls can be captured into a
 * HIP graph.  Results are the same bits for the same inputs.
 */
#ifndef FLINT_OPS_H
#define FLINT_OPS_H

#include "flint_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
    FLINT_DT_BF16 = 0,
    FLINT_DT_FP32 = 1
};

/* ---- linear layer with 4-bit weights ------------------------------------------------- */
/* W: [out_features][in_features] in the INT4 layout of flint_moe.h with a choice of group:
     codes   uint8 [out][in / 2], signed nibbles (two's complement), the even column low;
     scales  bf16 [out][in / group], one per row and `group` consecutive columns;
   value = q * scale.  group: 32, 64 or 128.  in_features % 128 == 0, 128 .. 32768;
   1 <= out_features <= 2^24. */
typedef struct {
    int32_t in_features, out_features, group;
    const uint8_t *codes;
    const uint16_t *scales;
} flint_int4_linear;

/* y[t][n] = sum_k W[n][k] x[t][k] (+ residual[t][n]) for a decode batch, 0 <= T <= 64.
     x: bf16, row stride ldx (elements, a multiple of 8, >= in_features);
     residual: bf16 or NULL, row stride ldr >= out_features (2-byte aligned; may be y itself
       when y is bf16 with the same stride: each element is read before it is written);
     y: y_type FLINT_DT_BF16 or FLINT_DT_FP32, row stride ldy >= out_features (aligned to
       its element), rounded once.
   Products of codes and x are exact, a group's sum and the sum over groups are fp32.  An
   infinity or a NaN in x stays in its token's row, as the products and sums of such numbers
   have it (an infinity times a code of zero is NaN). */
int flint_linear_int4(const flint_int4_linear *w, int64_t T, const uint16_t *x, int64_t ldx,
                      const uint16_t *residual, int64_t ldr, void *y, int64_t ldy, int32_t y_type,
                      void *stream);

/* ---- paged cache ---------------------------------------------------------------------- */
/* Keys and values of one layer in pages of page_size tokens (16, 32, 64 or 128):
     k: bf16 [n_pages][n_kv_heads][page_size][head_dim]
     v: bf16 [n_pages][n_kv_heads][head_dim][page_size]   (transposed, see below)
   A page's block is dense; pages are page_stride elements apart (a multiple of 8, at least
   n_kv_heads * page_size * head_dim; 0 means exactly that), so the layers of a model can
   share one allocation page by page.  head_dim: 64 or 128; n_kv_heads 1 .. 64;
   n_q_heads a multiple of n_kv_heads, at most 32 per key/value head; n_pages >= 1.
   Token j of a sequence lives in page table[j / page_size] at j % page_size; slot
   = page * page_size + that.  The values are stored transposed because the matrix
   instruction of the second product takes 8 consecutive tokens of one channel per lane. */
typedef struct {
    int32_t n_q_heads, n_kv_heads, head_dim, page_size;
    int64_t n_pages, page_stride;
    uint16_t *k, *v;
} flint_kv_cache;

enum {
    FLINT_ROPE_HALF = 0,   /* channel i is rotated with i + rot_dim / 2 */
    FLINT_ROPE_PAIRS = 1   /* channel 2 i is rotated with 2 i + 1       */
};

/* What happens to a query or key head before it is used, in this order:
     RMSNorm over head_dim: x * w / sqrt(mean(x^2) + eps), with q_norm / k_norm (bf16
       [head_dim]; either may be NULL: that kind is not normalised); eps >= 0;
     rotation of the first rot_dim channels by the position's angles: for i < rot_dim / 2 the
       pair (a, b) becomes (a c - b s, b c + a s) with c = cos[position][i], s = sin[..][i]
       (fp32 [max_position][rot_dim / 2]); rot_dim even, 0 .. head_dim, 0 = no rotation
       (then cos, sin and positions are not read).
   All in fp32, rounded to bf16 once. */
typedef struct {
    const uint16_t *q_norm, *k_norm;
    float eps;
    int32_t rot_dim, rope_style;
    int32_t max_position;
    const float *cos, *sin;
} flint_qk_transform;

/* T tokens' projections into the cache: qkv (bf16 [T][n_q_heads + 2 n_kv_heads][head_dim],
   row stride ldqkv, a multiple of 8) holds each token's queries, keys and values.
     q (bf16 [T][n_q_heads][head_dim], row stride ldq, a multiple of 8) receives the
       transformed queries; it may be the query part of qkv itself (q == qkv, ldq == ldqkv);
     the cache's k and v receive the transformed keys and the values at slots[t] (int64 [T]).
   A slot outside [0, n_pages * page_size) is skipped: that token's key and value go nowhere
   (-1 for the padding of a batch).  A position (int32 [T]) outside [0, max_position) is a
   caller error: the token's key and value go nowhere and its queries become zeros.  Slots
   are distinct.  0 <= T <= 2^20. */
int flint_kv_append(const flint_kv_cache *cache, const flint_qk_transform *transform, int64_t T,
                    const uint16_t *qkv, int64_t ldqkv, const int32_t *positions,
                    const int64_t *slots, uint16_t *q, int64_t ldq, void *stream);

/* ---- decode attention ------------------------------------------------------------------ */
/* scale multiplies q . k; window > 0 lets a query see the last `window` tokens only (its own
   included), 0 all; sinks: fp32 [n_q_heads] or NULL, one more score per query head, whose
   value is zero (it joins the softmax's denominator). */
typedef struct {
    float scale;
    int32_t window;
    const float *sinks;
} flint_attn;

/* Bytes of workspace for any batch of up to B_max sequences; 0 for invalid arguments. */
size_t flint_attn_decode_workspace_bytes(const flint_kv_cache *cache, int64_t B_max);

/* One query token per sequence, B sequences (0 <= B <= 1024):
     out[b][h] = sum_j p_j v_j,  p = softmax over j in [max(0, n - window), n) of
     scale q[b][h] . k_j  (and the sink),  n = kv_len[b]
   with k_j, v_j of key/value head h / (n_q_heads / n_kv_heads).
     q: bf16 [B][n_q_heads][head_dim], row stride ldq (a multiple of 8);
     table: int32 [B][ldt], ldt >= 1 the row stride and the pages that a row can name
       (4-byte aligned), ldt * page_size <= 2^25;
     kv_len: int32 [B] on the device, the current token included (4-byte aligned); read as
       0 if negative and as ldt * page_size if longer.  A sequence of length 0 gets zeros;
     prefix_len: the first prefix_len tokens of every sequence that takes part are the same keys
       and values (0 = nothing shared).  Their pages are read through the table row of the first
       of these, once for the whole batch; the result is that of the unshared call up to
       rounding.  Sequences shorter than the prefix, or whose window has left it, do not take
       part: their rows name their own pages, and those of an empty one nothing;
     out: bf16 [B][n_q_heads][head_dim], row stride ldo (a multiple of 8).
   A table entry outside [0, n_pages) masks its tokens; a query that sees no token gets zeros,
   whatever its sink, and so does one whose sink is +infinity.  Scores and sums are fp32, probabilities enter the second product as
   two bf16 parts, each rounded to nearest (17 bits), and the result is rounded once.  Cache places
   that no query sees may hold anything, infinities and NaN included; a value that a query sees
   and that is not finite makes its channel of the result NaN.
   ws: flint_attn_decode_workspace_bytes(cache, B) bytes. */
int flint_attn_decode(const flint_kv_cache *cache, const flint_attn *attn, int64_t B,
                      const uint16_t *q, int64_t ldq, const int32_t *table, int64_t ldt,
                      const int32_t *kv_len, int32_t prefix_len, uint16_t *out, int64_t ldo,
                      void *ws, size_t ws_bytes, void *stream);

/* ---- log probabilities ------------------------------------------------------------------ */
/* Bytes of workspace for any T <= T_max rows of `vocab` logits and `top_n` alternatives;
   0 for invalid arguments. */
size_t flint_token_logprobs_workspace_bytes(int64_t T_max, int32_t vocab, int32_t top_n);

/* Rows of logits (dtype FLINT_DT_BF16 or FLINT_DT_FP32, [T][vocab], row stride ld >= vocab,
   aligned to its element; 1 <= vocab <= 2^20, 0 <= T <= 2^20):
     logprob[t]  = logits[t][tokens[t]] - lse(logits[t])      (tokens: int32 [T])
     entropy[t]  = -sum_v p_v log p_v, in nats
     top_ids[t][0..top_n), top_logprobs[t][0..top_n): the largest logits, descending, equal
       values by ascending index (-0 == +0, NaN below -inf); 0 <= top_n <= min(32, vocab)
   Outputs are fp32 (top_ids int32), 4-byte aligned; logprob with tokens, entropy, and
   top_ids with top_logprobs may be NULL (not computed).  All sums fp32.  A logit of -inf has
   probability 0 and adds nothing to the entropy.  A token outside [0, vocab) has
   log probability -inf.  A row of -inf alone: every log probability -inf, entropy 0.  A row
   with a NaN or +inf: NaN for every log probability and the entropy, top_ids still ordered. */
int flint_token_logprobs(int64_t T, int32_t vocab, const void *logits, int64_t ld, int32_t dtype,
                         const int32_t *tokens, float *logprob, float *entropy, int32_t top_n,
                         int32_t *top_ids, float *top_logprobs, void *ws, size_t ws_bytes,
                         void *stream);

#ifdef __cplusplus
}
#endif
#endif
