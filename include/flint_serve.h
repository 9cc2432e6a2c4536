/*
 * flint_serve.h -- C ABI of what a server of many requests runs beside the decode-step
 * operators of flint_ops.h: a paged cache held in 4 bits with its append and its decode
 * attention, the pages of either cache forked, freed and compacted, low-rank adapters of many
 * requests beside a shared projection, and penalties, biases and grammar masks on logits.
 *
 * Conventions are those of flint_ops.h: device pointers, all work queued on `stream` and
 * nothing allocated or synchronised, bf16 values as uint16 bits, FLINT_* status codes with
 * the arguments checked before any HIP call, inputs never written and not aliased by
 * outputs (the exceptions are named), a batch of 0 a no-op once the rest is valid.
 * Pointers are 16-byte aligned unless stated; a row stride `ld*` counts elements.  Workspaces
 * need no initialisation and hold nothing between calls; calls that share one must not
 * overlap.  All calls can be captured into a HIP graph.  Results are the same bits for the
 * same inputs.
 */
#ifndef FLINT_SERVE_H
#define FLINT_SERVE_H

#include "flint_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- paged cache held in 4 bits -------------------------------------------------------- */
/* Keys and values of one layer in the OCP MXFP4 format: per token and head, blocks of 32
   channels share a power of two.  A code is E2M1: bit 3 the sign, bits 0 .. 2 one of
   {0, 0.5, 1, 1.5, 2, 3, 4, 6}; a scale byte s stands for 2^(s - 127), and 255 for NaN.
     value = code * 2^(s - 127)
   A page of page_size tokens (16, 32, 64 or 128) is one block of bytes, in this order:
     key codes     [n_kv_heads][page_size][head_dim / 2]    the even channel in the low nibble
     value codes   [n_kv_heads][page_size][head_dim / 2]
     key scales    [n_kv_heads][head_dim / 32][page_size]
     value scales  [n_kv_heads][head_dim / 32][page_size]
   2 * n_kv_heads * page_size * (head_dim / 2 + head_dim / 32) bytes; pages are page_stride
   bytes apart (a multiple of 16, at least a block; 0 means exactly that).  The limits on heads
   (head_dim 64 or 128), pages, tables and slots are those of flint_kv_cache. */
typedef struct {
    int32_t n_q_heads, n_kv_heads, head_dim, page_size;
    int64_t n_pages, page_stride;
    uint8_t *data;
} flint_kv4_cache;

/* flint_kv_append into this cache: queries are normalised, rotated and rounded to bf16 as
   there, to the same bits.  Keys are normalised and rotated in 64 bits and rounded once, to the
   cache's format; values come as they are.  A block's power of two is the least with
   max |x| <= 7 times it, 2^-125 .. 2^125 (2^0 where all are zero), and a code the nearest (an
   even one at a tie), so that no value is off by more than half of its code's step unless it is
   over 7 * 2^125 (those saturate).  A block with an infinity or a NaN gets the scale byte 255 and
   codes of 0.
     k, v: bf16 [T][n_kv_heads][head_dim] or NULL, row strides ldk, ldv (multiples of 8):
       receive the values that the new codes stand for (a prompt's own attention can then use
       what later steps will read; NaN for a byte of 255).  They are written for skipped slots
       too, but for a position outside the table they are zeros, like the queries.
   Slots are distinct; one outside the cache is skipped. */
int flint_kv4_append(const flint_kv4_cache *cache, const flint_qk_transform *transform, int64_t T,
                     const uint16_t *qkv, int64_t ldqkv, const int32_t *positions,
                     const int64_t *slots, uint16_t *q, int64_t ldq, uint16_t *k, int64_t ldk,
                     uint16_t *v, int64_t ldv, void *stream);

/* flint_attn_decode over this cache: the same arguments, masks, prefix and result, with k_j and
   v_j the values that the codes stand for (a NaN among them makes what it reaches NaN).  Scale
   bytes are 2 .. 252 or 255; others may overflow or lose small values.  As there, a row's weighted
   values are summed before they are divided: 2^8 times their sum has to stay in fp32's range. */
size_t flint_kv4_attn_decode_workspace_bytes(const flint_kv4_cache *cache, int64_t B_max);
int flint_kv4_attn_decode(const flint_kv4_cache *cache, const flint_attn *attn, int64_t B,
                          const uint16_t *q, int64_t ldq, const int32_t *table, int64_t ldt,
                          const int32_t *kv_len, int32_t prefix_len, uint16_t *out, int64_t ldo,
                          void *ws, size_t ws_bytes, void *stream);

/* ---- pages of a cache ------------------------------------------------------------------ */
/* The memory of a pool's pages: page p of array i is `bytes` bytes (a multiple of 16) at
   base + p * stride (bytes, a multiple of 16, at least `bytes`).  A bf16 cache is two arrays (k
   and v) per layer, a 4-bit one a single one.  Arrays do not overlap.  n_arrays 0 .. 1024;
   `arrays` is read by the host during the call.  n_pages 1 .. 2^24; page_size 16, 32, 64 or
   128 tokens. */
typedef struct {
    void *base;
    int64_t bytes, stride;
} flint_kv_array;

typedef struct {
    int32_t page_size;
    int32_t n_arrays;
    int64_t n_pages;
    const flint_kv_array *arrays;
} flint_kv_pages;

/* Who holds which page, on the device (int32, 4-byte aligned):
     refs [n_pages]       rows (or other owners) that hold a page; 0 = free
     free_list [n_pages]  the free pages: a stack, taken from entry n_free - 1 downwards
     n_free [1]
     table [rows][ldt]    pages of each row: a sequence of n tokens holds the first
                          ceil(n / page_size) entries; an entry outside [0, n_pages) is nobody's
     kv_len [rows]        tokens of each row (read as 0 if negative, as ldt * page_size if longer)
   Calls read one state and write another, which shares no memory with it: the old one can be
   gone back to as long as no page has been written since. */
typedef struct {
    int32_t *refs, *free_list, *n_free, *table, *kv_len;
} flint_kv_state;

/* Bytes of workspace for either call on up to rows_max old and new rows; 0 for invalid
   arguments. */
size_t flint_kv_pages_workspace_bytes(const flint_kv_pages *pages, int64_t rows_max);

/* The next step of a batch: new row r (of `rows`, 0 .. 1024) continues old row parent[r] (of
   rows_old, 0 .. 1024; int32 [rows], outside [0, rows_old): a new, empty sequence) and gets
   room for grow[r] more tokens (int32 [rows], negative read as 0).  Several rows may continue
   one (a fork); a row that none continues gives its pages back.
     Pages: refs of an old row's pages change by its continuing rows less one.  Those that reach
       0 go onto the free list, by ascending number, before any page is taken.
     Copy on write: a row that grows and whose last page is not full gets a copy of that page
       unless it is the last holder: of the growing rows with that last page, in order, each
       takes a copy while more holders than one are left.  All arrays are copied.
     New pages come from the top of the free list, row after row (a row's copy first) and have
       one holder.  A row that needs more than ldt entries does not grow.  Nor does one that
       needs pages, or keeps a page that rows ahead of it copy, where its needs and those of the
       rows ahead are more than there are.  Such a row takes no page and keeps its parent's
       pages and length; rows that do not fit ldt entries count as not growing.
     new->kv_len[r]: its tokens, the growth included; new->table: entries beyond a row's pages
       are -1; new->free_list: entries from n_free on are -1.
     slots (int64 [rows][lds], 8-byte aligned, or NULL): slots[r][i] = page * page_size + offset
       of the row's token i of grow[r]; -1 for i >= grow[r], where the row did not grow or where
       the entry is no page.
   Both tables have the row stride and width ldt >= 1, ldt * page_size <= 2^25. */
int flint_kv_advance(const flint_kv_pages *pages, int64_t ldt, int64_t rows_old, const flint_kv_state *old,
                     int64_t rows, const flint_kv_state *state, const int32_t *parent, const int32_t *grow,
                     int64_t *slots, int64_t lds, void *ws, size_t ws_bytes, void *stream);

/* Live pages (refs > 0) to the front: with n of them, the i-th live page from n on moves to the
   i-th free place below n, in all arrays (what a page holds stays at its old place too, until
   that is taken).  moved (int32 [n_pages]): the page's new number, -1 for a free one; the new
   state's refs, tables (rows x ldt; entries beyond a row's pages are -1) and lengths follow, and
   its free list is n_pages - 1 down to n, -1 behind that.  Tables that are not passed are brought
   up to date with `moved`. */
int flint_kv_compact(const flint_kv_pages *pages, int64_t ldt, int64_t rows, const flint_kv_state *old,
                     const flint_kv_state *state, int32_t *moved, void *ws, size_t ws_bytes, void *stream);

/* ---- low-rank adapters ------------------------------------------------------------------- */
/* Adapter i adds scales[i] * B_i (A_i x):
     a: bf16 [n_adapters][max_rank][in_features]      in_features % 8 == 0, 8 .. 32768
     b: bf16 [n_adapters][out_features][max_rank]     1 <= out_features <= 2^24
     ranks: int32 [n_adapters] or NULL (max_rank): rows of A_i and columns of B_i that count,
       the others may hold anything; read as 0 if negative, as max_rank if larger
     scales: fp32 [n_adapters] or NULL (1)
   max_rank: a multiple of 8, 8 .. 128; n_adapters 1 .. 2^20. */
typedef struct {
    int32_t in_features, out_features, max_rank, n_adapters;
    const uint16_t *a, *b;
    const int32_t *ranks;
    const float *scales;
} flint_lora_adapters;

/* Bytes of workspace for up to T_max tokens; 0 for invalid arguments. */
size_t flint_lora_workspace_bytes(const flint_lora_adapters *adapters, int64_t T_max);

/* y[t] = base[t] + scales[i] B_i (A_i x[t]) with i = ids[t], 0 <= T <= 65536.
     x: bf16, row stride ldx (a multiple of 8, >= in_features);
     ids: int32 [T] (4-byte aligned); outside [0, n_adapters): y = base;
     base: base_type FLINT_DT_BF16 or FLINT_DT_FP32, or NULL (zero), row stride ldb >=
       out_features, aligned to its element (a shared projection's result, in fp32 where y is to
       be rounded once); may be y itself if type and stride are the same;
     y: y_type, row stride ldy >= out_features, aligned to its element, rounded once.
   Products are exact, sums fp32; scales[i] A x enters the second product as three bf16 parts, in
   all as fp32.  A token's result depends on its own x and adapter only, the order of its sums on T as
   well; an infinity or a NaN in its A x makes its results NaN, and so does a scaled value that bf16
   rounds to an infinity (from 2^128 - 2^119 on). */
int flint_lora(const flint_lora_adapters *adapters, int64_t T, const uint16_t *x, int64_t ldx,
               const int32_t *ids, const void *base, int64_t ldb, int32_t base_type, void *y,
               int64_t ldy, int32_t y_type, void *ws, size_t ws_bytes, void *stream);

/* ---- logits ------------------------------------------------------------------------------ */
/* What happens to row t's logits, in this order (all in fp32, rounded once; any group may be
   absent, its pointers NULL; everything is 4-byte aligned):
     history: int32 [T][ldh], of which the first total_len[t] count (read as 0 if negative, as ldh if
       larger), the first prompt_len[t] of them the prompt's, the rest the model's own.  Tokens
       outside [0, vocab) are skipped.  With c the times that v occurs in the own part:
         repetition[t]: if v occurs in the history, x = x > 0 ? x / r : x * r
         frequency[t], presence[t]: x -= frequency * c, and presence once if c > 0
       (total_len may be NULL: ldh; prompt_len: 0)
     bias: entries bias_start[t] .. bias_start[t + 1] (int32 [T + 1]) of bias_ids and bias (fp32):
       x += bias; of a token that is listed more than once the last entry counts.  Entries
       outside [0, n_bias) and tokens outside [0, vocab) are skipped.
     masks: uint32 [n_masks][ldm], ldm >= ceil(vocab / 32): token v is allowed if bit v % 32 of
       word v / 32 is set; the others become -inf, whatever they were.  mask_rows: int32 [T], the
       mask of each row, outside [0, n_masks): none; NULL: mask t (rows from n_masks on: none). */
typedef struct {
    const int32_t *history;
    int64_t ldh;
    const int32_t *prompt_len, *total_len;
    const float *repetition, *frequency, *presence;
    const int32_t *bias_start, *bias_ids;
    const float *bias;
    int64_t n_bias;
    const uint32_t *masks;
    int64_t ldm, n_masks;
    const int32_t *mask_rows;
} flint_logit_rules;

/* logits -> out, both of type dtype (FLINT_DT_BF16 or FLINT_DT_FP32), [T][vocab], row strides
   ld, ldo >= vocab, aligned to the element; out may be logits itself with the same stride, and
   then only what changes is read and written.  1 <= vocab <= 2^20, 0 <= T <= 65536. */
int flint_logits_adjust(const flint_logit_rules *rules, int64_t T, int32_t vocab, const void *logits,
                        int64_t ld, void *out, int64_t ldo, int32_t dtype, void *stream);

#ifdef __cplusplus
}
#endif
#endif
