// serve.h -- internal launch interface of the operators of include/flint_serve.h.
#pragma once
#include "ops.h"

namespace flint {

// The 4-bit cache as the kernels see it: Cache::k is its data, page_stride counts bytes.

// attn_decode4.hip
size_t attn_decode4_ws_bytes(const Cache &c, int64_t B);    // any batch of up to B sequences
size_t attn_decode4_call_bytes(const Cache &c, int64_t B);  // a call with B sequences
hipError_t launch_attn_decode4(const AttnArgs &a, hipStream_t st);

// kv_append4.hip
struct Append4Args {
    AppendArgs a;
    uint16_t *k, *v;  // the new codes' values, or null
    int64_t ldk, ldv;
};
hipError_t launch_kv_append4(const Append4Args &a, hipStream_t st);

// kv_pages.hip
struct PageArray {
    uint8_t *base;
    int64_t bytes, stride;
};
struct PageState {
    int32_t *refs, *free_list, *n_free, *table, *kv_len;
};
struct PagesArgs {
    int page, page_shift, n_arrays, n_pages;
    const PageArray *arrays;  // host
    int64_t ldt;
    int rows_old, rows;
    PageState old, state;
    const int32_t *parent, *grow;
    int64_t *slots;
    int64_t lds;
    int32_t *moved;
    int32_t *ws;
};
constexpr int kPagesMaxRows = 1024;
size_t kv_pages_ws_bytes(int64_t n_pages, int64_t rows);
hipError_t launch_kv_advance(const PagesArgs &a, hipStream_t st);
hipError_t launch_kv_compact(const PagesArgs &a, hipStream_t st);

// lora.hip
struct LoraArgs {
    int T, K, N, R, n;  // tokens, in, out, max_rank, adapters
    const uint16_t *a, *b;
    const int32_t *ranks;
    const float *scales;
    const uint16_t *x;
    int64_t ldx;
    const int32_t *ids;
    const void *base;
    int64_t ldb;
    int base_fp32;
    void *y;
    int64_t ldy;
    int y_fp32;
    float *ws;
};
size_t lora_ws_bytes(int64_t T, int K, int R);    // up to T tokens
size_t lora_call_bytes(int64_t T, int K, int R);  // T tokens
hipError_t launch_lora(const LoraArgs &a, hipStream_t st);

// logits.hip
struct LogitsArgs {
    int T, V;
    const void *logits;
    int64_t ld;
    void *out;
    int64_t ldo;
    int fp32;
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
};
hipError_t launch_logits_adjust(const LogitsArgs &a, hipStream_t st);

}  // namespace flint
