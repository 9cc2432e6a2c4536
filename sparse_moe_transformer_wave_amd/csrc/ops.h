// ops.h -- internal launch interface of the decode-step operators (include/flint_ops.h).
#pragma once
#include "common.h"

namespace flint {

// Records a launch error for flint_moe_status_string and maps it to a status (api.hip).
int hip_status(hipError_t e);

// linear.hip
struct LinearArgs {
    int T, K, N, group;
    const uint8_t *codes;
    const uint16_t *scales;
    const uint16_t *x;
    int64_t ldx;
    const uint16_t *residual;
    int64_t ldr;
    void *y;
    int64_t ldy;
    int y_fp32;
};
hipError_t launch_linear_int4(const LinearArgs &a, hipStream_t st);

// The paged cache as the kernels see it (strides in elements).
struct Cache {
    int Hq, Hkv, D, page, page_shift;
    int64_t n_pages, page_stride;
    uint16_t *k, *v;
};

// kv_append.hip
struct AppendArgs {
    Cache c;
    const uint16_t *q_norm, *k_norm;
    float eps;
    int rot, pairs, max_pos;
    const float *cos, *sin;
    int T;
    const uint16_t *qkv;
    int64_t ldqkv;
    const int32_t *positions;
    const int64_t *slots;
    uint16_t *q;
    int64_t ldq;
};
hipError_t launch_kv_append(const AppendArgs &a, hipStream_t st);

// attn_decode.hip
struct AttnArgs {
    Cache c;
    float scale;
    int window;
    const float *sinks;
    int B, prefix;
    const uint16_t *q;
    int64_t ldq;
    const int32_t *table;
    int64_t ldt;
    const int32_t *kv_len;
    uint16_t *out;
    int64_t ldo;
    float *ws;
};
constexpr int kAttnMaxB = 1024;
size_t attn_decode_ws_bytes(const Cache &c, int64_t B);    // any batch of up to B sequences
size_t attn_decode_call_bytes(const Cache &c, int64_t B);  // a call with B sequences
hipError_t launch_attn_decode(const AttnArgs &a, hipStream_t st);

// logprobs.hip
struct LogprobArgs {
    int T, V;
    const void *logits;
    int64_t ld;
    int fp32;
    const int32_t *tokens;
    float *logprob, *entropy;
    int n;
    int32_t *top_ids;
    float *top_logprobs;
    void *ws;
};
size_t logprobs_ws_bytes(int64_t T, int V, int n);    // any batch of up to T rows
size_t logprobs_call_bytes(int64_t T, int V, int n);  // a call with T rows
hipError_t launch_token_logprobs(const LogprobArgs &a, hipStream_t st);

}  // namespace flint
