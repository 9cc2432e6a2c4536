// ops.h -- internal launch interface of the decode-step operators (include/flint_ops.h).
#pragma once
#include "common.h"

namespace flint {

// Two values as bf16, rounded to nearest, the first in the low half; and 8 of them.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}
__device__ __forceinline__ u32x4 pack8(const float *v)
{
    return u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}

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
// Where a lane's 8 channels are rotated with 8 whole channels of one other lane (half style,
// multiples of 8) or among themselves (pairs), or not at all.
inline bool lane_rotation(int rot, bool pairs) { return pairs ? rot % 8 == 0 : rot % 16 == 0; }

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
