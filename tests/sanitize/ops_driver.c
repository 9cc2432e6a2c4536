/* Every refusal path of include/flint_ops.h, and the sizing functions over their ranges; no
 * call here reaches a launch.  Pointers are addresses that are never read. */
#include <limits.h>
#include <stdio.h>
#include <stdlib.h>

#include "../../include/flint_ops.h"

#define WANT(call, code)                                                                                      \
    do {                                                                                                      \
        const int got_ = (call);                                                                              \
        if (got_ != (code)) {                                                                                 \
            printf("line %d: %s gave %d, not %d\n", __LINE__, #call, got_, (code));                           \
            exit(1);                                                                                          \
        }                                                                                                     \
    } while (0)

int main(void)
{
    uint8_t *const a = (uint8_t *)((uintptr_t)1 << 20);
    uint16_t *const p = (uint16_t *)a;
    int32_t *const i = (int32_t *)a;
    float *const f = (float *)a;

    flint_int4_linear w = {256, 8, 128, a, p};
    const int64_t Ts[] = {INT64_MIN, -1, 65, INT64_MAX}, lds[] = {INT64_MIN, -1, 0, 255, 257, INT64_MAX};
    for (int k = 0; k < 4; k++) WANT(flint_linear_int4(&w, Ts[k], p, 256, 0, 0, a, 8, 0, 0), FLINT_ERR_SHAPE);
    for (int k = 0; k < 6; k++) WANT(flint_linear_int4(&w, 1, p, lds[k], 0, 0, a, 8, 0, 0), FLINT_ERR_SHAPE);
    WANT(flint_linear_int4(0, 1, p, 256, 0, 0, a, 8, 0, 0), FLINT_ERR_NULL);
    WANT(flint_linear_int4(&w, 0, 0, 256, 0, 0, 0, 8, 0, 0), FLINT_OK);
    const int32_t bad[] = {INT32_MIN, -1, 0, 100, INT32_MAX};
    for (int k = 0; k < 5; k++) {
        flint_int4_linear b = w;
        b.in_features = bad[k];
        WANT(flint_linear_int4(&b, 1, p, 256, 0, 0, a, 8, 0, 0), FLINT_ERR_SHAPE);
        b = w;
        b.group = bad[k];
        WANT(flint_linear_int4(&b, 1, p, 256, 0, 0, a, 8, 0, 0), FLINT_ERR_SHAPE);
    }

    flint_kv_cache c = {32, 4, 128, 64, 100, 0, p, p};
    flint_qk_transform t = {0, 0, 0.f, 0, 0, 0, 0, 0};
    WANT(flint_kv_append(&c, &t, 0, 0, 5120, 0, 0, 0, 4096, 0), FLINT_OK);
    WANT(flint_kv_append(&c, 0, 1, p, 5120, 0, (int64_t *)a, p, 4096, 0), FLINT_ERR_NULL);
    for (int k = 0; k < 5; k++) {
        flint_kv_cache b = c;
        b.n_q_heads = bad[k] == 100 ? 33 : bad[k];
        WANT(flint_kv_append(&b, &t, 1, p, 5120, 0, (int64_t *)a, p, 4096, 0), FLINT_ERR_SHAPE);
        if (flint_attn_decode_workspace_bytes(&b, 4)) return 1;
        b = c;
        b.n_kv_heads = bad[k];
        WANT(flint_kv_append(&b, &t, 1, p, 5120, 0, (int64_t *)a, p, 4096, 0), FLINT_ERR_SHAPE);
        b = c;
        b.page_size = bad[k];
        WANT(flint_kv_append(&b, &t, 1, p, 5120, 0, (int64_t *)a, p, 4096, 0), FLINT_ERR_SHAPE);
    }
    for (int k = 0; k < 6; k++) WANT(flint_kv_append(&c, &t, 1, p, lds[k] == INT64_MAX ? 5121 : lds[k], 0, (int64_t *)a, p, 4096, 0), FLINT_ERR_SHAPE);
    flint_kv_cache wide = c;
    wide.page_stride = INT64_MAX / 8 * 8;
    WANT(flint_kv_append(&wide, &t, 1, p, 5120, 0, (int64_t *)a, p, 4096, 0), FLINT_ERR_SHAPE);

    const flint_attn at = {1.f, 0, 0};
    WANT(flint_attn_decode(&c, &at, 0, 0, 4096, 0, 4, 0, 0, 0, 4096, 0, 0, 0), FLINT_OK);
    WANT(flint_attn_decode(&c, &at, 1, p, 4096, i, 4, i, 0, p, 4096, a, 0, 0), FLINT_ERR_WORKSPACE);
    WANT(flint_attn_decode(&c, &at, 1, p, 4096, i, INT64_MAX, i, 0, p, 4096, a, 0, 0), FLINT_ERR_SHAPE);
    WANT(flint_attn_decode(&c, &at, 1, p, 4096, i, 4, i, INT32_MAX, p, 4096, a, 0, 0), FLINT_ERR_SHAPE);
    WANT(flint_attn_decode(&c, &at, INT64_MAX, p, 4096, i, 4, i, 0, p, 4096, a, 0, 0), FLINT_ERR_SHAPE);
    size_t last = 0;
    for (int64_t B = 0; B <= 1024; B += 31) {
        const size_t n = flint_attn_decode_workspace_bytes(&c, B);
        if (n < last) return 1;
        last = n;
    }
    if (flint_attn_decode_workspace_bytes(&c, 1025) || flint_attn_decode_workspace_bytes(&c, INT64_MIN)) return 1;

    WANT(flint_token_logprobs(0, 100, 0, 100, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0), FLINT_OK);
    WANT(flint_token_logprobs(1, 1 << 20, p, 1 << 20, 0, i, f, f, 32, i, f, a, 0, 0), FLINT_ERR_WORKSPACE);
    for (int k = 0; k < 3; k++) WANT(flint_token_logprobs(1, bad[k], p, 100, 0, i, f, f, 0, 0, 0, a, 0, 0), FLINT_ERR_SHAPE);
    WANT(flint_token_logprobs(1, 100, p, 100, 0, i, f, f, INT32_MAX, i, f, a, 0, 0), FLINT_ERR_SHAPE);
    for (int64_t T = 1; T <= 1 << 20; T *= 4)
        for (int32_t V = 1; V <= 1 << 20; V *= 8)
            if (!flint_token_logprobs_workspace_bytes(T, V, V < 32 ? V : 32)) return 1;
    if (flint_token_logprobs_workspace_bytes((1 << 20) + 1, 10, 0) || flint_token_logprobs_workspace_bytes(1, 10, 11)) return 1;
    printf("ops driver: ok\n");
    return 0;
}
