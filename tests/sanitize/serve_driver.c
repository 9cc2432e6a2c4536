/* Every refusal path of include/flint_serve.h, and the sizing functions over their ranges; no
 * call here reaches a launch.  Pointers are addresses that are never read. */
#include <limits.h>
#include <stdio.h>
#include <stdlib.h>

#include "../../include/flint_serve.h"

#define WANT(call, code)                                                                                      \
    do {                                                                                                      \
        const int got_ = (call);                                                                              \
        if (got_ != (code)) {                                                                                 \
            printf("line %d: %s gave %d, not %d\n", __LINE__, #call, got_, (code));                           \
            exit(1);                                                                                          \
        }                                                                                                     \
    } while (0)
#define HAVE(cond)                                                                                            \
    do {                                                                                                      \
        if (!(cond)) {                                                                                        \
            printf("line %d: %s\n", __LINE__, #cond);                                                         \
            exit(1);                                                                                          \
        }                                                                                                     \
    } while (0)

int main(void)
{
    uint8_t *const a = (uint8_t *)((uintptr_t)1 << 20);
    uint16_t *const p = (uint16_t *)a;
    int32_t *const i = (int32_t *)a;
    float *const f = (float *)a;
    const int32_t bad[] = {INT32_MIN, -1, 0, 100, INT32_MAX};
    const int64_t far[] = {INT64_MIN, -1, (int64_t)1 << 40, INT64_MAX};

    /* the 4-bit cache */
    const flint_kv4_cache c = {32, 4, 128, 64, 100, 0, a};
    const flint_qk_transform t = {0, 0, 0.f, 0, 0, 0, 0, 0};
    const flint_attn at = {1.f, 0, 0};
    WANT(flint_kv4_append(&c, &t, 0, 0, 5120, 0, 0, 0, 4096, 0, 0, 0, 0, 0), FLINT_OK);
    WANT(flint_kv4_append(&c, 0, 1, p, 5120, 0, (int64_t *)a, p, 4096, 0, 0, 0, 0, 0), FLINT_ERR_NULL);
    WANT(flint_kv4_attn_decode(&c, &at, 0, 0, 4096, 0, 4, 0, 0, 0, 4096, 0, 0, 0), FLINT_OK);
    WANT(flint_kv4_attn_decode(&c, &at, 1, p, 4096, i, 4, i, 0, p, 4096, a, 0, 0), FLINT_ERR_WORKSPACE);
    for (int k = 0; k < 5; k++) {
        flint_kv4_cache b[6] = {c, c, c, c, c, c};
        b[0].n_q_heads = bad[k] == 100 ? 33 : bad[k];
        b[1].n_kv_heads = bad[k];
        b[2].head_dim = bad[k];
        b[3].page_size = bad[k];
        b[4].n_pages = bad[k] > 0 ? INT64_MAX : bad[k];
        b[5].page_stride = bad[k] ? bad[k] : INT64_MAX / 16 * 16;
        for (int j = 0; j < 6; j++) {
            WANT(flint_kv4_append(&b[j], &t, 1, p, 5120, 0, (int64_t *)a, p, 4096, 0, 0, 0, 0, 0), FLINT_ERR_SHAPE);
            WANT(flint_kv4_attn_decode(&b[j], &at, 1, p, 4096, i, 4, i, 0, p, 4096, a, 0, 0), FLINT_ERR_SHAPE);
            HAVE(flint_kv4_attn_decode_workspace_bytes(&b[j], 4) == 0);
        }
    }
    for (int k = 0; k < 4; k++) {
        WANT(flint_kv4_append(&c, &t, far[k], p, 5120, 0, (int64_t *)a, p, 4096, 0, 0, 0, 0, 0), FLINT_ERR_SHAPE);
        WANT(flint_kv4_attn_decode(&c, &at, far[k], p, 4096, i, 4, i, 0, p, 4096, a, 0, 0), FLINT_ERR_SHAPE);
        WANT(flint_kv4_attn_decode(&c, &at, 1, p, 4096, i, far[k], i, 0, p, 4096, a, 0, 0), FLINT_ERR_SHAPE);
        HAVE(flint_kv4_attn_decode_workspace_bytes(&c, far[k]) == 0);
    }
    size_t last = 0;
    for (int64_t B = 0; B <= 1024; B += 31) {
        const size_t n = flint_kv4_attn_decode_workspace_bytes(&c, B);
        HAVE(n >= last);
        last = n;
    }

    /* pages */
    const flint_kv_array arr[2] = {{a, 1024, 1024}, {a + (1 << 20), 2048, 4096}};
    const flint_kv_pages pg = {64, 2, 100, arr};
    const flint_kv_state s0 = {i, i + 64, i + 128, i + 192, i + 256}, s1 = {i + 1024, i + 1088, i + 1152, i + 1216, i + 1280};
    WANT(flint_kv_advance(&pg, 8, 2, &s0, 3, &s1, i, i, 0, 0, a, 0, 0), FLINT_ERR_WORKSPACE);
    WANT(flint_kv_compact(&pg, 8, 3, &s0, &s1, i, a, 0, 0), FLINT_ERR_WORKSPACE);
    WANT(flint_kv_advance(&pg, 8, 2, &s0, 3, &s0, i, i, 0, 0, a, 0, 0), FLINT_ERR_SHAPE);
    WANT(flint_kv_compact(&pg, 8, 3, &s0, &s0, i, a, 0, 0), FLINT_ERR_SHAPE);
    for (int k = 0; k < 5; k++) {
        flint_kv_pages b[3] = {pg, pg, pg};
        b[0].page_size = bad[k];
        b[1].n_arrays = bad[k] > 0 ? 1025 : bad[k] ? bad[k] : -1;
        b[2].n_pages = bad[k] == 100 ? INT64_MAX : bad[k];
        for (int j = 0; j < 3; j++) {
            WANT(flint_kv_advance(&b[j], 8, 2, &s0, 3, &s1, i, i, 0, 0, a, 1 << 30, 0), FLINT_ERR_SHAPE);
            WANT(flint_kv_compact(&b[j], 8, 3, &s0, &s1, i, a, 1 << 30, 0), FLINT_ERR_SHAPE);
            HAVE(flint_kv_pages_workspace_bytes(&b[j], 1) == 0);
        }
    }
    for (int k = 0; k < 4; k++) {
        const flint_kv_array one = {a, far[k] > 0 ? far[k] / 16 * 16 : far[k], far[k]};
        flint_kv_pages b = pg;
        b.n_arrays = 1;
        b.arrays = &one;
        WANT(flint_kv_advance(&b, 8, 2, &s0, 3, &s1, i, i, 0, 0, a, 1 << 30, 0), FLINT_ERR_SHAPE);
        WANT(flint_kv_advance(&pg, far[k], 2, &s0, 3, &s1, i, i, 0, 0, a, 1 << 30, 0), FLINT_ERR_SHAPE);
        WANT(flint_kv_advance(&pg, 8, far[k], &s0, 3, &s1, i, i, 0, 0, a, 1 << 30, 0), FLINT_ERR_SHAPE);
        WANT(flint_kv_advance(&pg, 8, 2, &s0, far[k], &s1, i, i, 0, 0, a, 1 << 30, 0), FLINT_ERR_SHAPE);
        WANT(flint_kv_advance(&pg, 8, 2, &s0, 3, &s1, i, i, (int64_t *)a, far[k], a, 1 << 30, 0), FLINT_ERR_SHAPE);
        WANT(flint_kv_compact(&pg, far[k], 3, &s0, &s1, i, a, 1 << 30, 0), FLINT_ERR_SHAPE);
        WANT(flint_kv_compact(&pg, 8, far[k], &s0, &s1, i, a, 1 << 30, 0), FLINT_ERR_SHAPE);
        HAVE(flint_kv_pages_workspace_bytes(&pg, far[k]) == 0);
    }
    for (int64_t n = 1; n <= 1 << 24; n *= 2) {
        const flint_kv_pages b = {16, 0, n, 0};
        HAVE(flint_kv_pages_workspace_bytes(&b, 0) >= 12 * (size_t)n);
        HAVE(flint_kv_pages_workspace_bytes(&b, 1024) >= flint_kv_pages_workspace_bytes(&b, 0));
    }

    /* adapters */
    const flint_lora_adapters l = {2048, 5120, 16, 4, p, p, 0, 0};
    WANT(flint_lora(&l, 0, 0, 2048, 0, 0, 0, 0, 0, 5120, 0, 0, 0, 0), FLINT_OK);
    WANT(flint_lora(&l, 8, p, 2048, i, 0, 0, 0, a, 5120, 0, a, 0, 0), FLINT_ERR_WORKSPACE);
    WANT(flint_lora(&l, 8, p, 2048, i, a, 5121, 0, a, 5120, 0, a, 1 << 20, 0), FLINT_ERR_SHAPE);
    for (int k = 0; k < 5; k++) {
        flint_lora_adapters b[4] = {l, l, l, l};
        b[0].in_features = bad[k];
        b[1].out_features = bad[k] == 100 ? INT32_MAX : bad[k];
        b[2].max_rank = bad[k];
        b[3].n_adapters = bad[k] == 100 ? INT32_MAX : bad[k];
        for (int j = 0; j < 4; j++) {
            WANT(flint_lora(&b[j], 8, p, 2048, i, 0, 0, 0, a, 5120, 0, a, 1 << 30, 0), FLINT_ERR_SHAPE);
            HAVE(flint_lora_workspace_bytes(&b[j], 8) == 0);
        }
        WANT(flint_lora(&l, 8, p, 2048, i, 0, 0, 0, a, 5120, bad[k] ? bad[k] : 7, a, 1 << 30, 0), FLINT_ERR_FORMAT);
    }
    for (int k = 0; k < 4; k++) {
        WANT(flint_lora(&l, far[k], p, 2048, i, 0, 0, 0, a, 5120, 0, a, 1 << 30, 0), FLINT_ERR_SHAPE);
        HAVE(flint_lora_workspace_bytes(&l, far[k]) == 0);
        if (far[k] < 0) {
            WANT(flint_lora(&l, 8, p, far[k], i, 0, 0, 0, a, 5120, 0, a, 1 << 30, 0), FLINT_ERR_SHAPE);
            WANT(flint_lora(&l, 8, p, 2048, i, a, far[k], 0, a, 5120, 0, a, 1 << 30, 0), FLINT_ERR_SHAPE);
            WANT(flint_lora(&l, 8, p, 2048, i, 0, 0, 0, a, far[k], 0, a, 1 << 30, 0), FLINT_ERR_SHAPE);
        }
    }
    for (int K = 8; K <= 32768; K *= 8)
        for (int R = 8; R <= 128; R += 24)
            for (int64_t T = 1; T <= 65536; T *= 4) {
                const flint_lora_adapters b = {K, 5120, R, 4, p, p, 0, 0};
                HAVE(flint_lora_workspace_bytes(&b, T) >= 16);
            }

    /* logits */
    flint_logit_rules r = {0};
    WANT(flint_logits_adjust(&r, 0, 100, 0, 100, 0, 100, 0, 0), FLINT_OK);
    WANT(flint_logits_adjust(0, 1, 100, a, 100, a, 100, 0, 0), FLINT_ERR_NULL);
    for (int k = 0; k < 5; k++)
        if (bad[k] != 100) WANT(flint_logits_adjust(&r, 1, bad[k], a, INT64_MAX, a, INT64_MAX, 0, 0), FLINT_ERR_SHAPE);
    for (int k = 0; k < 4; k++) {
        WANT(flint_logits_adjust(&r, far[k], 100, a, 100, a, 100, 0, 0), FLINT_ERR_SHAPE);
        if (far[k] < 0) {
            WANT(flint_logits_adjust(&r, 1, 100, a, far[k], a, 100, 0, 0), FLINT_ERR_SHAPE);
            WANT(flint_logits_adjust(&r, 1, 100, a, 100, a, far[k], 0, 0), FLINT_ERR_SHAPE);
            flint_logit_rules b = r;
            b.history = i;
            b.ldh = far[k];
            WANT(flint_logits_adjust(&b, 1, 100, a, 100, a, 100, 0, 0), FLINT_ERR_SHAPE);
            b = r;
            b.masks = (const uint32_t *)a;
            b.ldm = far[k];
            b.n_masks = 1;
            WANT(flint_logits_adjust(&b, 1, 100, a, 100, a, 100, 0, 0), FLINT_ERR_SHAPE);
        }
    }
    (void)f;
    printf("serve driver: ok\n");
    return 0;
}
