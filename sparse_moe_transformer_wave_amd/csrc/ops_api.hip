// ops_api.hip -- the C ABI declared in include/flint_ops.h: argument validation and dispatch.
// Like api.hip, validation runs before any HIP call.
#include "../../include/flint_ops.h"
#include "ops.h"

using namespace flint;

namespace {

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int check_cache(const flint_kv_cache *c)
{
    if (!c) return FLINT_ERR_NULL;
    if (c->head_dim != 64 && c->head_dim != 128) return FLINT_ERR_SHAPE;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return FLINT_ERR_SHAPE;
    if (c->n_kv_heads < 1 || c->n_kv_heads > 64) return FLINT_ERR_SHAPE;
    if (c->n_q_heads < 1 || c->n_q_heads % c->n_kv_heads || c->n_q_heads / c->n_kv_heads > 32) return FLINT_ERR_SHAPE;
    if (c->n_pages < 1 || c->n_pages > INT32_MAX) return FLINT_ERR_SHAPE;
    const int64_t block = (int64_t)c->n_kv_heads * c->page_size * c->head_dim;
    if (c->page_stride != 0 && (c->page_stride < block || c->page_stride % 8)) return FLINT_ERR_SHAPE;
    if (c->page_stride > INT64_MAX / 2 / c->n_pages) return FLINT_ERR_SHAPE;  // byte offsets fit 64 bits
    return FLINT_OK;
}

int check_cache_pointers(const flint_kv_cache *c)
{
    if (!c->k || !c->v) return FLINT_ERR_NULL;
    return aligned(c->k, 16) && aligned(c->v, 16) ? FLINT_OK : FLINT_ERR_ALIGN;
}

Cache cache_of(const flint_kv_cache *c)
{
    Cache r;
    r.Hq = c->n_q_heads;
    r.Hkv = c->n_kv_heads;
    r.D = c->head_dim;
    r.page = c->page_size;
    r.page_shift = __builtin_ctz((unsigned)c->page_size);
    r.n_pages = c->n_pages;
    r.page_stride = c->page_stride ? c->page_stride : (int64_t)c->n_kv_heads * c->page_size * c->head_dim;
    r.k = c->k;
    r.v = c->v;
    return r;
}

}  // namespace

extern "C" {

int flint_linear_int4(const flint_int4_linear *w, int64_t T, const uint16_t *x, int64_t ldx,
                      const uint16_t *residual, int64_t ldr, void *y, int64_t ldy, int32_t y_type,
                      void *stream)
{
    if (!w) return FLINT_ERR_NULL;
    if (w->in_features < 128 || w->in_features > 32768 || w->in_features % 128) return FLINT_ERR_SHAPE;
    if (w->out_features < 1 || w->out_features > (1 << 24)) return FLINT_ERR_SHAPE;
    if (w->group != 32 && w->group != 64 && w->group != 128) return FLINT_ERR_SHAPE;
    if (T < 0 || T > 64) return FLINT_ERR_SHAPE;
    if (y_type != FLINT_DT_BF16 && y_type != FLINT_DT_FP32) return FLINT_ERR_FORMAT;
    if (ldx < w->in_features || ldx % 8 || ldy < w->out_features || (residual && ldr < w->out_features))
        return FLINT_ERR_SHAPE;
    if (T == 0) return FLINT_OK;
    if (!w->codes || !w->scales || !x || !y) return FLINT_ERR_NULL;
    if (!aligned(w->codes, 16) || !aligned(w->scales, 16) || !aligned(x, 16) || !aligned(residual, 2) ||
        !aligned(y, y_type == FLINT_DT_FP32 ? 4 : 2))
        return FLINT_ERR_ALIGN;
    const LinearArgs a{(int)T, w->in_features, w->out_features, w->group, w->codes, w->scales,
                       x, ldx, residual, ldr, y, ldy, y_type == FLINT_DT_FP32};
    return hip_status(launch_linear_int4(a, (hipStream_t)stream));
}

int flint_kv_append(const flint_kv_cache *cache, const flint_qk_transform *transform, int64_t T,
                    const uint16_t *qkv, int64_t ldqkv, const int32_t *positions,
                    const int64_t *slots, uint16_t *q, int64_t ldq, void *stream)
{
    int rc = check_cache(cache);
    if (rc) return rc;
    if (!transform) return FLINT_ERR_NULL;
    const flint_qk_transform &t = *transform;
    if (t.rot_dim < 0 || t.rot_dim > cache->head_dim || t.rot_dim % 2) return FLINT_ERR_SHAPE;
    if (t.rope_style != FLINT_ROPE_HALF && t.rope_style != FLINT_ROPE_PAIRS) return FLINT_ERR_FORMAT;
    if (t.rot_dim && t.max_position < 1) return FLINT_ERR_SHAPE;
    if (!(t.eps >= 0.f)) return FLINT_ERR_SHAPE;
    if (T < 0 || T > (1 << 20)) return FLINT_ERR_SHAPE;
    const int64_t D = cache->head_dim;
    if (ldqkv < (cache->n_q_heads + 2 * (int64_t)cache->n_kv_heads) * D || ldqkv % 8) return FLINT_ERR_SHAPE;
    if (ldq < cache->n_q_heads * D || ldq % 8) return FLINT_ERR_SHAPE;
    if (T == 0) return FLINT_OK;
    rc = check_cache_pointers(cache);
    if (rc) return rc;
    if (!qkv || !slots || !q) return FLINT_ERR_NULL;
    if (t.rot_dim && (!t.cos || !t.sin || !positions)) return FLINT_ERR_NULL;
    if (!aligned(qkv, 16) || !aligned(q, 16) || !aligned(t.q_norm, 16) || !aligned(t.k_norm, 16) ||
        !aligned(t.cos, 16) || !aligned(t.sin, 16) || !aligned(positions, 4) || !aligned(slots, 8))
        return FLINT_ERR_ALIGN;
    AppendArgs a;
    a.c = cache_of(cache);
    a.q_norm = t.q_norm;
    a.k_norm = t.k_norm;
    a.eps = t.eps;
    a.rot = t.rot_dim;
    a.pairs = t.rope_style == FLINT_ROPE_PAIRS;
    a.max_pos = t.max_position;
    a.cos = t.cos;
    a.sin = t.sin;
    a.T = (int)T;
    a.qkv = qkv;
    a.ldqkv = ldqkv;
    a.positions = positions;
    a.slots = slots;
    a.q = q;
    a.ldq = ldq;
    return hip_status(launch_kv_append(a, (hipStream_t)stream));
}

size_t flint_attn_decode_workspace_bytes(const flint_kv_cache *cache, int64_t B_max)
{
    if (check_cache(cache) != FLINT_OK || B_max < 0 || B_max > kAttnMaxB) return 0;
    return attn_decode_ws_bytes(cache_of(cache), B_max);
}

int flint_attn_decode(const flint_kv_cache *cache, const flint_attn *attn, int64_t B,
                      const uint16_t *q, int64_t ldq, const int32_t *table, int64_t ldt,
                      const int32_t *kv_len, int32_t prefix_len, uint16_t *out, int64_t ldo,
                      void *ws, size_t ws_bytes, void *stream)
{
    int rc = check_cache(cache);
    if (rc) return rc;
    if (!attn) return FLINT_ERR_NULL;
    if (B < 0 || B > kAttnMaxB || attn->window < 0 || prefix_len < 0) return FLINT_ERR_SHAPE;
    const int64_t width = (int64_t)cache->n_q_heads * cache->head_dim;
    if (ldq < width || ldq % 8 || ldo < width || ldo % 8) return FLINT_ERR_SHAPE;
    if (ldt < 1 || ldt > (1 << 25) / cache->page_size || prefix_len > ldt * cache->page_size) return FLINT_ERR_SHAPE;
    if (B == 0) return FLINT_OK;
    rc = check_cache_pointers(cache);
    if (rc) return rc;
    if (!q || !table || !kv_len || !out || !ws) return FLINT_ERR_NULL;
    if (!aligned(q, 16) || !aligned(table, 4) || !aligned(kv_len, 4) || !aligned(out, 16) || !aligned(ws, 16) ||
        !aligned(attn->sinks, 4))
        return FLINT_ERR_ALIGN;
    AttnArgs a;
    a.c = cache_of(cache);
    if (ws_bytes < attn_decode_call_bytes(a.c, B)) return FLINT_ERR_WORKSPACE;
    a.scale = attn->scale;
    a.window = attn->window;
    a.sinks = attn->sinks;
    a.B = (int)B;
    a.prefix = prefix_len;
    a.q = q;
    a.ldq = ldq;
    a.table = table;
    a.ldt = ldt;
    a.kv_len = kv_len;
    a.out = out;
    a.ldo = ldo;
    a.ws = (float *)ws;
    return hip_status(launch_attn_decode(a, (hipStream_t)stream));
}

size_t flint_token_logprobs_workspace_bytes(int64_t T_max, int32_t vocab, int32_t top_n)
{
    if (T_max < 0 || T_max > (1 << 20) || vocab < 1 || vocab > (1 << 20)) return 0;
    if (top_n < 0 || top_n > 32 || top_n > vocab) return 0;
    return logprobs_ws_bytes(T_max, vocab, top_n);
}

int flint_token_logprobs(int64_t T, int32_t vocab, const void *logits, int64_t ld, int32_t dtype,
                         const int32_t *tokens, float *logprob, float *entropy, int32_t top_n,
                         int32_t *top_ids, float *top_logprobs, void *ws, size_t ws_bytes,
                         void *stream)
{
    if (T < 0 || T > (1 << 20) || vocab < 1 || vocab > (1 << 20) || ld < vocab) return FLINT_ERR_SHAPE;
    if (top_n < 0 || top_n > 32 || top_n > vocab) return FLINT_ERR_SHAPE;
    if (dtype != FLINT_DT_BF16 && dtype != FLINT_DT_FP32) return FLINT_ERR_FORMAT;
    if (T == 0) return FLINT_OK;
    if (!logits || !ws || (logprob && !tokens)) return FLINT_ERR_NULL;
    if ((top_ids != nullptr) != (top_logprobs != nullptr) && top_n) return FLINT_ERR_NULL;
    if (!aligned(logits, dtype == FLINT_DT_FP32 ? 4 : 2) || !aligned(tokens, 4) || !aligned(logprob, 4) ||
        !aligned(entropy, 4) || !aligned(top_ids, 4) || !aligned(top_logprobs, 4) || !aligned(ws, 16))
        return FLINT_ERR_ALIGN;
    if (ws_bytes < logprobs_call_bytes(T, vocab, top_n)) return FLINT_ERR_WORKSPACE;
    const LogprobArgs a{(int)T, vocab, logits, ld, dtype == FLINT_DT_FP32, tokens, logprob, entropy,
                        top_ids ? top_n : 0, top_ids, top_logprobs, ws};
    return hip_status(launch_token_logprobs(a, (hipStream_t)stream));
}

}  // extern "C"
