// serve_api.hip -- the C ABI declared in include/flint_serve.h: argument validation and dispatch.
// Validation runs before any HIP call.
#include "../../include/flint_serve.h"
#include "serve.h"

using namespace flint;

namespace {

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool page_size_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }

// ---- 4-bit cache ---------------------------------------------------------------------------
int64_t block_bytes(const flint_kv4_cache *c)
{
    return 2 * (int64_t)c->n_kv_heads * c->page_size * (c->head_dim / 2 + c->head_dim / 32);
}

int check_cache(const flint_kv4_cache *c)
{
    if (!c) return FLINT_ERR_NULL;
    if (c->head_dim != 64 && c->head_dim != 128) return FLINT_ERR_SHAPE;
    if (!page_size_ok(c->page_size)) return FLINT_ERR_SHAPE;
    if (c->n_kv_heads < 1 || c->n_kv_heads > 64) return FLINT_ERR_SHAPE;
    if (c->n_q_heads < 1 || c->n_q_heads % c->n_kv_heads || c->n_q_heads / c->n_kv_heads > 32) return FLINT_ERR_SHAPE;
    if (c->n_pages < 1 || c->n_pages > INT32_MAX) return FLINT_ERR_SHAPE;
    if (c->page_stride != 0 && (c->page_stride < block_bytes(c) || c->page_stride % 16)) return FLINT_ERR_SHAPE;
    if (c->page_stride > INT64_MAX / c->n_pages) return FLINT_ERR_SHAPE;  // offsets fit 64 bits
    return FLINT_OK;
}

int check_cache_pointer(const flint_kv4_cache *c)
{
    if (!c->data) return FLINT_ERR_NULL;
    return aligned(c->data, 16) ? FLINT_OK : FLINT_ERR_ALIGN;
}

Cache cache_of(const flint_kv4_cache *c)
{
    Cache r;
    r.Hq = c->n_q_heads;
    r.Hkv = c->n_kv_heads;
    r.D = c->head_dim;
    r.page = c->page_size;
    r.page_shift = __builtin_ctz((unsigned)c->page_size);
    r.n_pages = c->n_pages;
    r.page_stride = c->page_stride ? c->page_stride : block_bytes(c);
    r.k = (uint16_t *)c->data;
    r.v = nullptr;
    return r;
}

// ---- pages -----------------------------------------------------------------------------------
int check_pages(const flint_kv_pages *p)
{
    if (!p) return FLINT_ERR_NULL;
    if (!page_size_ok(p->page_size) || p->n_arrays < 0 || p->n_arrays > 1024) return FLINT_ERR_SHAPE;
    if (p->n_pages < 1 || p->n_pages > (1 << 24)) return FLINT_ERR_SHAPE;
    if (p->n_arrays && !p->arrays) return FLINT_ERR_NULL;
    for (int i = 0; i < p->n_arrays; i++) {
        const flint_kv_array &a = p->arrays[i];
        if (a.bytes < 16 || a.bytes > (1 << 30) || a.bytes % 16 || a.stride < a.bytes || a.stride % 16) return FLINT_ERR_SHAPE;
        if (a.stride > INT64_MAX / p->n_pages) return FLINT_ERR_SHAPE;
    }
    return FLINT_OK;
}

int check_arrays(const flint_kv_pages *p)
{
    for (int i = 0; i < p->n_arrays; i++) {
        if (!p->arrays[i].base) return FLINT_ERR_NULL;
        if (!aligned(p->arrays[i].base, 16)) return FLINT_ERR_ALIGN;
    }
    return FLINT_OK;
}

// A state of `rows` rows: its tables may be absent where there are none.
int check_state(const flint_kv_state *s, int64_t rows)
{
    if (!s) return FLINT_ERR_NULL;
    if (!s->refs || !s->free_list || !s->n_free || (rows && (!s->table || !s->kv_len))) return FLINT_ERR_NULL;
    if (!aligned(s->refs, 4) || !aligned(s->free_list, 4) || !aligned(s->n_free, 4) || !aligned(s->table, 4) || !aligned(s->kv_len, 4))
        return FLINT_ERR_ALIGN;
    return FLINT_OK;
}

// Whether a state of `rows` rows and one of `rows_b` have memory in common.
bool shares(const flint_kv_pages *p, int64_t ldt, const flint_kv_state *a, int64_t rows, const flint_kv_state *b, int64_t rows_b)
{
    struct Array {
        uintptr_t at;
        uint64_t bytes;
    };
    auto arrays = [&](const flint_kv_state *s, int64_t r, Array *to) {
        const uint64_t pages = 4 * (uint64_t)p->n_pages;
        to[0] = {(uintptr_t)s->refs, pages};
        to[1] = {(uintptr_t)s->free_list, pages};
        to[2] = {(uintptr_t)s->n_free, 4};
        to[3] = {(uintptr_t)s->table, 4 * (uint64_t)r * (uint64_t)ldt};
        to[4] = {(uintptr_t)s->kv_len, 4 * (uint64_t)r};
    };
    Array x[5], y[5];
    arrays(a, rows, x);
    arrays(b, rows_b, y);
    for (const Array &i : x)
        for (const Array &j : y)
            if (i.at <= j.at ? j.at - i.at < i.bytes && j.bytes : i.at - j.at < j.bytes && i.bytes) return true;
    return false;
}

PageState state_of(const flint_kv_state *s) { return PageState{s->refs, s->free_list, s->n_free, s->table, s->kv_len}; }

static_assert(sizeof(PageArray) == sizeof(flint_kv_array), "the arrays are passed on as they are");

PagesArgs pages_args(const flint_kv_pages *p, int64_t ldt, const flint_kv_state *old, const flint_kv_state *state, void *ws)
{
    PagesArgs a{};
    a.page = p->page_size;
    a.page_shift = __builtin_ctz((unsigned)p->page_size);
    a.n_arrays = p->n_arrays;
    a.n_pages = (int)p->n_pages;
    a.arrays = reinterpret_cast<const PageArray *>(p->arrays);
    a.ldt = ldt;
    a.old = state_of(old);
    a.state = state_of(state);
    a.ws = (int32_t *)ws;
    return a;
}

// ---- adapters ----------------------------------------------------------------------------------
int check_adapters(const flint_lora_adapters *l)
{
    if (!l) return FLINT_ERR_NULL;
    if (l->in_features < 8 || l->in_features > 32768 || l->in_features % 8) return FLINT_ERR_SHAPE;
    if (l->out_features < 1 || l->out_features > (1 << 24)) return FLINT_ERR_SHAPE;
    if (l->max_rank < 8 || l->max_rank > 128 || l->max_rank % 8) return FLINT_ERR_SHAPE;
    if (l->n_adapters < 1 || l->n_adapters > (1 << 20)) return FLINT_ERR_SHAPE;
    return FLINT_OK;
}
constexpr int64_t kLoraMaxT = 65536;

bool type_ok(int32_t t) { return t == FLINT_DT_BF16 || t == FLINT_DT_FP32; }
uintptr_t type_size(int32_t t) { return t == FLINT_DT_FP32 ? 4 : 2; }

}  // namespace

extern "C" {

int flint_kv4_append(const flint_kv4_cache *cache, const flint_qk_transform *transform, int64_t T,
                     const uint16_t *qkv, int64_t ldqkv, const int32_t *positions,
                     const int64_t *slots, uint16_t *q, int64_t ldq, uint16_t *k, int64_t ldk,
                     uint16_t *v, int64_t ldv, void *stream)
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
    const int64_t D = cache->head_dim, kv = cache->n_kv_heads * D;
    if (ldqkv < cache->n_q_heads * D + 2 * kv || ldqkv % 8) return FLINT_ERR_SHAPE;
    if (ldq < cache->n_q_heads * D || ldq % 8) return FLINT_ERR_SHAPE;
    if ((k && (ldk < kv || ldk % 8)) || (v && (ldv < kv || ldv % 8))) return FLINT_ERR_SHAPE;
    if (T == 0) return FLINT_OK;
    rc = check_cache_pointer(cache);
    if (rc) return rc;
    if (!qkv || !slots || !q) return FLINT_ERR_NULL;
    if (t.rot_dim && (!t.cos || !t.sin || !positions)) return FLINT_ERR_NULL;
    if (!aligned(qkv, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(t.q_norm, 16) ||
        !aligned(t.k_norm, 16) || !aligned(t.cos, 16) || !aligned(t.sin, 16) || !aligned(positions, 4) || !aligned(slots, 8))
        return FLINT_ERR_ALIGN;
    Append4Args x;
    AppendArgs &a = x.a;
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
    x.k = k;
    x.ldk = ldk;
    x.v = v;
    x.ldv = ldv;
    return hip_status(launch_kv_append4(x, (hipStream_t)stream));
}

size_t flint_kv4_attn_decode_workspace_bytes(const flint_kv4_cache *cache, int64_t B_max)
{
    if (check_cache(cache) != FLINT_OK || B_max < 0 || B_max > kAttnMaxB) return 0;
    return attn_decode4_ws_bytes(cache_of(cache), B_max);
}

int flint_kv4_attn_decode(const flint_kv4_cache *cache, const flint_attn *attn, int64_t B,
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
    rc = check_cache_pointer(cache);
    if (rc) return rc;
    if (!q || !table || !kv_len || !out || !ws) return FLINT_ERR_NULL;
    if (!aligned(q, 16) || !aligned(table, 4) || !aligned(kv_len, 4) || !aligned(out, 16) || !aligned(ws, 16) ||
        !aligned(attn->sinks, 4))
        return FLINT_ERR_ALIGN;
    AttnArgs a;
    a.c = cache_of(cache);
    if (ws_bytes < attn_decode4_call_bytes(a.c, B)) return FLINT_ERR_WORKSPACE;
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
    return hip_status(launch_attn_decode4(a, (hipStream_t)stream));
}

size_t flint_kv_pages_workspace_bytes(const flint_kv_pages *pages, int64_t rows_max)
{
    if (check_pages(pages) != FLINT_OK || rows_max < 0 || rows_max > kPagesMaxRows) return 0;
    return kv_pages_ws_bytes(pages->n_pages, rows_max);
}

int flint_kv_advance(const flint_kv_pages *pages, int64_t ldt, int64_t rows_old, const flint_kv_state *old,
                     int64_t rows, const flint_kv_state *state, const int32_t *parent, const int32_t *grow,
                     int64_t *slots, int64_t lds, void *ws, size_t ws_bytes, void *stream)
{
    int rc = check_pages(pages);
    if (rc) return rc;
    if (rows_old < 0 || rows_old > kPagesMaxRows || rows < 0 || rows > kPagesMaxRows) return FLINT_ERR_SHAPE;
    if (ldt < 1 || ldt > (1 << 25) / pages->page_size) return FLINT_ERR_SHAPE;
    if (slots && (lds < 1 || lds > (1 << 25))) return FLINT_ERR_SHAPE;
    rc = check_arrays(pages);
    if (!rc) rc = check_state(old, rows_old);
    if (!rc) rc = check_state(state, rows);
    if (rc) return rc;
    if (!ws || (rows && (!parent || !grow))) return FLINT_ERR_NULL;
    if (!aligned(parent, 4) || !aligned(grow, 4) || !aligned(slots, 8) || !aligned(ws, 16)) return FLINT_ERR_ALIGN;
    if (shares(pages, ldt, old, rows_old, state, rows)) return FLINT_ERR_SHAPE;
    if (ws_bytes < kv_pages_ws_bytes(pages->n_pages, rows_old > rows ? rows_old : rows)) return FLINT_ERR_WORKSPACE;
    PagesArgs a = pages_args(pages, ldt, old, state, ws);
    a.rows_old = (int)rows_old;
    a.rows = (int)rows;
    a.parent = parent;
    a.grow = grow;
    a.slots = slots;
    a.lds = lds;
    return hip_status(launch_kv_advance(a, (hipStream_t)stream));
}

int flint_kv_compact(const flint_kv_pages *pages, int64_t ldt, int64_t rows, const flint_kv_state *old,
                     const flint_kv_state *state, int32_t *moved, void *ws, size_t ws_bytes, void *stream)
{
    int rc = check_pages(pages);
    if (rc) return rc;
    if (rows < 0 || rows > kPagesMaxRows) return FLINT_ERR_SHAPE;
    if (ldt < 1 || ldt > (1 << 25) / pages->page_size) return FLINT_ERR_SHAPE;
    rc = check_arrays(pages);
    if (!rc) rc = check_state(old, rows);
    if (!rc) rc = check_state(state, rows);
    if (rc) return rc;
    if (!ws || !moved) return FLINT_ERR_NULL;
    if (!aligned(moved, 4) || !aligned(ws, 16)) return FLINT_ERR_ALIGN;
    if (shares(pages, ldt, old, rows, state, rows)) return FLINT_ERR_SHAPE;
    if (ws_bytes < kv_pages_ws_bytes(pages->n_pages, rows)) return FLINT_ERR_WORKSPACE;
    PagesArgs a = pages_args(pages, ldt, old, state, ws);
    a.rows_old = a.rows = (int)rows;
    a.moved = moved;
    return hip_status(launch_kv_compact(a, (hipStream_t)stream));
}

size_t flint_lora_workspace_bytes(const flint_lora_adapters *adapters, int64_t T_max)
{
    if (check_adapters(adapters) != FLINT_OK || T_max < 0 || T_max > kLoraMaxT) return 0;
    return lora_ws_bytes(T_max, adapters->in_features, adapters->max_rank);
}

int flint_lora(const flint_lora_adapters *adapters, int64_t T, const uint16_t *x, int64_t ldx,
               const int32_t *ids, const void *base, int64_t ldb, int32_t base_type, void *y,
               int64_t ldy, int32_t y_type, void *ws, size_t ws_bytes, void *stream)
{
    int rc = check_adapters(adapters);
    if (rc) return rc;
    if (T < 0 || T > kLoraMaxT) return FLINT_ERR_SHAPE;
    if (!type_ok(y_type) || (base && !type_ok(base_type))) return FLINT_ERR_FORMAT;
    const flint_lora_adapters &l = *adapters;
    if (ldx < l.in_features || ldx % 8 || ldy < l.out_features || (base && ldb < l.out_features)) return FLINT_ERR_SHAPE;
    if (base && base == y && (base_type != y_type || ldb != ldy)) return FLINT_ERR_SHAPE;
    if (T == 0) return FLINT_OK;
    if (!l.a || !l.b || !x || !ids || !y || !ws) return FLINT_ERR_NULL;
    if (!aligned(l.a, 16) || !aligned(l.b, 16) || !aligned(l.ranks, 4) || !aligned(l.scales, 4) || !aligned(x, 16) || !aligned(ids, 4) ||
        !aligned(y, type_size(y_type)) || (base && !aligned(base, type_size(base_type))) || !aligned(ws, 16))
        return FLINT_ERR_ALIGN;
    if (ws_bytes < lora_call_bytes(T, l.in_features, l.max_rank)) return FLINT_ERR_WORKSPACE;
    const LoraArgs a{(int)T, l.in_features, l.out_features, l.max_rank, l.n_adapters, l.a, l.b, l.ranks, l.scales,
                     x, ldx, ids, base, base ? ldb : 0, base_type == FLINT_DT_FP32, y, ldy, y_type == FLINT_DT_FP32, (float *)ws};
    return hip_status(launch_lora(a, (hipStream_t)stream));
}

int flint_logits_adjust(const flint_logit_rules *rules, int64_t T, int32_t vocab, const void *logits,
                        int64_t ld, void *out, int64_t ldo, int32_t dtype, void *stream)
{
    if (!rules) return FLINT_ERR_NULL;
    if (!type_ok(dtype)) return FLINT_ERR_FORMAT;
    if (T < 0 || T > 65536 || vocab < 1 || vocab > (1 << 20) || ld < vocab || ldo < vocab) return FLINT_ERR_SHAPE;
    const flint_logit_rules &r = *rules;
    if (r.history && (r.ldh < 0 || r.ldh > INT32_MAX)) return FLINT_ERR_SHAPE;
    if (r.bias_start && (r.n_bias < 0 || r.n_bias > INT32_MAX)) return FLINT_ERR_SHAPE;
    if (r.masks && (r.ldm < (vocab + 31) / 32 || r.n_masks < 0 || r.n_masks > INT64_MAX / 8 / r.ldm)) return FLINT_ERR_SHAPE;
    if (T == 0) return FLINT_OK;
    if (!logits || !out) return FLINT_ERR_NULL;
    if (r.bias_start && r.n_bias && (!r.bias_ids || !r.bias)) return FLINT_ERR_NULL;
    const uintptr_t size = type_size(dtype);
    if (!aligned(logits, size) || !aligned(out, size)) return FLINT_ERR_ALIGN;
    const void *words[] = {r.history, r.prompt_len, r.total_len, r.repetition, r.frequency, r.presence,
                           r.bias_start, r.bias_ids, r.bias, r.masks, r.mask_rows};
    for (const void *p : words)
        if (!aligned(p, 4)) return FLINT_ERR_ALIGN;
    if (logits == out && ld != ldo) return FLINT_ERR_SHAPE;
    const LogitsArgs a{(int)T, vocab, logits, ld, out, ldo, dtype == FLINT_DT_FP32, r.history, r.ldh, r.prompt_len, r.total_len,
                       r.repetition, r.frequency, r.presence, r.bias_start, r.bias_ids, r.bias, r.n_bias, r.masks, r.ldm, r.n_masks,
                       r.mask_rows};
    return hip_status(launch_logits_adjust(a, (hipStream_t)stream));
}

}  // extern "C"
