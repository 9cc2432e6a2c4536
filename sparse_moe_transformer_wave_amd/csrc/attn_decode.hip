// attn_decode.hip -- decode attention over the paged cache, a prefix shared by the batch read
// once: out[b][h] = sum_j p_j v_j, p = softmax_j(scale q . k_j) with an optional sink.
//
// Sequences that can only be short (a window, or a table of few pages) are one workgroup per
// sequence, key/value head and 16 rows, which writes the result: one launch.  Otherwise the
// work of a call is a list of items, one workgroup each.  A prefix item takes a chunk of the shared prefix for up to 256 query
// rows of one key/value head (all the batch's queries of that head); an own item takes a
// chunk of one sequence's own tokens for 16 rows (its G = Hq / Hkv queries); the workgroups of
// the own items derive their list from kv_len, all the same one.  An item leaves
// its rows' maximum, sum and weighted values in the workspace, and a second launch joins
// each row's items and the sink.
//
// Scores are computed transposed, S^T (tokens x rows) = K Q^T, with the tokens of a tile
// taken in an order that leaves 8 consecutive tokens of a row in each lane's results.  That is
// the B operand of O^T (channels x rows) = V^T P^T, so probabilities never leave their lane,
// a row's statistics are per-lane numbers, and with values stored transposed both products'
// A operands are 16-byte pieces of the cache as it lies.
#include "ops.h"

#include <algorithm>

namespace flint {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kWaves = 8;
constexpr int kTok = 32;        // tokens of a register tile
constexpr int kRows = 16;       // query rows of an own item
constexpr int kStageTok = 64;   // tokens of an LDS stage (prefix items)
constexpr int kPreRows = 256;   // query rows of a prefix item: 32 per wave
constexpr int kCut = 64;        // stages between refills of the page list
constexpr int kPreTarget = 256; // prefix items of a call: one per CU, beyond one per row tile
constexpr int kOwnTarget = 1024;  // own items of a call, beyond one per sequence and row tile
constexpr int kWhole = 1024;    // a sequence of up to so many visible tokens is one workgroup's work

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// A batch whose rows of one key/value head fit one 16-row tile takes its prefix through the
// own-item path (the bytes are the same, and every wave works); one sequence shares nothing.
__host__ __device__ inline bool wide_prefix(int B, int G) { return B * G > kRows; }
__host__ __device__ inline int prefix_rows(int B, int G)
{
    if (!wide_prefix(B, G)) return kRows;
    const int r = ceil_div(B * G, 32) * 32;
    return r < kPreRows ? r : kPreRows;
}

// The prefix items of a call, known to the host.
struct Pre {
    int P, wide;             // shared tokens that are taken as such; 32x32 path or own-item path
    int rows, rtp;           // rows of an item and row tiles
    int tiles, chunk, nc;    // LDS stages (wide) or register tiles; per item; chunks
    int items;               // workgroups, all heads (some empty)
};
__host__ __device__ inline Pre pre_of(const AttnArgs &a)
{
    const int G = a.c.Hq / a.c.Hkv, unit = a.c.page > kStageTok ? a.c.page : kStageTok;
    Pre p;
    p.P = a.B == 1 ? 0 : a.prefix / unit * unit;
    p.wide = wide_prefix(a.B, G);
    p.rows = prefix_rows(a.B, G);
    p.rtp = ceil_div(a.B * G, p.rows);
    p.tiles = p.P / (p.wide ? kStageTok : kTok);
    const int64_t work = (int64_t)p.tiles * p.rtp * a.c.Hkv;
    const int least = p.wide ? 4 : kWaves, even = (int)((work + kPreTarget - 1) / kPreTarget);
    p.chunk = even > least ? even : least;
    p.nc = ceil_div(p.tiles, p.chunk);
    // chunks are dealt in eights, so that a chunk's row tiles meet on one XCD and its L2
    p.items = ceil_div(p.nc * a.c.Hkv, 8) * 8 * p.rtp;
    return p;
}

// The own items: 16-row tiles of a sequence, register tiles per item, items per key/value head.
struct Own {
    int G, rts, chunk, items;
};

struct Seq {
    int n, lo, start, part;  // length, first visible token, first own token, takes part in the prefix
};

__device__ __forceinline__ Seq seq_of(const AttnArgs &a, int b, int P)
{
    Seq s;
    const int64_t most = a.ldt * a.c.page;
    s.n = max(a.kv_len[b], 0);
    if (s.n > most) s.n = (int)most;
    s.lo = a.window ? max(0, s.n - a.window) : 0;
    s.part = P > 0 && s.lo == 0 && s.n >= P;
    s.start = s.part ? P : s.lo / kTok * kTok;
    return s;
}

// Integer sum and inclusive scan over a wave.
__device__ __forceinline__ int wave_sum_i(int v)
{
    v += FLINT_DPP(v, 0xB1);
    v += FLINT_DPP(v, 0x4E);
    v += FLINT_DPP(v, 0x141);
    v += FLINT_DPP(v, 0x140);
    return __builtin_amdgcn_readlane(v, 0) + __builtin_amdgcn_readlane(v, 16) + __builtin_amdgcn_readlane(v, 32) +
           __builtin_amdgcn_readlane(v, 48);
}
__device__ __forceinline__ int wave_scan_i(int v)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
        const int u = __shfl_up(v, m);
        if (lane >= m) v += u;
    }
    return v;
}

// First own item (per key/value head) of each sequence: cum[0 .. B].
struct PlanShared {
    int cum[kAttnMaxB + 1];
    int tot[kWaves], inc[kWaves];
};

__device__ __forceinline__ Own make_plan(const AttnArgs &a, int P, PlanShared &sh)
{
    constexpr int PER = kAttnMaxB / (64 * kWaves);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    Own p;
    p.G = a.c.Hq / a.c.Hkv;
    p.rts = ceil_div(p.G, kRows);
    int tiles[PER], sum = 0;  // at most 2^20 tiles a sequence
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const int b = PER * tid + i;
        tiles[i] = 0;
        if (b < a.B) {
            const Seq s = seq_of(a, b, P);
            tiles[i] = ceil_div(s.n - s.start, kTok);
        }
        sum += tiles[i];
    }
    sum = wave_sum_i(sum);
    if (lane == 0) sh.tot[wave] = sum;
    __syncthreads();
    sum = 0;
#pragma unroll
    for (int w = 0; w < kWaves; w++) sum += sh.tot[w];
    p.chunk = (int)max((int64_t)kWaves, ((int64_t)sum * p.rts * a.c.Hkv + kOwnTarget - 1) / kOwnTarget);
    int items = 0;
#pragma unroll
    for (int i = 0; i < PER; i++) items += ceil_div(tiles[i], p.chunk) * p.rts;
    const int inc = wave_scan_i(items);
    if (lane == 63) sh.inc[wave] = inc;
    __syncthreads();
    int at = inc - items;
    for (int w = 0; w < wave; w++) at += sh.inc[w];
#pragma unroll
    for (int i = 0; i < PER; i++) {
        if (PER * tid + i < a.B) sh.cum[PER * tid + i] = at;
        at += ceil_div(tiles[i], p.chunk) * p.rts;
        if (PER * tid + i == a.B - 1) sh.cum[a.B] = at;
    }
    __syncthreads();
    p.items = sh.cum[a.B];
    return p;
}

// Bounds of the items of any call with B sequences, and the workspace: the own items' plan
// (cum[0 .. B]), then {m, l} per row, then D weighted sums per row; prefix rows first.
__host__ __device__ inline int64_t plan_words(int64_t B) { return (B + 1 + 3) / 4 * 4; }
__host__ __device__ inline int64_t max_pre_items(int Hq, int Hkv, int64_t B)
{
    const int G = Hq / Hkv, rows = prefix_rows((int)B, G);
    const int64_t rtp = ceil_div((int)B * G, rows);
    return B < 2 ? 0 : (ceil_div(kPreTarget, (int)rtp) + Hkv + 8) * rtp;
}
__host__ __device__ inline int64_t max_own_items(int Hq, int Hkv, int64_t B)
{
    return kOwnTarget + (int64_t)Hkv * B * ceil_div(Hq / Hkv, kRows);
}
__host__ __device__ inline int64_t max_rows(int Hq, int Hkv, int64_t B)
{
    return max_pre_items(Hq, Hkv, B) * prefix_rows((int)B, Hq / Hkv) + max_own_items(Hq, Hkv, B) * kRows;
}
// A call's workspace pointers.
struct Work {
    int *cum;
    float *ml, *o;
};

// Probabilities as two bf16 parts, each the upper half of an fp32 (truncated): together they
// hold 16 bits.  A single bf16 would leave up to 2^-8 of sum p |v|, which a row of few tokens
// does not average away; the second product is free beside the cache's bytes.
__device__ __forceinline__ void split8(const float *p, u32x4 &hi, u32x4 &lo)
{
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t a = __float_as_uint(p[2 * i]), b = __float_as_uint(p[2 * i + 1]);
        const float ra = p[2 * i] - __uint_as_float(a & 0xffff0000u);
        const float rb = p[2 * i + 1] - __uint_as_float(b & 0xffff0000u);
        hi[i] = __builtin_amdgcn_perm(b, a, 0x07060302u);
        lo[i] = __builtin_amdgcn_perm(__float_as_uint(rb), __float_as_uint(ra), 0x07060302u);
    }
}

// A query fragment; a negative scale is taken into the (exact) sign of the query, so that
// maxima of products are maxima of scores.
__device__ __forceinline__ bf16x8 query_frag(const uint16_t *q, bool negate)
{
    u32x4 v = *reinterpret_cast<const u32x4 *>(q);
    if (negate)
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] ^= 0x80008000u;
    return as_bf16x8(v);
}

__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float finite_max(float m) { return m == -__builtin_inff() ? 0.f : m; }

// ---- own items -------------------------------------------------------------------------
// One wave: register tiles first, first + step, ... < end for 16 query rows, K and V straight
// from the cache into the A operands of the 16x16x32 MFMA.
// lane: row l % 16, lane group g = l / 16.  The two 16-token score products of a tile take the
// tokens 8 (r / 4) + r % 4 (+ 4) as their row r, so lane group g holds tokens 8 g .. 8 g + 7.
// m in the exponent's base-2 domain, l this lane's part of the sum (its 8 tokens of each
// tile), o[d / 16]: O^T, channel 16 dt + 4 g + i.
template <int D>
struct Acc {
    float m, l;
    f32x4 o[D / 16];
};

template <int D>
__device__ __forceinline__ void attend(const AttnArgs &a, int h, const int32_t *table, int lo, int hi, int first,
                                       int step, int end, const bf16x8 *qf, Acc<D> &acc)
{
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int sh = a.c.page_shift, page = a.c.page;
    const float scale = fabsf(a.scale) * kLog2e;
    for (int tile = first; tile < end; tile += step) {
        const int tb = tile * kTok;
        const int kt = tb + 8 * (r >> 2) + (r & 3), vt = tb + 8 * g;  // this lane's K rows kt, kt + 4; V tokens vt ..
        const int last = (hi - 1) >> sh;                              // the range's last table entry
        const int kp0 = table[min(kt >> sh, last)], vp0 = table[min(vt >> sh, last)];
        const bool vok = (uint32_t)vp0 < (uint64_t)a.c.n_pages;
        const int64_t kp = (uint32_t)kp0 < (uint64_t)a.c.n_pages ? kp0 : 0, vp = vok ? vp0 : 0;
        const uint16_t *kr = a.c.k + kp * a.c.page_stride + (int64_t)(h * page + (kt & (page - 1))) * D + 8 * g;
        const uint16_t *vr = a.c.v + vp * a.c.page_stride + (int64_t)(h * D + r) * page + (vt & (page - 1));
        u32x4 kf[2][D / 32], vf[D / 16];
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
            for (int kk = 0; kk < D / 32; kk++) kf[j][kk] = *reinterpret_cast<const u32x4 *>(kr + 4 * j * D + 32 * kk);
#pragma unroll
        for (int dt = 0; dt < D / 16; dt++) vf[dt] = *reinterpret_cast<const u32x4 *>(vr + 16 * dt * page);
        f32x4 s[2];
#pragma unroll
        for (int j = 0; j < 2; j++) {
            s[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kk = 0; kk < D / 32; kk++) s[j] = mfma16x16x32(as_bf16x8(kf[j][kk]), qf[kk], s[j]);
        }
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; i++) x[i] = s[i >> 2][i & 3] * scale;
        if (tb < lo || tb + kTok > hi || __any(!vok)) {
            // a tile with masked tokens: no score, and values that must not meet a zero
            // probability as an infinity or a NaN
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const bool see = vok && vt + i >= lo && vt + i < hi;
                x[i] = see ? x[i] : -__builtin_inff();
#pragma unroll
                for (int dt = 0; dt < D / 16; dt++)
                    if (!see) vf[dt][i >> 1] &= (i & 1) ? 0x0000ffffu : 0xffff0000u;
            }
        }
        float mx = x[0];
#pragma unroll
        for (int i = 1; i < 8; i++) mx = fmaxf(mx, x[i]);
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        mx = fmaxf(mx, acc.m);
        const float base = finite_max(mx);  // nothing visible so far
        const float al = ex2(acc.m - base);
        acc.m = mx;
        float p[8], ps = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            p[i] = ex2(x[i] - base);
            ps += p[i];
        }
        u32x4 ph, pl;
        split8(p, ph, pl);
        acc.l = acc.l * al + ps;
#pragma unroll
        for (int dt = 0; dt < D / 16; dt++) {
#pragma unroll
            for (int e = 0; e < 4; e++) acc.o[dt][e] *= al;
            acc.o[dt] = mfma16x16x32(as_bf16x8(vf[dt]), as_bf16x8(ph), acc.o[dt]);
            acc.o[dt] = mfma16x16x32(as_bf16x8(vf[dt]), as_bf16x8(pl), acc.o[dt]);
        }
    }
}

template <int D>
struct OwnShared {
    float m[kWaves][kRows], l[kWaves][kRows];
    f32x4 o[kWaves][D / 4][kRows];  // [wave][channel / 4][row]
};

// 16 rows over register tiles t0 .. t1 of a token range [lo, hi): the waves take tiles in turn
// and meet in LDS; done(row, c4, m, l, o) gets the sums of channels 4 c4 .. 4 c4 + 3.
template <int D, typename F>
__device__ __forceinline__ void own_item(const AttnArgs &a, int h, const int32_t *table, int lo, int hi, int t0, int t1,
                                         const uint16_t *q, OwnShared<D> &sh, F done)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15,
              g = lane >> 4;
    bf16x8 qf[D / 32];
#pragma unroll
    for (int kk = 0; kk < D / 32; kk++) qf[kk] = query_frag(q + 32 * kk + 8 * g, a.scale < 0.f);
    Acc<D> acc;
    acc.m = -__builtin_inff();
    acc.l = 0.f;
#pragma unroll
    for (int dt = 0; dt < D / 16; dt++) acc.o[dt] = f32x4{0.f, 0.f, 0.f, 0.f};
    attend<D>(a, h, table, lo, hi, t0 + wave, kWaves, t1, qf, acc);
    acc.l += __shfl_xor(acc.l, 16);
    acc.l += __shfl_xor(acc.l, 32);
    if (g == 0) {
        sh.m[wave][r] = acc.m;
        sh.l[wave][r] = acc.l;
    }
#pragma unroll
    for (int dt = 0; dt < D / 16; dt++) sh.o[wave][4 * dt + g][r] = acc.o[dt];
    __syncthreads();
    if (tid < kRows * (D / 4)) {
        const int rr = tid / (D / 4), c4 = tid % (D / 4);
        float m = sh.m[0][rr];
#pragma unroll
        for (int w = 1; w < kWaves; w++) m = fmaxf(m, sh.m[w][rr]);
        const float base = finite_max(m);
        float l = 0.f;
        f32x4 o{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWaves; w++) {
            const float f = ex2(sh.m[w][rr] - base);
            l = fmaf(f, sh.l[w][rr], l);
            const f32x4 v = sh.o[w][c4][rr];
#pragma unroll
            for (int e = 0; e < 4; e++) o[e] = fmaf(f, v[e], o[e]);
        }
        done(rr, c4, m, l, o);
    }
}

// ---- prefix items ------------------------------------------------------------------------
// Stages of 64 tokens are copied HBM -> LDS (no registers), three ahead of the one in use, and
// every wave multiplies its own 32 rows with all of them on the 32x32x16 MFMA.
//
// LDS stage: K rows in the order the score product wants (row 8 q + 4 h + i of a 32-token tile
// is token 16 (q / 2) + 8 h + 4 (q % 2) + i, so lane half h gets tokens 8 h .. 8 h + 7 of each
// 16), then V rows (one per channel, 64 tokens).  Row R keeps its 16-byte chunk c at
// c ^ swz(R): the 32 rows that a fragment read touches fall on distinct banks.
constexpr int kStages = 4;
constexpr int kCutPages = kCut * kStageTok / 16;
constexpr int stage_bytes(int D) { return 2 * kStageTok * D * 2; }

template <int CH>  // 16-byte chunks of a row
__device__ __forceinline__ int swz(int row) { return CH == 16 ? (row & 15) : ((row ^ (row >> 3)) & 7); }

__device__ __forceinline__ void copy16(const void *g, uint8_t *lds)
{
    __builtin_amdgcn_global_load_lds(g, (__attribute__((address_space(3))) void *)lds, 16, 0, 0);
}

// Waits until at most N of the wave's copies are in flight.
template <int N>
__device__ __forceinline__ void wait_copies()
{
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}
__device__ __forceinline__ void stage_barrier()
{
    // the barrier orders LDS accesses for the hardware; the signal fences keep the compiler
    // from moving fragment reads or copies across it
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// One wave's 32 rows: m (base 2, shared by the lanes l and l + 32 of a row), this lane's part
// of the sum, O^T: channel 32 dt + 8 (i / 4) + 4 (l / 32) + i % 4.
template <int D>
struct Acc32 {
    float m, l;
    f32x16 o[D / 32];
};

// One 64-token stage in LDS.  MASK: tokens whose page is not valid (ok, per 8 tokens).
template <int D, bool MASK>
__device__ __forceinline__ void pre_stage(const uint8_t *st, const bf16x8 *qf, float scale, uint32_t ok, Acc32<D> &acc)
{
    constexpr int KCH = D / 8, VCH = kStageTok / 8;
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const uint8_t *vs = st + kStageTok * D * 2;
#pragma unroll 1
    for (int t = 0; t < kStageTok / 32; t++) {
        f32x16 s;
#pragma unroll
        for (int i = 0; i < 16; i++) s[i] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; kk++) {
            const int c = 2 * kk + h;
            const u32x4 kf = *reinterpret_cast<const u32x4 *>(st + (32 * t + r) * (2 * D) + 16 * (c ^ swz<KCH>(r)));
            s = mfma32(as_bf16x8(kf), qf[kk], s);
        }
        bool see[2] = {true, true};  // registers 0 .. 7, 8 .. 15: eight tokens of one page each
        if (MASK)
#pragma unroll
            for (int k = 0; k < 2; k++) see[k] = (ok >> (4 * t + 2 * k + h)) & 1;
        float mx = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < 16; i++)
            if (!MASK || see[i >> 3]) mx = fmaxf(mx, s[i]);
        mx *= scale;
        // The reference maximum moves only when a score has left it 8 behind (a factor of 256,
        // harmless in fp32), so most tiles neither exchange maxima nor rescale.
        if (__any(!(mx <= acc.m + 8.f) && mx != -__builtin_inff())) {
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            mx = fmaxf(mx, acc.m);
            const float al = ex2(acc.m - finite_max(mx));
            acc.m = mx;
            acc.l *= al;
#pragma unroll
            for (int dt = 0; dt < D / 32; dt++)
#pragma unroll
                for (int i = 0; i < 16; i++) acc.o[dt][i] *= al;
        }
        const float base = finite_max(acc.m);
        float p[16];
#pragma unroll
        for (int i = 0; i < 16; i++) {
            p[i] = ex2(fmaf(s[i], scale, -base));
            if (MASK && !see[i >> 3]) p[i] = 0.f;
        }
        float ps = 0.f;
#pragma unroll
        for (int i = 0; i < 16; i++) ps += p[i];
        acc.l += ps;
#pragma unroll
        for (int k = 0; k < 2; k++) {
            u32x4 ph, pl;
            split8(p + 8 * k, ph, pl);
            const int c = 4 * t + 2 * k + h;
#pragma unroll
            for (int dt = 0; dt < D / 32; dt++) {
                const int d = 32 * dt + r;
                u32x4 vf = *reinterpret_cast<const u32x4 *>(vs + d * (2 * kStageTok) + 16 * (c ^ swz<VCH>(d)));
                if (MASK && !see[k]) vf = u32x4{0u, 0u, 0u, 0u};
                acc.o[dt] = mfma32(as_bf16x8(vf), as_bf16x8(ph), acc.o[dt]);
                acc.o[dt] = mfma32(as_bf16x8(vf), as_bf16x8(pl), acc.o[dt]);
            }
        }
    }
}

// Stages t0 .. t1 of the prefix for row tile rt of key/value head h; rows to workspace row out + r.
template <int D>
__device__ __forceinline__ void prefix_item(const AttnArgs &a, const Pre &p, int h, int rt, int t0, int t1, int64_t out,
                                            const Work &w, uint8_t *stages, int *pages)
{
    constexpr int KPC = 1024 / (2 * D);   // K rows of one copy instruction (1 KB)
    constexpr int NK = kStageTok / KPC / kWaves, NV = D / 8 / kWaves;  // a wave's copies per stage: K, V
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 31, hh = lane >> 5, G = a.c.Hq / a.c.Hkv, rows = a.B * G;
    const int row = rt * kPreRows + wave * 32 + r;
    const bool live = rt * kPreRows + wave * 32 < rows;  // this wave has rows
    const float scale = fabsf(a.scale) * kLog2e;
    const int page = a.c.page, sft = a.c.page_shift;
    bf16x8 qf[D / 16];
    {
        const int q = min(row, rows - 1);
        const uint16_t *qp = a.q + (q / G) * a.ldq + (h * G + q % G) * D;
#pragma unroll
        for (int kk = 0; kk < D / 16; kk++) qf[kk] = query_frag(qp + 16 * kk + 8 * hh, a.scale < 0.f);
    }
    Acc32<D> acc;
    acc.m = -__builtin_inff();
    acc.l = 0.f;
#pragma unroll
    for (int dt = 0; dt < D / 32; dt++)
#pragma unroll
        for (int i = 0; i < 16; i++) acc.o[dt][i] = 0.f;

    for (int c0 = t0; c0 < t1; c0 += kCut) {
        const int c1 = min(c0 + kCut, t1);
        // the cut's pages; entries outside the cache read page 0 and mask their tokens
        const int e0 = (c0 * kStageTok) >> sft, ne = ((c1 * kStageTok - 1) >> sft) - e0 + 1;
        if (c0 != t0) __syncthreads();
        bool bad = false;
        for (int i = tid; i < ne; i += 64 * kWaves) {
            const int pg = a.table[e0 + i];
            const bool good = (uint32_t)pg < (uint64_t)a.c.n_pages;
            pages[i] = good ? pg : -1;
            bad |= !good;
        }
        bad = __syncthreads_or(bad);
        // Copies of stage s into its slot: lane l of K copy i fills row KPC (NK wave + i) + l /
        // (D / 8), chunk l % (D / 8); of V copy i, channel 8 (NV wave + i) + l / 8, chunk l % 8.
        auto issue = [&](int s) {
            uint8_t *st = stages + s % kStages * stage_bytes(D);
            const int tb = s * kStageTok;
#pragma unroll
            for (int i = 0; i < NK; i++) {
                const int rr = KPC * (NK * wave + i) + lane / (D / 8);
                const int r32 = rr & 31, tok = tb + (rr & 32) + (r32 & 0x13) + ((r32 & 8) >> 1) + ((r32 & 4) << 1);
                const int64_t pg = max(pages[(tok >> sft) - e0], 0);
                const int c = (lane % (D / 8)) ^ swz<D / 8>(r32);
                copy16(a.c.k + pg * a.c.page_stride + (int64_t)(h * page + (tok & (page - 1))) * D + 8 * c,
                       st + 1024 * (NK * wave + i));
            }
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int d = 8 * (NV * wave + i) + lane / 8, c = (lane % 8) ^ swz<8>(d), tok = tb + 8 * c;
                const int64_t pg = max(pages[(tok >> sft) - e0], 0);
                copy16(a.c.v + pg * a.c.page_stride + (int64_t)(h * D + d) * page + (tok & (page - 1)),
                       st + kStageTok * D * 2 + 1024 * (NV * wave + i));
            }
        };
        for (int s = c0; s < min(c0 + kStages - 1, c1); s++) issue(s);
        for (int s = c0; s < c1; s++) {
            // Stage s has landed for this wave once only the later stages' copies are in flight;
            // the barrier makes it true for every wave and frees the slot read in the previous
            // iteration, which stage s + kStages - 1 refills.
            const int later = min(kStages - 2, c1 - 1 - s);
            if (later == 2)
                wait_copies<2 * (NK + NV)>();
            else if (later == 1)
                wait_copies<NK + NV>();
            else
                wait_copies<0>();
            stage_barrier();
            if (s + kStages - 1 < c1) issue(s + kStages - 1);
            if (!live) continue;
            const uint8_t *st = stages + s % kStages * stage_bytes(D);
            if (!bad) {
                pre_stage<D, false>(st, qf, scale, 0, acc);
            } else {
                uint32_t ok = 0;
                for (int c = 0; c < 8; c++) ok |= (uint32_t)(pages[((s * kStageTok + 8 * c) >> sft) - e0] >= 0) << c;
                pre_stage<D, true>(st, qf, scale, ok, acc);
            }
        }
    }
    if (!live) return;
    acc.l += __shfl_xor(acc.l, 32);
    const int64_t dst = out + wave * 32 + r;
    if (hh == 0) {
        w.ml[2 * dst] = acc.m;
        w.ml[2 * dst + 1] = acc.l;
    }
    float *o = w.o + dst * D;
#pragma unroll
    for (int dt = 0; dt < D / 32; dt++)
#pragma unroll
        for (int q = 0; q < 4; q++)
            *reinterpret_cast<f32x4 *>(o + 32 * dt + 8 * q + 4 * hh) =
                f32x4{acc.o[dt][4 * q], acc.o[dt][4 * q + 1], acc.o[dt][4 * q + 2], acc.o[dt][4 * q + 3]};
}

// The head, row tile and chunk of prefix workgroup `it`; false for a padding one.
__device__ __forceinline__ bool pre_item_of(const Pre &p, int Hkv, int it, int &h, int &rt, int &c)
{
    const int cc = it / (8 * p.rtp) * 8 + it % 8;
    rt = it / 8 % p.rtp;
    h = cc / p.nc;
    c = cc % p.nc;
    return h < Hkv;
}
__device__ __forceinline__ int pre_item_at(const Pre &p, int h, int rt, int c)
{
    const int cc = h * p.nc + c;
    return (cc / 8 * p.rtp + rt) * 8 + cc % 8;
}

// ---- launches ------------------------------------------------------------------------------
// The result of 4 channels of a query from its joined sums; a row that saw nothing is zero.
__device__ __forceinline__ void sink_in(const AttnArgs &a, int hq, float &m, float &l, float &f)
{
    f = 1.f;
    if (!a.sinks || l == 0.f) return;
    const float sk = a.sinks[hq] * kLog2e, mn = fmaxf(m, sk), base = finite_max(mn);
    f = ex2(m - base);
    l = l * f + ex2(sk - base);
    m = mn;
}
__device__ __forceinline__ void store4(uint16_t *dst, f32x4 o, float f, float l)
{
    const float r = l == 0.f ? 0.f : f / l;
    u32x2 v;
#pragma unroll
    for (int i = 0; i < 2; i++)
        v[i] = l == 0.f ? 0u : f2bf(o[2 * i] * r) | (f2bf(o[2 * i + 1] * r) << 16);
    *reinterpret_cast<u32x2 *>(dst) = v;
}

// One workgroup per sequence, key/value head and 16 rows: the whole sequence.
template <int D>
__global__ __launch_bounds__(64 * kWaves) void attn_whole_kernel(AttnArgs a)
{
    __shared__ __attribute__((aligned(16))) OwnShared<D> sh;
    const int G = a.c.Hq / a.c.Hkv, rts = ceil_div(G, kRows), r = threadIdx.x & 15;
    const int rt = blockIdx.x % rts, h = blockIdx.x / rts % a.c.Hkv, b = blockIdx.x / (rts * a.c.Hkv);
    const Seq s = seq_of(a, b, 0);
    const int qh = h * G + min(rt * kRows + r, G - 1);
    own_item<D>(a, h, a.table + b * a.ldt, s.lo, s.n, s.start / kTok, ceil_div(s.n, kTok), a.q + b * a.ldq + qh * D, sh,
                [&](int rr, int c4, float m, float l, f32x4 o) {
                    if (rt * kRows + rr >= G) return;
                    const int hq = h * G + rt * kRows + rr;
                    float f;
                    sink_in(a, hq, m, l, f);
                    store4(a.out + b * a.ldo + hq * D + 4 * c4, o, f, l);
                });
}

template <int D>
__global__ __launch_bounds__(64 * kWaves) void attn_items_kernel(AttnArgs a, Pre p, Work w)
{
    // the stages of a prefix item or an own item's exchange; the rest apart from them, so that
    // reading it does not wait for copies in flight
    extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
    __shared__ PlanShared plan;
    __shared__ int pages[kCutPages];
    OwnShared<D> &own_sh = *reinterpret_cast<OwnShared<D> *>(dyn);
    const int it = blockIdx.x, r = threadIdx.x & 15, G = a.c.Hq / a.c.Hkv;
    int64_t out;
    auto done = [&](int rr, int c4, float m, float l, f32x4 o) {
        if (c4 == 0) {
            w.ml[2 * (out + rr)] = m;
            w.ml[2 * (out + rr) + 1] = l;
        }
        *reinterpret_cast<f32x4 *>(w.o + (out + rr) * D + 4 * c4) = o;
    };
    if (it < p.items) {
        int h, rt, c;
        if (!pre_item_of(p, a.c.Hkv, it, h, rt, c)) return;
        const int t0 = c * p.chunk, t1 = min(t0 + p.chunk, p.tiles);
        out = (int64_t)it * p.rows;
        if (p.wide) {
            prefix_item<D>(a, p, h, rt, t0, t1, out, w, dyn, pages);
        } else {
            const int q = min(r, a.B * G - 1);
            own_item<D>(a, h, a.table, 0, p.P, t0, t1, a.q + (q / G) * a.ldq + (h * G + q % G) * D, own_sh, done);
        }
        return;
    }
    const int item = it - p.items;
    const Own n = make_plan(a, p.P, plan);
    if (item == 0)  // for the join
        for (int b = threadIdx.x; b <= a.B; b += 64 * kWaves) w.cum[b] = plan.cum[b];
    if (item >= n.items * a.c.Hkv) return;
    const int h = item / n.items, own = item % n.items;
    int b = 0, y = a.B - 1;  // the last sequence that starts at or before this item: it has items
    while (b < y) {
        const int mid = (b + y + 1) >> 1;
        if (plan.cum[mid] <= own)
            b = mid;
        else
            y = mid - 1;
    }
    const Seq s = seq_of(a, b, p.P);
    const int at = own - plan.cum[b], rt = at % n.rts, c = at / n.rts;
    const int t0 = s.start / kTok + c * n.chunk, t1 = min(t0 + n.chunk, ceil_div(s.n, kTok));
    const int qh = h * G + min(rt * kRows + r, G - 1);
    out = (int64_t)p.items * p.rows + (int64_t)item * kRows;
    own_item<D>(a, h, a.table + b * a.ldt, max(s.lo, s.start), s.n, t0, t1, a.q + b * a.ldq + qh * D, own_sh, done);
}

// One workgroup per query row: joins the row's items and the sink.  Eight items at a time per
// wave, then the waves.
template <int D>
__global__ __launch_bounds__(64 * kWaves) void attn_join_kernel(AttnArgs a, Pre p, Work w)
{
    __shared__ float sm[kWaves], sl[kWaves];
    __shared__ float so[kWaves][D];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int G = a.c.Hq / a.c.Hkv, rts = ceil_div(G, kRows);
    const int b = blockIdx.x / a.c.Hq, hq = blockIdx.x % a.c.Hq, h = hq / G, gi = hq % G;
    const int c0 = w.cum[b], c1 = w.cum[b + 1], per_head = w.cum[a.B];
    const Seq s = seq_of(a, b, p.P);
    const int prow = b * G + gi, np = s.part ? p.nc : 0, total = np + (c1 - c0) / rts;
    auto row_of = [&](int i) {
        return i < np ? (int64_t)pre_item_at(p, h, prow / p.rows, i) * p.rows + prow % p.rows
                      : (int64_t)p.items * p.rows + ((int64_t)h * per_head + c0 + gi / kRows + (i - np) * rts) * kRows + gi % kRows;
    };
    float m = -__builtin_inff(), l = 0.f, o[D / 64] = {};
    for (int i0 = 8 * wave; i0 < total; i0 += 8 * kWaves) {
        float mi[8], li[8], v[8][D / 64], mx = m;
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const bool have = i0 + k < total;
            const int64_t row = row_of(min(i0 + k, total - 1));
            mi[k] = have ? w.ml[2 * row] : -__builtin_inff();
            li[k] = have ? w.ml[2 * row + 1] : 0.f;
#pragma unroll
            for (int e = 0; e < D / 64; e++) v[k][e] = have ? w.o[row * D + lane * (D / 64) + e] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < 8; k++) mx = fmaxf(mx, mi[k]);
        const float base = finite_max(mx), al = ex2(m - base);
        m = mx;
        l *= al;
#pragma unroll
        for (int e = 0; e < D / 64; e++) o[e] *= al;
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const float f = ex2(mi[k] - base);
            l = fmaf(f, li[k], l);
#pragma unroll
            for (int e = 0; e < D / 64; e++) o[e] = fmaf(f, v[k][e], o[e]);
        }
    }
    if (lane == 0) {
        sm[wave] = m;
        sl[wave] = l;
    }
#pragma unroll
    for (int e = 0; e < D / 64; e++) so[wave][lane * (D / 64) + e] = o[e];
    __syncthreads();
    if (threadIdx.x >= D / 4) return;
    m = sm[0];
#pragma unroll
    for (int i = 1; i < kWaves; i++) m = fmaxf(m, sm[i]);
    const float base = finite_max(m);
    f32x4 r{0.f, 0.f, 0.f, 0.f};
    l = 0.f;
#pragma unroll
    for (int i = 0; i < kWaves; i++) {
        const float f = ex2(sm[i] - base);
        l = fmaf(f, sl[i], l);
#pragma unroll
        for (int e = 0; e < 4; e++) r[e] = fmaf(f, so[i][4 * threadIdx.x + e], r[e]);
    }
    float f;
    sink_in(a, hq, m, l, f);
    store4(a.out + b * a.ldo + hq * D + 4 * threadIdx.x, r, f, l);
}

}  // namespace

static int64_t call_rows(const Cache &c, int64_t B) { return (max_rows(c.Hq, c.Hkv, B) + 1) / 2 * 2; }

size_t attn_decode_call_bytes(const Cache &c, int64_t B)
{
    return ((size_t)plan_words(B) + (size_t)call_rows(c, B) * (c.D + 2)) * 4;
}

size_t attn_decode_ws_bytes(const Cache &c, int64_t B)
{
    // fewer sequences may fill more rows of a prefix item: the largest over all batches up to B
    size_t most = 16;
    for (int64_t b = 1; b <= B; b++) most = std::max(most, attn_decode_call_bytes(c, b));
    return most;
}

template <int D>
static hipError_t launch_d(const AttnArgs &a, hipStream_t st)
{
    const int64_t G = a.c.Hq / a.c.Hkv, rts = (G + kRows - 1) / kRows, most = a.ldt * a.c.page;
    // the tokens of a sequence that its own items can span, from lengths the host knows
    const int64_t seen = a.window ? std::min<int64_t>(most, a.window + kTok) : most;
    const Pre p = pre_of(a);
    if (seen <= kWhole || (a.window && a.window <= kWhole)) {
        attn_whole_kernel<D><<<(unsigned)(a.B * a.c.Hkv * rts), 64 * kWaves, 0, st>>>(a);
        return hipGetLastError();
    }
    Work w;
    w.cum = (int *)a.ws;
    w.ml = a.ws + plan_words(a.B);
    w.o = w.ml + 2 * call_rows(a.c, a.B);
    // no more items than the longest possible lengths give
    const int64_t own = std::min<int64_t>(max_own_items(a.c.Hq, a.c.Hkv, a.B),
                                          a.c.Hkv * a.B * rts * (seen / (kTok * kWaves) + 1));
    const size_t lds = p.items && p.wide ? (size_t)kStages * stage_bytes(D) : sizeof(OwnShared<D>);
    static_assert(kStages * stage_bytes(D) >= (int)sizeof(OwnShared<D>), "own items share the stages' LDS");
    attn_items_kernel<D><<<(unsigned)(p.items + own), 64 * kWaves, lds, st>>>(a, p, w);
    attn_join_kernel<D><<<(unsigned)(a.B * a.c.Hq), 64 * kWaves, 0, st>>>(a, p, w);
    return hipGetLastError();
}

hipError_t launch_attn_decode(const AttnArgs &a, hipStream_t st)
{
    return a.c.D == 128 ? launch_d<128>(a, st) : launch_d<64>(a, st);
}

}  // namespace flint
