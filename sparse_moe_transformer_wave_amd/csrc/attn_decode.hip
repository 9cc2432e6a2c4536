// attn_decode.hip -- decode attention over the paged cache, a prefix shared by the batch read
// once: out[b][h] = sum_j p_j v_j, p = softmax_j(scale q . k_j) with an optional sink.
//
// The work of a call is a list of items, one workgroup each; every workgroup derives the same
// list from kv_len.  A prefix item takes a chunk of the shared prefix for up to 256 query
// rows of one key/value head (all the batch's queries of that head); an own item takes a
// chunk of one sequence's own tokens for 16 rows (its G = Hq / Hkv queries).  An item leaves
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

// The items of a call, the same in every workgroup of both launches.
struct Plan {
    int G, rts;              // query heads per key/value head; 16-row tiles of a sequence
    int rows, rtp;           // rows and row tiles of the prefix
    int pre_tiles;           // stages (wide) or register tiles of the shared prefix; 0: none
    int pre_chunk, pre_nc;   // tiles per prefix item, chunks
    int pre_items;           // workgroups of the prefix, all heads (some empty)
    int chunk;               // register tiles per own item
    int own_items;           // per key/value head
};

struct Seq {
    int n, lo, start, part;  // length, first visible token, first own token, takes part in the prefix
};

__device__ __forceinline__ int prefix_tokens(const AttnArgs &a)
{
    const int unit = a.c.page > kStageTok ? a.c.page : kStageTok;
    return a.B == 1 ? 0 : a.prefix / unit * unit;
}

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

// Workspace of the plan's own: the first own item (per key/value head) of each sequence.
struct PlanShared {
    int cum[kAttnMaxB + 1];
    int64_t tot[kWaves];
    int parts[kWaves], inc[kWaves];
};

__device__ __forceinline__ Plan make_plan(const AttnArgs &a, PlanShared &sh)
{
    constexpr int PER = kAttnMaxB / (64 * kWaves);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    Plan p;
    p.G = a.c.Hq / a.c.Hkv;
    p.rts = ceil_div(p.G, kRows);
    const int P = prefix_tokens(a);
    int tiles[PER], parts = 0;
    int64_t sum = 0;
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const int b = PER * tid + i;
        tiles[i] = 0;
        if (b < a.B) {
            const Seq s = seq_of(a, b, P);
            tiles[i] = ceil_div(s.n - s.start, kTok);
            parts += s.part;
        }
        sum += tiles[i];
    }
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
        sum += __shfl_xor(sum, m);
        parts += __shfl_xor(parts, m);
    }
    if (lane == 0) {
        sh.tot[wave] = sum;
        sh.parts[wave] = parts;
    }
    __syncthreads();
    sum = parts = 0;
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
        sum += sh.tot[w];
        parts += sh.parts[w];
    }
    const bool wide = wide_prefix(a.B, p.G);
    p.rows = prefix_rows(a.B, p.G);
    p.rtp = ceil_div(a.B * p.G, p.rows);
    p.pre_tiles = parts ? P / (wide ? kStageTok : kTok) : 0;
    p.pre_chunk = max(wide ? 4 : kWaves, ceil_div(p.pre_tiles * p.rtp * a.c.Hkv, kPreTarget));
    p.pre_nc = ceil_div(p.pre_tiles, p.pre_chunk);
    // chunks are dealt in eights, so that a chunk's row tiles meet on one XCD and its L2
    p.pre_items = ceil_div(p.pre_nc * a.c.Hkv, 8) * 8 * p.rtp;
    p.chunk = (int)max((int64_t)kWaves, (sum * p.rts * a.c.Hkv + kOwnTarget - 1) / kOwnTarget);
    // exclusive scan of the sequences' items
    int items = 0;
#pragma unroll
    for (int i = 0; i < PER; i++) items += ceil_div(tiles[i], p.chunk) * p.rts;
    int inc = items;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
        const int v = __shfl_up(inc, m);
        if (lane >= m) inc += v;
    }
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
    p.own_items = sh.cum[a.B];
    return p;
}

// Bounds of the items of any call with B sequences, and the workspace:
//   ml: {m, l} per row (fp32 pairs), o: D weighted sums per row; prefix rows first.
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
__device__ __forceinline__ int64_t pre_row(const Plan &p, int item, int r) { return (int64_t)item * p.rows + r; }
__device__ __forceinline__ int64_t own_row(const Plan &p, int item, int r)
{
    return (int64_t)p.pre_items * p.rows + (int64_t)item * kRows + r;
}

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
// and meet in LDS.  Results of row r go to workspace row out + r.
template <int D>
__device__ __forceinline__ void own_item(const AttnArgs &a, int h, const int32_t *table, int lo, int hi, int t0, int t1,
                                         const uint16_t *q, int64_t out, int64_t all_rows, OwnShared<D> &sh)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
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
        if (c4 == 0) {
            a.ws[2 * (out + rr)] = m;
            a.ws[2 * (out + rr) + 1] = l;
        }
        *reinterpret_cast<f32x4 *>(a.ws + 2 * all_rows + (out + rr) * D + 4 * c4) = o;
    }
}

// ---- prefix items ------------------------------------------------------------------------
// Stages of 64 tokens are copied HBM -> LDS (no registers), one ahead of the one in use, and
// every wave multiplies its own 32 rows with all of them on the 32x32x16 MFMA.
//
// LDS stage: K rows in the order the score product wants (row 8 q + 4 h + i of a 32-token tile
// is token 16 (q / 2) + 8 h + 4 (q % 2) + i, so lane half h gets tokens 8 h .. 8 h + 7 of each
// 16), then V rows (one per channel, 64 tokens).  Row R keeps its 16-byte chunk c at
// c ^ swz(R): the 32 rows that a fragment read touches fall on distinct banks.
template <int D>
struct PreShared {
    uint8_t stage[2][2 * kStageTok * D * 2];
    int page[kCut * kStageTok / 16];
    int bad;
};

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

// Stages t0 .. t1 of the prefix for row tile rt of key/value head h.
template <int D>
__device__ __forceinline__ void prefix_item(const AttnArgs &a, const Plan &p, int h, int rt, int t0, int t1, int64_t out,
                                            int64_t all_rows, PreShared<D> &sh)
{
    constexpr int KPC = 1024 / (2 * D);   // K rows of one copy instruction (1 KB)
    constexpr int NK = kStageTok / KPC / kWaves, NV = D / 8 / kWaves;  // a wave's copies per stage: K, V
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 31, hh = lane >> 5, rows = a.B * p.G;
    const int row = rt * kPreRows + wave * 32 + r;
    const bool live = rt * kPreRows + wave * 32 < rows;  // this wave has rows
    bf16x8 qf[D / 16];
    {
        const int q = min(row, rows - 1);
        const uint16_t *qp = a.q + (q / p.G) * a.ldq + (h * p.G + q % p.G) * D;
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
    const float scale = fabsf(a.scale) * kLog2e;
    const int page = a.c.page, sft = a.c.page_shift;

    for (int c0 = t0; c0 < t1; c0 += kCut) {
        const int c1 = min(c0 + kCut, t1);
        // the cut's pages; entries outside the cache read page 0 and mask their tokens
        const int e0 = (c0 * kStageTok) >> sft, ne = ((c1 * kStageTok - 1) >> sft) - e0 + 1;
        __syncthreads();
        if (tid == 0) sh.bad = 0;
        __syncthreads();
        for (int i = tid; i < ne; i += 64 * kWaves) {
            const int pg = a.table[e0 + i];
            const bool good = (uint32_t)pg < (uint64_t)a.c.n_pages;
            sh.page[i] = good ? pg : -1;
            if (!good) sh.bad = 1;
        }
        __syncthreads();
        const bool bad = sh.bad;
        // Copies of stage s into slot s % 2: lane l of K copy i fills row KPC (NK wave + i) + l /
        // (D / 8), chunk l % (D / 8); of V copy i, channel 8 (NV wave + i) + l / 8, chunk l % 8.
        auto issue = [&](int s) {
            uint8_t *st = sh.stage[s & 1];
            const int tb = s * kStageTok;
#pragma unroll
            for (int i = 0; i < NK; i++) {
                const int rr = KPC * (NK * wave + i) + lane / (D / 8);
                const int r32 = rr & 31, tok = tb + (rr & 32) + (r32 & 0x13) + ((r32 & 8) >> 1) + ((r32 & 4) << 1);
                const int64_t pg = max(sh.page[(tok >> sft) - e0], 0);
                const int c = (lane % (D / 8)) ^ swz<D / 8>(r32);
                copy16(a.c.k + pg * a.c.page_stride + (int64_t)(h * page + (tok & (page - 1))) * D + 8 * c,
                       st + 1024 * (NK * wave + i));
            }
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int d = 8 * (NV * wave + i) + lane / 8, c = (lane % 8) ^ swz<8>(d), tok = tb + 8 * c;
                const int64_t pg = max(sh.page[(tok >> sft) - e0], 0);
                copy16(a.c.v + pg * a.c.page_stride + (int64_t)(h * D + d) * page + (tok & (page - 1)),
                       st + kStageTok * D * 2 + 1024 * (NV * wave + i));
            }
        };
        issue(c0);
        for (int s = c0; s < c1; s++) {
            // slot (s + 1) % 2 was read in the previous iteration, which the barrier has ended
            if (s + 1 < c1) {
                issue(s + 1);
                wait_copies<NK + NV>();
            } else {
                wait_copies<0>();
            }
            stage_barrier();  // stage s is in LDS for every wave
            if (live) {
                if (!bad) {
                    pre_stage<D, false>(sh.stage[s & 1], qf, scale, 0, acc);
                } else {
                    uint32_t ok = 0;
                    for (int c = 0; c < 8; c++)
                        ok |= (uint32_t)(sh.page[((s * kStageTok + 8 * c) >> sft) - e0] >= 0) << c;
                    pre_stage<D, true>(sh.stage[s & 1], qf, scale, ok, acc);
                }
            }
            stage_barrier();  // stage s has been read by every wave
        }
    }
    if (!live) return;
    acc.l += __shfl_xor(acc.l, 32);
    const int64_t dst = out + wave * 32 + r;
    if (hh == 0) {
        a.ws[2 * dst] = acc.m;
        a.ws[2 * dst + 1] = acc.l;
    }
    float *o = a.ws + 2 * all_rows + dst * D;
#pragma unroll
    for (int dt = 0; dt < D / 32; dt++)
#pragma unroll
        for (int q = 0; q < 4; q++)
            *reinterpret_cast<f32x4 *>(o + 32 * dt + 8 * q + 4 * hh) =
                f32x4{acc.o[dt][4 * q], acc.o[dt][4 * q + 1], acc.o[dt][4 * q + 2], acc.o[dt][4 * q + 3]};
}

// The head, row tile and chunk of prefix workgroup `it`; false for a padding one.
__device__ __forceinline__ bool pre_item_of(const Plan &p, int Hkv, int it, int &h, int &rt, int &c)
{
    const int cc = it / (8 * p.rtp) * 8 + it % 8;
    rt = it / 8 % p.rtp;
    h = cc / p.pre_nc;
    c = cc % p.pre_nc;
    return h < Hkv;
}
__device__ __forceinline__ int pre_item_at(const Plan &p, int h, int rt, int c)
{
    const int cc = h * p.pre_nc + c;
    return (cc / 8 * p.rtp + rt) * 8 + cc % 8;
}

template <int D>
__global__ __launch_bounds__(64 * kWaves) void attn_items_kernel(AttnArgs a, int64_t all_rows)
{
    __shared__ PlanShared ps;
    __shared__ __attribute__((aligned(16))) union {
        OwnShared<D> own;
        PreShared<D> pre;
    } sh;
    const Plan p = make_plan(a, ps);
    const int it = blockIdx.x, r = threadIdx.x & 15;
    if (it < p.pre_items) {
        int h, rt, c;
        if (!pre_item_of(p, a.c.Hkv, it, h, rt, c)) return;
        const int t0 = c * p.pre_chunk, t1 = min(t0 + p.pre_chunk, p.pre_tiles);
        if (wide_prefix(a.B, p.G)) {
            prefix_item<D>(a, p, h, rt, t0, t1, pre_row(p, it, 0), all_rows, sh.pre);
        } else {
            const int q = min(r, a.B * p.G - 1);
            own_item<D>(a, h, a.table, 0, p.pre_tiles * kTok, t0, t1, a.q + (q / p.G) * a.ldq + (h * p.G + q % p.G) * D,
                        pre_row(p, it, 0), all_rows, sh.own);
        }
        return;
    }
    const int item = it - p.pre_items;
    if (item >= p.own_items * a.c.Hkv) return;
    const int h = item / p.own_items, own = item % p.own_items;
    int b = 0, y = a.B - 1;  // the last sequence that starts at or before this item: it has items
    while (b < y) {
        const int mid = (b + y + 1) >> 1;
        if (ps.cum[mid] <= own)
            b = mid;
        else
            y = mid - 1;
    }
    const Seq s = seq_of(a, b, prefix_tokens(a));
    const int rt = (own - ps.cum[b]) % p.rts, c = (own - ps.cum[b]) / p.rts;
    const int t0 = s.start / kTok + c * p.chunk, t1 = min(t0 + p.chunk, ceil_div(s.n, kTok));
    const int qh = h * p.G + min(rt * kRows + r, p.G - 1);
    own_item<D>(a, h, a.table + b * a.ldt, max(s.lo, s.start), s.n, t0, t1, a.q + b * a.ldq + qh * D, own_row(p, item, 0),
                all_rows, sh.own);
}

// One wave per query row: joins the row's items and the sink.
template <int D>
__global__ __launch_bounds__(64 * kWaves) void attn_join_kernel(AttnArgs a, int64_t all_rows)
{
    __shared__ PlanShared ps;
    const Plan p = make_plan(a, ps);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t q = (int64_t)blockIdx.x * kWaves + wave;
    if (q >= (int64_t)a.B * a.c.Hq) return;
    const int b = (int)(q / a.c.Hq), hq = (int)(q % a.c.Hq), h = hq / p.G, gi = hq % p.G;
    const Seq s = seq_of(a, b, prefix_tokens(a));
    const int prow = b * p.G + gi, prt = prow / p.rows;
    const int np = s.part ? p.pre_nc : 0, ns = (ps.cum[b + 1] - ps.cum[b]) / p.rts;
    const int own0 = h * p.own_items + ps.cum[b] + gi / kRows;
    auto row_of = [&](int i) {
        return i < np ? pre_row(p, pre_item_at(p, h, prt, i), prow % p.rows)
                      : own_row(p, own0 + (i - np) * p.rts, gi % kRows);
    };
    const float *ml = a.ws, *os = a.ws + 2 * all_rows;
    float m = -__builtin_inff(), l = 0.f, o[D / 64] = {};
    for (int i0 = 0; i0 < np + ns; i0 += 64) {
        // the lanes fetch 64 items' statistics at once; their rows follow with weights known
        const int n = min(64, np + ns - i0);
        const int64_t mine = row_of(i0 + min(lane, n - 1));
        const float mi = lane < n ? ml[2 * mine] : -__builtin_inff(), li = lane < n ? ml[2 * mine + 1] : 0.f;
        float mx = mi;
#pragma unroll
        for (int k = 1; k < 64; k *= 2) mx = fmaxf(mx, __shfl_xor(mx, k));
        mx = fmaxf(mx, m);
        const float base = finite_max(mx), al = ex2(m - base), f = ex2(mi - base);
        float lw = f * li;
#pragma unroll
        for (int k = 1; k < 64; k *= 2) lw += __shfl_xor(lw, k);
        m = mx;
        l = l * al + lw;
#pragma unroll
        for (int e = 0; e < D / 64; e++) o[e] *= al;
        for (int i = 0; i < n; i += 8) {  // eight rows in flight; lanes past n hold weight 0
            float v[8][D / 64], fi[8];
#pragma unroll
            for (int k = 0; k < 8; k++) {
                fi[k] = i + k < n ? __shfl(f, i + k) : 0.f;
                const float *src = os + __shfl(mine, min(i + k, n - 1)) * D + lane * (D / 64);
#pragma unroll
                for (int e = 0; e < D / 64; e++) v[k][e] = src[e];
            }
#pragma unroll
            for (int k = 0; k < 8; k++)
                if (i + k < n)
#pragma unroll
                    for (int e = 0; e < D / 64; e++) o[e] = fmaf(fi[k], v[k][e], o[e]);
        }
    }
    if (a.sinks && l != 0.f) {
        const float sk = a.sinks[hq] * kLog2e, mn = fmaxf(m, sk);
        const float base = finite_max(mn), f0 = ex2(m - base);
        l = l * f0 + ex2(sk - base);
#pragma unroll
        for (int e = 0; e < D / 64; e++) o[e] *= f0;
    }
    uint16_t *dst = a.out + b * a.ldo + hq * D + lane * (D / 64);
#pragma unroll
    for (int e = 0; e < D / 64; e++) dst[e] = (uint16_t)f2bf(l == 0.f ? 0.f : o[e] / l);
}

}  // namespace

// The sums start after the statistics, 16-byte aligned.
static int64_t call_rows(const Cache &c, int64_t B) { return (max_rows(c.Hq, c.Hkv, B) + 1) / 2 * 2; }

size_t attn_decode_call_bytes(const Cache &c, int64_t B) { return (size_t)call_rows(c, B) * (c.D + 2) * 4; }

size_t attn_decode_ws_bytes(const Cache &c, int64_t B)
{
    // fewer sequences may fill more rows of a prefix item: the largest over all batches up to B
    size_t most = 16;
    for (int64_t b = 1; b <= B; b++) most = std::max(most, attn_decode_call_bytes(c, b));
    return most;
}

hipError_t launch_attn_decode(const AttnArgs &a, hipStream_t st)
{
    const int64_t rows = call_rows(a.c, a.B);
    // no more items than the longest possible lengths give
    const int64_t G = a.c.Hq / a.c.Hkv, most = a.ldt * a.c.page;
    const int64_t seen = a.window ? std::min<int64_t>(most, a.window + kTok) : most;
    const int64_t own = std::min<int64_t>(max_own_items(a.c.Hq, a.c.Hkv, a.B),
                                          a.c.Hkv * a.B * ((G + kRows - 1) / kRows) * (seen / (kTok * kWaves) + 1));
    const unsigned grid = (unsigned)((a.prefix ? max_pre_items(a.c.Hq, a.c.Hkv, a.B) : 0) + own);
    const unsigned joins = (unsigned)(((int64_t)a.B * a.c.Hq + kWaves - 1) / kWaves);
    if (a.c.D == 128) {
        attn_items_kernel<128><<<grid, 64 * kWaves, 0, st>>>(a, rows);
        attn_join_kernel<128><<<joins, 64 * kWaves, 0, st>>>(a, rows);
    } else {
        attn_items_kernel<64><<<grid, 64 * kWaves, 0, st>>>(a, rows);
        attn_join_kernel<64><<<joins, 64 * kWaves, 0, st>>>(a, rows);
    }
    return hipGetLastError();
}

}  // namespace flint
