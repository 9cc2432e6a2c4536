// attn_decode.hip -- decode attention over the paged cache, a prefix shared by the batch read
// once: out[b][h] = sum_j p_j v_j, p = softmax_j(scale q . k_j) with an optional sink.
//
// The work of a call is a list of items, one workgroup each, that the host can count.  A prefix
// item takes a chunk of the shared prefix for up to 128 query rows of one key/value head (all
// the batch's queries of that head); an own item takes a part of one sequence's own tokens for
// 16 rows (its G = Hq / Hkv queries).  An item leaves its rows' maximum, sum and weighted values
// in the workspace, and a second launch joins each row's items and the sink.  Where every
// sequence is one item, that writes the result itself: one launch.
//
// Scores are computed transposed, S^T (tokens x rows) = K Q^T, with the tokens of a tile
// taken in an order that leaves 8 consecutive tokens of a row in each lane's results.  That is
// the B operand of O^T (channels x rows) = V^T P^T, so probabilities never leave their lane,
// a row's statistics are per-lane numbers, and with values stored transposed both products'
// A operands are 16-byte pieces of the cache as it lies.
//
// Bound by the cache's bytes where a key is read for few queries, by the matrix products where
// the prefix has many: 16 rows per key/value head make 16 products of a byte's worth each, 256
// rows the pipe's whole rate.  Measured (32 query and 4 key/value heads of 128, 64-token pages):
// 8 sequences, 96K shared and up to 4000 own tokens: 58 + 7 us, 238 MB, 4.1 TB/s (6.1 between
// 96K and 192K shared); 32 sequences, 32K shared and up to 1000 own: 50 + 8 us, 17.5 GFLOP; 32
// sequences, from 64K to 128K shared: 52 us, 660 TFLOP/s of products, 990 with the probabilities'
// second part; one sequence, a window of 513: 7 + 4 us, two dependent reads of memory and a join.
#include "ops.h"

#include <algorithm>

namespace flint {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kWaves = 8;       // of a whole short sequence
constexpr int kOwnWaves = 4;    // of an own item
constexpr int kPreWaves = 4;    // of a prefix item
constexpr int kTok = 32;        // tokens of a register tile
constexpr int kRows = 16;       // query rows of an own item
constexpr int kStageTok = 64;   // tokens of an LDS stage (prefix items)
constexpr int kPreRows = 128;   // query rows of a prefix item at most: 32 per wave
constexpr int kCut = 64;        // stages between refills of the page list
constexpr int kCUs = 256;       // prefix items of a call, or twice as many (pre_target), beyond one per row tile
constexpr int kOwnItems = 512;  // own items of a call, beyond one per sequence, head and row tile
constexpr int kMaxChunks = 256;  // prefix items of a query row: more take its join longer than they save
constexpr int kMaxSplit = 128;  // own items of a sequence, head and row tile
constexpr int kWhole = 256;     // a sequence of up to so many visible tokens is one workgroup's work in any case

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }
__host__ __device__ inline int max_of(int a, int b) { return a > b ? a : b; }

// A batch whose rows of one key/value head fit one 16-row tile takes its prefix through the
// own-item path (the bytes are the same, and every wave works); one sequence shares nothing.
__host__ __device__ inline bool wide_prefix(int B, int G) { return B * G > kRows; }
__host__ __device__ inline int prefix_rows(int B, int G)
{
    if (!wide_prefix(B, G)) return kRows;
    const int r = ceil_div(B * G, 32) * 32;
    return r < kPreRows ? r : kPreRows;
}

// The prefix items that a call is cut into: two workgroups per CU or one.  Two are faster in
// themselves, one computing while the other waits or forms probabilities (64 rows, 96K tokens: 58
// us against 64; 256 rows, 128K: 118 against 152), but leave twice the partial results to write
// and join.  A full item of fewer than 16 stages does not make up for that (128 rows, 32K tokens:
// 27 + 7 us with one workgroup against 33 + 11; 256 rows, 32K: 45 + 8 against 45 + 11; 256 rows,
// 64K, 16 stages: 81 + 8 against 66 + 11).
__host__ __device__ inline int pre_target(int rows, int64_t stages)
{
    return rows < kPreRows || stages >= 16 * 2 * kCUs ? 2 * kCUs : kCUs;
}

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
    if (a.window && a.window < p.P) p.P = 0;  // every window has left it
    p.wide = wide_prefix(a.B, G);
    p.rows = prefix_rows(a.B, G);
    p.rtp = ceil_div(a.B * G, p.rows);
    p.tiles = p.P / (p.wide ? kStageTok : kTok);
    const int64_t work = (int64_t)p.tiles * p.rtp * a.c.Hkv;
    const int target = pre_target(p.rows, work), least = p.wide ? 2 : kOwnWaves, even = (int)((work + target - 1) / target);
    p.chunk = max_of(max_of(even, least), ceil_div(p.tiles, kMaxChunks));
    p.nc = ceil_div(p.tiles, p.chunk);
    // chunks are dealt in eights, so that a chunk's row tiles meet on one XCD and its L2
    p.items = ceil_div(p.nc * a.c.Hkv, 8) * 8 * p.rtp;
    return p;
}

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

// The first sequence that takes part in the prefix: its table row names the prefix's pages (the rows
// of others need not).  -1: none does.
__device__ __forceinline__ int prefix_seq(const AttnArgs &a, int P)
{
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        const int b = b0 + (threadIdx.x & 63);
        const uint64_t part = __ballot(b < a.B && seq_of(a, min(b, a.B - 1), P).part);
        if (part) return b0 + __builtin_ctzll(part);
    }
    return -1;
}

// A sequence's own register tiles in nsplit parts, whole rounds of the workgroup's waves each.
struct Split {
    int t0, per, n;  // first tile, tiles per part, parts that are not empty
};
__device__ __forceinline__ Split split_of(const Seq &s, int nsplit)
{
    const int t0 = s.start / kTok, tiles = ceil_div(s.n, kTok) - t0;
    const int per = ceil_div(ceil_div(tiles, nsplit), kOwnWaves) * kOwnWaves;
    return Split{t0, per, tiles > 0 ? ceil_div(tiles, per) : 0};
}

// Parts per sequence, head and row tile: enough items for the GPU, at least one tile per wave.
__host__ inline int own_parts(int Hq, int Hkv, int64_t B, int64_t seen)
{
    const int64_t pairs = B * Hkv * ceil_div(Hq / Hkv, kRows);
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(kMaxSplit, kOwnItems / pairs));
    return (int)std::min<int64_t>(want, (seen + kTok * kOwnWaves - 1) / (kTok * kOwnWaves));
}

// Bounds of the items of any call with B sequences, and the workspace: {m, l} per row, then D
// weighted sums per row; prefix rows first.
__host__ inline int64_t max_pre_items(int Hq, int Hkv, int64_t B)
{
    const int G = Hq / Hkv, rows = prefix_rows((int)B, G);
    const int64_t rtp = ceil_div((int)B * G, rows);
    return B < 2 ? 0 : (ceil_div(2 * kCUs, (int)rtp) + Hkv + 8) * rtp;
}
__host__ inline int64_t max_rows(int Hq, int Hkv, int64_t B)
{
    const int64_t pairs = B * Hkv * ceil_div(Hq / Hkv, kRows);
    return max_pre_items(Hq, Hkv, B) * prefix_rows((int)B, Hq / Hkv) +
           pairs * own_parts(Hq, Hkv, B, INT32_MAX) * kRows;
}
struct Work {
    float *ml, *o;
};

// Probabilities as two bf16 parts, each rounded to nearest: together they hold 17 bits, and what
// is left has no sign of its own (parts cut off instead of rounded leave up to 2^-15, always
// missing, where the sum that divides has it; rounding takes the same six instructions for two).
// A single bf16 would leave up to 2^-8 of sum p |v|, which a row of few tokens does not average
// away.  The second product is free where the cache's bytes are the bound; where a prefix has 256
// rows it is a third of the products.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}
__device__ __forceinline__ void split8(const float *p, u32x4 &hi, u32x4 &lo)
{
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t h = pack_bf16(p[2 * i], p[2 * i + 1]);
        hi[i] = h;
        lo[i] = pack_bf16(p[2 * i] - bf2f(h), p[2 * i + 1] - __uint_as_float(h & 0xffff0000u));
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
    if (first >= end) return;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int sh = a.c.page_shift, page = a.c.page, last = (hi - 1) >> sh;  // the range's last table entry
    const int kt0 = 8 * (r >> 2) + (r & 3), vt0 = 8 * g;  // this lane's K rows kt0, kt0 + 4 of a tile; V tokens vt0 ..
    const float scale = fabsf(a.scale) * kLog2e;
    const uint16_t *kb = a.c.k + (int64_t)h * page * D + 8 * g, *vb = a.c.v + (int64_t)(h * D + r) * page;
    u32x4 kf[2][D / 32], vf[D / 16];
    int kp, vp;  // table entries of the tile to load next
    auto pages = [&](int tile) {
        kp = table[min((tile * kTok + kt0) >> sh, last)];
        vp = table[min((tile * kTok + vt0) >> sh, last)];
    };
    auto valid = [&](int pg) { return (uint32_t)pg < (uint64_t)a.c.n_pages; };
    auto load_k = [&](int tile) {
        const uint16_t *kr = kb + (valid(kp) ? kp : 0) * a.c.page_stride + ((tile * kTok + kt0) & (page - 1)) * D;
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
            for (int kk = 0; kk < D / 32; kk++) kf[j][kk] = *reinterpret_cast<const u32x4 *>(kr + 4 * j * D + 32 * kk);
    };
    auto load_v = [&](int tile) {
        const uint16_t *vr = vb + (valid(vp) ? vp : 0) * a.c.page_stride + ((tile * kTok + vt0) & (page - 1));
#pragma unroll
        for (int dt = 0; dt < D / 16; dt++) vf[dt] = *reinterpret_cast<const u32x4 *>(vr + 16 * dt * page);
    };
    pages(first);
    load_k(first);
    load_v(first);
    bool vok = valid(vp);
    if (first + step < end) pages(first + step);
    // Each operand's registers take the next tile's as soon as their products are issued, and
    // its table entries are a tile ahead of that.
    for (int tile = first; tile < end; tile += step) {
        const int tb = tile * kTok, vt = tb + vt0;
        const bool more = tile + step < end;
        f32x4 s[2];
#pragma unroll
        for (int j = 0; j < 2; j++) {
            s[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kk = 0; kk < D / 32; kk++) s[j] = mfma16x16x32(as_bf16x8(kf[j][kk]), qf[kk], s[j]);
        }
        if (more) load_k(tile + step);
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
        if (more) {
            load_v(tile + step);
            vok = valid(vp);
            if (tile + 2 * step < end) pages(tile + 2 * step);
        }
    }
}

template <int D, int W>
struct OwnShared {
    float m[W][kRows], l[W][kRows];
    f32x4 o[W][D / 4][kRows];  // [wave][channel / 4][row]
};

// 16 rows over register tiles t0 .. t1 of a token range [lo, hi): the waves take tiles in turn
// and meet in LDS; done(row, c4, m, l, o) gets the sums of channels 4 c4 .. 4 c4 + 3.
template <int D, int W, typename F>
__device__ __forceinline__ void own_item(const AttnArgs &a, int h, const int32_t *table, int lo, int hi, int t0, int t1,
                                         const uint16_t *q, OwnShared<D, W> &sh, F done)
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
    attend<D>(a, h, table, lo, hi, t0 + wave, W, t1, qf, acc);
    acc.l += __shfl_xor(acc.l, 16);
    acc.l += __shfl_xor(acc.l, 32);
    if (g == 0) {
        sh.m[wave][r] = acc.m;
        sh.l[wave][r] = acc.l;
    }
#pragma unroll
    for (int dt = 0; dt < D / 16; dt++) sh.o[wave][4 * dt + g][r] = acc.o[dt];
    __syncthreads();
    for (int i = tid; i < kRows * (D / 4); i += 64 * W) {
        const int rr = i / (D / 4), c4 = i % (D / 4);
        float m = sh.m[0][rr];
#pragma unroll
        for (int w = 1; w < W; w++) m = fmaxf(m, sh.m[w][rr]);
        const float base = finite_max(m);
        float l = 0.f;
        f32x4 o{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < W; w++) {
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
// Stages of 64 tokens are copied HBM -> LDS (no registers), one ahead of the one in use, and
// every wave multiplies its own 32 rows with all of them on the 32x32x16 MFMA.  Two workgroups
// share a CU: one multiplies while the other waits, forms probabilities or writes.
//
// LDS stage: K rows in the order the score product wants (row 8 q + 4 h + i of a 32-token tile
// is token 16 (q / 2) + 8 h + 4 (q % 2) + i, so lane half h gets tokens 8 h .. 8 h + 7 of each
// 16), then V rows (one per channel, 64 tokens).  Row R keeps its 16-byte chunk c at
// c ^ swz(R mod 32): the 32 rows that a fragment read touches fall on distinct banks.
constexpr int kStages = 2;
constexpr int kCutPages = kCut * kStageTok / 16;
constexpr int stage_bytes(int D) { return 2 * kStageTok * D * 2; }

template <int CH>  // 16-byte chunks of a row
__device__ __forceinline__ int swz(int row) { return CH == 16 ? (row & 15) : ((row ^ (row >> 3)) & 7); }

__device__ __forceinline__ void copy16(const void *g, uint8_t *lds)
{
    __builtin_amdgcn_global_load_lds(g, (__attribute__((address_space(3))) void *)lds, 16, 0, 0);
}

// Waits for the wave's copies (vmcnt 0).
__device__ __forceinline__ void wait_copies() { __builtin_amdgcn_s_waitcnt(0x0F70); }
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

// 32 of a wave's rows: m (base 2, shared by the lanes l and l + 32 of a row), this lane's part
// of the sum, O^T: channel 32 dt + 8 (i / 4) + 4 (l / 32) + i % 4.
template <int D>
struct Acc32 {
    float m, l;
    f32x16 o[D / 32];
};

// Fragments of 32-token tile t of a stage: K columns 16 kk .., V channels 32 dt .. at tokens 16 k ..
template <int D>
__device__ __forceinline__ bf16x8 k_frag(const uint8_t *st, int t, int kk)
{
    const int r = threadIdx.x & 31, c = 2 * kk + ((threadIdx.x >> 5) & 1);
    return as_bf16x8(*reinterpret_cast<const u32x4 *>(st + (32 * t + r) * (2 * D) + 16 * (c ^ swz<D / 8>(r))));
}
template <int D>
__device__ __forceinline__ u32x4 v_frag(const uint8_t *st, int t, int k, int dt)
{
    const int r = threadIdx.x & 31, c = 4 * t + 2 * k + ((threadIdx.x >> 5) & 1);
    return *reinterpret_cast<const u32x4 *>(st + kStageTok * D * 2 + (32 * dt + r) * (2 * kStageTok) + 16 * (c ^ swz<8>(r)));
}

template <int D>
__device__ __forceinline__ f32x16 scores(const uint8_t *st, int t, const bf16x8 *qf)
{
    f32x16 s;
#pragma unroll
    for (int i = 0; i < 16; i++) s[i] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; kk++) s = mfma32(k_frag<D>(st, t, kk), qf[kk], s);
    return s;
}

// The factor al that the sums so far take when scores with maximum mx (this lane's, scaled)
// join them; true if it is not one.  The reference maximum moves only when a score has left it
// 8 behind (a factor of 256, harmless in fp32), so most tiles neither exchange maxima nor rescale.
template <int D>
__device__ __forceinline__ bool raise_max(float mx, Acc32<D> &acc, float &al)
{
    if (!__any(!(mx <= acc.m + 8.f) && mx != -__builtin_inff())) return false;
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    mx = fmaxf(mx, acc.m);
    al = ex2(acc.m - finite_max(mx));
    acc.m = mx;
    acc.l *= al;
    return true;
}
template <int D>
__device__ __forceinline__ void rescale(Acc32<D> &acc, float al)
{
#pragma unroll
    for (int dt = 0; dt < D / 32; dt++)
#pragma unroll
        for (int i = 0; i < 16; i++) acc.o[dt][i] *= al;
}

// The probabilities of a tile, in two bf16 parts per 16 tokens.
struct Prob {
    u32x4 hi[2], lo[2];
};

// Values of a tile; see: whether this lane's 8 tokens of each 16 are valid.
template <int D, bool MASK>
__device__ __forceinline__ void add_values(const uint8_t *st, int t, const Prob &p, const bool *see, Acc32<D> &acc)
{
#pragma unroll
    for (int k = 0; k < 2; k++)
#pragma unroll
        for (int dt = 0; dt < D / 32; dt++) {
            u32x4 v = v_frag<D>(st, t, k, dt);
            if (MASK && !see[k]) v = u32x4{0u, 0u, 0u, 0u};
            acc.o[dt] = mfma32(as_bf16x8(v), as_bf16x8(p.hi[k]), acc.o[dt]);
            acc.o[dt] = mfma32(as_bf16x8(v), as_bf16x8(p.lo[k]), acc.o[dt]);
        }
}

// This lane's maximum of a tile's scores, scaled; only those seen.
template <bool MASK>
__device__ __forceinline__ float max_score(f32x16 s, float scale, const bool *see)
{
    float mx = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < 16; i++)
        if (!MASK || see[i >> 3]) mx = fmaxf(mx, s[i]);
    return MASK && mx == -__builtin_inff() ? mx : mx * scale;
}

// Scores to probabilities against the present reference maximum.
template <int D, bool MASK>
__device__ __forceinline__ void weigh(f32x16 s, float scale, const bool *see, Prob &pr, Acc32<D> &acc)
{
    const float base = finite_max(acc.m);
    float p[16], ps = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i++) {
        p[i] = ex2(fmaf(s[i], scale, -base));
        if (MASK && !see[i >> 3]) p[i] = 0.f;
        ps += p[i];
    }
    acc.l += ps;
#pragma unroll
    for (int k = 0; k < 2; k++) split8(p + 8 * k, pr.hi[k], pr.lo[k]);
}

// The order of a basic block with MFMAs, READS LDS reads for them and the vector work of
// weigh(): reads run four ahead of their products, and each of the first BESIDE MFMAs is
// followed by its share of the vector instructions.
template <int MFMA, int READS, int BESIDE>
__device__ __forceinline__ void overlap()
{
    constexpr int kVector = 96 / BESIDE + 1, kPer = MFMA / READS;
    __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);  // LDS reads
#pragma unroll
    for (int i = 0; i < MFMA; i++) {
        if (i % kPer == 0 && i / kPer + 4 < READS) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                        // MFMA
        if (i < BESIDE) __builtin_amdgcn_sched_group_barrier(0x402, kVector, 0);  // vector, exponentials
    }
}
__device__ __forceinline__ void formed_here(Prob &p)
{
#pragma unroll
    for (int k = 0; k < 2; k++) asm volatile("" : "+v"(p.hi[k]), "+v"(p.lo[k]));
}

// One 64-token stage: two tiles.  The second tile's scores are multiplied while the first's
// probabilities are formed, the first's values while the second's are.
template <int D>
__device__ __forceinline__ void pre_stage(const uint8_t *st, const bf16x8 *qf, float scale, Acc32<D> &acc)
{
    const bool see[2] = {true, true};
    float al;
    const f32x16 s0 = scores<D>(st, 0, qf);
    if (raise_max(max_score<false>(s0, scale, see), acc, al)) rescale(acc, al);
    Prob p0, p1;
    f32x16 s1 = scores<D>(st, 1, qf);
    weigh<D, false>(s0, scale, see, p0, acc);
    overlap<D / 16, D / 16, D / 16>();
    formed_here(p0);
    if (raise_max(max_score<false>(s1, scale, see), acc, al)) {
        add_values<D, false>(st, 0, p0, see, acc);  // weighted by the old maximum: added here, and
        rescale(acc, al);                           // nothing of it below
#pragma unroll
        for (int k = 0; k < 2; k++) p0.hi[k] = p0.lo[k] = u32x4{0u, 0u, 0u, 0u};
    }
    add_values<D, false>(st, 0, p0, see, acc);
    weigh<D, false>(s1, scale, see, p1, acc);
    add_values<D, false>(st, 1, p1, see, acc);
    overlap<D / 4, D / 8, D / 8>();
}

// A stage with tokens whose page is not valid (ok: a bit per 8 tokens).
template <int D>
__device__ __forceinline__ void masked_stage(const uint8_t *st, const bf16x8 *qf, float scale, uint32_t ok, Acc32<D> &acc)
{
#pragma unroll 1
    for (int t = 0; t < 2; t++) {
        bool see[2];
#pragma unroll
        for (int k = 0; k < 2; k++) see[k] = (ok >> (4 * t + 2 * k + ((threadIdx.x >> 5) & 1))) & 1;
        const f32x16 s = scores<D>(st, t, qf);
        float al;
        if (raise_max(max_score<true>(s, scale, see), acc, al)) rescale(acc, al);
        Prob p;
        weigh<D, true>(s, scale, see, p, acc);
        add_values<D, true>(st, t, p, see, acc);
    }
}

// Stages t0 .. t1 of the prefix for row tile rt of key/value head h; rows to workspace row out + r.
template <int D>
__device__ __forceinline__ void prefix_item(const AttnArgs &a, const Pre &p, int h, int rt, int t0, int t1, int64_t out,
                                            const Work &w, uint8_t *stages, int *pages)
{
    constexpr int KPC = 1024 / (2 * D);   // K rows of one copy instruction (1 KB)
    constexpr int NK = kStageTok / KPC / kPreWaves, NV = D / 8 / kPreWaves;  // a wave's copies per stage: K, V
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 31, hh = lane >> 5, G = a.c.Hq / a.c.Hkv, rows = a.B * G;
    const int row0 = wave * 32;                                     // the wave's first row of the item
    const bool live = row0 < p.rows && rt * p.rows + row0 < rows;   // it has rows
    const float scale = fabsf(a.scale) * kLog2e;
    const int page = a.c.page, sft = a.c.page_shift;
    // Sequence 0 takes part as a rule: its entries of the first cut are on their way while the lengths
    // come, which costs 0 to 0.5 us of a call.
    const int e_first = (t0 * kStageTok) >> sft, n_first = ((min(t0 + kCut, t1) * kStageTok - 1) >> sft) - e_first + 1;
    static_assert(kCutPages <= 64 * kPreWaves, "an entry of a cut per thread");
    const int32_t early = a.table[e_first + min(tid, n_first - 1)];
    const int seq = prefix_seq(a, p.P);
    if (seq < 0) return;  // nothing here is joined to any row
    const int32_t *table = a.table + seq * a.ldt;
    // The wave's copies: K copy i fills LDS rows KPC (NK wave + i) + l / (D / 8) from tokens ktok
    // + (l / (D / 8)) and, past 4, + 8 of the stage, chunk l % (D / 8); V copy i fills channels
    // 8 (NV wave + i) + l / 8, chunk l % 8.  What a lane adds to the copy's scalar address:
    int koff[NK], voff[NV], vpage[NV];  // vpage: where pages are smaller than a stage, from its first
#pragma unroll
    for (int i = 0; i < NK; i++) {
        const int r0 = KPC * (NK * wave + i), lr = lane / (D / 8), r32 = (r0 + lr) & 31;
        koff[i] = ((lr & 3) + 2 * (lr & 4)) * D + 8 * ((lane % (D / 8)) ^ swz<D / 8>(r32));
    }
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int d = 8 * (NV * wave + i) + lane / 8, c = (lane % 8) ^ swz<8>(d & 31);
        voff[i] = d * page + ((8 * c) & (page - 1));
        vpage[i] = (8 * c) >> sft;
    }
    bf16x8 qf[D / 16];
    {
        const int row = min(rt * p.rows + row0 + r, rows - 1);
        const uint16_t *qp = a.q + (row / G) * a.ldq + (h * G + row % G) * D;
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
        for (int i = tid; i < ne; i += 64 * kPreWaves) {
            const int pg = c0 == t0 && seq == 0 ? early : table[e0 + i];
            const bool good = (uint32_t)pg < (uint64_t)a.c.n_pages;
            pages[i] = good ? pg : -1;
            bad |= !good;
        }
        bad = __syncthreads_or(bad);
        // Copies of stage s into its slot.  A K copy's rows lie in one page and a V copy's
        // channels too where a page holds a stage's tokens, so the page and its address are
        // scalar; smaller pages give each lane its own.
        auto page_at = [&](int i) { return max(pages[i], 0); };
        auto issue = [&](int s) {
            uint8_t *st = stages + s % kStages * stage_bytes(D);
            const int tb = s * kStageTok, e = (tb >> sft) - e0;
#pragma unroll
            for (int i = 0; i < NK; i++) {
                const int r0 = KPC * (NK * wave + i);
                const int tok = tb + (r0 & 32) + (r0 & 0x13) + ((r0 & 8) >> 1) + ((r0 & 4) << 1);
                const int64_t pg = __builtin_amdgcn_readfirstlane(page_at((tok >> sft) - e0));
                copy16(a.c.k + pg * a.c.page_stride + (h * page + (tok & (page - 1))) * D + koff[i], st + 1024 * (NK * wave + i));
            }
            const int64_t pv = page >= kStageTok ? __builtin_amdgcn_readfirstlane(page_at(e)) : 0;
            const uint16_t *vb = a.c.v + pv * a.c.page_stride + h * page * D + (tb & (page - 1));
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const uint16_t *src = vb + voff[i];
                if (page < kStageTok) src += (int64_t)page_at(e + vpage[i]) * a.c.page_stride;
                copy16(src, st + kStageTok * D * 2 + 1024 * (NV * wave + i));
            }
        };
        issue(c0);
        for (int s = c0; s < c1; s++) {
            // Stage s is in LDS for every wave once each has seen its own copies land and met the
            // barrier, which also ends every wave's use of the other slot: it takes stage s + 1.
            wait_copies();
            stage_barrier();
            if (s + 1 < c1) issue(s + 1);
            if (!live) continue;
            const uint8_t *st = stages + s % kStages * stage_bytes(D);
            if (!bad) {
                pre_stage<D>(st, qf, scale, acc);
            } else {
                uint32_t ok = 0;
                for (int c = 0; c < 8; c++) ok |= (uint32_t)(pages[((s * kStageTok + 8 * c) >> sft) - e0] >= 0) << c;
                masked_stage<D>(st, qf, scale, ok, acc);
            }
        }
    }
    if (!live) return;
    acc.l += __shfl_xor(acc.l, 32);
    const int64_t dst = out + row0 + r;
    if (hh == 0) {
        w.ml[2 * dst] = acc.m;
        w.ml[2 * dst + 1] = acc.l;
    }
    float *o = w.o + dst * D;
#pragma unroll
    for (int dt = 0; dt < D / 32; dt++)
#pragma unroll
        for (int i = 0; i < 4; i++)
            *reinterpret_cast<f32x4 *>(o + 32 * dt + 8 * i + 4 * hh) =
                f32x4{acc.o[dt][4 * i], acc.o[dt][4 * i + 1], acc.o[dt][4 * i + 2], acc.o[dt][4 * i + 3]};
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

constexpr int join_waves(int per) { return per > 8 ? per : 8; }  // of a workgroup: one row's, or several rows'

// ---- launches ------------------------------------------------------------------------------
// The sink joins a row's sums: f is the factor that its weighted values take.  An infinite one
// leaves nothing: l = 0, unless it is NaN.
__device__ __forceinline__ void sink_in(const AttnArgs &a, int hq, float &m, float &l, float &f)
{
    f = 1.f;
    if (!a.sinks || l == 0.f) return;
    const float sk = a.sinks[hq] * kLog2e, mn = fmaxf(m, sk), base = finite_max(mn);
    if (sk == __builtin_inff() && l == l) {
        l = 0.f;
        return;
    }
    f = ex2(m - base);
    l = l * f + ex2(sk - base);
    m = mn;
}
// The result of 4 channels of a query from its joined sums; a row that saw nothing is zero.
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
    __shared__ __attribute__((aligned(16))) OwnShared<D, kWaves> sh;
    const int G = a.c.Hq / a.c.Hkv, rts = ceil_div(G, kRows), r = threadIdx.x & 15;
    const int rt = blockIdx.x % rts, h = blockIdx.x / rts % a.c.Hkv, b = blockIdx.x / (rts * a.c.Hkv);
    const Seq s = seq_of(a, b, 0);
    const int qh = h * G + min(rt * kRows + r, G - 1);
    own_item<D, kWaves>(a, h, a.table + b * a.ldt, s.lo, s.n, s.start / kTok, ceil_div(s.n, kTok), a.q + b * a.ldq + qh * D,
                        sh, [&](int rr, int c4, float m, float l, f32x4 o) {
                            if (rt * kRows + rr >= G) return;
                            const int hq = h * G + rt * kRows + rr;
                            float f;
                            sink_in(a, hq, m, l, f);
                            store4(a.out + b * a.ldo + hq * D + 4 * c4, o, f, l);
                        });
}

template <int D, bool WIDE>
__global__ __launch_bounds__(64 * kOwnWaves, 2) void attn_items_kernel(AttnArgs a, Pre p, int nsplit, Work w)
{
    // a prefix item's stages or an own item's exchange; the pages apart from them, so that
    // reading those does not wait for copies in flight
    extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
    __shared__ int pages[WIDE ? kCutPages : 1];
    OwnShared<D, kOwnWaves> &own_sh = *reinterpret_cast<OwnShared<D, kOwnWaves> *>(dyn);
    const int r = threadIdx.x & 15, G = a.c.Hq / a.c.Hkv;
    int64_t out;
    auto done = [&](int rr, int c4, float m, float l, f32x4 o) {
        if (c4 == 0) {
            w.ml[2 * (out + rr)] = m;
            w.ml[2 * (out + rr) + 1] = l;
        }
        *reinterpret_cast<f32x4 *>(w.o + (out + rr) * D + 4 * c4) = o;
    };
    int item = blockIdx.x;
    if (item < p.items) {  // the long ones first
        int h, rt, c;
        if (!pre_item_of(p, a.c.Hkv, item, h, rt, c)) return;
        const int t0 = c * p.chunk, t1 = min(t0 + p.chunk, p.tiles);
        out = (int64_t)item * p.rows;
        if constexpr (WIDE) {
            prefix_item<D>(a, p, h, rt, t0, t1, out, w, dyn, pages);
        } else {  // all rows in one tile: the own items' path over that sequence's table row
            const int q = min(r, a.B * G - 1), seq = prefix_seq(a, p.P);
            if (seq < 0) return;
            own_item<D, kOwnWaves>(a, h, a.table + seq * a.ldt, 0, p.P, t0, t1, a.q + (q / G) * a.ldq + (h * G + q % G) * D, own_sh, done);
        }
        return;
    }
    item -= p.items;
    const int rts = ceil_div(G, kRows), c = item % nsplit, pair = item / nsplit;
    const int rt = pair % rts, h = pair / rts % a.c.Hkv, b = pair / (rts * a.c.Hkv);
    const Seq s = seq_of(a, b, p.P);
    const Split sp = split_of(s, nsplit);
    if (c >= sp.n) return;
    const int t0 = sp.t0 + c * sp.per, t1 = min(t0 + sp.per, ceil_div(s.n, kTok));
    const int qh = h * G + min(rt * kRows + r, G - 1);
    out = (int64_t)p.items * p.rows + (int64_t)item * kRows;
    own_item<D, kOwnWaves>(a, h, a.table + b * a.ldt, max(s.lo, s.start), s.n, t0, t1, a.q + b * a.ldq + qh * D, own_sh, done);
}

// Joins a query row's items and the sink.  PER waves take a row, eight items at a time each.
template <int D, int PER>
__global__ __launch_bounds__(64 * join_waves(PER)) void attn_join_kernel(AttnArgs a, Pre p, int nsplit, Work w)
{
    constexpr int W = join_waves(PER);
    __shared__ float sm[W], sl[W];
    __shared__ float so[W][D];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), part = wave % PER;
    const int G = a.c.Hq / a.c.Hkv, rts = ceil_div(G, kRows), rows = a.B * a.c.Hq;
    const int at = blockIdx.x * (W / PER) + wave / PER, q = min(at, rows - 1);
    const int b = q / a.c.Hq, hq = q % a.c.Hq, h = hq / G, gi = hq % G;
    const Seq s = seq_of(a, b, p.P);
    const int prow = b * G + gi, np = s.part ? p.nc : 0, total = np + split_of(s, nsplit).n;
    const int64_t own = (int64_t)p.items * p.rows + (int64_t)((b * a.c.Hkv + h) * rts + gi / kRows) * nsplit * kRows + gi % kRows;
    auto row_of = [&](int i) {
        return i < np ? (int64_t)pre_item_at(p, h, prow / p.rows, i) * p.rows + prow % p.rows : own + (int64_t)(i - np) * kRows;
    };
    float m = -__builtin_inff(), l = 0.f, o[D / 64] = {};
    for (int i0 = 8 * part; i0 < total; i0 += 8 * PER) {
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
    if (part || lane >= D / 4 || at >= rows) return;
    m = sm[wave];
#pragma unroll
    for (int i = 1; i < PER; i++) m = fmaxf(m, sm[wave + i]);
    const float base = finite_max(m);
    f32x4 r{0.f, 0.f, 0.f, 0.f};
    l = 0.f;
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const float f = ex2(sm[wave + i] - base);
        l = fmaf(f, sl[wave + i], l);
#pragma unroll
        for (int e = 0; e < 4; e++) r[e] = fmaf(f, so[wave + i][4 * lane + e], r[e]);
    }
    float f;
    sink_in(a, hq, m, l, f);
    store4(a.out + b * a.ldo + hq * D + 4 * lane, r, f, l);
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

template <int D, int PER>
static void launch_join(const AttnArgs &a, const Pre &p, int nsplit, const Work &w, hipStream_t st)
{
    constexpr int W = join_waves(PER);
    attn_join_kernel<D, PER><<<(unsigned)ceil_div(a.B * a.c.Hq * PER, W), 64 * W, 0, st>>>(a, p, nsplit, w);
}

template <int D>
static hipError_t launch_d(const AttnArgs &a, hipStream_t st)
{
    const int64_t pairs = (int64_t)a.B * a.c.Hkv * ceil_div(a.c.Hq / a.c.Hkv, kRows), most = a.ldt * a.c.page;
    // the tokens of a sequence that its own items can span, from lengths the host knows
    const int64_t seen = a.window ? std::min<int64_t>(most, (int64_t)a.window + kTok - 1) : most;
    const Pre p = pre_of(a);
    const int nsplit = own_parts(a.c.Hq, a.c.Hkv, a.B, seen);
    // One launch where a sequence is a workgroup's work: short, or so many sequences that they fill
    // the GPU as they are.  Windows of 513 tokens: 64 sequences 15 us, two launches 18 + 8; 16: 12.7
    // against 9.6 + 4; one: 11.9 against 7.1 + 4.  Of 1000: 32 sequences 20 us against 16 + 5, 16: 19
    // against 12 + 4.
    if (seen <= kWhole || (!p.items && (nsplit == 1 || seen <= 8 * pairs))) {
        attn_whole_kernel<D><<<(unsigned)pairs, 64 * kWaves, 0, st>>>(a);
        return hipGetLastError();
    }
    Work w;
    w.ml = a.ws;
    w.o = w.ml + 2 * call_rows(a.c, a.B);
    const unsigned grid = (unsigned)(p.items + pairs * nsplit);
    static_assert(kPreWaves == kOwnWaves, "prefix and own items share a launch");
    if (p.items && p.wide) {
        constexpr size_t lds = std::max<size_t>((size_t)kStages * stage_bytes(D), sizeof(OwnShared<D, kOwnWaves>));
        attn_items_kernel<D, true><<<grid, 64 * kOwnWaves, lds, st>>>(a, p, nsplit, w);
    } else {
        attn_items_kernel<D, false><<<grid, 64 * kOwnWaves, sizeof(OwnShared<D, kOwnWaves>), st>>>(a, p, nsplit, w);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // Waves per row by the items that a row can have (4096 rows of 9 items: two 6 us, eight 14; 8 rows
    // of 380: 16).
    const int most_items = p.nc + nsplit;
    if (most_items <= 8)
        launch_join<D, 1>(a, p, nsplit, w, st);
    else if (most_items <= 16)
        launch_join<D, 2>(a, p, nsplit, w, st);
    else if (most_items <= 32)
        launch_join<D, 4>(a, p, nsplit, w, st);
    else if (most_items <= 64)
        launch_join<D, 8>(a, p, nsplit, w, st);
    else
        launch_join<D, 16>(a, p, nsplit, w, st);
    return hipGetLastError();
}

hipError_t launch_attn_decode(const AttnArgs &a, hipStream_t st)
{
    return a.c.D == 128 ? launch_d<128>(a, st) : launch_d<64>(a, st);
}

}  // namespace flint
