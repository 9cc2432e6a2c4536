// attn_decode.hip -- decode attention over the paged cache, a prefix shared by the batch read
// once: out[b][h] = sum_j p_j v_j, p = softmax_j(scale q . k_j) with an optional sink.
//
// The work of a call is a list of items (key/value head, segment, tile of 16 query rows,
// chunk of tokens).  Segments are the shared prefix, whose rows are all the batch's queries
// of that head, and each sequence's own tokens, whose rows are its G = Hq / Hkv queries.
// Every workgroup derives the same list from kv_len; an item leaves its rows' running
// maximum, sum and weighted values in the workspace, and a second launch joins each row's
// items and the sink.
//
// Scores are computed transposed, S^T (tokens x rows) = K Q^T, so a lane of the 16x16x32
// MFMA result holds 4 consecutive tokens of one row.  The two 16-token products of a 32-token
// tile take the tokens in the order 8 (r / 4) + r % 4 (+ 4): lane group g then holds tokens
// 8 g .. 8 g + 7 of its row, which is the B operand of O^T (channels x rows) = V^T P^T, and
// with values stored transposed both operands load straight from the cache, 16 bytes a lane.
#include "ops.h"

#include <algorithm>

namespace flint {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kTok = 32;        // tokens of a tile
constexpr int kRows = 16;       // query rows of an item
constexpr int kTarget = 1024;   // items that a call is cut into, beyond one per segment

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// The items of a call, the same in every workgroup of both launches.
struct Plan {
    int G, rts, rtp;         // query heads per key/value head; row tiles of a sequence, of the prefix
    int prefix_tiles;        // 32-token tiles of the shared prefix (0: none)
    int chunk;               // tiles per item
    int prefix_items;        // per key/value head
};

struct Seq {
    int n, lo, start, part;  // length, first visible token, first own token, takes part in the prefix
};

__device__ __forceinline__ int prefix_tokens(const AttnArgs &a)
{
    const int unit = a.c.page > 64 ? a.c.page : 64;
    return a.prefix / unit * unit;
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

// Fills cum[0 .. B]: the first own item (per key/value head) of each sequence.
__device__ __forceinline__ Plan make_plan(const AttnArgs &a, int *cum, int64_t *scratch)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    Plan p;
    p.G = a.c.Hq / a.c.Hkv;
    p.rts = ceil_div(p.G, kRows);
    p.rtp = ceil_div(a.B * p.G, kRows);
    const int P = prefix_tokens(a);
    int tiles[4], parts = 0;
    int64_t sum = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int b = 4 * tid + i;
        tiles[i] = 0;
        if (b < a.B) {
            const Seq s = seq_of(a, b, P);
            tiles[i] = ceil_div(s.n - s.start, kTok);
            parts += s.part;
        }
        sum += tiles[i];
    }
    // totals over the workgroup
    int64_t tot = sum;
    int np = parts;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
        tot += __shfl_xor(tot, m);
        np += __shfl_xor(np, m);
    }
    if (lane == 0) {
        scratch[wave] = tot;
        scratch[4 + wave] = np;
    }
    __syncthreads();
    tot = scratch[0] + scratch[1] + scratch[2] + scratch[3];
    np = (int)(scratch[4] + scratch[5] + scratch[6] + scratch[7]);
    p.prefix_tiles = np ? P / kTok : 0;
    const int64_t work = (tot * p.rts + (int64_t)p.prefix_tiles * p.rtp) * a.c.Hkv;
    p.chunk = (int)max((int64_t)8, (work + kTarget - 1) / kTarget);
    p.prefix_items = p.rtp * ceil_div(p.prefix_tiles, p.chunk);
    // exclusive scan of the sequences' items
    int items = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) items += ceil_div(tiles[i], p.chunk) * p.rts;
    int inc = items;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
        const int v = __shfl_up(inc, m);
        if (lane >= m) inc += v;
    }
    __syncthreads();
    if (lane == 63) scratch[wave] = inc;
    __syncthreads();
    int at = inc - items;
    for (int w = 0; w < wave; w++) at += (int)scratch[w];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if (4 * tid + i < a.B) cum[4 * tid + i] = at;
        at += ceil_div(tiles[i], p.chunk) * p.rts;
        if (4 * tid + i == a.B - 1) cum[a.B] = at;
    }
    __syncthreads();
    return p;
}

// Eight probabilities as two bf16 parts, each the upper half of an fp32 (truncated): together
// they hold 16 bits.  A single bf16 would leave up to 2^-8 of sum p |v|, which a row of few
// tokens does not average away; the second product is free beside the cache's bytes.
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

// One wave: tiles first, first + step, ... < end of a token range for 16 query rows.
// lane: row l % 16, lane group g = l / 16.  m in the exponent's base-2 domain, l this lane's
// part of the sum (its 8 tokens of each tile), o[d / 16]: O^T, channel 16 dt + 4 g + i.
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
    const float scale = a.scale * kLog2e;
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
        const float base = mx == -__builtin_inff() ? 0.f : mx;  // nothing visible so far
        const float al = exp2f(acc.m - base);
        acc.m = mx;
        float p[8], ps = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            p[i] = exp2f(x[i] - base);
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

// Workspace: per item and row {m, l} and the row's D weighted sums.
template <int D>
__device__ __forceinline__ float *item_row(const AttnArgs &a, int64_t item, int r)
{
    return a.ws + (item * kRows + r) * (D + 4);
}

template <int D>
__global__ __launch_bounds__(256) void attn_items_kernel(AttnArgs a)
{
    __shared__ int cum[kAttnMaxB + 1];
    __shared__ int64_t scratch[8];
    __shared__ float sm[4][kRows], sl[4][kRows];
    __shared__ f32x4 so[4][D / 4][kRows + 1];  // [wave][channel / 4][row]
    const Plan p = make_plan(a, cum, scratch);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
    const int P = p.prefix_tiles * kTok;
    const int per_head = p.prefix_items + cum[a.B], total = per_head * a.c.Hkv;
    for (int item = blockIdx.x; item < total; item += gridDim.x) {
        const int h = item / per_head, it = item % per_head;
        int rt, c, b = 0, lo, hi, t0, t1;
        if (it < p.prefix_items) {
            rt = it % p.rtp;
            c = it / p.rtp;
            lo = 0;
            hi = P;
            t0 = c * p.chunk;
            t1 = min(t0 + p.chunk, p.prefix_tiles);
        } else {
            const int own = it - p.prefix_items;
            int x = 0, y = a.B - 1;  // the last sequence that starts at or before this item and has items
            while (x < y) {
                const int mid = (x + y + 1) >> 1;
                if (cum[mid] <= own)
                    x = mid;
                else
                    y = mid - 1;
            }
            b = x;
            const Seq s = seq_of(a, b, prefix_tokens(a));
            rt = (own - cum[b]) % p.rts;
            c = (own - cum[b]) / p.rts;
            lo = max(s.lo, s.start);
            hi = s.n;
            t0 = s.start / kTok + c * p.chunk;
            t1 = min(t0 + p.chunk, ceil_div(s.n, kTok));
        }
        // this lane's query row
        const bool pre = it < p.prefix_items;
        const int row = rt * kRows + r, rows = pre ? a.B * p.G : p.G;
        const int qb = pre ? min(row, rows - 1) / p.G : b, qh = h * p.G + min(row, rows - 1) % p.G;
        bf16x8 qf[D / 32];
#pragma unroll
        for (int kk = 0; kk < D / 32; kk++)
            qf[kk] = as_bf16x8(*reinterpret_cast<const u32x4 *>(a.q + qb * a.ldq + qh * D + 32 * kk + 8 * g));
        Acc<D> acc;
        acc.m = -__builtin_inff();
        acc.l = 0.f;
#pragma unroll
        for (int dt = 0; dt < D / 16; dt++) acc.o[dt] = f32x4{0.f, 0.f, 0.f, 0.f};
        attend<D>(a, h, a.table + (pre ? 0 : b * a.ldt), lo, hi, t0 + wave, 4, t1, qf, acc);
        acc.l += __shfl_xor(acc.l, 16);
        acc.l += __shfl_xor(acc.l, 32);
        __syncthreads();  // the previous item's LDS has been read
        if (g == 0) {
            sm[wave][r] = acc.m;
            sl[wave][r] = acc.l;
        }
#pragma unroll
        for (int dt = 0; dt < D / 16; dt++) so[wave][4 * dt + g][r] = acc.o[dt];
        __syncthreads();
        for (int i = tid; i < kRows * (D / 4); i += 256) {
            const int rr = i % kRows, c4 = i / kRows;
            float m = sm[0][rr];
            for (int w = 1; w < 4; w++) m = fmaxf(m, sm[w][rr]);
            const float base = m == -__builtin_inff() ? 0.f : m;
            float l = 0.f;
            f32x4 o{0.f, 0.f, 0.f, 0.f};
            for (int w = 0; w < 4; w++) {
                const float f = exp2f(sm[w][rr] - base);
                l += f * sl[w][rr];
                const f32x4 v = so[w][c4][rr];
#pragma unroll
                for (int e = 0; e < 4; e++) o[e] += f * v[e];
            }
            float *dst = item_row<D>(a, item, rr);
            if (c4 == 0) {
                dst[0] = m;
                dst[1] = l;
            }
            *reinterpret_cast<f32x4 *>(dst + 4 + 4 * c4) = o;
        }
    }
}

// One wave per query row: joins the row's items and the sink.
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a)
{
    __shared__ int cum[kAttnMaxB + 1];
    __shared__ int64_t scratch[8];
    const Plan p = make_plan(a, cum, scratch);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t q = (int64_t)blockIdx.x * 4 + wave;
    if (q >= (int64_t)a.B * a.c.Hq) return;
    const int b = (int)(q / a.c.Hq), hq = (int)(q % a.c.Hq), h = hq / p.G, gi = hq % p.G;
    const int per_head = p.prefix_items + cum[a.B];
    const Seq s = seq_of(a, b, prefix_tokens(a));
    const int64_t base_item = (int64_t)h * per_head;
    const int prow = b * p.G + gi;
    const int np = s.part && p.prefix_items ? p.prefix_items / p.rtp : 0;
    const int ns = (cum[b + 1] - cum[b]) / p.rts;
    float m = -__builtin_inff(), l = 0.f, o[D / 64] = {};
    for (int i = 0; i < np + ns; i++) {
        const int64_t item = i < np ? base_item + i * p.rtp + prow / kRows
                                    : base_item + p.prefix_items + cum[b] + (i - np) * p.rts + gi / kRows;
        const float *src = item_row<D>(a, item, (i < np ? prow : gi) % kRows);
        const float mi = src[0], li = src[1], mn = fmaxf(m, mi);
        const float base = mn == -__builtin_inff() ? 0.f : mn;
        const float f0 = exp2f(m - base), f1 = exp2f(mi - base);
        m = mn;
        l = l * f0 + li * f1;
#pragma unroll
        for (int e = 0; e < D / 64; e++) o[e] = o[e] * f0 + src[4 + lane + 64 * e] * f1;
    }
    if (a.sinks && l != 0.f) {
        const float sk = a.sinks[hq] * kLog2e, mn = fmaxf(m, sk);
        const float base = mn == -__builtin_inff() ? 0.f : mn;
        const float f0 = exp2f(m - base);
        l = l * f0 + exp2f(sk - base);
#pragma unroll
        for (int e = 0; e < D / 64; e++) o[e] *= f0;
    }
#pragma unroll
    for (int e = 0; e < D / 64; e++)
        a.out[b * a.ldo + hq * D + lane + 64 * e] = (uint16_t)f2bf(l == 0.f ? 0.f : o[e] / l);
}

// Bound of the items of any call with B sequences.
int64_t max_items(const Cache &c, int64_t B)
{
    const int64_t G = c.Hq / c.Hkv;
    return kTarget + c.Hkv * ((B * G + kRows - 1) / kRows + B * ((G + kRows - 1) / kRows));
}

}  // namespace

size_t attn_decode_ws_bytes(const Cache &c, int64_t B)
{
    return (size_t)max_items(c, B) * kRows * (c.D + 4) * 4;
}

hipError_t launch_attn_decode(const AttnArgs &a, hipStream_t st)
{
    const unsigned grid = (unsigned)std::min<int64_t>(max_items(a.c, a.B), 2048);
    const unsigned joins = (unsigned)(((int64_t)a.B * a.c.Hq + 3) / 4);
    if (a.c.D == 128) {
        attn_items_kernel<128><<<grid, 256, 0, st>>>(a);
        attn_join_kernel<128><<<joins, 256, 0, st>>>(a);
    } else {
        attn_items_kernel<64><<<grid, 256, 0, st>>>(a);
        attn_join_kernel<64><<<joins, 256, 0, st>>>(a);
    }
    return hipGetLastError();
}

}  // namespace flint
