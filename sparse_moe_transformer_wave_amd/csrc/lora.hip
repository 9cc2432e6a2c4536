// lora.hip -- low-rank adapters of many requests: y[t] = base[t] + s_i B_i (A_i x[t]), i = ids[t].
//
// Two launches: h[t] = A_i x[t] (in fp32, in the workspace), then y.  Tokens go through the matrix
// products 16 at a time as the columns of an operand, whatever their adapters: for each adapter
// among them its weights are the other operand, and a column is kept by the tokens that have it.
// So one adapter's tokens share its weights, mixed ones read every adapter's once per tile, nothing
// is sorted, and no token's numbers meet another's.
//
// Bound by the launches for a decode batch, by the bytes of x, base and y for prompts.  h enters the
// second product as three bf16 parts, each rounded to nearest and the rest exact, so as fp32 (two
// leave 2^-17 of every term: eight times what fp32 sums do); the further parts are free beside the
// second product's bytes.
#include "serve.h"

#include <algorithm>

namespace flint {

namespace {

constexpr int kDownWaves = 8;  // of an h workgroup: they share its columns of x
constexpr int kUpWaves = 4;
constexpr int kMaxRankTiles = 8;
constexpr int kUpCols = 64;    // outputs of a wave's round

__device__ __forceinline__ int rank_of(const LoraArgs &a, int id)
{
    return a.ranks ? min(max(a.ranks[id], 0), a.R) : a.R;
}

// The adapters of a tile of 16 tokens: this lane's token's (-1: none), and a bit for the first
// token of each.  Every lane of the wave takes part.
__device__ __forceinline__ uint32_t tile_adapters(const LoraArgs &a, int t0, int &id)
{
    const int c = threadIdx.x & 15, t = t0 + c;
    id = t < a.T ? a.ids[t] : -1;
    if (id < 0 || id >= a.n) id = -1;
    bool first = id >= 0;
#pragma unroll
    for (int j = 0; j < 16; j++) {
        const int other = __shfl(id, j);
        if (j < c && other == id) first = false;
    }
    return (uint32_t)__ballot(first) & 0xffffu;
}

// Workgroup (tile of 16 MT tokens, slot of its adapters, part of the columns of x): h of its tokens.
// A wave takes every kDownWaves-th 32 columns of the part, all rank tiles of 16; the waves meet in LDS.
template <int MT>
__global__ __launch_bounds__(64 * kDownWaves) void lora_down_kernel(LoraArgs a, int slots, int splits)
{
    __shared__ f32x4 sh[kDownWaves][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15, g = lane >> 4;
    const int split = blockIdx.x % splits, slot = blockIdx.x / splits % slots, tile = blockIdx.x / (splits * slots);
    const int steps = (a.K + 31) / 32, s0 = (int)((int64_t)steps * split / splits), s1 = (int)((int64_t)steps * (split + 1) / splits);
    int id[MT];
    uint32_t todo[MT];
    const uint16_t *xp[MT];
#pragma unroll
    for (int m = 0; m < MT; m++) {
        const int t0 = (tile * MT + m) * 16;
        todo[m] = tile_adapters(a, t0, id[m]);
        xp[m] = a.x + (int64_t)min(t0 + r, a.T - 1) * a.ldx + 8 * g;
    }
    float *h = a.ws + (int64_t)split * a.T * a.R;
    for (int seen = 0;; seen++) {
        // the next adapter: the first of the first 16 tokens that have any left
        int now = -1;
#pragma unroll
        for (int m = 0; m < MT; m++)
            if (now < 0 && todo[m]) now = __shfl(id[m], __builtin_ctz(todo[m]));
        if (now < 0) return;
        now = __builtin_amdgcn_readfirstlane(now);
        bool has[MT];
#pragma unroll
        for (int m = 0; m < MT; m++) {
            const uint32_t mine = (uint32_t)__ballot(id[m] == now) & 0xffffu;
            has[m] = mine != 0;
            if (mine) todo[m] &= ~(mine & -mine);
        }
        if (seen % slots != slot) continue;
        const int rank = rank_of(a, now), rts = (rank + 15) / 16;
        for (int rt = 0; rt < rts; rt++) {
            const int row = rt * 16 + r;
            const uint16_t *ap = a.a + ((int64_t)now * a.R + min(row, rank - 1)) * a.K + 8 * g;
            f32x4 acc[MT];
#pragma unroll
            for (int m = 0; m < MT; m++) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
            for (int s = s0 + wave; s < s1; s += kDownWaves) {
                const bool in = 32 * s + 8 * g < a.K;
                u32x4 w = u32x4{0u, 0u, 0u, 0u};
                if (in) w = *reinterpret_cast<const u32x4 *>(ap + 32 * s);
#pragma unroll
                for (int m = 0; m < MT; m++) {
                    u32x4 v = u32x4{0u, 0u, 0u, 0u};
                    if (has[m] && in) v = *reinterpret_cast<const u32x4 *>(xp[m] + 32 * s);
                    if (has[m]) acc[m] = mfma16x16x32(as_bf16x8(w), as_bf16x8(v), acc[m]);
                }
            }
#pragma unroll
            for (int m = 0; m < MT; m++) {
                __syncthreads();
                sh[wave][lane] = acc[m];
                __syncthreads();
                if (wave == 0) {
                    f32x4 sum = sh[0][lane];
#pragma unroll
                    for (int w = 1; w < kDownWaves; w++) sum += sh[w][lane];
                    // ranks 16 rt + 4 g .. + 3 of token r; those past the adapter's are not read
                    const int t = (tile * MT + m) * 16 + r;
                    if (id[m] == now && rt * 16 + 4 * g < a.R)
                        *reinterpret_cast<f32x4 *>(h + (int64_t)t * a.R + rt * 16 + 4 * g) = sum;
                }
            }
        }
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}

// 16 consecutive values of a row at p, as fp32; whole: all are there and 16-byte aligned.
__device__ __forceinline__ void load16(const void *p, int fp32, bool whole, int n, float *v)
{
    if (fp32) {
        const float *f = (const float *)p;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            f32x4 x{0.f, 0.f, 0.f, 0.f};
            if (whole)
                x = *reinterpret_cast<const f32x4 *>(f + 4 * i);
            else
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (4 * i + e < n) x[e] = f[4 * i + e];
#pragma unroll
            for (int e = 0; e < 4; e++) v[4 * i + e] = x[e];
        }
        return;
    }
    const uint16_t *b = (const uint16_t *)p;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        u32x4 x{0u, 0u, 0u, 0u};
        if (whole)
            x = *reinterpret_cast<const u32x4 *>(b + 8 * i);
        else
#pragma unroll
            for (int e = 0; e < 8; e++)
                if (8 * i + e < n) x[e >> 1] |= (uint32_t)b[8 * i + e] << (16 * (e & 1));
#pragma unroll
        for (int e = 0; e < 4; e++) {
            v[8 * i + 2 * e] = bf2f(x[e] & 0xffffu);
            v[8 * i + 2 * e + 1] = bf2f(x[e] >> 16);
        }
    }
}
__device__ __forceinline__ void store16(void *p, int fp32, bool whole, int n, const float *v)
{
    if (fp32) {
        float *f = (float *)p;
        if (whole)
#pragma unroll
            for (int i = 0; i < 4; i++) *reinterpret_cast<f32x4 *>(f + 4 * i) = f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
        else
#pragma unroll
            for (int i = 0; i < 16; i++)
                if (i < n) f[i] = v[i];
        return;
    }
    uint16_t *b = (uint16_t *)p;
    uint32_t x[8];
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    if (whole)
#pragma unroll
        for (int i = 0; i < 2; i++) *reinterpret_cast<u32x4 *>(b + 8 * i) = u32x4{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
    else
#pragma unroll
        for (int i = 0; i < 16; i++)
            if (i < n) b[i] = (uint16_t)(x[i >> 1] >> (16 * (i & 1)));
}

// A wave: 16 tokens, `rounds` rounds of 64 outputs.  Row q of product j is output 16 (q / 4) + 4 j + q % 4
// of the round, so a lane's results are 16 consecutive outputs of its token.  RS: steps of 32 ranks.
template <int RS>
__global__ __launch_bounds__(64 * kUpWaves) void lora_up_kernel(LoraArgs a, int tiles, int rounds, int splits, int vec)
{
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int item = __builtin_amdgcn_readfirstlane(blockIdx.x * kUpWaves + (threadIdx.x >> 6));
    const int tile = item % tiles, n_first = item / tiles * rounds * kUpCols, t = tile * 16 + r;
    if (n_first >= a.N) return;
    int id;
    const uint32_t all = tile_adapters(a, tile * 16, id);
    const int tc = min(t, a.T - 1);
    // the token's h as the other operand: ranks 32 k + 8 g .. + 7, three parts
    u32x4 part[3][RS];
    const float scale = id >= 0 && a.scales ? a.scales[id] : 1.f;
    const int rank = id >= 0 ? rank_of(a, id) : 0;
#pragma unroll
    for (int k = 0; k < RS; k++) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = 0.f;
        if (32 * k + 8 * g < rank)
            for (int s = 0; s < splits; s++) {
                const float *h = a.ws + ((int64_t)s * a.T + tc) * a.R + 32 * k + 8 * g;
                const f32x4 x = *reinterpret_cast<const f32x4 *>(h), y = *reinterpret_cast<const f32x4 *>(h + 4);
#pragma unroll
                for (int i = 0; i < 4; i++) v[i] += x[i], v[4 + i] += y[i];
            }
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = 32 * k + 8 * g + i < rank ? v[i] * scale : 0.f;
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int e = 0; e < 3; e++) {
                const uint32_t p = pack_bf16(v[2 * i], v[2 * i + 1]);
                part[e][k][i] = p;
                v[2 * i] -= bf2f(p & 0xffffu);
                v[2 * i + 1] -= __uint_as_float(p & 0xffff0000u);
            }
    }
    const int es_b = a.base_fp32 ? 4 : 2, es_y = a.y_fp32 ? 4 : 2;
    for (int n0 = n_first; n0 < min(n_first + rounds * kUpCols, a.N); n0 += kUpCols) {
        const int n = n0 + 16 * g, have = a.N - n;  // this lane's outputs
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; i++) y[i] = 0.f;
        if (a.base && t < a.T && have > 0)
            load16((const uint8_t *)a.base + (t * a.ldb + n) * es_b, a.base_fp32, (vec & 1) && have >= 16, have, y);
        f32x4 acc[4];
#pragma unroll
        for (int j = 0; j < 4; j++) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (uint32_t todo = all; todo; todo &= todo - 1) {
            const int now = __builtin_amdgcn_readfirstlane(__shfl(id, __builtin_ctz(todo)));
            const int rn = rank_of(a, now);
            f32x4 c[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                c[j] = f32x4{0.f, 0.f, 0.f, 0.f};
                const int row = min(n0 + 16 * (r >> 2) + 4 * j + (r & 3), a.N - 1);
                const uint16_t *bp = a.b + ((int64_t)now * a.N + row) * a.R + 8 * g;
#pragma unroll
                for (int k = 0; k < RS; k++) {
                    u32x4 w = u32x4{0u, 0u, 0u, 0u};
                    const int left = rn - 32 * k - 8 * g;  // columns that count
                    if (left > 0) w = *reinterpret_cast<const u32x4 *>(bp + 32 * k);
                    if (left > 0 && left < 8)
#pragma unroll
                        for (int i = 0; i < 4; i++) w[i] &= (2 * i < left ? 0xffffu : 0u) | (2 * i + 1 < left ? 0xffff0000u : 0u);
#pragma unroll
                    for (int e = 0; e < 3; e++) c[j] = mfma16x16x32(as_bf16x8(w), as_bf16x8(part[e][k]), c[j]);
                }
            }
            if (id == now)
#pragma unroll
                for (int j = 0; j < 4; j++) acc[j] = c[j];
        }
        if (t >= a.T || have <= 0) continue;
        if (id >= 0)
#pragma unroll
            for (int i = 0; i < 16; i++) y[i] += acc[i >> 2][i & 3];
        store16((uint8_t *)a.y + (t * a.ldy + n) * es_y, a.y_fp32, (vec & 2) && have >= 16, have, y);
    }
}

struct Split {
    int mt, tiles, slots, splits;
};
// Tiles of 64 tokens where there are enough of them, or of 16; the adapters of a tile over as many
// workgroups, and the columns of x, as the GPU has room for.
Split plan_of(int64_t T, int K)
{
    Split p;
    p.mt = T >= 4096 ? 4 : 1;
    p.tiles = (int)((T + 16 * p.mt - 1) / (16 * p.mt));
    p.slots = std::max(1, std::min(16, 512 / p.tiles));
    const int want = std::max(1, 512 / p.tiles);
    p.splits = std::max(1, std::min({want, 8, K / (32 * kDownWaves * 4)}));
    return p;
}

}  // namespace

size_t lora_call_bytes(int64_t T, int K, int R) { return (size_t)plan_of(T, K).splits * T * R * 4; }

size_t lora_ws_bytes(int64_t T, int K, int R)
{
    // fewer tokens may be split over more workgroups: the largest over all batches up to T
    size_t most = 16;
    for (int64_t t = 1; t <= T; t = t < 1024 ? t + 1 : std::min(t + 16, std::max(T, t + 1))) most = std::max(most, lora_call_bytes(t, K, R));
    return std::max(most, T > 0 ? lora_call_bytes(T, K, R) : 0);
}

hipError_t launch_lora(const LoraArgs &a, hipStream_t st)
{
    const Split p = plan_of(a.T, a.K);
    const unsigned grid = (unsigned)(p.tiles * p.slots * p.splits);
    if (p.mt == 4)
        lora_down_kernel<4><<<grid, 64 * kDownWaves, 0, st>>>(a, p.slots, p.splits);
    else
        lora_down_kernel<1><<<grid, 64 * kDownWaves, 0, st>>>(a, p.slots, p.splits);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int tiles = (a.T + 15) / 16;
    const int64_t chunks = (a.N + kUpCols - 1) / kUpCols;
    // rounds of a wave: it splits h once for all of them; 4096 waves fill the GPU
    const int rounds = (int)std::max<int64_t>(1, std::min<int64_t>(chunks, tiles * chunks / 4096));
    const int64_t items = tiles * ((chunks + rounds - 1) / rounds);
    const auto wide = [](const void *q, int64_t ld, int fp32) { return ((uintptr_t)q | (uintptr_t)(ld * (fp32 ? 4 : 2))) % 16 == 0; };
    const int vec = (wide(a.base, a.ldb, a.base_fp32) ? 1 : 0) | (wide(a.y, a.ldy, a.y_fp32) ? 2 : 0);
    const unsigned wgs = (unsigned)((items + kUpWaves - 1) / kUpWaves);
    if (a.R <= 32)
        lora_up_kernel<1><<<wgs, 64 * kUpWaves, 0, st>>>(a, tiles, rounds, p.splits, vec);
    else if (a.R <= 64)
        lora_up_kernel<2><<<wgs, 64 * kUpWaves, 0, st>>>(a, tiles, rounds, p.splits, vec);
    else
        lora_up_kernel<4><<<wgs, 64 * kUpWaves, 0, st>>>(a, tiles, rounds, p.splits, vec);
    return hipGetLastError();
}

}  // namespace flint
