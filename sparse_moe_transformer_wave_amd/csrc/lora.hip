// lora.hip -- low-rank adapters of many requests: y[t] = base[t] + s_i B_i (A_i x[t]), i = ids[t].
//
// Tokens go through the matrix products 16 at a time, whatever their adapters: for each adapter among
// them its weights are the other operand, and a token keeps the results of its own.  So one adapter's
// tokens share its weights as far as a tile goes, nothing is sorted, and no token's numbers meet another's.
//
// Two launches: h = A_i x in fp32 to the workspace, then y.  Both stage rows through registers into LDS:
// loads in a fragment's own order take 16 rows in 16 lanes, and so 64 cycles of a CU's address unit where
// rows in order take 16 (4099 tokens, 8 adapters of rank 64, 4096 -> 2048: 31 + 29 us, staged 20 + 18).
// A small batch is one launch instead: every workgroup computes its adapter's h by itself (8 tokens, 6
// adapters of rank 16, 2048 -> 5120: 7.6 us, in two launches 9.5), and its weights of the second product
// and its part of base are on their way meanwhile.
//
// Bound by the chain of dependent reads for a decode batch.  A prompt's first launch is bound by the starts of
// its workgroups: of rank 64 one takes 151 KB of LDS, so a CU has one at a time, and 4099 tokens are 65 tiles of
// 4 parts, 260 workgroups for 256 CUs, and as many again of the second slot; each waits for its ids and its
// first loads and then has four stages (with one of them 17.6 of the 20 us are left).  The second's 18 us are 16
// without the stores; x, base and y take 13 at a copy's rate.  h enters the second product as three bf16 parts,
// each rounded to nearest and the rest exact, so as fp32 (two leave 2^-17 of every term: eight times what fp32
// sums do).
#include "serve.h"

#include <algorithm>

namespace flint {

namespace {

constexpr int kWaves = 8;    // of a small batch's workgroup: they share its columns of x
constexpr int kUpCols = 64;  // outputs of such a wave
constexpr int kSteps = 4;    // steps of 32 columns that such a wave has on their way
constexpr int kTile = 64;    // tokens of a workgroup of the two launches: 16 to each of its four waves
constexpr int kCols = 128;   // outputs of a round of the second

// Workgroup b of `grid`, a multiple of 8, takes place (b % 8) grid / 8 + b / 8: consecutive places, which
// are consecutive tokens and so the same adapters, meet on one XCD and its L2.
__device__ __forceinline__ int place_on_xcd(int b, int grid) { return b % 8 * (grid / 8) + b / 8; }
inline int grid_of(int64_t places) { return (int)((places + 7) / 8 * 8); }

__device__ __forceinline__ int rank_of(const LoraArgs &a, int id)
{
    return a.ranks ? min(max(a.ranks[id], 0), a.R) : a.R;
}

// The adapters of N tokens from t0 on, lane l that of token l mod N (-1: none); returns a bit for the first
// token of each.
template <int N>
__device__ __forceinline__ uint64_t first_tokens(const LoraArgs &a, int t0, int &id)
{
    const int t = t0 + (threadIdx.x & (N - 1));
    id = t < a.T ? a.ids[t] : -1;
    if (id < 0 || id >= a.n) id = -1;
    uint64_t firsts = 0, rest = __ballot(id >= 0) & (N == 64 ? ~0ull : (1ull << (N & 63)) - 1);
    while (rest) {
        const int first = __builtin_ctzll(rest);
        firsts |= 1ull << first;
        rest &= ~__ballot(id == __builtin_amdgcn_readlane(id, first));
    }
    return firsts;
}
// Of those first tokens the ones whose adapters are a slot's: every slots-th.
__device__ __forceinline__ uint64_t slot_tokens(uint64_t firsts, int slot, int slots)
{
    const int lane = threadIdx.x & 63, order = __popcll(firsts & ((1ull << lane) - 1));
    return __ballot(((firsts >> lane) & 1) && order % slots == slot);
}

// 8 values as an operand's three parts.
__device__ __forceinline__ void split8(float *v, u32x4 *part)
{
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int e = 0; e < 3; e++) {
            const uint32_t p = pack_bf16(v[2 * i], v[2 * i + 1]);
            part[e][i] = p;
            v[2 * i] -= bf2f(p & 0xffffu);
            v[2 * i + 1] -= __uint_as_float(p & 0xffff0000u);
        }
}
// 8 columns of B of which `left` count.
__device__ __forceinline__ u32x4 first_columns(u32x4 w, int left)
{
    if (left < 8)
#pragma unroll
        for (int i = 0; i < 4; i++) w[i] &= (2 * i < left ? 0xffffu : 0u) | (2 * i + 1 < left ? 0xffff0000u : 0u);
    return w;
}

// N consecutive outputs of a token.  Bits of base are loaded where nothing has to wait for them and
// become numbers when they are used; wide: all N are there and aligned, otherwise the first `have` go one
// by one.
template <int N>
struct Outputs {
    u32x4 raw[N / 4];
    __device__ __forceinline__ void fetch(const LoraArgs &a, const uint8_t *base, bool wide)
    {
        if (!a.base || !wide) return;
        if (a.base_fp32) {
#pragma unroll
            for (int i = 0; i < N / 4; i++) raw[i] = *reinterpret_cast<const u32x4 *>(base + 16 * i);
        } else {
#pragma unroll
            for (int i = 0; i < N / 8; i++) raw[i] = *reinterpret_cast<const u32x4 *>(base + 16 * i);
        }
    }
    __device__ __forceinline__ void store(const LoraArgs &a, const uint8_t *base, uint8_t *y, bool wide, int have, float *v) const
    {
        if (!wide) {
#pragma unroll 1
            for (int i = 0; i < min(have, N); i++) {
                float x = 0.f;
#pragma unroll
                for (int k = 0; k < N; k++) x = k == i ? v[k] : x;
                if (a.base) x += a.base_fp32 ? ((const float *)base)[i] : bf2f(((const uint16_t *)base)[i]);
                if (a.y_fp32)
                    ((float *)y)[i] = x;
                else
                    ((uint16_t *)y)[i] = (uint16_t)pack_bf16(x, 0.f);
            }
            return;
        }
        if (a.base)
#pragma unroll
            for (int i = 0; i < N; i++) {
                const uint32_t b = raw[i >> 3][(i >> 1) & 3], f = raw[i >> 2][i & 3];
                v[i] += __uint_as_float(a.base_fp32 ? f : i & 1 ? b & 0xffff0000u : b << 16);
            }
        if (a.y_fp32) {
#pragma unroll
            for (int i = 0; i < N / 4; i++) reinterpret_cast<f32x4 *>(y)[i] = f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
        } else {
#pragma unroll
            for (int i = 0; i < N / 8; i++)
                reinterpret_cast<u32x4 *>(y)[i] = pack8(v + 8 * i);
        }
    }
};

// ---- two launches --------------------------------------------------------------------------
// Workgroup (slot of the adapters, tile of 64 tokens, part of the columns of x): h of its tokens, RT rank
// tiles of 16.  A stage is KC columns of the adapter's rows and the tokens', in LDS with a pitch that puts
// 16 rows on different banks; the next stage is on its way while one is in use.  Four of the eight waves take
// the first half of its columns and four the other: parts of x that are not summed here are read again by
// every workgroup of the second launch (512 tokens, rank 64, 8192 -> 8192: 21.7 us for both, with four waves
// and twice the parts 23.2; 4099 tokens 39.1 and 38.4).  KC 256 where that leaves a CU one workgroup anyway
// or the rows are few; of rank 32 two share a CU (2048 tokens of 16 adapters 55 us, with 256 columns 60).
template <int RT, int KC>
__global__ __launch_bounds__(512) void lora_down_kernel(LoraArgs a, int grid, int slots, int splits)
{
    constexpr int TPR = KC / 8, RPP = 512 / TPR;  // threads to a row, rows of a pass of the workgroup
    constexpr int ROWS = 16 * RT + kTile, APASSES = 16 * RT / RPP, XPASSES = kTile / RPP, PITCH = 2 * KC + 16;
    static_assert(16 * RT % RPP == 0 && kTile % RPP == 0, "a pass has rows of one kind");
    __shared__ __attribute__((aligned(16))) uint8_t lds[2][ROWS * PITCH];
    __shared__ f32x4 half_sum[4][RT][64];
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) & 3, half = __builtin_amdgcn_readfirstlane(tid >> 8);  // of a stage's columns
    const int slot = blockIdx.x / grid, place = place_on_xcd(blockIdx.x % grid, grid), split = place % splits, tile = place / splits;
    if (tile * kTile >= a.T) return;
    const int chunks = (a.K + KC - 1) / KC, c0 = (int)((int64_t)chunks * split / splits), c1 = (int)((int64_t)chunks * (split + 1) / splits);
    const int row0 = tid / TPR, col0 = tid % TPR * 8;
    u32x4 va[APASSES], vx[XPASSES];
    auto load_x = [&](int c, uint64_t groups) {  // a bit for each 16 tokens that are wanted, at its first
        const int col = min(c * KC + col0, a.K - 8);
#pragma unroll
        for (int p = 0; p < XPASSES; p++) {
            const int tok = row0 + p * RPP;
            if ((groups >> (tok & 48)) & 1) vx[p] = *reinterpret_cast<const u32x4 *>(a.x + (int64_t)min(tile * kTile + tok, a.T - 1) * a.ldx + col);
        }
    };
#pragma unroll
    for (int p = 0; p < XPASSES; p++) vx[p] = u32x4{0u, 0u, 0u, 0u};
    constexpr uint64_t kAll = 0x0001000100010001ull;
    if (slot == 0) load_x(c0, kAll);  // while it finds out about their adapters
    int all;
    uint64_t todo = slot_tokens(first_tokens<64>(a, tile * kTile, all), slot, slots);
    const int ranks = all >= 0 ? rank_of(a, all) : 0;
    const int id = __shfl(all, 16 * wave + r), t = tile * kTile + 16 * wave + r;
    float *h = a.ws + (int64_t)split * a.T * a.R;
    bool early = slot == 0;
    for (; todo; todo &= todo - 1) {
        const int first = __builtin_ctzll(todo), now = __builtin_amdgcn_readlane(all, first), rank = __builtin_amdgcn_readlane(ranks, first);
        const uint64_t mine = __ballot(all == now);
        if (rank == 0) continue;
        uint64_t groups = 0;
#pragma unroll
        for (int i = 0; i < 64; i += 16) groups |= (uint64_t)(((mine >> i) & 0xffff) != 0) << i;
        auto load_a = [&](int c) {
            const int col = min(c * KC + col0, a.K - 8);
#pragma unroll
            for (int p = 0; p < APASSES; p++)
                va[p] = *reinterpret_cast<const u32x4 *>(a.a + ((int64_t)now * a.R + min(row0 + p * RPP, rank - 1)) * a.K + col);
        };
        f32x4 acc[RT];
#pragma unroll
        for (int rt = 0; rt < RT; rt++) acc[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
        const bool has = (mine >> (16 * wave)) & 0xffff;
        load_a(c0);
        if (!early) load_x(c0, groups);
        early = false;
        for (int c = c0; c < c1; c++) {
            uint8_t *st = lds[c & 1];
            const bool in = c * KC + col0 < a.K;  // behind the last column both count as zeros
#pragma unroll
            for (int p = 0; p < APASSES; p++)
                *reinterpret_cast<u32x4 *>(st + (row0 + p * RPP) * PITCH + 2 * col0) = in ? va[p] : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int p = 0; p < XPASSES; p++)
                *reinterpret_cast<u32x4 *>(st + (16 * RT + row0 + p * RPP) * PITCH + 2 * col0) = in ? vx[p] : u32x4{0u, 0u, 0u, 0u};
            __syncthreads();  // and every wave is done with the stage before, whose place the next takes
            if (c + 1 < c1) {
                load_a(c + 1);
                load_x(c + 1, groups);
            }
            if (!has) continue;
#pragma unroll
            for (int k = 0; k < KC / 64; k++) {
                const uint8_t *at = st + KC * half + 64 * k + 16 * g;
                const u32x4 x = *reinterpret_cast<const u32x4 *>(at + (16 * RT + 16 * wave + r) * PITCH);
#pragma unroll
                for (int rt = 0; rt < RT; rt++) {
                    const u32x4 w = *reinterpret_cast<const u32x4 *>(at + (16 * rt + r) * PITCH);
                    acc[rt] = mfma16x16x32(as_bf16x8(w), as_bf16x8(x), acc[rt]);
                }
            }
        }
        if (half)
#pragma unroll
            for (int rt = 0; rt < RT; rt++) half_sum[wave][rt][lane] = acc[rt];
        __syncthreads();
        // ranks 16 rt + 4 g .. + 3 of token r; those past the adapter's are not read
        if (!half && id == now)
#pragma unroll
            for (int rt = 0; rt < RT; rt++)
                if (16 * rt + 4 * g < a.R)
                    *reinterpret_cast<f32x4 *>(h + (int64_t)t * a.R + 16 * rt + 4 * g) = acc[rt] + half_sum[wave][rt][lane];
    }
}

// Workgroup (slot of the adapters, tile of 64 tokens, `rounds` rounds of 128 outputs); a token's outputs are
// written by the slot of its adapter, or by the first.  RS: steps of 32 ranks.
//
// Column c of product j is output 8 c + j of the round, so that a lane's results are 8 consecutive outputs
// of tokens 4 g .. 4 g + 3 and 16 lanes' 128 of one.  The round's rows of B, which lie together, go to LDS in
// that order (row 8 c + j to 16 j + c) with a pitch of 16 bytes more, which keeps 16 columns on different
// banks; the next round's or adapter's are on their way meanwhile.
template <int RS>
__global__ __launch_bounds__(256) void lora_up_kernel(LoraArgs a, int grid, int slots, int rounds, int splits, int vec)
{
    constexpr int PR = 4 * RS, PIECES = kCols * PR / 256, PITCH = 16 * PR + 16;  // pieces of 16 bytes, of a row and a thread
    constexpr int QR = 8 * RS, QUADS = kTile * QR / 256, HP = 32 * RS + 4;       // four ranks of h, likewise
    __shared__ __attribute__((aligned(16))) uint8_t lds[kCols * PITCH];
    static_assert(kTile * HP * 4 <= kCols * PITCH, "h has the rows' place before they come");
    float *hs = reinterpret_cast<float *>(lds);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15, g = lane >> 4;
    const int slot = blockIdx.x / grid, place = place_on_xcd(blockIdx.x % grid, grid);
    const int parts = (a.N + rounds * kCols - 1) / (rounds * kCols), tile = place / parts;
    const int n_first = place % parts * rounds * kCols, n_end = min(n_first + rounds * kCols, a.N);
    if (tile * kTile >= a.T) return;
    // the tile's h: its first part while this finds out about the tokens' adapters
    f32x4 hv[QUADS];
    const float *hsrc[QUADS];
#pragma unroll
    for (int i = 0; i < QUADS; i++) {
        const int q = tid + 256 * i;
        hsrc[i] = a.ws + (int64_t)min(tile * kTile + q / QR, a.T - 1) * a.R + min(q % QR * 4, a.R - 4);
        hv[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (slot == 0) hv[i] = *reinterpret_cast<const f32x4 *>(hsrc[i]);
    }
    int all;
    const uint64_t firsts = slot_tokens(first_tokens<64>(a, tile * kTile, all), slot, slots);
    // the tokens that this workgroup writes; those without an adapter are there already where y is base
    uint64_t writes = slot == 0 && !(vec & 4) ? __ballot(all < 0 && tile * kTile + lane < a.T) : 0;
    for (uint64_t todo = firsts; todo; todo &= todo - 1) writes |= __ballot(all == __builtin_amdgcn_readlane(all, __builtin_ctzll(todo)));
    if (!writes) return;
    u32x4 next[PIECES];
    auto fetch_rows = [&](int now, int n0) {  // of B, as they lie
        const uint16_t *src = a.b + ((int64_t)now * a.N + n0) * a.R;
#pragma unroll
        for (int i = 0; i < PIECES; i++) {
            const int p = tid + 256 * i, row = min(p / PR, a.N - n0 - 1), col = min(p % PR * 8, a.R - 8);
            next[i] = *reinterpret_cast<const u32x4 *>(src + row * a.R + col);
        }
    };
    const int ranks = all >= 0 ? rank_of(a, all) : 0;
    const float scales = all >= 0 && a.scales ? a.scales[all] : 1.f;
    const int t0 = tile * kTile + 16 * wave;
    u32x4 part[RS][3];
    if (firsts) {
        fetch_rows(__builtin_amdgcn_readlane(all, __builtin_ctzll(firsts)), n_first);
        // the parts' sum, scaled, through LDS to an operand: token r, ranks 32 k + 8 g .. + 7
#pragma unroll 4
        for (int s = slot == 0; s < splits; s++)
#pragma unroll
            for (int i = 0; i < QUADS; i++) hv[i] += *reinterpret_cast<const f32x4 *>(hsrc[i] + (int64_t)s * a.T * a.R);
#pragma unroll
        for (int i = 0; i < QUADS; i++) {
            const int q = tid + 256 * i, row = q / QR, left = __shfl(ranks, row) - q % QR * 4;  // ranks that count
            const float scale = __shfl(scales, row);
#pragma unroll
            for (int e = 0; e < 4; e++) hv[i][e] = e < left ? hv[i][e] * scale : 0.f;
            *reinterpret_cast<f32x4 *>(hs + row * HP + q % QR * 4) = hv[i];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < RS; k++) {
            const float *src = hs + (16 * wave + r) * HP + 32 * k + 8 * g;
            const f32x4 lo = *reinterpret_cast<const f32x4 *>(src), hi = *reinterpret_cast<const f32x4 *>(src + 4);
            float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            split8(v, part[k]);
        }
    }
    int mine[4];  // adapters of the tokens whose results this lane gets
#pragma unroll
    for (int e = 0; e < 4; e++) mine[e] = __shfl(all, 16 * wave + 4 * g + e);
    const uint32_t put = (uint32_t)(writes >> (16 * wave + 4 * g)) & 15u;  // which of them it writes
    const int es_b = a.base_fp32 ? 4 : 2, es_y = a.y_fp32 ? 4 : 2;
    for (int n0 = n_first; n0 < n_end; n0 += kCols) {
        const int n = n0 + 8 * r, have = a.N - n;  // this lane's outputs
        const bool wide = (vec & 3) == 3 && n0 + kCols <= a.N;
        const uint8_t *base = (const uint8_t *)a.base + ((int64_t)(t0 + 4 * g) * a.ldb + n) * es_b;
        uint8_t *y = (uint8_t *)a.y + ((int64_t)(t0 + 4 * g) * a.ldy + n) * es_y;
        Outputs<8> o[4];
        float v[4][8];
#pragma unroll
        for (int e = 0; e < 4; e++) {
            if ((put >> e) & 1) o[e].fetch(a, base + e * a.ldb * es_b, wide);
#pragma unroll
            for (int j = 0; j < 8; j++) v[e][j] = 0.f;
        }
        for (uint64_t todo = firsts; todo; todo &= todo - 1) {
            const int first = __builtin_ctzll(todo), now = __builtin_amdgcn_readlane(all, first), rank = __builtin_amdgcn_readlane(ranks, first);
            __syncthreads();  // every wave is done with what was there
#pragma unroll
            for (int i = 0; i < PIECES; i++) {
                const int p = tid + 256 * i, row = p / PR, piece = p % PR;
                *reinterpret_cast<u32x4 *>(lds + (16 * (row & 7) + (row >> 3)) * PITCH + 16 * piece) = first_columns(next[i], rank - 8 * piece);
            }
            __syncthreads();
            const uint64_t rest = todo & (todo - 1);
            if (rest || n0 + kCols < n_end)
                fetch_rows(__builtin_amdgcn_readlane(all, __builtin_ctzll(rest ? rest : firsts)), rest ? n0 : n0 + kCols);
            if (!((__ballot(all == now) >> (16 * wave)) & 0xffff)) continue;
#pragma unroll
            for (int j = 0; j < 8; j++) {
                f32x4 c{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < RS; k++) {
                    const u32x4 w = *reinterpret_cast<const u32x4 *>(lds + (16 * j + r) * PITCH + 64 * k + 16 * g);
#pragma unroll
                    for (int e = 0; e < 3; e++) c = mfma16x16x32(as_bf16x8(part[k][e]), as_bf16x8(w), c);
                }
#pragma unroll
                for (int e = 0; e < 4; e++) v[e][j] = mine[e] == now ? c[e] : v[e][j];
            }
        }
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (((put >> e) & 1) && have > 0) o[e].store(a, base + e * a.ldb * es_b, y + e * a.ldy * es_y, wide, have, v[e]);
    }
}

// ---- a small batch ---------------------------------------------------------------------------
// Workgroup (tile of 16 tokens, slot of its adapters, 512 outputs), fragments straight from memory and h in
// LDS.  Row q of product j is output 16 (q / 4) + 4 j + q % 4 of a wave's 64, so that a lane's results are 16
// consecutive outputs of its token.
template <int RT>
__global__ __launch_bounds__(64 * kWaves) void lora_small_kernel(LoraArgs a, int slots, int parts, int vec)
{
    constexpr int RS = (RT + 1) / 2;
    __shared__ f32x4 sh[kWaves][RT][64];
    __shared__ __attribute__((aligned(16))) float hs[16][16 * RT + 4];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15, g = lane >> 4;
    const int part_n = blockIdx.x % parts, slot = blockIdx.x / parts % slots, tile = blockIdx.x / (parts * slots);
    const int t = tile * 16 + r, n0 = (part_n * kWaves + wave) * kUpCols, n = n0 + 16 * g, have = t < a.T ? a.N - n : 0;
    const bool wide = (vec & 3) == 3 && n0 + kUpCols <= a.N;
    const uint8_t *base = (const uint8_t *)a.base + ((int64_t)t * a.ldb + n) * (a.base_fp32 ? 4 : 2);
    uint8_t *y = (uint8_t *)a.y + ((int64_t)t * a.ldy + n) * (a.y_fp32 ? 4 : 2);
    int id;
    const uint64_t all = first_tokens<16>(a, tile * 16, id);
    Outputs<16> o;
    if (slot == 0 && !(vec & 4) && __any(id < 0)) {  // tokens without an adapter
        float v[16] = {};
        if (id < 0 && have > 0) {
            o.fetch(a, base, wide);
            o.store(a, base, y, wide, have, v);
        }
    }
    const uint16_t *xp = a.x + (int64_t)min(t, a.T - 1) * a.ldx + 8 * g;
    const int steps = (a.K + 31) / 32;
    for (uint64_t todo = slot_tokens(all, slot, slots); todo; todo &= todo - 1) {
        const int now = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo)), rank = rank_of(a, now);
        const bool mine = id == now && have > 0;
        if (mine) o.fetch(a, base, wide);
        u32x4 w[4][RS];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int row = min(n0 + 16 * (r >> 2) + 4 * j + (r & 3), a.N - 1);
            const uint16_t *bp = a.b + ((int64_t)now * a.N + row) * a.R + 8 * g;
#pragma unroll
            for (int k = 0; k < RS; k++) {
                w[j][k] = u32x4{0u, 0u, 0u, 0u};
                if (32 * k + 8 * g < rank) w[j][k] = *reinterpret_cast<const u32x4 *>(bp + 32 * k);
            }
        }
        // h: a wave's steps of 32 columns lie together, since a step is half a cache line of each row
        f32x4 acc[RT];
        const uint16_t *ap[RT];
#pragma unroll
        for (int rt = 0; rt < RT; rt++) {
            ap[rt] = a.a + ((int64_t)now * a.R + min(16 * rt + r, max(rank, 1) - 1)) * a.K + 8 * g;
            acc[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        for (int s = kSteps * wave; s < steps; s += kSteps * kWaves) {
            u32x4 f[kSteps][RT], x[kSteps];
#pragma unroll
            for (int u = 0; u < kSteps; u++) {
                // K ends inside a step where it is no multiple of 32; there and behind it columns count as zeros
                const int col = 32 * (s + u) + 8 * g < a.K ? 32 * (s + u) : 0;
                x[u] = *reinterpret_cast<const u32x4 *>(xp + (col ? col : 8 * g < a.K ? 0 : -8 * g));
#pragma unroll
                for (int rt = 0; rt < RT; rt++) f[u][rt] = *reinterpret_cast<const u32x4 *>(ap[rt] + (col ? col : 8 * g < a.K ? 0 : -8 * g));
            }
#pragma unroll
            for (int u = 0; u < kSteps; u++) {
                const bool in = 32 * (s + u) + 8 * g < a.K;
                if (!in) x[u] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
                for (int rt = 0; rt < RT; rt++) {
                    if (!in) f[u][rt] = u32x4{0u, 0u, 0u, 0u};
                    acc[rt] = mfma16x16x32(as_bf16x8(f[u][rt]), as_bf16x8(x[u]), acc[rt]);
                }
            }
        }
#pragma unroll
        for (int rt = 0; rt < RT; rt++) sh[wave][rt][lane] = acc[rt];
        __syncthreads();
        for (int rt = wave; rt < RT; rt += kWaves) {
            f32x4 sum = sh[0][rt][lane];
#pragma unroll
            for (int v = 1; v < kWaves; v++) sum += sh[v][rt][lane];
            *reinterpret_cast<f32x4 *>(&hs[r][16 * rt + 4 * g]) = sum;
        }
        __syncthreads();
        const float scale = a.scales ? a.scales[now] : 1.f;
        u32x4 part[RS][3];
#pragma unroll
        for (int k = 0; k < RS; k++) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const int rk = 32 * k + 8 * g + i;
                v[i] = rk < rank ? hs[r][min(rk, 16 * RT - 1)] * scale : 0.f;
            }
            split8(v, part[k]);
        }
        float v[16];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            f32x4 c{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < RS; k++) {
                const u32x4 b = first_columns(w[j][k], rank - 32 * k - 8 * g);
#pragma unroll
                for (int e = 0; e < 3; e++) c = mfma16x16x32(as_bf16x8(b), as_bf16x8(part[k][e]), c);
            }
#pragma unroll
            for (int i = 0; i < 4; i++) v[4 * j + i] = c[i];
        }
        if (mine) o.store(a, base, y, wide, have, v);
    }
}

// How a call is cut.  small: one launch.  Otherwise tiles of 64 tokens, whose adapters and whose columns
// of x are shared out over as many workgroups as the GPU has room for.
struct Split {
    bool small;
    int tiles, slots, splits;
};
int rank_tiles(int R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8; }
Split split_of(int64_t T, int K, int R)
{
    Split p;
    // one launch reads A again for each 512 outputs, in its fragments' order: us against two launches, 8
    // tokens, 7.6 : 9.5 at rank 16 and K 2048, 10.3 : 9.7 at 4096, 16.0 : 10.7 at 8192; 9.5 : 9.6 at rank
    // 32 and K 2048, 23 : 12 at rank 64 and K 4096; 16 tokens 8.5 : 10.1, 32 tokens 13.3 : 13.8
    p.small = T <= 32 && R <= 32 && rank_tiles(R) * K <= 4096;
    p.tiles = (int)((T + kTile - 1) / kTile);
    // a slot without an adapter costs its workgroups' start, an adapter more in a slot the others' time
    // again: 64 tokens of 64 adapters 36, 18 and 21 us with 4, 16 and 64; 2048 of 16 74, 60 and 70 with
    // 2, 4 and 8; 4099 in runs 43, 39 and 41 with 1, 2 and 4
    p.slots = p.tiles <= 4 ? 16 : p.tiles <= 32 ? 4 : 2;
    // parts of at least two stages, 256 workgroups in all or a few more
    p.splits = std::max(1, std::min({8, K / 512, (255 + p.tiles) / p.tiles}));
    return p;
}

template <int RT, int KC>
void launch_down(const LoraArgs &a, const Split &p, hipStream_t st)
{
    const int grid = grid_of((int64_t)p.tiles * p.splits);
    lora_down_kernel<RT, KC><<<(unsigned)(grid * p.slots), 512, 0, st>>>(a, grid, p.slots, p.splits);
}
template <int RS>
void launch_up(const LoraArgs &a, const Split &p, int vec, hipStream_t st)
{
    const int64_t chunks = (a.N + kCols - 1) / kCols;
    // rounds of a workgroup, which reads h once for all of them, as long as there are 256 of them:
    // 46, 39 and 41 us for 4099 tokens with 128, 256 and 512
    const int rounds = (int)std::max<int64_t>(1, std::min<int64_t>(chunks, p.tiles * chunks / 256));
    const int grid = grid_of(p.tiles * ((chunks + rounds - 1) / rounds));
    lora_up_kernel<RS><<<(unsigned)(grid * p.slots), 256, 0, st>>>(a, grid, p.slots, rounds, p.splits, vec);
}

}  // namespace

size_t lora_call_bytes(int64_t T, int K, int R)
{
    const Split p = split_of(T, K, R);
    return p.small ? 16 : std::max<size_t>(16, (size_t)p.splits * T * R * 4);
}

size_t lora_ws_bytes(int64_t T, int K, int R)
{
    // fewer tokens may be split over more workgroups: the largest over all batches up to T
    size_t most = 16;
    for (int64_t t = 1; t <= T; t = t < 1024 ? t + 1 : std::min(t + 64, std::max(T, t + 1))) most = std::max(most, lora_call_bytes(t, K, R));
    return most;
}

hipError_t launch_lora(const LoraArgs &a, hipStream_t st)
{
    const Split p = split_of(a.T, a.K, a.R);
    const int RT = rank_tiles(a.R);
    const auto wide = [](const void *q, int64_t ld, int fp32) { return ((uintptr_t)q | (uintptr_t)(ld * (fp32 ? 4 : 2))) % 16 == 0; };
    // rows whose pieces of 16 bytes are aligned, of base and of y; and whether y is base
    const int vec = (wide(a.base, a.ldb, a.base_fp32) ? 1 : 0) | (wide(a.y, a.ldy, a.y_fp32) ? 2 : 0) | (a.base == a.y ? 4 : 0);
    if (p.small) {
        const int parts = (a.N + kWaves * kUpCols - 1) / (kWaves * kUpCols), slots = std::min(16, a.T);
        const unsigned grid = (unsigned)((a.T + 15) / 16 * slots * parts);
        if (RT == 1)
            lora_small_kernel<1><<<grid, 64 * kWaves, 0, st>>>(a, slots, parts, vec);
        else
            lora_small_kernel<2><<<grid, 64 * kWaves, 0, st>>>(a, slots, parts, vec);
        return hipGetLastError();
    }
    if (RT == 1)
        launch_down<1, 256>(a, p, st);
    else if (RT == 2)
        launch_down<2, 128>(a, p, st);
    else if (RT == 4)
        launch_down<4, 256>(a, p, st);
    else
        launch_down<8, 128>(a, p, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.R <= 32)
        launch_up<1>(a, p, vec, st);
    else if (a.R <= 64)
        launch_up<2>(a, p, vec, st);
    else
        launch_up<4>(a, p, vec, st);
    return hipGetLastError();
}

}  // namespace flint
