// linear.hip -- a decode batch (T <= 64 tokens) through a linear layer with INT4 weights and
// group scales: y[t][n] = sum over groups of s[n][group] * sum_k q[n][k] x[t][k].
//
// Bound by the weights' bytes (0.5 + 2 / group per weight, each read once): codes stream from
// HBM straight into the MFMA B operand with 16-byte loads, 16 rows of W per tile, a batch of
// 4 KB per wave ahead of the one in use.  What competes with the bytes is the vector work of
// making codes bf16: 8 MFMA operands of 8 codes leave about 100 instructions per KB.  So a code
// becomes a bf16 by its bits alone: with its sign bit flipped it is q + 8, which below the
// exponent of 8 reads 8 + (q + 8) / 2 = q / 2 + 12 (exact; one shift and one and-or for two
// codes), and the 12 is taken out of the group's sum by starting it at -12 sum(x) rather than 0.
// The group's scale multiplies that fp32 sum, so no weight is ever rounded.  x is staged once
// per workgroup in LDS in the A operand's order, with its group sums.
#include "ops.h"

#include <algorithm>

namespace flint {

namespace {

constexpr int kWaves = 8;
// Eight codes of a word (sign bits flipped) as bf16 q / 2 + 12: columns (0, 4), (1, 5), (2, 6), (3, 7).
// (nibble, eight: those constants in registers, where one instruction takes both.)
__device__ __forceinline__ u32x4 codes_bf16(uint32_t q, uint32_t nibble, uint32_t eight)
{
    const uint32_t u = q ^ 0x88888888u;
    return u32x4{((u << 3) & nibble) | eight, ((u >> 1) & nibble) | eight, ((u >> 5) & nibble) | eight,
                 ((u >> 9) & nibble) | eight};
}
constexpr uint32_t kNibble = 0x00780078u, kEight = 0x41004100u;  // two bf16: mantissa bits 3 .. 6; 8.0
// Eight bf16 of x in that order of columns.
__device__ __forceinline__ u32x4 pair_columns(u32x4 v)
{
    return u32x4{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u), __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
                 __builtin_amdgcn_perm(v[3], v[1], 0x05040100u), __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
}

// Dwords of four lane groups transposed: afterwards dword j of lane group g is what dword g
// of lane group j was.
__device__ __forceinline__ void transpose4(u32x4 &d)
{
    auto swap32 = [](uint32_t &a, uint32_t &b) {
        auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
        a = r[0];
        b = r[1];
    };
    auto swap16 = [](uint32_t &a, uint32_t &b) {
        auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
        a = r[0];
        b = r[1];
    };
    uint32_t a = d[0], b = d[1], c = d[2], e = d[3];
    swap32(a, c);
    swap32(b, e);
    swap16(a, b);
    swap16(c, e);
    d = u32x4{a, b, c, e};
}

// LDS of a chunk of kc columns: x as [block][j][g][t] 16-byte pieces, then the group sums
// [group][t] times -12, t padded to TP (a power of two, so that offsets are constants).
__host__ __device__ constexpr int pad4(int t) { return t < 4 ? 4 : t; }
constexpr int chunk_bytes(int group, int TP) { return 128 * TP * 2 + (128 / group) * pad4(TP) * 4; }  // of 128 columns
constexpr int exchange_bytes(int TP, int RT) { return kWaves * RT * (TP < 16 ? 1 : TP / 16) * 1024; }
// A CU's 160 KB for two workgroups, or for one where the tokens are many and a chunk would be short.
constexpr int lds_budget(int TP) { return (TP < 32 ? 80 : 160) * 1024; }
constexpr int max_chunk(int group, int TP, int RT)
{
    return (lds_budget(TP) - exchange_bytes(TP, RT)) / chunk_bytes(group, TP) * 128;
}

// One workgroup: 8 / wpt times RT row tiles at a time (RT share the fragments of x that a wave reads
// from LDS), the K columns of each split over wpt = 2^lw waves.
// K is taken in chunks of kc columns whose x fits the LDS.
template <int GROUP, int TP, int RT>
__global__ __launch_bounds__(64 * kWaves) void linear_int4_kernel(LinearArgs a, int kc, int lw)
{
    constexpr int TT = TP < 16 ? 1 : TP / 16;  // token tiles
    constexpr int SPB = 128 / GROUP;           // scales per block
    constexpr int kBatch = 4 / RT;             // 128-column blocks of a batch
    extern __shared__ __attribute__((aligned(16))) uint8_t xs[];
    float *const sums = reinterpret_cast<float *>(xs + (size_t)kc * TP * 2);
    __shared__ f32x4 red[kWaves][RT * TT][64];
    static_assert(sizeof red == exchange_bytes(TP, RT), "counted by the host");
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n16 = lane & 15, g = lane >> 4;
    const int wpt = 1 << lw, per = kWaves >> lw;  // row tiles of a workgroup
    const int sub = wave >> lw, part = wave & (wpt - 1);
    const int tiles = (a.N + 16 * RT - 1) / (16 * RT), groups = (tiles + per - 1) >> (3 - lw);
    const int T = a.T;
    uint32_t nibble = kNibble, eight = kEight;
    asm volatile("" : "+v"(nibble));
    asm volatile("" : "+s"(eight));
    const size_t srow = (size_t)a.K / GROUP;

    // The wave's batches in order: of a chunk its part of the blocks, chunk by chunk, row group by
    // row group.
    auto blocks = [&](int k0) { return min(kc, a.K - k0) >> 7; };
    auto first = [&](int k0) { return (blocks(k0) * part) >> lw; };
    auto end = [&](int k0) { return (blocks(k0) * (part + 1)) >> lw; };
    struct Pos {
        int grp, k0, b;
    };
    auto settle = [&](Pos &p) {  // to the next batch that exists
        while (p.grp < groups && p.b >= end(p.k0)) {
            p.k0 += kc;
            if (p.k0 >= a.K) {
                p.k0 = 0;
                p.grp += gridDim.x;
            }
            p.b = first(p.k0);
        }
    };
    u32x4 w[RT][kBatch], nw[RT][kBatch];
    uint16_t sc[RT][kBatch * SPB], nsc[RT][kBatch * SPB];
    auto load = [&](const Pos &p) {  // into nw, nsc
        if (p.grp >= groups) return;
        const int n = end(p.k0) - p.b;
#pragma unroll
        for (int r = 0; r < RT; r++) {
            const int row = min(((p.grp * per + sub) * RT + r) * 16 + n16, a.N - 1);
            const uint8_t *wr = a.codes + (size_t)row * (a.K / 2) + p.k0 / 2 + 64 * p.b + 16 * g;
            const uint16_t *sr = a.scales + (size_t)row * srow + (p.k0 / 128 + p.b) * SPB;
            if (n >= kBatch) {
#pragma unroll
                for (int i = 0; i < kBatch; i++)
                    nw[r][i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(wr + 64 * i));
                __builtin_memcpy(nsc[r], sr, sizeof nsc[r]);
            } else {
#pragma unroll
                for (int i = 0; i < kBatch; i++)
                    if (i < n) {
                        nw[r][i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(wr + 64 * i));
#pragma unroll
                        for (int u = 0; u < SPB; u++) nsc[r][i * SPB + u] = sr[i * SPB + u];
                    }
            }
        }
    };
    Pos pos{(int)blockIdx.x, 0, first(0)};
    settle(pos);
    load(pos);  // on its way while x is staged

    int staged = -1;  // first column of the chunk in LDS
    for (int grp = blockIdx.x; grp < groups; grp += gridDim.x) {
        f32x4 acc[RT][TT];
#pragma unroll
        for (int r = 0; r < RT; r++)
#pragma unroll
            for (int tt = 0; tt < TT; tt++) acc[r][tt] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int k0 = 0; k0 < a.K; k0 += kc) {
            if (staged != k0) {
                if (staged >= 0) __syncthreads();  // the previous chunk has been read
                const int p8 = blocks(k0) * 16;    // pieces of a token
                for (int i = tid; i < T * p8; i += 64 * kWaves) {
                    const int t = i / p8, c8 = i % p8, blk = c8 / 16, p = c8 % 16;
                    // piece p = columns 8 p of the block: (g, j) = (p / 4, p % 4), and (p % 4, p / 4)
                    // where the codes are transposed
                    const int pg = GROUP == 128 ? p / 4 : p % 4, pj = GROUP == 128 ? p % 4 : p / 4;
                    const u32x4 v = *reinterpret_cast<const u32x4 *>(a.x + t * a.ldx + k0 + 8 * c8);
                    *reinterpret_cast<u32x4 *>(xs + ((size_t)((blk * 4 + pj) * 4 + pg) * TP + t) * 16) = pair_columns(v);
                    float sum = 0.f;  // of the piece, then of the group's pieces (neighbouring lanes)
#pragma unroll
                    for (int e = 0; e < 4; e++) sum += bf2f(v[e] & 0xffffu) + bf2f(v[e] >> 16);
#pragma unroll
                    for (int m = 1; m < GROUP / 8; m *= 2) sum += __shfl_xor(sum, m);
                    if (p % (GROUP / 8) == 0) sums[(c8 / (GROUP / 8)) * pad4(TP) + t] = -12.f * sum;
                }
                __syncthreads();
                staged = k0;
            }
            const int be = end(k0);
            for (int b = first(k0); b < be; b += kBatch) {
#pragma unroll
                for (int r = 0; r < RT; r++) {
#pragma unroll
                    for (int i = 0; i < kBatch; i++) w[r][i] = nw[r][i];
#pragma unroll
                    for (int i = 0; i < kBatch * SPB; i++) sc[r][i] = nsc[r][i];
                }
                pos.b += kBatch;
                settle(pos);
                load(pos);
                const uint8_t *xb = xs + (size_t)b * 256 * TP + g * (16 * TP);
                const float *sb = sums + b * SPB * pad4(TP);
#pragma unroll
                for (int i = 0; i < kBatch; i++) {
                    if (b + i >= be) break;
                    if (GROUP != 128)
#pragma unroll
                        for (int r = 0; r < RT; r++) transpose4(w[r][i]);
#pragma unroll
                    for (int u = 0; u < SPB; u++) {
                        f32x4 p[RT][TT];
#pragma unroll
                        for (int tt = 0; tt < TT; tt++) {  // rows past T hold anything; their results are not written
                            p[0][tt] = *reinterpret_cast<const f32x4 *>(sb + (i * SPB + u) * pad4(TP) +
                                                                        min(16 * tt + 4 * g, pad4(TP) - 4));
#pragma unroll
                            for (int r = 1; r < RT; r++) p[r][tt] = p[0][tt];
                        }
#pragma unroll
                        for (int jj = 0; jj < 4 / SPB; jj++) {
                            const int j = u * (4 / SPB) + jj;
                            bf16x8 wb[RT];
#pragma unroll
                            for (int r = 0; r < RT; r++) wb[r] = as_bf16x8(codes_bf16(w[r][i][j], nibble, eight));
#pragma unroll
                            for (int tt = 0; tt < TT; tt++) {
                                const bf16x8 xv = as_bf16x8(*reinterpret_cast<const u32x4 *>(
                                    xb + (i * 16 + j * 4) * (16 * TP) + min(16 * tt + n16, TP - 1) * 16));
#pragma unroll
                                for (int r = 0; r < RT; r++) p[r][tt] = mfma16x16x32(xv, wb[r], p[r][tt]);
                            }
                        }
#pragma unroll
                        for (int r = 0; r < RT; r++) {
                            const float s = bf2f(sc[r][i * SPB + u]);
#pragma unroll
                            for (int tt = 0; tt < TT; tt++)
#pragma unroll
                                for (int e = 0; e < 4; e++) acc[r][tt][e] = fmaf(p[r][tt][e], s, acc[r][tt][e]);
                        }
                    }
                }
            }
        }
        if (wpt > 1) {  // the parts of a row tile meet in LDS, summed in wave order
#pragma unroll
            for (int r = 0; r < RT; r++)
#pragma unroll
                for (int tt = 0; tt < TT; tt++) red[wave][r * TT + tt][lane] = acc[r][tt];
            __syncthreads();
            if (part == 0)
#pragma unroll
                for (int r = 0; r < RT; r++)
#pragma unroll
                    for (int tt = 0; tt < TT; tt++) {
                        for (int q = 1; q < wpt; q++) {
                            const f32x4 v = red[wave + q][r * TT + tt][lane];
#pragma unroll
                            for (int e = 0; e < 4; e++) acc[r][tt][e] += v[e];
                        }
                    }
            __syncthreads();
        }
        if (part) continue;
#pragma unroll
        for (int r = 0; r < RT; r++) {
            const int n = ((grp * per + sub) * RT + r) * 16 + n16;
            if (n >= a.N) continue;
#pragma unroll
            for (int tt = 0; tt < TT; tt++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int t = 16 * tt + 4 * g + e;
                    if (t >= T) continue;
                    float v = acc[r][tt][e] * 2.f;
                    if (a.residual) v += bf2f(a.residual[t * a.ldr + n]);
                    if (a.y_fp32)
                        ((float *)a.y)[t * a.ldy + n] = v;
                    else
                        ((uint16_t *)a.y)[t * a.ldy + n] = (uint16_t)f2bf(v);
                }
        }
    }
}

template <int GROUP, int TP, int RT>
hipError_t launch_group(const LinearArgs &a, hipStream_t st)
{
    const int kc = std::min(a.K, max_chunk(GROUP, TP, RT));
    static_assert(max_chunk(GROUP, TP, RT) >= 128, "a chunk fits");
    const int tiles = (a.N + 16 * RT - 1) / (16 * RT);
    // Enough waves to cover the GPU, eight per CU: K is split over up to 8 of them where rows are few
    // (twice as many waves: 2048 x 5120, T = 8, 8.6 us instead of 7.2, each workgroup staging x).
    int lw = 3;
    while (lw > 0 && (tiles << lw) > 2048) lw--;
    static_assert(kWaves == 8, "a workgroup's waves in powers of two");
    const int groups = (tiles + (kWaves >> lw) - 1) / (kWaves >> lw);
    const size_t lds = (size_t)kc / 128 * chunk_bytes(GROUP, TP);
    linear_int4_kernel<GROUP, TP, RT><<<std::min(groups, TP < 32 ? 512 : 256), 64 * kWaves, lds, st>>>(a, kc, lw);
    return hipGetLastError();
}
template <int TP, int RT>
hipError_t launch_rt(const LinearArgs &a, hipStream_t st)
{
    return a.group == 128  ? launch_group<128, TP, RT>(a, st)
           : a.group == 64 ? launch_group<64, TP, RT>(a, st)
                           : launch_group<32, TP, RT>(a, st);
}
template <int TP>
hipError_t launch_tp(const LinearArgs &a, hipStream_t st)
{
    // Two row tiles to a wave where reading x from LDS bounds it and rows are many (64 tokens, 2048 x
    // 131072: 91 us, one 125; 4096 x 4096: 48 us, one 38; 32 tokens, 2048 x 131072: 58 us, one 49).
    if constexpr (TP == 64)
        if (a.N >= 16384) return launch_rt<TP, 2>(a, st);
    return launch_rt<TP, 1>(a, st);
}

}  // namespace

hipError_t launch_linear_int4(const LinearArgs &a, hipStream_t st)
{
    return a.T == 1    ? launch_tp<1>(a, st)
           : a.T <= 4  ? launch_tp<4>(a, st)
           : a.T <= 8  ? launch_tp<8>(a, st)
           : a.T <= 16 ? launch_tp<16>(a, st)
           : a.T <= 32 ? launch_tp<32>(a, st)
                       : launch_tp<64>(a, st);
}

}  // namespace flint
