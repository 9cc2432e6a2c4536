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
constexpr int kBatch = 4;           // 128-column blocks of a batch
constexpr int kXBytes = 64 * 1024;  // LDS for x: one K chunk of all T tokens

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
constexpr size_t lds_bytes(int kc, int group, int TP) { return (size_t)kc * TP * 2 + (size_t)(kc / group) * pad4(TP) * 4; }

// One workgroup: 8 / wpt row tiles at a time, the K columns of each split over wpt = 2^lw waves.
// K is taken in chunks of kc columns whose x fits the LDS.
template <int GROUP, int TP>
__global__ __launch_bounds__(64 * kWaves) void linear_int4_kernel(LinearArgs a, int kc, int lw)
{
    constexpr int TT = TP < 16 ? 1 : TP / 16;  // token tiles
    constexpr int SPB = 128 / GROUP;           // scales per block
    extern __shared__ __attribute__((aligned(16))) uint8_t xs[];
    float *const sums = reinterpret_cast<float *>(xs + (size_t)kc * TP * 2);
    __shared__ f32x4 red[kWaves][TT][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n16 = lane & 15, g = lane >> 4;
    const int wpt = 1 << lw, per = kWaves >> lw;  // row tiles of a workgroup
    const int sub = wave >> lw, part = wave & (wpt - 1);
    const int tiles = (a.N + 15) / 16, groups = (tiles + per - 1) >> (3 - lw);
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
    u32x4 w[kBatch], nw[kBatch];
    uint16_t sc[kBatch * SPB], nsc[kBatch * SPB];
    auto load = [&](const Pos &p) {  // into nw, nsc
        if (p.grp >= groups) return;
        const int row = min((p.grp * per + sub) * 16 + n16, a.N - 1), n = end(p.k0) - p.b;
        const uint8_t *wr = a.codes + (size_t)row * (a.K / 2) + p.k0 / 2 + 64 * p.b + 16 * g;
        const uint16_t *sr = a.scales + (size_t)row * srow + (p.k0 / 128 + p.b) * SPB;
        if (n >= kBatch) {
#pragma unroll
            for (int i = 0; i < kBatch; i++)
                nw[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(wr + 64 * i));
            __builtin_memcpy(nsc, sr, sizeof nsc);
        } else {
#pragma unroll
            for (int i = 0; i < kBatch; i++)
                if (i < n) {
                    nw[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(wr + 64 * i));
#pragma unroll
                    for (int u = 0; u < SPB; u++) nsc[i * SPB + u] = sr[i * SPB + u];
                }
        }
    };
    Pos pos{(int)blockIdx.x, 0, first(0)};
    settle(pos);
    load(pos);  // on its way while x is staged

    int staged = -1;  // first column of the chunk in LDS
    for (int grp = blockIdx.x; grp < groups; grp += gridDim.x) {
        f32x4 acc[TT];
#pragma unroll
        for (int tt = 0; tt < TT; tt++) acc[tt] = f32x4{0.f, 0.f, 0.f, 0.f};
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
                for (int i = 0; i < kBatch; i++) w[i] = nw[i];
#pragma unroll
                for (int i = 0; i < kBatch * SPB; i++) sc[i] = nsc[i];
                pos.b += kBatch;
                settle(pos);
                load(pos);
                const uint8_t *xb = xs + (size_t)b * 256 * TP + g * (16 * TP);
                const float *sb = sums + b * SPB * pad4(TP);
#pragma unroll
                for (int i = 0; i < kBatch; i++) {
                    if (b + i >= be) break;
                    if (GROUP != 128) transpose4(w[i]);
#pragma unroll
                    for (int u = 0; u < SPB; u++) {
                        f32x4 p[TT];
#pragma unroll
                        for (int tt = 0; tt < TT; tt++)  // rows past T hold anything; their results are not written
                            p[tt] = *reinterpret_cast<const f32x4 *>(sb + (i * SPB + u) * pad4(TP) +
                                                                     min(16 * tt + 4 * g, pad4(TP) - 4));
#pragma unroll
                        for (int jj = 0; jj < 4 / SPB; jj++) {
                            const int j = u * (4 / SPB) + jj;
                            const bf16x8 wb = as_bf16x8(codes_bf16(w[i][j], nibble, eight));
#pragma unroll
                            for (int tt = 0; tt < TT; tt++) {
                                const u32x4 xv = *reinterpret_cast<const u32x4 *>(
                                    xb + (i * 16 + j * 4) * (16 * TP) + min(16 * tt + n16, TP - 1) * 16);
                                p[tt] = mfma16x16x32(as_bf16x8(xv), wb, p[tt]);
                            }
                        }
                        const float s = bf2f(sc[i * SPB + u]);
#pragma unroll
                        for (int tt = 0; tt < TT; tt++)
#pragma unroll
                            for (int e = 0; e < 4; e++) acc[tt][e] = fmaf(p[tt][e], s, acc[tt][e]);
                    }
                }
            }
        }
        if (wpt > 1) {  // the parts of a row tile meet in LDS, summed in wave order
#pragma unroll
            for (int tt = 0; tt < TT; tt++) red[wave][tt][lane] = acc[tt];
            __syncthreads();
            if (part == 0)
#pragma unroll
                for (int tt = 0; tt < TT; tt++) {
                    for (int q = 1; q < wpt; q++) {
                        const f32x4 v = red[wave + q][tt][lane];
#pragma unroll
                        for (int e = 0; e < 4; e++) acc[tt][e] += v[e];
                    }
                }
            __syncthreads();
        }
        const int n = (grp * per + sub) * 16 + n16;
        if (part == 0 && n < a.N) {
#pragma unroll
            for (int tt = 0; tt < TT; tt++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int t = 16 * tt + 4 * g + e;
                    if (t >= T) continue;
                    float v = acc[tt][e] * 2.f;
                    if (a.residual) v += bf2f(a.residual[t * a.ldr + n]);
                    if (a.y_fp32)
                        ((float *)a.y)[t * a.ldy + n] = v;
                    else
                        ((uint16_t *)a.y)[t * a.ldy + n] = (uint16_t)f2bf(v);
                }
        }
    }
}

template <int TP>
hipError_t launch_tp(const LinearArgs &a, hipStream_t st)
{
    const int kc = std::min(a.K, kXBytes / (2 * TP) / 128 * 128);
    const int tiles = (a.N + 15) / 16;
    // enough waves to cover the GPU: K is split over up to 8 waves where rows are few
    int lw = 3;
    while (lw > 0 && (tiles << lw) > 4096) lw--;
    static_assert(kWaves == 8, "a workgroup's waves in powers of two");
    const int groups = (tiles + (kWaves >> lw) - 1) / (kWaves >> lw);
    const size_t lds = lds_bytes(kc, a.group, TP);
    const dim3 grid(std::min(groups, 512)), block(64 * kWaves);
    if (a.group == 128)
        linear_int4_kernel<128, TP><<<grid, block, lds, st>>>(a, kc, lw);
    else if (a.group == 64)
        linear_int4_kernel<64, TP><<<grid, block, lds, st>>>(a, kc, lw);
    else
        linear_int4_kernel<32, TP><<<grid, block, lds, st>>>(a, kc, lw);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_int4(const LinearArgs &a, hipStream_t st)
{
    return a.T == 1   ? launch_tp<1>(a, st)
           : a.T <= 4 ? launch_tp<4>(a, st)
           : a.T <= 8 ? launch_tp<8>(a, st)
           : a.T <= 16 ? launch_tp<16>(a, st)
           : a.T <= 32 ? launch_tp<32>(a, st)
                       : launch_tp<64>(a, st);
}

}  // namespace flint
