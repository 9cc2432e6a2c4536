// linear.hip -- a decode batch (T <= 64 tokens) through a linear layer with INT4 weights and
// group scales: y[t][n] = sum over groups of s[n][group] * sum_k q[n][k] x[t][k].
//
// Bound by the weights' bytes (0.5 + 2 / group per weight, each read once): codes stream from
// HBM straight into the MFMA B operand with 16-byte loads, 16 rows of W per tile, and are
// made exact bf16 integers / 16 on the way (v_cvt_off_f32_i4 gives q / 16 from a nibble); the
// group's scale multiplies the group's fp32 sum, so no weight is ever rounded.  x is staged
// once per workgroup in LDS in the A operand's order.
#include "ops.h"

#include <algorithm>

namespace flint {

namespace {

constexpr int kWaves = 8;
constexpr int kBatch = 4;                 // 128-column blocks a wave has in flight
constexpr int kXBytes = 64 * 1024;        // LDS for x: one K chunk of all T tokens

// Eight signed nibbles of a word as bf16 q / 16 (exact), columns in order.
__device__ __forceinline__ u32x4 nibbles_bf16(uint32_t q)
{
    const uint32_t h = q >> 4;
    auto cvt = [](uint32_t v, int byte) { return __float_as_uint(__builtin_amdgcn_cvt_off_f32_i4((int)(v >> (8 * byte)))); };
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; i++) r[i] = __builtin_amdgcn_perm(cvt(h, i), cvt(q, i), 0x07060302u);
    return r;
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

// One workgroup: 8 / wpt row tiles at a time, the K columns of each split over wpt waves.
// TT token tiles of 16.  K is taken in chunks of kc columns whose x fits the LDS.
template <int GROUP, int TT>
__global__ __launch_bounds__(64 * kWaves) void linear_int4_kernel(LinearArgs a, int kc, int wpt)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t xs[];  // [block][j][g][t] 16-byte pieces
    __shared__ f32x4 red[kWaves][TT][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n16 = lane & 15, g = lane >> 4;
    const int per = kWaves / wpt;                       // row tiles of a workgroup
    const int sub = wave / wpt, part = wave % wpt;
    const int tiles = (a.N + 15) / 16, groups = (tiles + per - 1) / per;
    const int T = a.T;
    constexpr int SPB = 128 / GROUP;                    // scales per block
    const size_t srow = (size_t)a.K / GROUP;
    int staged = -1;                                    // first column of the chunk in LDS
    for (int grp = blockIdx.x; grp < groups; grp += gridDim.x) {
        const int tile = grp * per + sub;
        const bool live = tile < tiles;
        const int row = live ? min(tile * 16 + n16, a.N - 1) : 0;
        const uint8_t *wr = a.codes + (size_t)row * (a.K / 2) + 16 * g;
        const uint16_t *sr = a.scales + (size_t)row * srow;
        f32x4 acc[TT];
#pragma unroll
        for (int tt = 0; tt < TT; tt++) acc[tt] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int k0 = 0; k0 < a.K; k0 += kc) {
            const int cols = min(kc, a.K - k0), nb = cols / 128;
            if (staged != k0) {
                if (staged >= 0) __syncthreads();  // the previous chunk has been read
                for (int i = tid; i < T * (cols / 8); i += 64 * kWaves) {
                    const int t = i / (cols / 8), c8 = i % (cols / 8), blk = c8 / 16, p = c8 % 16;
                    // piece p = columns 8 p of the block: (g, j) = (p / 4, p % 4), and (p % 4, p / 4)
                    // where the codes are transposed
                    const int pg = GROUP == 128 ? p / 4 : p % 4, pj = GROUP == 128 ? p % 4 : p / 4;
                    *reinterpret_cast<u32x4 *>(xs + ((size_t)((blk * 4 + pj) * 4 + pg) * T + t) * 16) =
                        *reinterpret_cast<const u32x4 *>(a.x + t * a.ldx + k0 + 8 * c8);
                }
                __syncthreads();
                staged = k0;
            }
            if (!live) continue;
            const int b0 = nb * part / wpt, b1 = nb * (part + 1) / wpt;
            for (int b = b0; b < b1; b += kBatch) {
                u32x4 w[kBatch];
                float s[kBatch][SPB];
#pragma unroll
                for (int i = 0; i < kBatch; i++)
                    if (b + i < b1) {
                        w[i] = *reinterpret_cast<const u32x4 *>(wr + (k0 + 128 * (b + i)) / 2);
#pragma unroll
                        for (int u = 0; u < SPB; u++)
                            s[i][u] = bf2f(sr[(k0 / 128 + b + i) * SPB + u]);
                    }
#pragma unroll
                for (int i = 0; i < kBatch; i++)
                    if (b + i < b1) {
                        if (GROUP != 128) transpose4(w[i]);
#pragma unroll
                        for (int u = 0; u < SPB; u++) {
                            f32x4 p[TT];
#pragma unroll
                            for (int tt = 0; tt < TT; tt++) p[tt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int jj = 0; jj < 4 / SPB; jj++) {
                                const int j = u * (4 / SPB) + jj;
                                const bf16x8 wb = as_bf16x8(nibbles_bf16(w[i][j]));
#pragma unroll
                                for (int tt = 0; tt < TT; tt++) {
                                    // rows past T repeat the last token; their results are not written
                                    const int t = min(16 * tt + n16, T - 1);
                                    const u32x4 xv = *reinterpret_cast<const u32x4 *>(
                                        xs + ((size_t)(((b + i) * 4 + j) * 4 + g) * T + t) * 16);
                                    p[tt] = mfma16x16x32(as_bf16x8(xv), wb, p[tt]);
                                }
                            }
#pragma unroll
                            for (int tt = 0; tt < TT; tt++)
#pragma unroll
                                for (int e = 0; e < 4; e++) acc[tt][e] = fmaf(p[tt][e], s[i][u], acc[tt][e]);
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
        const int n = tile * 16 + n16;
        if (part == 0 && live && n < a.N) {
#pragma unroll
            for (int tt = 0; tt < TT; tt++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int t = 16 * tt + 4 * g + e;
                    if (t >= T) continue;
                    float v = acc[tt][e] * 16.f;
                    if (a.residual) v += bf2f(a.residual[t * a.ldr + n]);
                    if (a.y_fp32)
                        ((float *)a.y)[t * a.ldy + n] = v;
                    else
                        ((uint16_t *)a.y)[t * a.ldy + n] = (uint16_t)f2bf(v);
                }
        }
    }
}

template <int TT>
hipError_t launch_tt(const LinearArgs &a, hipStream_t st)
{
    const int kc = std::min(a.K, kXBytes / (2 * a.T) / 128 * 128);
    const int tiles = (a.N + 15) / 16;
    // enough waves to cover the GPU: K is split over up to 8 waves where rows are few
    int wpt = 8;
    while (wpt > 1 && tiles * wpt > 4096) wpt /= 2;
    const int groups = (tiles + kWaves / wpt - 1) / (kWaves / wpt);
    const size_t lds = (size_t)a.T * kc * 2;
    const dim3 grid(std::min(groups, 512)), block(64 * kWaves);
    if (a.group == 128)
        linear_int4_kernel<128, TT><<<grid, block, lds, st>>>(a, kc, wpt);
    else if (a.group == 64)
        linear_int4_kernel<64, TT><<<grid, block, lds, st>>>(a, kc, wpt);
    else
        linear_int4_kernel<32, TT><<<grid, block, lds, st>>>(a, kc, wpt);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_int4(const LinearArgs &a, hipStream_t st)
{
    return a.T <= 16 ? launch_tt<1>(a, st) : a.T <= 32 ? launch_tt<2>(a, st) : launch_tt<4>(a, st);
}

}  // namespace flint
