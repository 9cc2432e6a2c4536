// linear.hip -- a decode batch (T <= 64 tokens) through a linear layer with INT4 weights and
// group scales: y[t][n] = sum over groups of s[n][group] * sum_k q[n][k] x[t][k].
//
// Bound by the weights' bytes (0.5 + 2 / group per weight, each read once): codes stream from
// HBM straight into the MFMA B operand with 16-byte loads, 16 rows of W per tile, a batch per
// wave ahead of the one in use.  What competes with the bytes is the vector work of making
// codes bf16: 15 instructions for 8 codes, half of them at half rate.  A code becomes q
// itself, exactly, so a group's products are exact and its fp32 sum holds nothing that is not in
// the result.  (A bf16 with an offset of 12 takes 9 instructions for 8, but the offset times x
// stays in the sum until it is taken out again: an x of some thousands left 1e-3 in rows whose codes
// there are zero.  64 tokens, 2048 x 131072: 75 us so, exact 85; one token 30, exact 31.)
// The group's scale multiplies that fp32 sum, so no weight is ever rounded.
//
// Two kernels.  With few rows of W every wave has its own part of K and reads that part of x for
// itself; with many, whole workgroups need the same x and share it in LDS.
// Codes are loaded into the caches: a row of 64 (2 k + 1) bytes ends inside a cache line, whose other
// half the next batch takes (with loads past the caches 36295 x 3968: 26 us, so 22).
// Measured: one token, 2048 x 130953, groups of 64, fp32 out: 31.3 us, 4.6 TB/s of weights; 8
// tokens, 2048 x 5120: 5.3 us; 64 tokens, 4096 x 4096: 11.7 us; 64 tokens, 2048 x 131072: 86 us,
// where the vector work no longer hides behind bytes.
#include "ops.h"

#include <algorithm>
#include <type_traits>

namespace flint {

namespace {

constexpr int kWaves = 8;
constexpr int kNarrow = 1536;    // row tiles up to which K is split over a workgroup's waves
constexpr int kNarrowOne = 256;  // row tiles up to which each is a workgroup of its own
// Eight codes of a word as bf16, exactly q: columns (0, 2), (4, 6), (1, 3), (5, 7).  All eight become
// magnitudes 0 .. 8 at once, then bytes magnitude | sign << 7, which as E4M3 count in steps of 2^-9
// (up to 15: the subnormals and the binade above them); the conversion's scale takes that out.
__device__ __forceinline__ u32x4 codes_bf16(uint32_t q)
{
    const uint32_t sign = q & 0x88888888u, one = sign >> 3;
    const uint32_t mag = (q ^ (sign | (sign - one))) + one;  // 16 - q where negative
    const uint32_t even = (mag & 0x0f0f0f0fu) | ((sign << 4) & 0xf0f0f0f0u), odd = ((mag >> 4) & 0x0f0f0f0fu) | (sign & 0xf0f0f0f0u);
    auto two = [](uint32_t b, auto half) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.f, decltype(half)::value));
    };
    return u32x4{two(even, std::false_type{}), two(even, std::true_type{}), two(odd, std::false_type{}), two(odd, std::true_type{})};
}
// Eight bf16 of x in that order of columns.
__device__ __forceinline__ u32x4 pair_columns(u32x4 v)
{
    return u32x4{__builtin_amdgcn_perm(v[1], v[0], 0x05040100u), __builtin_amdgcn_perm(v[3], v[2], 0x05040100u),
                 __builtin_amdgcn_perm(v[1], v[0], 0x07060302u), __builtin_amdgcn_perm(v[3], v[2], 0x07060302u)};
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

// Results of row n of W for tokens t .. t + 3.
__device__ __forceinline__ void store(const LinearArgs &a, int n, int t, f32x4 v)
{
    if (n >= a.N) return;
#pragma unroll
    for (int e = 0; e < 4; e++) {
        if (t + e >= a.T) break;
        float y = v[e];
        if (a.residual) y += bf2f(a.residual[(t + e) * a.ldr + n]);
        if (a.y_fp32)
            ((float *)a.y)[(t + e) * a.ldy + n] = y;
        else
            ((uint16_t *)a.y)[(t + e) * a.ldy + n] = (uint16_t)f2bf(y);
    }
}

// Orders a wave's own LDS accesses for the compiler; the hardware keeps them in order.
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// ---- few rows of W ------------------------------------------------------------------------
// A workgroup takes RT row tiles, its waves an eighth of K each, and each wave reads its own part of
// x, a block of 128 columns ahead: 4 rows of 256 bytes with an instruction, turned into the A
// operand's order in LDS of its own (piece p of row n at p ^ n: no bank is asked twice).  Loads
// straight into that order ask for 64 cache lines each and were the bound (64 tokens, 8320 x 2048: 33
// us).
template <int GROUP, int TP, int RT>
__global__ __launch_bounds__(64 * kWaves) void linear_narrow_kernel(LinearArgs a)
{
    constexpr int TT = TP < 16 ? 1 : TP / 16;          // token tiles
    constexpr int Q = TP < 16 ? (TP + 3) / 4 : 4;      // four-row loads of a tile
    constexpr int SPB = 128 / GROUP;    // scales per block of 128 columns
    constexpr int kX = TT * 256, kRed = RT * TT * 64;  // 16-byte pieces of a wave: its block of x, then its sums
    __shared__ u32x4 lds[kWaves][kX > kRed ? kX : kRed];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n16 = lane & 15, g = lane >> 4, row0 = blockIdx.x * (16 * RT);
    const int nb = a.K / 128, b0 = nb * wave / kWaves, b1 = nb * (wave + 1) / kWaves;
    const size_t srow = (size_t)a.K / GROUP;
    u32x4 w[RT], x[TT][4], nw[RT], nx[TT][Q];
    uint16_t sc[RT][SPB], nsc[RT][SPB];
    auto load = [&](int b) {  // block b into nw, nsc, nx
        if (b >= b1) return;
#pragma unroll
        for (int r = 0; r < RT; r++) {
            const int row = min(row0 + 16 * r + n16, a.N - 1);
            nw[r] = *reinterpret_cast<const u32x4 *>(a.codes + (size_t)row * (a.K / 2) + 64 * b + 16 * g);
            __builtin_memcpy(nsc[r], a.scales + row * srow + b * SPB, sizeof nsc[r]);
        }
#pragma unroll
        for (int tt = 0; tt < TT; tt++)
#pragma unroll
            for (int q = 0; q < Q; q++)  // rows past T hold anything; their results are not written
                nx[tt][q] = *reinterpret_cast<const u32x4 *>(a.x + min(16 * tt + 4 * q + g, a.T - 1) * a.ldx + 128 * b + 8 * n16);
    };
    f32x4 acc[RT][TT];
#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int tt = 0; tt < TT; tt++) acc[r][tt] = f32x4{0.f, 0.f, 0.f, 0.f};
    load(b0);
    for (int b = b0; b < b1; b++) {
#pragma unroll
        for (int r = 0; r < RT; r++) {
            w[r] = nw[r];
#pragma unroll
            for (int u = 0; u < SPB; u++) sc[r][u] = nsc[r][u];
        }
        wave_fence();  // the last block has been read
#pragma unroll
        for (int tt = 0; tt < TT; tt++)
#pragma unroll
            for (int q = 0; q < Q; q++) lds[wave][tt * 256 + (4 * q + g) * 16 + (n16 ^ (4 * q + g))] = pair_columns(nx[tt][q]);
        wave_fence();
        load(b + 1);
#pragma unroll
        for (int tt = 0; tt < TT; tt++)
#pragma unroll
            for (int j = 0; j < 4; j++) x[tt][j] = lds[wave][tt * 256 + n16 * 16 + ((GROUP == 128 ? 4 * g + j : 4 * j + g) ^ n16)];
        if (GROUP != 128)
#pragma unroll
            for (int r = 0; r < RT; r++) transpose4(w[r]);
#pragma unroll
        for (int u = 0; u < SPB; u++) {
            f32x4 p[RT][TT];
#pragma unroll
            for (int r = 0; r < RT; r++)
#pragma unroll
                for (int tt = 0; tt < TT; tt++) p[r][tt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int jj = 0; jj < 4 / SPB; jj++) {
                const int j = u * (4 / SPB) + jj;
#pragma unroll
                for (int r = 0; r < RT; r++) {
                    const bf16x8 wb = as_bf16x8(codes_bf16(w[r][j]));
#pragma unroll
                    for (int tt = 0; tt < TT; tt++) p[r][tt] = mfma16x16x32(as_bf16x8(x[tt][j]), wb, p[r][tt]);
                }
            }
#pragma unroll
            for (int r = 0; r < RT; r++) {
                const float s = bf2f(sc[r][u]);
#pragma unroll
                for (int tt = 0; tt < TT; tt++)
#pragma unroll
                    for (int e = 0; e < 4; e++) acc[r][tt][e] = fmaf(p[r][tt][e], s, acc[r][tt][e]);
            }
        }
    }
    // The waves' sums meet in LDS, added in wave order.
    wave_fence();
#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int tt = 0; tt < TT; tt++)
            lds[wave][(r * TT + tt) * 64 + lane] = __builtin_bit_cast(u32x4, acc[r][tt]);
    __syncthreads();
    for (int q = wave; q < RT * TT; q += kWaves) {
        f32x4 v = __builtin_bit_cast(f32x4, lds[0][q * 64 + lane]);
#pragma unroll
        for (int k = 1; k < kWaves; k++) {
            const f32x4 o = __builtin_bit_cast(f32x4, lds[k][q * 64 + lane]);
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] += o[e];
        }
        store(a, row0 + 16 * (q / TT) + n16, 16 * (q % TT) + 4 * g, v);
    }
}

// ---- many rows of W -----------------------------------------------------------------------
// LDS of a chunk of kc columns: x as [block][j][g][t] 16-byte pieces, t padded to TP (a power of two,
// so that offsets are constants).
constexpr int chunk_bytes(int TP) { return 128 * TP * 2; }  // of 128 columns
// A CU's 160 KB for two workgroups, or for one where the tokens are many and a chunk would be short.
constexpr int lds_budget(int TP) { return (TP < 32 ? 80 : 160) * 1024; }
constexpr int exchange_bytes(int KS) { return KS > 1 ? kWaves * 1024 : 0; }
constexpr int max_chunk(int TP, int KS) { return (lds_budget(TP) - exchange_bytes(KS)) / chunk_bytes(TP) * 128; }

// Where token t lies in piece p of a block: the pieces of one token, written by neighbouring lanes,
// on distinct banks.
template <int TP>
__device__ __forceinline__ int slot_of(int t, int p) { return t ^ (p & (TP < 16 ? TP - 1 : 15)); }

// KS waves take RT row tiles (which share the fragments of x that they read from LDS) and a KS-th of
// K each, in chunks of kc columns whose x fits the LDS.
template <int GROUP, int TP, int RT, int KS>
__global__ __launch_bounds__(64 * kWaves, TP < 32 ? 4 : 2) void linear_int4_kernel(LinearArgs a, int kc)
{
    constexpr int TT = TP < 16 ? 1 : TP / 16;        // token tiles
    constexpr int SPB = 128 / GROUP;                 // scales per block
    constexpr int kStage = 4;                        // pieces of x that a thread has in flight while it stages them
    constexpr int kBatch = (TP < 32 ? 4 : 8) / RT;   // blocks of a batch: 64 KB ahead per CU
    extern __shared__ __attribute__((aligned(16))) uint8_t xs[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n16 = lane & 15, g = lane >> 4;
    constexpr int PER = kWaves / KS;  // row tiles (times RT) of a workgroup
    const int sub = wave / KS, part = wave % KS;
    const int tiles = (a.N + 16 * RT - 1) / (16 * RT), groups = (tiles + PER - 1) / PER;
    const int T = a.T;
    const size_t srow = (size_t)a.K / GROUP;

    // The wave's batches in order: chunk by chunk, row group by row group.
    auto blocks = [&](int k0) { return min(kc, a.K - k0) >> 7; };
    auto first = [&](int k0) { return blocks(k0) * part / KS; };
    auto end = [&](int k0) { return blocks(k0) * (part + 1) / KS; };
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
            const int row = min(((p.grp * PER + sub) * RT + r) * 16 + n16, a.N - 1);
            const uint8_t *wr = a.codes + (size_t)row * (a.K / 2) + p.k0 / 2 + 64 * p.b + 16 * g;
            const uint16_t *sr = a.scales + (size_t)row * srow + (p.k0 / 128 + p.b) * SPB;
            if (n >= kBatch) {
#pragma unroll
                for (int i = 0; i < kBatch; i++)
                    nw[r][i] = *reinterpret_cast<const u32x4 *>(wr + 64 * i);
                __builtin_memcpy(nsc[r], sr, sizeof nsc[r]);
            } else {
#pragma unroll
                for (int i = 0; i < kBatch; i++)
                    if (i < n) {
                        nw[r][i] = *reinterpret_cast<const u32x4 *>(wr + 64 * i);
#pragma unroll
                        for (int u = 0; u < SPB; u++) nsc[r][i * SPB + u] = sr[i * SPB + u];
                    }
            }
        }
    };
    int xat[4];  // this lane's piece of x in block column j, token tile 0
#pragma unroll
    for (int j = 0; j < 4; j++) xat[j] = (g * TP + slot_of<TP>(min(n16, TP - 1), 4 * j + g)) * 16;
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
                const int row = blocks(k0) * 16, pieces = row * T;  // 16-byte pieces, token by token
                for (int i0 = tid; i0 < pieces; i0 += kStage * 64 * kWaves) {
                    u32x4 v[kStage];
#pragma unroll
                    for (int q = 0; q < kStage; q++) {
                        const int i = min(i0 + q * 64 * kWaves, pieces - 1);
                        v[q] = *reinterpret_cast<const u32x4 *>(a.x + i / row * a.ldx + k0 + 8 * (i % row));
                    }
#pragma unroll
                    for (int q = 0; q < kStage; q++) {
                        const int i = i0 + q * 64 * kWaves;
                        if (i >= pieces) break;
                        const int t = i / row, c8 = i % row, blk = c8 / 16, p = c8 % 16;
                        // piece p = columns 8 p of the block: (g, j) = (p / 4, p % 4), and (p % 4, p / 4)
                        // where the codes are transposed
                        const int pg = GROUP == 128 ? p / 4 : p % 4, pj = GROUP == 128 ? p % 4 : p / 4;
                        *reinterpret_cast<u32x4 *>(xs + ((size_t)((blk * 4 + pj) * 4 + pg) * TP + slot_of<TP>(t, 4 * pj + pg)) * 16) = pair_columns(v[q]);
                    }
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
                const uint8_t *xb = xs + (size_t)b * 256 * TP;
                auto block = [&](int i) {
                    if (GROUP != 128)
#pragma unroll
                        for (int r = 0; r < RT; r++) transpose4(w[r][i]);
#pragma unroll
                    for (int u = 0; u < SPB; u++) {
                        f32x4 p[RT][TT];
#pragma unroll
                        for (int r = 0; r < RT; r++)
#pragma unroll
                            for (int tt = 0; tt < TT; tt++) p[r][tt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int jj = 0; jj < 4 / SPB; jj++) {
                            const int j = u * (4 / SPB) + jj;
                            bf16x8 wb[RT];
#pragma unroll
                            for (int r = 0; r < RT; r++) wb[r] = as_bf16x8(codes_bf16(w[r][i][j]));
#pragma unroll
                            for (int tt = 0; tt < TT; tt++) {  // rows past T hold anything; their results are not written
                                const bf16x8 xv = as_bf16x8(*reinterpret_cast<const u32x4 *>(
                                    xb + (i * 16 + j * 4) * (16 * TP) + 256 * tt + xat[j]));
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
                };
                if (TP < 32 && b + kBatch <= be) {  // one run of code, in which reads from LDS go ahead of their products
#pragma unroll
                    for (int i = 0; i < kBatch; i++) block(i);
                } else {  // (with many tokens that takes more registers than there are)
#pragma unroll
                    for (int i = 0; i < kBatch; i++)
                        if (b + i < be) block(i);
                }
            }
        }
        if constexpr (KS > 1) {  // the parts of a row tile meet in LDS, summed in wave order
            static_assert(RT == 1 && TT == 1, "counted by exchange_bytes");
            __shared__ f32x4 red[kWaves][64];
            if (part) red[wave][lane] = acc[0][0];
            __syncthreads();
            if (part == 0)
#pragma unroll
                for (int q = 1; q < KS; q++) {
                    const f32x4 v = red[wave + q][lane];
#pragma unroll
                    for (int e = 0; e < 4; e++) acc[0][0][e] += v[e];
                }
            __syncthreads();
            if (part) continue;
        }
#pragma unroll
        for (int r = 0; r < RT; r++)
#pragma unroll
            for (int tt = 0; tt < TT; tt++)
                store(a, ((grp * PER + sub) * RT + r) * 16 + n16, 16 * tt + 4 * g, acc[r][tt]);
    }
}

template <int GROUP, int TP, int RT, int KS>
hipError_t launch_wide(const LinearArgs &a, hipStream_t st)
{
    static_assert(max_chunk(TP, KS) >= 128, "a chunk fits");
    const int kc = std::min(a.K, max_chunk(TP, KS)), per = kWaves / KS;
    const int tiles = (a.N + 16 * RT - 1) / (16 * RT), groups = (tiles + per - 1) / per;
    const size_t lds = (size_t)kc / 128 * chunk_bytes(TP);
    linear_int4_kernel<GROUP, TP, RT, KS><<<std::min(groups, TP < 32 ? 512 : 256), 64 * kWaves, lds, st>>>(a, kc);
    return hipGetLastError();
}
template <int GROUP, int TP>
hipError_t launch_group(const LinearArgs &a, hipStream_t st)
{
    const int tiles = (a.N + 15) / 16;
    // Up to 24576 rows x is read anew by every workgroup (K = 2048, 1, 8, 16, 32 and 64 tokens: 24576
    // rows 9.5, 10.8, 11, 15.2 and 25.5 us, staged 10.8, 12.4, 13.6, 18.3 and 27.3; K = 8320: 27, 32,
    // 38, 52 and 80, staged 35, 42, 49, 67 and 104); with more of them that is no gain (32000 rows, K =
    // 2048: 11.2, 12.7, 13.4, 18.8 and 32.8, staged 11.2, 12.8, 13.9, 19.6 and 28.4).  Two row tiles to
    // a workgroup as soon as one each would take a second round of the CUs (5120 rows, 64 tokens: 9.5
    // us, one 12.3; 2048 rows, one token: one 3.4, two 4.7).
    if (tiles <= kNarrow) {
        if (tiles <= kNarrowOne)
            linear_narrow_kernel<GROUP, TP < 4 ? 4 : TP, 1><<<tiles, 64 * kWaves, 0, st>>>(a);
        else
            linear_narrow_kernel<GROUP, TP < 4 ? 4 : TP, 2><<<(tiles + 1) / 2, 64 * kWaves, 0, st>>>(a);
        return hipGetLastError();
    }
    // Two row tiles to a wave halve the reads of x from LDS where those bound it and the rows are
    // enough for every wave (K = 2048, 131072 rows: 64 tokens 85 us, one 114; 32 tokens 46, one 52;
    // 32000 rows: 64 tokens 39, one 29; 32 tokens 24, one 20).
    if constexpr (TP >= 32)
        if (tiles >= 2 * kWaves * 256) return launch_wide<GROUP, TP, 2, 1>(a, st);
    // 2048 waves are eight to a CU.  Where the last of them would be half the GPU's or less, two waves
    // take a row tile, half of K each (33673 rows, K = 6272: one token 33 us, whole 43; 8 tokens 43, 51;
    // 131072 rows, K = 2048, 8 tokens: 38, whole 36).  With more than 16 staging x twice as often costs
    // more (33673 rows, 64 tokens, with the codes' former conversion: 210, whole 173).
    if constexpr (TP < 32)
        if ((tiles - 1) % (kWaves * 256) < kWaves * 128) return launch_wide<GROUP, TP, 1, 2>(a, st);
    return launch_wide<GROUP, TP, 1, 1>(a, st);
}
template <int TP>
hipError_t launch_tp(const LinearArgs &a, hipStream_t st)
{
    return a.group == 128  ? launch_group<128, TP>(a, st)
           : a.group == 64 ? launch_group<64, TP>(a, st)
                           : launch_group<32, TP>(a, st);
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
