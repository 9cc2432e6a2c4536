// kv_append4.hip -- new tokens into the 4-bit paged cache: per-head RMSNorm and rotation of
// queries and keys, keys and values to blocks of 32 E2M1 codes under one power of two.
//
//   x' = x w / sqrt(mean(x^2) + eps);  (a, b) -> (a c - b s, b c + a s)
//   e = least with max |x'| <= 7 2^e;  code = nearest of {0, .5, 1, 1.5, 2, 3, 4, 6} to |x'| / 2^e
//
// Bound by the projections' bytes, a plain copy of the queries beside a few bytes of codes.  A lane
// holds 8 channels (16 bytes) of one head, a wave 512 / D heads of one token and kind; a block of
// 32 is four lanes.  Keys are computed in 64 bits: a value next to the border of two codes goes
// where the exact value does (32 bits would put one in 2^20 on the other side, and a code is a step
// of up to a half), and one head in nine has them.  Codes come from integer comparisons of the high
// word, whose exponent takes the scale, and a bit for what is below it.
#include "serve.h"

namespace flint {

namespace {

__device__ __forceinline__ u32x4 pack8(const float *v)
{
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const bf16x2_t b = __builtin_convertvector(f32x2_t{v[2 * i], v[2 * i + 1]}, bf16x2_t);
        r[i] = __builtin_bit_cast(uint32_t, b);
    }
    return r;
}

// Where a lane's 8 channels are rotated with 8 whole channels of one other lane (half style,
// multiples of 8) or among themselves (pairs), or not at all.
__host__ inline bool lane_rotation(int rot, bool pairs) { return pairs ? rot % 8 == 0 : rot % 16 == 0; }

// A token's place and angles, for the lane's 8 channels.
struct Place {
    bool ok, keep;      // the position is in the table; and the slot in the cache
    int64_t page;
    int off;
    const float *cp, *sp;
    float cs[8], sn[8];  // whole-lane rotation: the sines with the sign of the lane's side
};

template <int D>
__device__ __forceinline__ bool second_half(const AppendArgs &a, int c0) { return !a.pairs && c0 >= a.rot / 2; }

template <int D, bool PLAIN>
__device__ __forceinline__ Place place_of(const AppendArgs &a, int t)
{
    const int c0 = 8 * (threadIdx.x & (D / 8 - 1)), half = a.rot / 2;
    const bool second = second_half<D>(a, c0);
    Place p;
    p.ok = true;
    p.cp = p.sp = nullptr;
    if (a.rot) {
        const int at = a.positions[t];
        p.ok = at >= 0 && at < a.max_pos;
        p.cp = a.cos + (int64_t)(p.ok ? at : 0) * half;
        p.sp = a.sin + (int64_t)(p.ok ? at : 0) * half;
        if (PLAIN && c0 < a.rot) {
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                if (a.pairs) {
                    const float2 c = *reinterpret_cast<const float2 *>(p.cp + (c0 + i) / 2);
                    const float2 s = *reinterpret_cast<const float2 *>(p.sp + (c0 + i) / 2);
                    p.cs[i] = p.cs[i + 1] = c.x, p.cs[i + 2] = p.cs[i + 3] = c.y;
                    p.sn[i] = -s.x, p.sn[i + 1] = s.x, p.sn[i + 2] = -s.y, p.sn[i + 3] = s.y;
                } else {
                    const int at0 = (second ? c0 - half : c0) + i;
                    const float4 c = *reinterpret_cast<const float4 *>(p.cp + at0), s = *reinterpret_cast<const float4 *>(p.sp + at0);
                    p.cs[i] = c.x, p.cs[i + 1] = c.y, p.cs[i + 2] = c.z, p.cs[i + 3] = c.w;
                    p.sn[i] = s.x, p.sn[i + 1] = s.y, p.sn[i + 2] = s.z, p.sn[i + 3] = s.w;
                    if (!second)
#pragma unroll
                        for (int j = 0; j < 4; j++) p.sn[i + j] = -p.sn[i + j];
                }
            }
        }
    }
    const int64_t slot = a.slots[t];
    p.keep = p.ok && slot >= 0 && slot < a.c.n_pages * a.c.page;
    p.page = p.keep ? slot >> a.c.page_shift : 0;
    p.off = (int)(p.keep ? slot & (a.c.page - 1) : 0);
    return p;
}

__device__ __forceinline__ float root(float x) { return sqrtf(x); }
__device__ __forceinline__ double root(double x) { return sqrt(x); }
__device__ __forceinline__ float fma_of(float x, float y, float z) { return fmaf(x, y, z); }
__device__ __forceinline__ double fma_of(double x, double y, double z) { return fma(x, y, z); }

// 8 channels of a head, normalised and rotated in F.  buf: the wave's 512 values of LDS, used
// where the partner channels are not whole lanes.
template <int D, bool PLAIN, typename F>
__device__ __forceinline__ void norm_rotate(const AppendArgs &a, const Place &p, u32x4 raw, const uint16_t *nw, F *buf, F *v)
{
    constexpr int LPH = D / 8;
    const int lane = threadIdx.x & 63, li = lane % LPH, c0 = 8 * li, half = a.rot / 2;
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = bf2f((uint16_t)(raw[i >> 1] >> (16 * (i & 1))));
    if (nw) {
        const u32x4 w = *reinterpret_cast<const u32x4 *>(nw + c0);
        F ss = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) ss = fma_of(v[i], v[i], ss);
#pragma unroll
        for (int m = 1; m < LPH; m *= 2) ss += __shfl_xor(ss, m);
        const F r = F(1) / root(ss * F(1.0 / D) + F(a.eps));
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = v[i] * r * F(bf2f((uint16_t)(w[i >> 1] >> (16 * (i & 1)))));
    }
    if (!a.rot) return;
    if (PLAIN) {
        const int partner = lane - li + (second_half<D>(a, c0) ? li - half / 8 : li + half / 8);
        F o[8];
#pragma unroll
        for (int i = 0; i < 8; i++) o[i] = a.pairs ? v[i ^ 1] : __shfl(v[i], partner & 63);
        if (c0 < a.rot)
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = fma_of(v[i], F(p.cs[i]), o[i] * F(p.sn[i]));
        return;
    }
    // the head's lanes are in one wave, so its LDS row is complete in program order
    F *row = buf + (lane - li) * 8;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 8; i++) row[c0 + i] = v[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int c = c0 + i;
        if (c >= a.rot) continue;
        const bool up = a.pairs ? (c & 1) : c >= half;
        const int ang = a.pairs ? c / 2 : up ? c - half : c;
        const int other = a.pairs ? c ^ 1 : up ? c - half : c + half;
        const F x = row[other] * F(p.sp[ang]);
        v[i] = fma_of(v[i], F(p.cp[ang]), up ? x : -x);
    }
}

// The codes of a lane's 8 values, the first in the low nibble; its block is lanes 4 k .. 4 k + 3.
// byte: the block's scale.
__device__ __forceinline__ uint32_t quantise8(const double *v, int &byte)
{
    uint32_t hi[8], top = 0;
    bool low[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v[i]);
        hi[i] = (uint32_t)(u >> 32);
        low[i] = (uint32_t)u != 0;
        // high word and what is below it, ordered like |v|
        top = max(top, ((hi[i] & 0x7fffffffu) << 1) | (uint32_t)low[i]);
    }
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2));
    if (top >= 0xffe00000u) {  // an infinity or a NaN
        byte = 255;
        return 0;
    }
    // m 2^x with m <= 1.75: e = x - 2, else x - 1
    int e = (int)(top >> 21) - 1023 - ((top & 0x1fffffu) <= 0x180000u ? 2 : 1);
    e = top == 0 ? 0 : min(max(e, -125), 125);
    byte = e + 127;
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int h = max((int)(hi[i] & 0x7fffffffu) - (e << 20), 0);  // of |v| / 2^e; far below the first border 0
        const uint32_t key = ((uint32_t)h << 1) | (uint32_t)low[i];
        // high words of 0.25, 0.75, ... 5; a tie goes to the even code
        uint32_t c = (key > 0x3fd00000u * 2u) + (key >= 0x3fe80000u * 2u) + (key > 0x3ff40000u * 2u) + (key >= 0x3ffc0000u * 2u) +
                     (key > 0x40040000u * 2u) + (key >= 0x400c0000u * 2u) + (key > 0x40140000u * 2u);
        codes |= (c | (hi[i] >> 31) << 3) << (4 * i);
    }
    return codes;
}

// What 8 codes stand for, as bf16.
__device__ __forceinline__ u32x4 values8(uint32_t codes, int byte)
{
    const float s = __uint_as_float((uint32_t)byte << 23);
    u32x4 r;
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 0));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 1));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 2));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 3));
    return byte == 255 ? u32x4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u} : r;
}

// Groups of a token: 512 / D heads of one kind each; queries, keys, values.
struct Groups {
    int q, kv;
    __host__ __device__ Groups(const Cache &c)
    {
        const int hpw = 512 / c.D;
        q = (c.Hq + hpw - 1) / hpw;
        kv = (c.Hkv + hpw - 1) / hpw;
    }
    __host__ __device__ int all() const { return q + 2 * kv; }
};

template <int D, bool PLAIN>
__global__ __launch_bounds__(256) void kv_append4_kernel(Append4Args x, int parts)
{
    constexpr int LPH = D / 8, HPW = 64 / LPH;
    __shared__ double buf[PLAIN ? 1 : 4][PLAIN ? 1 : 512];
    const AppendArgs &a = x.a;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int sub = lane / LPH, li = lane % LPH, c0 = 8 * li;
    const int item = blockIdx.x * 4 + wave, t = item / parts;
    if (t >= a.T) return;
    const Groups gr(a.c);
    const Place p = place_of<D, PLAIN>(a, t);
    double *mine = buf[PLAIN ? 0 : wave];
    const uint16_t *row = a.qkv + (int64_t)t * a.ldqkv;
    for (int g = item % parts; g < gr.all(); g += parts) {
        if (g < gr.q) {
            const int h = g * HPW + sub, at = min(h, a.c.Hq - 1);
            float v[8];
            norm_rotate<D, PLAIN, float>(a, p, *reinterpret_cast<const u32x4 *>(row + at * D + c0), a.q_norm, (float *)mine, v);
            const u32x4 out = p.ok ? pack8(v) : u32x4{0u, 0u, 0u, 0u};
            if (h < a.c.Hq) *reinterpret_cast<u32x4 *>(a.q + t * a.ldq + h * D + c0) = out;
            continue;
        }
        const bool is_v = g >= gr.q + gr.kv;
        const int h = (g - gr.q - (is_v ? gr.kv : 0)) * HPW + sub, at = min(h, a.c.Hkv - 1);
        const u32x4 raw = *reinterpret_cast<const u32x4 *>(row + (a.c.Hq + (is_v ? a.c.Hkv : 0) + at) * D + c0);
        double v[8];
        if (is_v) {
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = bf2f((uint16_t)(raw[i >> 1] >> (16 * (i & 1))));
        } else {
            norm_rotate<D, PLAIN, double>(a, p, raw, a.k_norm, mine, v);
        }
        int byte;
        const uint32_t codes = quantise8(v, byte);
        if (h >= a.c.Hkv) continue;
        uint16_t *dst = is_v ? x.v : x.k;
        if (dst)
            *reinterpret_cast<u32x4 *>(dst + t * (is_v ? x.ldv : x.ldk) + h * D + c0) =
                p.ok ? values8(codes, byte) : u32x4{0u, 0u, 0u, 0u};
        if (!p.keep) continue;
        // a page's key codes, value codes, key scales, value scales
        uint8_t *pg = reinterpret_cast<uint8_t *>(a.c.k) + p.page * a.c.page_stride;
        const int part = a.c.Hkv * a.c.page * (D / 2), spart = a.c.Hkv * a.c.page * (D / 32);
        *reinterpret_cast<uint32_t *>(pg + (is_v ? part : 0) + (h * a.c.page + p.off) * (D / 2) + 4 * li) = codes;
        if ((li & 3) == 0) pg[2 * part + (is_v ? spart : 0) + (h * (D / 32) + li / 4) * a.c.page + p.off] = (uint8_t)byte;
    }
}

template <int D>
hipError_t launch_d(const Append4Args &x, hipStream_t st)
{
    const int groups = Groups(x.a.c).all();
    const int parts = x.a.T * (int64_t)groups <= 8192 ? groups : (groups + 2) / 3;
    const int64_t wgs = ((int64_t)x.a.T * parts + 3) / 4;
    if (wgs > INT32_MAX) return hipErrorInvalidValue;
    if (lane_rotation(x.a.rot, x.a.pairs))
        kv_append4_kernel<D, true><<<(unsigned)wgs, 256, 0, st>>>(x, parts);
    else
        kv_append4_kernel<D, false><<<(unsigned)wgs, 256, 0, st>>>(x, parts);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append4(const Append4Args &x, hipStream_t st)
{
    return x.a.c.D == 128 ? launch_d<128>(x, st) : launch_d<64>(x, st);
}

}  // namespace flint
