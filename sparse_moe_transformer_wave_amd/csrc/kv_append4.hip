// kv_append4.hip -- new tokens into the 4-bit paged cache: per-head RMSNorm and rotation of
// queries and keys, keys and values to blocks of 32 E2M1 codes under one power of two.
//
//   x' = x w / sqrt(mean(x^2) + eps);  (a, b) -> (a c - b s, b c + a s)
//   e = least with max |x'| <= 7 2^e;  code = nearest of {0, .5, 1, 1.5, 2, 3, 4, 6} to |x'| / 2^e
//
// Bound by the projections' bytes, a plain copy of the queries beside a few bytes of codes, and
// close behind by the vector pipe.  A wave takes one token's heads 512 channels of a kind at a time, 8
// (16 bytes) to a lane, a block of 32 being four lanes; the next group's are on their way meanwhile.
// Keys are computed in 64 bits: a code is that of the exact value, and not, for a value next to the
// border of two codes, that of 32 bits' rounding (a code is a step of up to a half).  They become fp32
// towards zero, with the last bit set where something is cut off, and the code's conversion rounds those
// as it would the exact value.
#include "serve.h"

#include <type_traits>

namespace flint {

namespace {

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

__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}
// The sum over the 8 or 16 lanes of a head.
template <int LPH>
__device__ __forceinline__ float head_sum(float v)
{
    v += __int_as_float(FLINT_DPP(__float_as_int(v), 0xB1));
    v += __int_as_float(FLINT_DPP(__float_as_int(v), 0x4E));
    v += __int_as_float(FLINT_DPP(__float_as_int(v), 0x141));
    if (LPH == 16) v += __int_as_float(FLINT_DPP(__float_as_int(v), 0x140));
    return v;
}
template <int LPH>
__device__ __forceinline__ double head_sum(double v)
{
    auto other = [](double x, auto C) {
        const uint64_t u = __builtin_bit_cast(uint64_t, x);
        const uint32_t lo = FLINT_DPP((int)(uint32_t)u, decltype(C)::value), hi = FLINT_DPP((int)(u >> 32), decltype(C)::value);
        return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
    };
    v += other(v, std::integral_constant<int, 0xB1>{});
    v += other(v, std::integral_constant<int, 0x4E>{});
    v += other(v, std::integral_constant<int, 0x141>{});
    if (LPH == 16) v += other(v, std::integral_constant<int, 0x140>{});
    return v;
}

// of a query: as kv_append.hip has it, so that its bits are those that the bf16 cache's append gives
__device__ __forceinline__ float rsqrt_of(float x) { return 1.0f / sqrtf(x); }
__device__ __forceinline__ double rsqrt_of(double x) { return rsqrt(x); }
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
        const F r = rsqrt_of(head_sum<LPH>(ss) * F(1.0 / D) + F(a.eps));
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
    wave_fence();
#pragma unroll
    for (int i = 0; i < 8; i++) row[c0 + i] = v[i];
    wave_fence();
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

// The largest of a block's 32 values, over its four lanes.
__device__ __forceinline__ uint32_t block_max(uint32_t v)
{
    v = max(v, (uint32_t)FLINT_DPP((int)v, 0xB1));
    return max(v, (uint32_t)FLINT_DPP((int)v, 0x4E));
}
// The scale byte of a block whose largest |x| has the biased exponent x and is above 1.75 of its
// power of two or not.
__device__ __forceinline__ int scale_byte(int x, bool above) { return min(max(x - (above ? 1 : 2), 2), 252); }

// The codes of a lane's 8 bf16 values, the first in the low nibble; its block is lanes 4 k .. 4 k + 3.
// byte: the block's scale.  The conversion divides by the scale, rounds to nearest (an even code at a
// tie) and stops at 6.
__device__ __forceinline__ uint32_t quantise8(u32x4 raw, int &byte)
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) top = max(top, max(raw[i] & 0x7fffu, (raw[i] >> 16) & 0x7fffu));
    top = block_max(top);
    byte = top == 0 ? 127 : scale_byte((int)(top >> 7), (top & 0x7fu) > 0x60u);
    const float s = __uint_as_float((uint32_t)byte << 23);
    auto pair = [](uint32_t two) { return __builtin_bit_cast(bf16x2_t, two); };  // (of a vector's element it takes the first)
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair(raw[0]), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair(raw[1]), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair(raw[2]), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair(raw[3]), s, 3);
    if (top < 0x7f80u) return c;
    byte = 255;  // an infinity or a NaN
    return 0;
}

// v as fp32, towards zero with the last bit set where that is not exact: on the same side of every
// border as v, since borders have fewer bits.
__device__ __forceinline__ float to_odd(double v)
{
    const float f = (float)v;
    const double d = f;
    uint32_t u = __float_as_uint(f);
    if (fabs(d) > fabs(v)) u--;
    if (d != v) u |= 1u;
    return __uint_as_float(u);
}
// The codes of a lane's 8 values in 64 bits.
__device__ __forceinline__ uint32_t quantise8(const double *v, int &byte)
{
    float f[8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        f[i] = to_odd(v[i]);
        top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
    }
    top = block_max(top);
    byte = top == 0 ? 127 : scale_byte((int)(top >> 23), (top & 0x7fffffu) > 0x600000u);
    const float s = __uint_as_float((uint32_t)byte << 23);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[0], f[1], s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[2], f[3], s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[4], f[5], s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[6], f[7], s, 3);
    if (top < 0x7f800000u) return c;
    byte = 255;
    return 0;
}

// What codes stand for, as bf16: byte S of them.
template <int S>
__device__ __forceinline__ uint32_t values2(uint32_t codes, int byte)
{
    const float s = __uint_as_float((uint32_t)byte << 23);
    return byte == 255 ? 0x7fc07fc0u : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, S));
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

// A wave takes every `parts`-th of a token's groups.  6 waves per SIMD: 47 us for 8192 tokens; 5 of them
// (the registers that the compiler takes by itself) 52, 7 50.
template <int D, bool PLAIN>
__global__ __launch_bounds__(256, PLAIN ? 6 : 4) void kv_append4_kernel(Append4Args x, int parts)
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
    auto load = [&](int g) {
        const bool is_q = g < gr.q, is_v = g >= gr.q + gr.kv;
        const int h = (g - (is_q ? 0 : is_v ? gr.q + gr.kv : gr.q)) * HPW + sub;
        const int at = is_q ? min(h, a.c.Hq - 1) : a.c.Hq + (is_v ? a.c.Hkv : 0) + min(h, a.c.Hkv - 1);
        return *reinterpret_cast<const u32x4 *>(row + at * D + c0);
    };
    u32x4 raw = load(item % parts), next;
    for (int g = item % parts; g < gr.all(); g += parts, raw = next) {
        if (g + parts < gr.all()) next = load(g + parts);
        if (g < gr.q) {
            const int h = g * HPW + sub;
            float v[8];
            norm_rotate<D, PLAIN, float>(a, p, raw, a.q_norm, (float *)mine, v);
            const u32x4 out = p.ok ? pack8(v) : u32x4{0u, 0u, 0u, 0u};
            if (h < a.c.Hq) *reinterpret_cast<u32x4 *>(a.q + t * a.ldq + h * D + c0) = out;
            continue;
        }
        const bool is_v = g >= gr.q + gr.kv;
        const int h = (g - gr.q - (is_v ? gr.kv : 0)) * HPW + sub;
        int byte;
        uint32_t codes;
        if (is_v || (!a.k_norm && !a.rot)) {
            codes = quantise8(raw, byte);
        } else {
            double v[8];
            norm_rotate<D, PLAIN, double>(a, p, raw, a.k_norm, mine, v);
            codes = quantise8(v, byte);
        }
        if (h >= a.c.Hkv) continue;
        uint16_t *dst = is_v ? x.v : x.k;
        if (dst) {
            const u32x4 out{values2<0>(codes, byte), values2<1>(codes, byte), values2<2>(codes, byte), values2<3>(codes, byte)};
            *reinterpret_cast<u32x4 *>(dst + t * (is_v ? x.ldv : x.ldk) + h * D + c0) = p.ok ? out : u32x4{0u, 0u, 0u, 0u};
        }
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
    // A wave each for a token's groups while there are few; otherwise five groups to a wave, which share
    // its angles and weights (8192 tokens of 10 groups: 47 us, three 52, ten 52, one 67).
    const int parts = x.a.T * (int64_t)groups <= 8192 ? groups : (groups + 4) / 5;
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
