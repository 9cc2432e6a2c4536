// kv_append.hip -- new tokens into the paged cache: per-head RMSNorm and rotation of queries
// and keys on the way, values transposed into their page.
//
//   x' = x w / sqrt(mean(x^2) + eps);  (a, b) -> (a c - b s, b c + a s)
//
// Bound by bytes (every element read and written once).  A lane holds 8 channels (16 bytes)
// of one head of one token, D / 8 lanes a head; the mean is reduced inside the DPP row and
// the rotation's partner channels are exchanged through the wave's own LDS rows.  Values go
// through LDS in tiles of 64 tokens so that 8 tokens of one channel leave as 16 bytes.
#include "ops.h"

namespace flint {

namespace {

constexpr int kTile = 64;  // value tokens per workgroup

// The queries and keys: 256 threads = 2048 / D heads of any token.
template <int D>
__device__ __forceinline__ void append_qk(const AppendArgs &a, int wg, float (*buf)[D])
{
    constexpr int LPH = D / 8;  // lanes per head
    const int tid = threadIdx.x, sub = tid / LPH, li = tid % LPH;
    const int heads = a.c.Hq + a.c.Hkv;
    const int64_t item = (int64_t)wg * (256 / LPH) + sub;
    const bool live = item < (int64_t)a.T * heads;
    const int t = live ? (int)(item / heads) : 0, h = live ? (int)(item % heads) : 0;
    const bool is_k = h >= a.c.Hq;
    const u32x4 raw = *reinterpret_cast<const u32x4 *>(a.qkv + t * a.ldqkv + h * D + 8 * li);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[2 * i] = bf2f(raw[i] & 0xffffu);
        v[2 * i + 1] = bf2f(raw[i] >> 16);
    }
    const uint16_t *nw = is_k ? a.k_norm : a.q_norm;
    if (nw) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++) ss = fmaf(v[i], v[i], ss);
#pragma unroll
        for (int m = 1; m < LPH; m *= 2) ss += __shfl_xor(ss, m);
        const float r = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
        const u32x4 wv = *reinterpret_cast<const u32x4 *>(nw + 8 * li);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = v[2 * i] * r * bf2f(wv[i] & 0xffffu);
            v[2 * i + 1] = v[2 * i + 1] * r * bf2f(wv[i] >> 16);
        }
    }
    bool ok = true;
    if (a.rot) {
        const int p = a.positions[t];
        ok = p >= 0 && p < a.max_pos;
        const int half = a.rot / 2;
        const float *cs = a.cos + (int64_t)(ok ? p : 0) * half, *sn = a.sin + (int64_t)(ok ? p : 0) * half;
#pragma unroll
        for (int i = 0; i < 8; i++) buf[sub][8 * li + i] = v[i];
        // the head's lanes are in one wave, so its LDS row is complete in program order
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int c = 8 * li + i;
            if (c < a.rot) {
                const bool second = a.pairs ? (c & 1) : c >= half;
                const int ang = a.pairs ? c / 2 : second ? c - half : c;
                const int partner = a.pairs ? c ^ 1 : second ? c - half : c + half;
                const float o = buf[sub][partner];
                v[i] = second ? fmaf(v[i], cs[ang], o * sn[ang]) : fmaf(v[i], cs[ang], -(o * sn[ang]));
            }
        }
    }
    if (!live) return;
    u32x4 out;
#pragma unroll
    for (int i = 0; i < 4; i++) out[i] = f2bf(v[2 * i]) | (f2bf(v[2 * i + 1]) << 16);
    if (!is_k) {
        if (!ok) out = u32x4{0u, 0u, 0u, 0u};
        *reinterpret_cast<u32x4 *>(a.q + t * a.ldq + h * D + 8 * li) = out;
        return;
    }
    const int64_t slot = a.slots[t];
    if (!ok || slot < 0 || slot >= a.c.n_pages * a.c.page) return;
    const int64_t page = slot >> a.c.page_shift;
    const int off = (int)(slot & (a.c.page - 1));
    uint16_t *dst = a.c.k + page * a.c.page_stride + ((h - a.c.Hq) * a.c.page + off) * D + 8 * li;
    *reinterpret_cast<u32x4 *>(dst) = out;
}

// The values of 64 tokens of one key/value head.
template <int D>
__device__ __forceinline__ void append_v(const AppendArgs &a, int tile, int h, uint16_t (*buf)[D + 2])
{
    __shared__ int64_t s_slot[kTile];
    const int tid = threadIdx.x, t0 = tile * kTile, n = min(kTile, a.T - t0);
    const uint16_t *src = a.qkv + (int64_t)(a.c.Hq + a.c.Hkv + h) * D;
    if (tid < n) {
        int64_t s = a.slots[t0 + tid];
        if (s < 0 || s >= a.c.n_pages * a.c.page) s = -1;
        if (a.rot) {
            const int p = a.positions[t0 + tid];
            if (p < 0 || p >= a.max_pos) s = -1;
        }
        s_slot[tid] = s;
    }
    for (int i = tid; i < n * (D / 8); i += 256) {
        const int t = i / (D / 8), c = i % (D / 8);
        const u32x4 v = *reinterpret_cast<const u32x4 *>(src + (int64_t)(t0 + t) * a.ldqkv + 8 * c);
#pragma unroll
        for (int j = 0; j < 4; j++) *reinterpret_cast<uint32_t *>(&buf[t][8 * c + 2 * j]) = v[j];
    }
    __syncthreads();
    for (int i = tid; i < n * D; i += 256) {
        const int t = i % n, d = i / n;
        const int64_t slot = s_slot[t];
        if (slot < 0) continue;
        const int64_t page = slot >> a.c.page_shift;
        const int off = (int)(slot & (a.c.page - 1));
        a.c.v[page * a.c.page_stride + (int64_t)(h * D + d) * a.c.page + off] = buf[t][d];
    }
}

template <int D>
__global__ __launch_bounds__(256) void kv_append_kernel(AppendArgs a, int qk_wgs)
{
    __shared__ union {
        float qk[2048 / D][D];
        uint16_t v[kTile][D + 2];
    } sh;
    if ((int)blockIdx.x < qk_wgs)
        append_qk<D>(a, blockIdx.x, sh.qk);
    else
        append_v<D>(a, (blockIdx.x - qk_wgs) / a.c.Hkv, (blockIdx.x - qk_wgs) % a.c.Hkv, sh.v);
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs &a, hipStream_t st)
{
    const int per = 2048 / a.c.D;  // heads per workgroup
    const int64_t qk = ((int64_t)a.T * (a.c.Hq + a.c.Hkv) + per - 1) / per;
    const int64_t v = (int64_t)((a.T + kTile - 1) / kTile) * a.c.Hkv;
    if (qk + v > INT32_MAX) return hipErrorInvalidValue;
    if (a.c.D == 128)
        kv_append_kernel<128><<<(unsigned)(qk + v), 256, 0, st>>>(a, (int)qk);
    else
        kv_append_kernel<64><<<(unsigned)(qk + v), 256, 0, st>>>(a, (int)qk);
    return hipGetLastError();
}

}  // namespace flint
