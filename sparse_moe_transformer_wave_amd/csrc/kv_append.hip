// kv_append.hip -- new tokens into the paged cache: per-head RMSNorm and rotation of queries
// and keys on the way, values transposed into their page.
//
//   x' = x w / sqrt(mean(x^2) + eps);  (a, b) -> (a c - b s, b c + a s)
//
// Bound by bytes (every element read and written once): 8192 tokens of 32 + 2 x 4 heads of 128 in 38
// us, 172 MB, 4.5 TB/s where a plain copy reaches 5.2; 562 tokens of 4 + 2 x 4 in 5.1 us; 8 tokens in
// 3.3 us, a launch.  A lane holds 8 channels (16 bytes) of
// one head; a wave takes one token's angles and norm weights once and its heads 512 / D at a
// time.  The mean is reduced inside a DPP row and the rotation's partner channels come from the
// partner lane.  Values go through LDS in tiles of 32 tokens, so that 8 tokens of one channel
// leave as 16 bytes where they are consecutive in a page, and the tiles start where the page's
// 8-token pieces do.
#include "ops.h"

namespace flint {

namespace {

constexpr int kTile = 32;       // value tokens per workgroup, for prompts (64: 1008 tokens 8.6 us, so 8.0; 8192: 40, 38)
constexpr int kSmallTile = 8;   // and for decode batches, whose values scatter channel by channel

__device__ __forceinline__ void unpack8(u32x4 r, float *v)
{
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[2 * i] = bf2f(r[i] & 0xffffu);
        v[2 * i + 1] = bf2f(r[i] >> 16);
    }
}
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
__device__ __forceinline__ void load8(const float *p, float *v)
{
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// Where a lane's 8 channels are rotated with 8 whole channels of one other lane (half style,
// multiples of 8) or among themselves (pairs), or not at all.
__host__ __device__ inline bool lane_rotation(int rot, bool pairs) { return pairs ? rot % 8 == 0 : rot % 16 == 0; }

// The queries and keys of one token, every `parts`-th group of 512 / D heads from `part` on.
// PLAIN: lane_rotation(); otherwise each channel finds its partner in the wave's LDS rows.
template <int D, bool PLAIN>
__device__ __forceinline__ void append_qk(const AppendArgs &a, int t, int part, int parts, float (*buf)[D])
{
    constexpr int LPH = D / 8, HPW = 64 / LPH;  // lanes per head, heads per wave
    const int lane = threadIdx.x & 63, sub = lane / LPH, li = lane % LPH, c0 = 8 * li;
    const int heads = a.c.Hq + a.c.Hkv, half = a.rot / 2;
    const int64_t slot = a.slots[t];
    bool ok = true;
    float cs[8], sn[8];  // PLAIN: this lane's angles, the sines with the sign of its side
    const float *cp = nullptr, *sp = nullptr;
    const bool turns = a.rot && c0 < a.rot;
    const bool second = !a.pairs && c0 >= half;
    if (a.rot) {
        const int p = a.positions[t];
        ok = p >= 0 && p < a.max_pos;
        cp = a.cos + (int64_t)(ok ? p : 0) * half;
        sp = a.sin + (int64_t)(ok ? p : 0) * half;
        if (PLAIN && turns) {
            if (a.pairs) {
                const float4 c = *reinterpret_cast<const float4 *>(cp + c0 / 2), s = *reinterpret_cast<const float4 *>(sp + c0 / 2);
                cs[0] = cs[1] = c.x, cs[2] = cs[3] = c.y, cs[4] = cs[5] = c.z, cs[6] = cs[7] = c.w;
                sn[0] = -s.x, sn[1] = s.x, sn[2] = -s.y, sn[3] = s.y, sn[4] = -s.z, sn[5] = s.z, sn[6] = -s.w, sn[7] = s.w;
            } else {
                load8(cp + (second ? c0 - half : c0), cs);
                load8(sp + (second ? c0 - half : c0), sn);
                if (!second)
#pragma unroll
                    for (int i = 0; i < 8; i++) sn[i] = -sn[i];
            }
        }
    }
    const bool keep = ok && slot >= 0 && slot < a.c.n_pages * a.c.page;
    const int64_t page = keep ? slot >> a.c.page_shift : 0;
    const int off = (int)(keep ? slot & (a.c.page - 1) : 0);
    const int partner = lane - li + (second ? li - half / 8 : li + half / 8);  // half style, PLAIN
    for (int h0 = part * HPW; h0 < heads; h0 += parts * HPW) {
        const int h = min(h0 + sub, heads - 1);
        const bool is_k = h >= a.c.Hq;
        const uint16_t *nw = is_k ? a.k_norm : a.q_norm;
        const u32x4 raw = *reinterpret_cast<const u32x4 *>(a.qkv + t * a.ldqkv + h * D + c0);
        const u32x4 wv = nw ? *reinterpret_cast<const u32x4 *>(nw + c0) : u32x4{0u, 0u, 0u, 0u};
        float v[8], o[8];
        unpack8(raw, v);
        if (nw) {
            float ss = 0.f, w[8];
#pragma unroll
            for (int i = 0; i < 8; i++) ss = fmaf(v[i], v[i], ss);
#pragma unroll
            for (int m = 1; m < LPH; m *= 2) ss += __shfl_xor(ss, m);
            const float r = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
            unpack8(wv, w);
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = v[i] * r * w[i];
        }
        if (a.rot && PLAIN) {
#pragma unroll
            for (int i = 0; i < 8; i++) o[i] = a.pairs ? v[i ^ 1] : __shfl(v[i], partner & 63);
            if (turns)
#pragma unroll
                for (int i = 0; i < 8; i++) v[i] = fmaf(v[i], cs[i], o[i] * sn[i]);
        } else if (a.rot) {
            // the head's lanes are in one wave, so its LDS row is complete in program order
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < 8; i++) buf[sub][c0 + i] = v[i];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const int c = c0 + i;
                if (c < a.rot) {
                    const bool up = a.pairs ? (c & 1) : c >= half;
                    const int ang = a.pairs ? c / 2 : up ? c - half : c;
                    const int other = a.pairs ? c ^ 1 : up ? c - half : c + half;
                    const float x = buf[sub][other] * sp[ang];
                    v[i] = fmaf(v[i], cp[ang], up ? x : -x);
                }
            }
        }
        if (h0 + sub >= heads) continue;
        u32x4 out = pack8(v);
        if (!is_k) {
            if (!ok) out = u32x4{0u, 0u, 0u, 0u};
            *reinterpret_cast<u32x4 *>(a.q + t * a.ldq + h * D + c0) = out;
        } else if (keep) {
            *reinterpret_cast<u32x4 *>(a.c.k + page * a.c.page_stride + ((h - a.c.Hq) * a.c.page + off) * D + c0) = out;
        }
    }
}

// The values of a tile of up to kTile tokens of one key/value head.
template <int D>
__device__ __forceinline__ void append_v(const AppendArgs &a, int tile, int size, int h, uint16_t (*buf)[D + 2], int64_t *s_slot,
                                         int *s_piece)
{
    // Tiles start where the first token's 8-token pieces do, so the pieces of one consecutive run
    // (a prompt) lie in one tile each.
    const int64_t first = a.slots[0];
    const int lead = first > 0 ? (int)(first & 7) : 0;
    const int tid = threadIdx.x, t0 = max(tile * size - lead, 0), n = min(tile * size - lead + size, a.T) - t0;
    const uint16_t *src = a.qkv + (int64_t)(a.c.Hq + a.c.Hkv + h) * D;
    if (tid < kTile) {
        int64_t s = -1;
        if (tid < n) {
            s = a.slots[t0 + tid];
            if (s < 0 || s >= a.c.n_pages * a.c.page) s = -1;
            if (a.rot) {
                const int p = a.positions[t0 + tid];
                if (p < 0 || p >= a.max_pos) s = -1;
            }
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
    auto dst = [&](int64_t slot, int d) {
        return a.c.v + (slot >> a.c.page_shift) * a.c.page_stride + (int64_t)(h * D + d) * a.c.page + (slot & (a.c.page - 1));
    };
    if (n >= 8) {  // whole pieces, 8 tokens apart from the first aligned slot: a thread per 8 tokens of two channels
        int first_at = 0;
        while (first_at < 8 && (s_slot[first_at] & 7) != 0) first_at++;
        if (tid < kTile / 8) {  // whether piece tid is whole
            const int p = first_at + 8 * tid;
            const int64_t s = s_slot[min(p, n - 1)];
            bool whole = p + 8 <= n && s >= 0 && (s & 7) == 0;
#pragma unroll
            for (int j = 1; j < 8; j++) whole = whole && s_slot[min(p + j, n - 1)] == s + j;
            s_piece[tid] = whole;
        }
        __syncthreads();
        for (int i = tid; i < kTile / 8 * (D / 2); i += 256) {
            const int q = i % (kTile / 8), p = first_at + 8 * q, d = 2 * (i / (kTile / 8));
            if (!s_piece[q]) continue;
            uint32_t x[8];
#pragma unroll
            for (int j = 0; j < 8; j++) x[j] = *reinterpret_cast<const uint32_t *>(&buf[p + j][d]);
            u32x4 lo, hi;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                lo[j] = __builtin_amdgcn_perm(x[2 * j + 1], x[2 * j], 0x05040100u);
                hi[j] = __builtin_amdgcn_perm(x[2 * j + 1], x[2 * j], 0x07060302u);
            }
            *reinterpret_cast<u32x4 *>(dst(s_slot[p], d)) = lo;
            *reinterpret_cast<u32x4 *>(dst(s_slot[p], d + 1)) = hi;
        }
        // the others one by one
        for (int t = tid / 64; t < n; t += 4) {
            const int64_t s = s_slot[t];
            if (s < 0 || (t >= first_at && t < first_at + kTile && s_piece[(t - first_at) / 8])) continue;
            for (int d = tid & 63; d < D; d += 64) *dst(s, d) = buf[t][d];
        }
        return;
    }
    for (int i = tid; i < n * D; i += 256) {
        const int t = i / D, d = i % D;
        if (s_slot[t] >= 0) *dst(s_slot[t], d) = buf[t][d];
    }
}

template <int D, bool PLAIN>
__global__ __launch_bounds__(256) void kv_append_kernel(AppendArgs a, int v_wgs, int size, int parts)
{
    __shared__ union {
        float qk[4][512 / D][D];
        uint16_t v[kTile][D + 2];
    } sh;
    __shared__ int64_t s_slot[kTile];
    __shared__ int s_piece[kTile / 8];
    if ((int)blockIdx.x < v_wgs) {  // the longer ones first
        append_v<D>(a, blockIdx.x / a.c.Hkv, size, blockIdx.x % a.c.Hkv, sh.v, s_slot, s_piece);
    } else {
        const int wave = threadIdx.x >> 6, item = (blockIdx.x - v_wgs) * 4 + wave, t = item / parts;
        if (t < a.T) append_qk<D, PLAIN>(a, t, item % parts, parts, sh.qk[wave]);
    }
}

template <int D>
hipError_t launch_d(const AppendArgs &a, hipStream_t st)
{
    const int groups = ((a.c.Hq + a.c.Hkv) * D + 511) / 512;  // groups of heads a token has
    // A wave each for a token's groups while there are few; otherwise three groups to a wave, which
    // share its angles and weights (8192 tokens of 9 groups: 38.4 us, one group 51.1, nine 43.3).
    const int parts = a.T * (int64_t)groups <= 8192 ? groups : (groups + 2) / 3;
    const int64_t qk = ((int64_t)a.T * parts + 3) / 4;
    const int size = a.T <= 512 ? kSmallTile : kTile;
    const int64_t v = (int64_t)((a.T + 7 + size - 1) / size) * a.c.Hkv;
    if (qk + v > INT32_MAX) return hipErrorInvalidValue;
    const unsigned grid = (unsigned)(qk + v);
    if (lane_rotation(a.rot, a.pairs))
        kv_append_kernel<D, true><<<grid, 256, 0, st>>>(a, (int)v, size, parts);
    else
        kv_append_kernel<D, false><<<grid, 256, 0, st>>>(a, (int)v, size, parts);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs &a, hipStream_t st)
{
    return a.c.D == 128 ? launch_d<128>(a, st) : launch_d<64>(a, st);
}

}  // namespace flint
