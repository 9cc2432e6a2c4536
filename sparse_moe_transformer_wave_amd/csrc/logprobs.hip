// logprobs.hip -- log probabilities of given tokens, entropy and the largest logits of a row.
//
// One pass over the row with a running maximum m and the sums
//   s = sum e^{x - m},   u = sum e^{x - m} (x - m)
// (m -> m': s' = e^{m - m'} s, u' = e^{m - m'} (u + (m - m') s)), from which
//   log p(v) = x_v - m - log s,   entropy = log s - u / s.
// Bound by the logits' bytes.  A wave owns a contiguous piece of the row (16-byte loads, per
// lane statistics) and, beside the sums, the candidates for the top n: 64-bit keys (order of
// the value, then the lower index) gathered in LDS behind a threshold that only rises.  A
// row of a large batch is one workgroup; with few rows a row is split over workgroups and a
// second launch joins the parts.
#include "ops.h"

#include <algorithm>

namespace flint {

namespace {

constexpr int kWaves = 4;
constexpr int kCand = 128;      // candidate keys of a wave
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kMaxTop = 32;

// Orders as (value descending, index ascending): -0 == +0, NaN below -inf.
__device__ __forceinline__ uint64_t order_key(float v, uint32_t idx)
{
    uint32_t u = __float_as_uint(v);
    u = u == 0x80000000u ? 0u : u;
    uint32_t ord = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    ord = (u & 0x7fffffffu) > 0x7f800000u ? 0u : ord;
    return ((uint64_t)ord << 32) | (uint64_t)(0xffffffffu - idx);
}
__device__ __forceinline__ uint32_t key_index(uint64_t k) { return 0xffffffffu - (uint32_t)k; }
__device__ __forceinline__ float key_value(uint64_t k)
{
    const uint32_t o = (uint32_t)(k >> 32);
    if (o == 0u) return __uint_as_float(0x7fc00000u);
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

struct Stat {
    float m, s, u;
};

// The statistics of two disjoint sets joined.  Maxima are finite or +inf (-FLT_MAX at the
// start), so their difference is clamped rather than allowed to overflow to -inf times zero.
__device__ __forceinline__ Stat join(Stat a, Stat b)
{
    const float m = fmaxf(a.m, b.m);
    const float da = fmaxf(a.m - m, -1e30f), db = fmaxf(b.m - m, -1e30f);
    const float ea = exp2f(da * kLog2e), eb = exp2f(db * kLog2e);
    return Stat{m, ea * a.s + eb * b.s, ea * (a.u + da * a.s) + eb * (b.u + db * b.s)};
}

// A wave's candidates: cnt keys in LDS, of which the n largest matter; tau = the n-th
// largest key once there are n (an element with a smaller key cannot be in the result).
struct Top {
    uint64_t *buf;
    int n, cnt;
    uint64_t tau;
};

// Keeps the n largest of the candidates, sorted: each key's rank is the number of larger
// ones (keys are distinct).
__device__ __forceinline__ void compact(Top &t)
{
    const int lane = threadIdx.x & 63;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const uint64_t k0 = lane < t.cnt ? t.buf[lane] : 0, k1 = lane + 64 < t.cnt ? t.buf[lane + 64] : 0;
    int r0 = 0, r1 = 0;
    for (int i = 0; i < t.cnt; i++) {
        const uint64_t o = t.buf[i];
        r0 += o > k0;
        r1 += o > k1;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (lane < t.cnt && r0 < t.n) t.buf[r0] = k0;
    if (lane + 64 < t.cnt && r1 < t.n) t.buf[r1] = k1;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    t.cnt = min(t.cnt, t.n);
    if (t.cnt == t.n) t.tau = t.buf[t.n - 1];
}

// Offers one key per lane (have: whether this lane has one).
__device__ __forceinline__ void offer(Top &t, bool have, uint64_t key)
{
    const int lane = threadIdx.x & 63;
    uint64_t mask = __ballot(have && key > t.tau);
    if (mask == 0) return;
    if (t.cnt + __popcll(mask) > kCand) {
        compact(t);
        mask = __ballot(have && key > t.tau);
    }
    if ((mask >> lane) & 1) t.buf[t.cnt + __popcll(mask & ((1ull << lane) - 1))] = key;
    t.cnt += __popcll(mask);
}

template <typename E>
__device__ __forceinline__ float load_one(const E *p);
template <>
__device__ __forceinline__ float load_one<uint16_t>(const uint16_t *p) { return bf2f(*p); }
template <>
__device__ __forceinline__ float load_one<float>(const float *p) { return *p; }

// A wave over elements [lo, hi) of a row.  EPC elements per 16-byte chunk; chunks are
// aligned, so the first and the last may be partial.
template <typename E>
__device__ __forceinline__ void scan(const E *row, int lo, int hi, Stat &st, Top &top)
{
    constexpr int EPC = 16 / sizeof(E), U = 16 / EPC;  // 16 elements per lane and step
    const int lane = threadIdx.x & 63;
    const int lead = (int)(((uintptr_t)(row + lo) & 15) / sizeof(E));  // elements before lo in its chunk
    const int base = lo - lead;                                       // index of chunk 0's first element
    const int chunks = (hi - base + EPC - 1) / EPC;
    for (int c0 = 0; c0 < chunks; c0 += 64 * U) {
        float x[U][EPC];
#pragma unroll
        for (int q = 0; q < U; q++) {
            const int e0 = base + (c0 + 64 * q + lane) * EPC;
            if (e0 >= lo && e0 + EPC <= hi) {
                const u32x4 v = *reinterpret_cast<const u32x4 *>(row + e0);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    if (EPC == 8) {
                        x[q][2 * i] = bf2f(v[i] & 0xffffu);
                        x[q][2 * i + 1] = bf2f(v[i] >> 16);
                    } else {
                        x[q][i] = __uint_as_float(v[i]);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < EPC; i++)
                    x[q][i] = e0 + i >= lo && e0 + i < hi ? load_one(row + e0 + i) : -__builtin_inff();
            }
        }
        float mx = st.m;
#pragma unroll
        for (int q = 0; q < U; q++)
#pragma unroll
            for (int i = 0; i < EPC; i++) mx = fmaxf(mx, x[q][i]);
        const float d = fmaxf(st.m - mx, -1e30f), r = exp2f(d * kLog2e);
        st.u = r * (st.u + d * st.s);
        st.s = r * st.s;
        st.m = mx;
#pragma unroll
        for (int q = 0; q < U; q++)
#pragma unroll
            for (int i = 0; i < EPC; i++) {
                const float t = x[q][i] - mx, e = exp2f(t * kLog2e);
                st.s += e;
                st.u = fmaf(e, fmaxf(t, -1e4f), st.u);  // -inf adds 0, not 0 * -inf
            }
        if (top.n) {
#pragma unroll
            for (int q = 0; q < U; q++)
#pragma unroll
                for (int i = 0; i < EPC; i++) {
                    const int e = base + (c0 + 64 * q + lane) * EPC + i;
                    offer(top, e >= lo && e < hi, order_key(x[q][i], (uint32_t)e));
                }
        }
    }
}

struct Part {
    float m, s, u, pad;
};

__device__ __forceinline__ Stat wave_join(Stat st)
{
#pragma unroll
    for (int m = 1; m < 64; m *= 2)
        st = join(st, Stat{__shfl_xor(st.m, m), __shfl_xor(st.s, m), __shfl_xor(st.u, m)});
    return st;
}

// The row's outputs from its statistics and its sorted top keys (one wave).
__device__ __forceinline__ void finish(const LogprobArgs &a, int t, Stat st, const uint64_t *keys)
{
    const int lane = threadIdx.x & 63;
    const float ls = logf(st.s);
    auto lp = [&](float x) { return st.s == 0.f ? -__builtin_inff() : x - st.m - ls; };
    if (lane < a.n) {
        const uint64_t k = keys[lane];
        a.top_ids[(int64_t)t * a.n + lane] = (int32_t)key_index(k);
        a.top_logprobs[(int64_t)t * a.n + lane] = lp(key_value(k));
    }
    if (lane == 0) {
        if (a.entropy) a.entropy[t] = st.s == 0.f ? 0.f : ls - st.u / st.s;
        if (a.logprob) {
            const int id = a.tokens[t];
            float x = -__builtin_inff();
            if (id >= 0 && id < a.V)
                x = a.fp32 ? ((const float *)a.logits)[t * a.ld + id] : bf2f(((const uint16_t *)a.logits)[t * a.ld + id]);
            a.logprob[t] = lp(x);
        }
    }
}

// Workgroup (part p of S, row t).  S == 1: the row's outputs; otherwise its part's
// statistics and top keys go to the workspace: Part [T][S], then keys [T][S][n].
template <typename E>
__global__ __launch_bounds__(64 * kWaves) void logprobs_kernel(LogprobArgs a, int S)
{
    __shared__ uint64_t cand[kWaves][kCand];
    __shared__ Stat stats[kWaves];
    __shared__ int counts[kWaves];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int t = blockIdx.x / S, p = blockIdx.x % S;
    const E *row = (const E *)a.logits + t * a.ld;
    const int pieces = S * kWaves, mine = p * kWaves + wave;
    const int lo = (int)((int64_t)a.V * mine / pieces), hi = (int)((int64_t)a.V * (mine + 1) / pieces);
    Stat st{-__FLT_MAX__, 0.f, 0.f};
    Top top{cand[wave], a.n, 0, 0};
    if (lo < hi) scan(row, lo, hi, st, top);
    st = wave_join(st);
    if (a.n) compact(top);
    if (lane == 0) {
        stats[wave] = st;
        counts[wave] = top.cnt;
    }
    __syncthreads();
    if (wave) return;
    for (int w = 1; w < kWaves; w++) {
        st = join(st, stats[w]);
        if (a.n) offer(top, lane < counts[w], lane < counts[w] ? cand[w][lane] : 0);
    }
    if (a.n) compact(top);
    if (S == 1) {
        finish(a, t, st, top.buf);
        return;
    }
    Part *ps = (Part *)a.ws;
    uint64_t *keys = (uint64_t *)(ps + (int64_t)a.T * S);
    const int64_t at = (int64_t)t * S + p;
    if (lane == 0) ps[at] = Part{st.m, st.s, st.u, 0.f};
    if (lane < a.n) keys[at * a.n + lane] = lane < top.cnt ? top.buf[lane] : 0;  // 0: no element
}

__global__ __launch_bounds__(64) void logprobs_join_kernel(LogprobArgs a, int S)
{
    __shared__ uint64_t cand[kCand];
    const int lane = threadIdx.x, t = blockIdx.x;
    const Part *ps = (const Part *)a.ws + (int64_t)t * S;
    const uint64_t *keys = (const uint64_t *)((const Part *)a.ws + (int64_t)a.T * S) + (int64_t)t * S * a.n;
    Stat st{-__FLT_MAX__, 0.f, 0.f};
    for (int i = lane; i < S; i += 64) st = join(st, Stat{ps[i].m, ps[i].s, ps[i].u});
    st = wave_join(st);
    Top top{cand, a.n, 0, 0};
    if (a.n) {
        for (int i = 0; i < S * a.n; i += 64) {
            const uint64_t k = i + lane < S * a.n ? keys[i + lane] : 0;
            offer(top, k != 0, k);
        }
        compact(top);
    }
    finish(a, t, st, cand);
}

// Parts per row: enough workgroups for the GPU, at least 4096 elements each.
int parts(int T, int V)
{
    int s = 1;
    while (s < 64 && (int64_t)T * s < 512 && V / (2 * s) >= 4096) s *= 2;
    return s;
}

}  // namespace

size_t logprobs_ws_bytes(int64_t T, int V, int n)
{
    size_t most = 16;
    // fewer rows may take more parts: the largest T * parts over all batches up to T
    for (int64_t t = 1; t <= T && t <= 512; t++) {
        const int s = parts((int)t, V);
        if (s > 1) most = std::max(most, (size_t)t * s * (sizeof(Part) + 8 * (size_t)n));
    }
    return most;
}

hipError_t launch_token_logprobs(const LogprobArgs &a, hipStream_t st)
{
    const int S = parts(a.T, a.V);
    if (a.fp32)
        logprobs_kernel<float><<<(unsigned)(a.T * S), 64 * kWaves, 0, st>>>(a, S);
    else
        logprobs_kernel<uint16_t><<<(unsigned)(a.T * S), 64 * kWaves, 0, st>>>(a, S);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || S == 1) return e;
    logprobs_join_kernel<<<(unsigned)a.T, 64, 0, st>>>(a, S);
    return hipGetLastError();
}

}  // namespace flint
