// logprobs.hip -- log probabilities of given tokens, entropy and the largest logits of a row.
//
// One pass over the row with a running maximum m and, to base 2 with R = m log2(e), the sums
//   s = sum 2^{x log2(e) - R},   u = sum 2^{x log2(e) - R} (x log2(e) - R)
// (R -> R': s' = 2^{R - R'} s, u' = 2^{R - R'} (u + (R - R') s)), from which
//   log2 p(v) = x_v log2(e) - R - log2 s,   entropy = ln 2 (log2 s - u / s).
// x log2(e) - R is one fused operation, exact against R as rounded.
//
// Bound by the logits' bytes; beside them the vector pipe, with an exponential (four times an
// instruction's cost) and five more instructions per value.  Measured in a loop of calls: 1024 x
// 131072 bf16 in 51 us, 5.2 TB/s, with the largest 54, with the 20 largest 64; half of the values
// masked 52, 57 and 68; 512 x 131072 fp32 with the largest 50; one row of 130953 fp32 in a graph
// with the 20 largest 10.8, without 4.7.
//
// A wave owns a contiguous piece of the row (16-byte loads, per lane statistics) and, beside the
// sums, the candidates for the top n: 64-bit keys (order of the value, then the lower index)
// gathered in LDS behind a threshold that only rises.  It starts as the n-th largest of the lanes'
// first maxima, so that a step compares one maximum per lane with it and rarely does more.  A row of
// a large batch, or a short one, is one workgroup; a long one of few is split over workgroups and a
// second launch joins the parts.  Waves sort their own keys and find their ranks among the others'
// by halving: one wave ranking all 128 took 2 us more.
#include "ops.h"

#include <algorithm>

namespace flint {

namespace {

constexpr int kWaves = 4;
constexpr int kMaxTop = 32;
constexpr int kCand = 128;  // candidate keys of a wave
constexpr float kLog2e = 1.44269504088896340736f;
static_assert(kMaxTop + 64 <= kCand, "a full step after a compaction fits");

__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }

// Orders as (value descending, index ascending): -0 == +0, NaN below -inf.
__device__ __forceinline__ uint32_t order_of(float v)
{
    uint32_t u = __float_as_uint(v);
    u = u == 0x80000000u ? 0u : u;
    const uint32_t ord = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return (u & 0x7fffffffu) > 0x7f800000u ? 0u : ord;
}
__device__ __forceinline__ uint64_t order_key(float v, uint32_t idx)
{
    return ((uint64_t)order_of(v) << 32) | (uint64_t)(0xffffffffu - idx);
}
__device__ __forceinline__ uint32_t key_index(uint64_t k) { return 0xffffffffu - (uint32_t)k; }
__device__ __forceinline__ float key_value(uint64_t k)
{
    const uint32_t o = (uint32_t)(k >> 32);
    if (o == 0u) return __uint_as_float(0x7fc00000u);
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

// m: the maximum itself (-FLT_MAX at the start, +inf if it occurred); R: what the sums stand against,
// m log2(e) as rounded.
struct Stat {
    float m, R, s, u;
};

// Beyond these log2(e) m could overflow: there only equal values are within reach of each other,
// and plain differences do.
__device__ __forceinline__ bool ordinary(float m) { return fabsf(m) < 1e38f; }

// Never contracted with what uses it: R is one number wherever it occurs, and equal maxima fall by 0
// (with a product left unrounded each raise() took the rounding of R, 6e-5 at m = 1000, into the sums).
__device__ __forceinline__ float reference(float m)
{
#pragma clang fp contract(off)
    return m * kLog2e;
}
__device__ __forceinline__ Stat nothing() { return Stat{-__FLT_MAX__, reference(-__FLT_MAX__), 0.f, 0.f}; }

// R(from) - R(to), clamped so that it never becomes -inf times zero.
__device__ __forceinline__ float fall(float from, float rf, float to, float rt)
{
    return fmaxf(ordinary(from) && ordinary(to) ? rf - rt : (from - to) * kLog2e, -1e30f);
}

// The statistics of two disjoint sets joined.
__device__ __forceinline__ Stat join(Stat a, Stat b)
{
    const float m = fmaxf(a.m, b.m), R = reference(m);
    const float da = fall(a.m, a.R, m, R), db = fall(b.m, b.R, m, R);
    const float ea = ex2(da), eb = ex2(db);
    return Stat{m, R, ea * a.s + eb * b.s, ea * (a.u + da * a.s) + eb * (b.u + db * b.s)};
}

__device__ __forceinline__ void lds_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// A wave's candidates: cnt keys in LDS (16-byte aligned), of which the n largest matter.  A key
// at or below tau cannot be among them; low is tau's value.
struct Top {
    uint64_t *buf;
    int n, cnt;
    uint64_t tau;
    float low;
};

// How many of the wave's candidates are larger than k0 and k1 (TWO: both wanted).
template <bool TWO>
__device__ __forceinline__ void larger(const Top &t, uint64_t k0, uint64_t k1, int &r0, int &r1)
{
    typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
    for (int i = 0; i < t.cnt; i += 8) {
        u64x2 o[4];
#pragma unroll
        for (int j = 0; j < 4; j++) o[j] = *reinterpret_cast<const u64x2 *>(t.buf + i + 2 * j);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            r0 += o[j >> 1][j & 1] > k0;
            if (TWO) r1 += o[j >> 1][j & 1] > k1;
        }
    }
}

// Keeps the n largest of the candidates, sorted: each key's rank is the number of larger ones
// (keys are distinct).
__device__ __forceinline__ void compact(Top &t)
{
    const int lane = threadIdx.x & 63;
    if (lane < 8 && t.cnt + lane < kCand) t.buf[t.cnt + lane] = 0;  // the last group of eight
    lds_fence();
    const uint64_t k0 = lane < t.cnt ? t.buf[lane] : 0, k1 = lane + 64 < t.cnt ? t.buf[lane + 64] : 0;
    int r0 = 0, r1 = 0;
    if (t.cnt > 64)
        larger<true>(t, k0, k1, r0, r1);
    else
        larger<false>(t, k0, k1, r0, r1);
    lds_fence();
    if (lane < t.cnt && r0 < t.n) t.buf[r0] = k0;
    if (lane + 64 < t.cnt && r1 < t.n) t.buf[r1] = k1;
    lds_fence();
    t.cnt = min(t.cnt, t.n);
    if (t.cnt == t.n) {
        t.tau = t.buf[t.n - 1];
        t.low = key_value(t.tau);
    }
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

// A first threshold from one value's order per lane (0 where it has none): the n-th largest of
// them, to 16 bits, downwards.  n lanes have a value at or above it, so nothing below can be in
// the result.
__device__ __forceinline__ void first_threshold(Top &t, uint32_t ord)
{
    uint32_t at = 0;
#pragma unroll
    for (int b = 31; b >= 16; b--) {
        const uint32_t up = at | (1u << b);
        if (__popcll(__ballot(ord >= up)) >= t.n) at = up;
    }
    if (at == 0) return;
    t.tau = (uint64_t)at << 32;  // below every key of that order
    t.low = key_value(t.tau);
}

__device__ __forceinline__ float load_one(const uint16_t *p) { return bf2f(*p); }
__device__ __forceinline__ float load_one(const float *p) { return *p; }

// The maximum rises to mx where that is higher.
__device__ __forceinline__ void raise(Stat &st, float mx)
{
    const float m = fmaxf(mx, st.m), R = reference(m), d = fall(st.m, st.R, m, R), r = ex2(d);
    st.u = r * (st.u + d * st.s);
    st.s = r * st.s;
    st.m = m;
    st.R = R;
}
// Adds a value; ord: the lane's maximum is ordinary.  -inf adds 0, not 0 * -inf.
__device__ __forceinline__ void add_any(Stat &st, float x, bool ord)
{
    const float t = ord ? fmaf(x, kLog2e, -st.R) : (x - st.m) * kLog2e, e = ex2(t);
    st.s += e;
    st.u = fmaf(e, fmaxf(t, -1e4f), st.u);
}

// The 16-byte pieces of a row: head elements before the first, n pieces, tail elements behind.
template <typename E>
struct Pieces {
    static constexpr int EPC = 16 / sizeof(E);
    int head, n, tail;
    __device__ __forceinline__ Pieces(const E *row, int V)
    {
        head = min((int)((16 - ((uintptr_t)row & 15)) & 15) / (int)sizeof(E), V);
        n = (V - head) / EPC;
        tail = V - head - n * EPC;
    }
};

constexpr int kU = 4;            // pieces per lane and step
constexpr int kStep = 64 * kU;   // pieces of a step

// Value `at` of a lane's pieces, chosen among registers a bit of its place at a time.
template <int EPC>
__device__ __forceinline__ float value_at(const u32x4 *v, int at)
{
    const int d = EPC == 8 ? at >> 1 : at;
    uint32_t r[4 * kU];
#pragma unroll
    for (int i = 0; i < 4 * kU; i++) r[i] = v[i >> 2][i & 3];
#pragma unroll
    for (int b = 3; b >= 0; b--) {
        const uint32_t m = 0u - (uint32_t)((d >> b) & 1);
#pragma unroll
        for (int i = 0; i < (1 << b); i++) r[i] = (m & r[i + (1 << b)]) | (~m & r[i]);
    }
    return __uint_as_float(EPC == 4 ? r[0] : (at & 1) ? r[0] & 0xffff0000u : r[0] << 16);
}

// A wave over pieces [c_lo, c_hi) of a row, in ascending order.
template <typename E>
__device__ __forceinline__ void scan(const E *row, const Pieces<E> &pc, int c_lo, int c_hi, Stat &st, Top &top)
{
    constexpr int EPC = Pieces<E>::EPC;
    const uint32_t none = EPC == 8 ? 0xff80ff80u : 0xff800000u;  // -inf
    const int lane = threadIdx.x & 63;
    for (int c0 = c_lo; c0 < c_hi; c0 += kStep) {
        const int e0 = pc.head + (c0 + lane) * EPC;  // this lane's piece q starts 64 q EPC further
        auto in = [&](int q) { return c0 + 64 * q + lane < c_hi; };
        u32x4 v[kU];
        if (c0 + kStep <= c_hi) {
#pragma unroll
            for (int q = 0; q < kU; q++)  // read once: nothing of it need stay in the caches
                v[q] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(row + e0 + 64 * q * EPC));
        } else {
#pragma unroll
            for (int q = 0; q < kU; q++) {
                v[q] = u32x4{none, none, none, none};
                if (in(q)) v[q] = *reinterpret_cast<const u32x4 *>(row + e0 + 64 * q * EPC);
            }
        }
        float x[kU][EPC];
#pragma unroll
        for (int q = 0; q < kU; q++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                if constexpr (EPC == 8) {
                    x[q][2 * i] = __uint_as_float(v[q][i] << 16);
                    x[q][2 * i + 1] = __uint_as_float(v[q][i] & 0xffff0000u);
                } else {
                    x[q][i] = __uint_as_float(v[q][i]);
                }
            }
        float mx = x[0][0], mn = x[0][0];
#pragma unroll
        for (int q = 0; q < kU; q++)
#pragma unroll
            for (int i = 0; i < EPC; i++) {
                mx = fmaxf(mx, x[q][i]);
                mn = fminf(mn, x[q][i]);
            }
        if (__any(mx > st.m)) raise(st, mx);
        const bool ord = ordinary(st.m);
        const float R = ord ? st.R : 0.f;  // not: far out, or nothing but -inf so far
        if (!__any(!(mn > -1e38f) || !ord)) {
#pragma unroll
            for (int q = 0; q < kU; q++)
#pragma unroll
                for (int i = 0; i < EPC; i++) {
                    const float t = fmaf(x[q][i], kLog2e, -R), e = ex2(t);
                    st.s += e;
                    st.u = fmaf(e, t, st.u);
                }
        } else if (!__any(!ord && mx != -__builtin_inff())) {  // masked values: -inf adds 0, not 0 * -inf
#pragma unroll
            for (int q = 0; q < kU; q++)
#pragma unroll
                for (int i = 0; i < EPC; i++) {
                    const float t = fmaf(x[q][i], kLog2e, -R), e = ex2(t);
                    st.s += e;
                    st.u = fmaf(e, fmaxf(t, -1e4f), st.u);
                }
        } else {
#pragma unroll
            for (int q = 0; q < kU; q++)
#pragma unroll
                for (int i = 0; i < EPC; i++) add_any(st, x[q][i], ord);
        }
        if (top.n == 0) continue;
        if (c0 == c_lo) {
            float best = mx;  // of values that are there: a missing piece's -inf are none
            if (c0 + kStep > c_hi) {
                best = __uint_as_float(0x7fc00000u);
#pragma unroll
                for (int q = 0; q < kU; q++)
#pragma unroll
                    for (int i = 0; i < EPC; i++)
                        if (in(q)) best = fmaxf(best, x[q][i]);
            }
            first_threshold(top, order_of(best));
            if (!(top.low > -__builtin_inff())) {  // most lanes have masked values alone: do enough others exist?
                float others = 0.f;
#pragma unroll
                for (int q = 0; q < kU; q++)
#pragma unroll
                    for (int i = 0; i < EPC; i++) others += x[q][i] > -__builtin_inff() ? 1.f : 0.f;
                if (wave_sum(others) >= (float)top.n) {  // then no -inf is in the result
                    top.tau = ((uint64_t)order_of(-__builtin_inff()) << 32) | 0xffffffffu;
                    top.low = -__FLT_MAX__;
                }
            }
        } else if (!__any(!(mx <= top.low))) {
            continue;  // equal values come later here: their indices are higher
        }
        // A bit for each value that may pass, the first in the highest place.  low is a number
        // once n candidates are known, a NaN before (every value passes).
        uint32_t may = 0;
#pragma unroll
        for (int q = 0; q < kU; q++)
#pragma unroll
            for (int i = 0; i < EPC; i++) may = 2 * may + !(x[q][i] < top.low);
        if (c0 + kStep > c_hi)
#pragma unroll
            for (int q = 0; q < kU; q++)
                if (!in(q)) may &= ~(((1u << EPC) - 1) << (EPC * (kU - 1 - q)));
        while (__any(may != 0)) {  // one value of each lane at a time
            const bool have = may != 0;
            const int at = have ? kU * EPC - 1 - (31 - __builtin_clz(may)) : 0;
            const int e = e0 + 64 * EPC * (at / EPC) + at % EPC;
            if (have) may ^= 1u << (kU * EPC - 1 - at);
            offer(top, have, order_key(value_at<EPC>(v, at), (uint32_t)e));
        }
        if (top.cnt >= 2 * top.n + 16) compact(top);  // a higher threshold for the steps to come
    }
}

// The at most 2 (EPC - 1) elements around the pieces, one per lane.
template <typename E>
__device__ __forceinline__ void scan_edges(const E *row, const Pieces<E> &pc, Stat &st, Top &top)
{
    const int lane = threadIdx.x & 63;
    const bool have = lane < pc.head + pc.tail;
    if (!__any(have)) return;
    const int e = lane < pc.head ? lane : pc.n * Pieces<E>::EPC + lane;
    const float x = have ? load_one(row + e) : -__builtin_inff();
    raise(st, x);
    add_any(st, x, ordinary(st.m));
    if (top.n) offer(top, have, order_key(x, (uint32_t)e));
}

struct Part {
    float m, R, s, u;
};

__device__ __forceinline__ float wave_max(float v)
{
    v = fmaxf(v, __int_as_float(FLINT_DPP(__float_as_int(v), 0xB1)));
    v = fmaxf(v, __int_as_float(FLINT_DPP(__float_as_int(v), 0x4E)));
    v = fmaxf(v, __int_as_float(FLINT_DPP(__float_as_int(v), 0x141)));
    v = fmaxf(v, __int_as_float(FLINT_DPP(__float_as_int(v), 0x140)));
    const float a = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 0));
    const float b = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16));
    const float c = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 32));
    const float d = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 48));
    return fmaxf(fmaxf(a, b), fmaxf(c, d));
}
__device__ __forceinline__ Stat wave_join(Stat st)
{
    raise(st, wave_max(st.m));
    return Stat{st.m, st.R, wave_sum(st.s), wave_sum(st.u)};
}

// The logit of the row's token, -inf outside the vocabulary (fetched ahead of its use).
__device__ __forceinline__ float token_logit(const LogprobArgs &a, int t)
{
    if (!a.logprob) return 0.f;
    const int id = a.tokens[t];
    if (id < 0 || id >= a.V) return -__builtin_inff();
    return a.fp32 ? ((const float *)a.logits)[t * a.ld + id] : bf2f(((const uint16_t *)a.logits)[t * a.ld + id]);
}

// The row's outputs from its statistics and its sorted top keys (one wave).
__device__ __forceinline__ void finish(const LogprobArgs &a, int t, Stat st, const uint64_t *keys, float x)
{
    const int lane = threadIdx.x & 63;
    constexpr float kLn2 = 0.693147180559945309417f;
    const float ls = log2f(st.s);
    auto lp = [&](float v) {
        if (st.s == 0.f) return -__builtin_inff();  // nothing in the row but -inf
        const bool ord = ordinary(st.m) && ordinary(v);
        return ord ? (fmaf(v, kLog2e, -st.R) - ls) * kLn2 : v - st.m - ls * kLn2;
    };
    if (lane < a.n) {
        const uint64_t k = keys[lane];
        a.top_ids[(int64_t)t * a.n + lane] = (int32_t)key_index(k);
        a.top_logprobs[(int64_t)t * a.n + lane] = lp(key_value(k));
    }
    if (lane == 0) {
        if (a.entropy) a.entropy[t] = st.s == 0.f ? 0.f : (ls - st.u / st.s) * kLn2;
        if (a.logprob) a.logprob[t] = lp(x);
    }
}

// LDS of a workgroup: its waves' candidates, statistics and counts, and the joined top keys.
struct Shared {
    alignas(16) uint64_t cand[kWaves][kCand];
    uint64_t best[kMaxTop];
    Stat stats[kWaves];
    int counts[kWaves];
};

// The workgroup's waves joined: wave 0 returns with the statistics of all, and sh.best holds the
// n largest candidates, sorted (cnt of them).  Each wave sorts its own, and a key's rank is the sum
// of its ranks in the waves' lists, found by halving.
__device__ __forceinline__ bool join_waves(Stat &st, Top &top, Shared &sh, int &cnt)
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    st = wave_join(st);
    if (top.n) compact(top);
    if (lane == 0) {
        sh.stats[wave] = st;
        sh.counts[wave] = top.cnt;
    }
    __syncthreads();
    cnt = 0;
    if (top.n) {
        const uint64_t key = lane < top.cnt ? top.buf[lane] : 0;
        int rank = lane;
#pragma unroll
        for (int w = 0; w < kWaves; w++) {
            const int have = sh.counts[w];
            cnt += have;
            if (w == wave) continue;
            int at = 0;  // keys of list w that are larger
#pragma unroll
            for (int by = kMaxTop; by; by /= 2)
                if (at + by <= have && sh.cand[w][at + by - 1] > key) at += by;
            rank += at;
        }
        if (lane < top.cnt && rank < top.n) sh.best[rank] = key;
        cnt = min(cnt, top.n);
        __syncthreads();
    }
    if (wave) return false;
#pragma unroll
    for (int w = 1; w < kWaves; w++) st = join(st, sh.stats[w]);
    return true;
}

// Workgroup (part p of S, row t).  S == 1: the row's outputs; otherwise its part's statistics
// and top keys go to the workspace: Part [T][S], then keys [T][S][n], 0 where there is none.
template <typename E>
__global__ __launch_bounds__(64 * kWaves) void logprobs_kernel(LogprobArgs a, int S)
{
    __shared__ Shared sh;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int t = blockIdx.x / S, p = blockIdx.x % S;
    const E *row = (const E *)a.logits + t * a.ld;
    const float x = S == 1 ? token_logit(a, t) : 0.f;
    const Pieces<E> pc(row, a.V);
    const int waves = S * kWaves, mine = p * kWaves + wave, steps = (pc.n + kStep - 1) / kStep;
    const int lo = steps * mine / waves * kStep, hi = min(steps * (mine + 1) / waves * kStep, pc.n);
    Stat st = nothing();
    Top top{sh.cand[wave], a.n, 0, 0, __uint_as_float(0x7fc00000u)};
    if (lo < hi) scan(row, pc, lo, hi, st, top);
    if (mine == waves - 1) scan_edges(row, pc, st, top);
    int cnt;
    if (!join_waves(st, top, sh, cnt)) return;
    if (S == 1) {
        finish(a, t, st, sh.best, x);
        return;
    }
    Part *ps = (Part *)a.ws;
    uint64_t *keys = (uint64_t *)(ps + (int64_t)a.T * S);
    const int64_t at = (int64_t)t * S + p;
    if (lane == 0) ps[at] = Part{st.m, st.R, st.s, st.u};
    if (lane < a.n) keys[at * a.n + lane] = lane < cnt ? sh.best[lane] : 0;
}

// One workgroup per row: its parts joined.
constexpr int kMaxParts = 64;
__global__ __launch_bounds__(64 * kWaves) void logprobs_join_kernel(LogprobArgs a, int S)
{
    __shared__ Shared sh;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), t = blockIdx.x;
    const float x = token_logit(a, t);
    const Part *ps = (const Part *)a.ws + (int64_t)t * S;
    const uint64_t *keys = (const uint64_t *)((const Part *)a.ws + (int64_t)a.T * S) + (int64_t)t * S * a.n;
    Stat st = nothing();
    if (tid < S) st = Stat{ps[tid].m, ps[tid].R, ps[tid].s, ps[tid].u};
    Top top{sh.cand[wave], a.n, 0, 0, 0.f};
    if (a.n) {
        constexpr int PER = kMaxParts * kMaxTop / (64 * kWaves);
        uint64_t k[PER], best = 0;
#pragma unroll
        for (int i = 0; i < PER; i++) {
            k[i] = tid + 64 * kWaves * i < S * a.n ? keys[tid + 64 * kWaves * i] : 0;
            best = max(best, k[i]);
        }
        first_threshold(top, (uint32_t)(best >> 32));
#pragma unroll
        for (int i = 0; i < PER; i++) offer(top, k[i] != 0, k[i]);
    }
    int cnt;
    if (join_waves(st, top, sh, cnt)) finish(a, t, st, sh.best, x);
}

// Parts per row: enough workgroups for the GPU, at least 2048 values each; but a short row is one
// launch's work (one row of 17000 values: 6.7 us with the largest, 9.8 with the 20 largest, in parts
// 5.2 + 3.8 and 6.6 + 5.1; 32 rows of 24000: 9.1 and 12.8, in parts 5.7 + 4.5 and 7.2 + 5.5; 32 rows
// of 32001: 10.9 and 14.6, in parts 6.0 + 4.6 and 7.3 + 5.8).  16 waves to a row were no faster: the
// vector pipes of one CU are busy with 4.
constexpr int kShortRow = 24576;
int parts(int T, int V)
{
    int s = 1;
    if (V <= kShortRow) return s;
    while (s < kMaxParts && (int64_t)T * s < 512 && V / (2 * s) >= 2048) s *= 2;
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

size_t logprobs_call_bytes(int64_t T, int V, int n)
{
    const int s = parts((int)T, V);
    return s > 1 ? (size_t)T * s * (sizeof(Part) + 8 * (size_t)n) : 0;
}

hipError_t launch_token_logprobs(const LogprobArgs &a, hipStream_t st)
{
    const int S = parts(a.T, a.V);
    if (a.fp32)
        logprobs_kernel<float><<<(unsigned)(a.T * S), 64 * kWaves, 0, st>>>(a, S);
    else
        logprobs_kernel<uint16_t><<<(unsigned)(a.T * S), 64 * kWaves, 0, st>>>(a, S);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || S == 1) return e;
    logprobs_join_kernel<<<(unsigned)a.T, 64 * kWaves, 0, st>>>(a, S);
    return hipGetLastError();
}

}  // namespace flint
