// logits.hip -- penalties for repeated tokens, biases and grammar masks on logits.
//
//   x = l;  seen: x > 0 ? x / r : x r;  x -= f c + p [c > 0];  x += bias;  not allowed: -inf
//
// A workgroup takes a range of one row's vocabulary: it counts the row's history in LDS (a word per
// token of its range: a bit for the prompt's, a count for the row's own; sums of whole numbers, so
// their order does not matter), then applies everything to its values in registers and rounds once.
// The biases take the same LDS words in a second turn, where the row has any: the highest entry of a
// token stays.  Every workgroup of a row reads the whole history, from L2.
//
// Bound by the logits' bytes, read and written once; in place only pieces of 16 bytes that something
// changes are touched.
#include "serve.h"

namespace flint {

namespace {

constexpr int kVals = 16;  // values of a thread
constexpr uint32_t kPrompt = 0x80000000u;
constexpr uint32_t kNegInf = 0xff800000u;

template <typename E>
__device__ __forceinline__ float widen(E v)
{
    if constexpr (sizeof(E) == 4)
        return v;
    else
        return bf2f(v);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}
template <typename E>
__device__ __forceinline__ E narrow(float v)
{
    if constexpr (sizeof(E) == 4)
        return v;
    else
        return (E)pack_bf16(v, 0.f);
}

// The rules of a row.
struct Row {
    const int32_t *history;
    int total, prompt;
    float rep, freq, pres;
    int b0, b1;             // its bias entries
    const uint32_t *mask;   // or null
};
__device__ __forceinline__ Row row_of(const LogitsArgs &a, int t)
{
    Row r;
    r.history = a.history ? a.history + t * a.ldh : nullptr;
    r.total = r.prompt = 0;
    if (a.history) {
        const int64_t n = a.total_len ? min((int64_t)max(a.total_len[t], 0), a.ldh) : a.ldh;
        r.total = (int)n;
        r.prompt = a.prompt_len ? min(max(a.prompt_len[t], 0), r.total) : 0;
    }
    r.rep = a.repetition ? a.repetition[t] : 1.f;
    r.freq = a.frequency ? a.frequency[t] : 0.f;
    r.pres = a.presence ? a.presence[t] : 0.f;
    r.b0 = r.b1 = 0;
    if (a.bias_start) {
        r.b0 = max(a.bias_start[t], 0);
        r.b1 = (int)min((int64_t)a.bias_start[t + 1], a.n_bias);
    }
    r.mask = nullptr;
    if (a.masks) {
        const int64_t m = a.mask_rows ? a.mask_rows[t] : t;
        if (m >= 0 && m < a.n_masks) r.mask = a.masks + m * a.ldm;
    }
    return r;
}

// The first launch parameter's ranges: W threads and 16 W values, from `head` on where pieces of 16
// bytes are aligned (VEC; the first range takes the elements before them too) or from 0.
// SAME: out is logits.
template <typename E, int W, bool VEC, bool SAME>
__global__ __launch_bounds__(W) void logits_kernel(LogitsArgs a, int ranges)
{
    constexpr int EPC = VEC ? 16 / sizeof(E) : 1, NP = kVals / EPC;
    __shared__ uint32_t word[kVals * W + 8];
    const int tid = threadIdx.x, t = blockIdx.x / ranges, c = blockIdx.x % ranges;
    const E *in = (const E *)a.logits + t * a.ld;
    E *out = (E *)a.out + t * a.ldo;
    const int head = VEC ? min((int)((16 - ((uintptr_t)in & 15)) & 15) / (int)sizeof(E), a.V) : 0;
    const int lo = c == 0 ? 0 : head + c * kVals * W, hi = min(head + (c + 1) * kVals * W, a.V), first = head + c * kVals * W;
    if (lo >= hi) return;
    const Row r = row_of(a, t);
    // this thread's pieces, and one element before them
    auto at = [&](int q) { return first + (tid + W * q) * EPC; };
    typedef E piece_t __attribute__((ext_vector_type(EPC == 1 ? 2 : EPC)));
    float x[NP][EPC], edge = 0.f;
    const bool has_edge = VEC && c == 0 && tid < head;
    auto load = [&](int q) {
        const int e = at(q);
        if (EPC > 1 && e + EPC <= hi) {
            const piece_t v = *reinterpret_cast<const piece_t *>(in + e);
#pragma unroll
            for (int i = 0; i < EPC; i++) x[q][i] = widen<E>(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < EPC; i++) x[q][i] = e + i < hi ? widen<E>(in[e + i]) : 0.f;
        }
    };
    if (!SAME) {  // on their way while the history is counted
#pragma unroll
        for (int q = 0; q < NP; q++) load(q);
        if (has_edge) edge = widen<E>(in[tid]);
    }
    const bool counted = r.total > 0, biased = r.b0 < r.b1;
    uint32_t touched = 0;  // a bit per piece that changes; the highest for the edge
    auto clear = [&] {
        for (int i = tid; i < hi - lo; i += W) word[i] = 0;
        __syncthreads();
    };
    if (counted) {
        clear();
        const uint32_t n = hi - lo;
        for (int i = tid; i < r.total; i += W) {
            const uint32_t v = (uint32_t)r.history[i] - (uint32_t)lo;
            if (v < n) {
                if (i < r.prompt)
                    atomicOr(&word[v], kPrompt);
                else
                    atomicAdd(&word[v], 1u);
            }
        }
        __syncthreads();
        auto penalise = [&](float &v, uint32_t w) {
            if (w == 0) return;
            v = v > 0.f ? v / r.rep : v * r.rep;
            const uint32_t own = w & ~kPrompt;
            if (own) v = v - r.freq * (float)own - r.pres;
        };
#pragma unroll
        for (int q = 0; q < NP; q++) {
            uint32_t w[EPC], any = 0;
#pragma unroll
            for (int i = 0; i < EPC; i++) {
                w[i] = at(q) + i < hi ? word[at(q) + i - lo] : 0;
                any |= w[i];
            }
            if (!any) continue;
            if (SAME) load(q);
            touched |= 1u << q;
#pragma unroll
            for (int i = 0; i < EPC; i++) penalise(x[q][i], w[i]);
        }
        if (has_edge && word[tid]) {
            if (SAME) edge = widen<E>(in[tid]);
            touched |= 1u << 31;
            penalise(edge, word[tid]);
        }
    }
    if (biased) {
        if (counted) __syncthreads();
        clear();
        const uint32_t n = hi - lo;
        for (int i = r.b0 + tid; i < r.b1; i += W) {
            const uint32_t v = (uint32_t)a.bias_ids[i] - (uint32_t)lo;
            if (v < n) atomicMax(&word[v], (uint32_t)(i - r.b0) + 1u);
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < NP; q++) {
            uint32_t w[EPC], any = 0;
#pragma unroll
            for (int i = 0; i < EPC; i++) {
                w[i] = at(q) + i < hi ? word[at(q) + i - lo] : 0;
                any |= w[i];
            }
            if (!any) continue;
            if (SAME && !((touched >> q) & 1)) load(q);
            touched |= 1u << q;
#pragma unroll
            for (int i = 0; i < EPC; i++)
                if (w[i]) x[q][i] += a.bias[r.b0 + w[i] - 1];
        }
        if (has_edge && word[tid]) {
            if (SAME && !(touched >> 31)) edge = widen<E>(in[tid]);
            touched |= 1u << 31;
            edge += a.bias[r.b0 + word[tid] - 1];
        }
    }
    auto store = [&](int q) {
        const int e = at(q);
        if (e >= hi) return;
        if (EPC > 1 && e + EPC <= hi) {
            piece_t v;
            if constexpr (sizeof(E) == 4) {
#pragma unroll
                for (int i = 0; i < EPC; i++) v[i] = x[q][i];
            } else {
#pragma unroll
                for (int i = 0; i + 1 < EPC; i += 2) {
                    const uint32_t p = pack_bf16(x[q][i], x[q][i + 1]);
                    v[i] = (E)p;
                    v[i + 1] = (E)(p >> 16);
                }
            }
            *reinterpret_cast<piece_t *>(out + e) = v;
        } else {
#pragma unroll
            for (int i = 0; i < EPC; i++)
                if (e + i < hi) out[e + i] = narrow<E>(x[q][i]);
        }
    };
    const float ninf = __uint_as_float(kNegInf);
#pragma unroll
    for (int q = 0; q < NP; q++) {
        const int e = at(q);
        if (e >= hi) continue;
        uint32_t keep = (1u << EPC) - 1;
        if (r.mask) {
            const int last = min(e + EPC, hi) - 1;
            const uint64_t w = (uint64_t)r.mask[last >> 5] << 32 | r.mask[e >> 5];  // the same word twice, or two
            keep = (uint32_t)((e >> 5) == (last >> 5) ? (uint32_t)w >> (e & 31) : w >> (e & 31)) & keep;
        }
        const bool masked = r.mask && keep != (1u << EPC) - 1;
        if (SAME) {
            if (!masked && !((touched >> q) & 1)) continue;
            if (keep && !((touched >> q) & 1)) load(q);
        }
        if (masked)
#pragma unroll
            for (int i = 0; i < EPC; i++)
                if (!((keep >> i) & 1)) x[q][i] = ninf;
        store(q);
    }
    if (has_edge) {
        const bool off = r.mask && !((r.mask[tid >> 5] >> (tid & 31)) & 1);
        if (off) edge = ninf;
        if (!SAME || off || touched >> 31) out[tid] = narrow<E>(edge);
    }
}

template <typename E, int W>
void launch_w(const LogitsArgs &a, hipStream_t st)
{
    const bool same = a.logits == a.out;
    // pieces of 16 bytes: rows of logits and out lie alike
    const bool vec = (((uintptr_t)a.logits ^ (uintptr_t)a.out) & 15) == 0 && ((a.ld - a.ldo) * sizeof(E)) % 16 == 0;
    const int ranges = (a.V + kVals * W - 1) / (kVals * W);
    const unsigned grid = (unsigned)(a.T * (int64_t)ranges);
    if (vec && same)
        logits_kernel<E, W, true, true><<<grid, W, 0, st>>>(a, ranges);
    else if (vec)
        logits_kernel<E, W, true, false><<<grid, W, 0, st>>>(a, ranges);
    else
        logits_kernel<E, W, false, false><<<grid, W, 0, st>>>(a, ranges);
}

}  // namespace

hipError_t launch_logits_adjust(const LogitsArgs &a, hipStream_t st)
{
    const bool wide = a.T * (int64_t)((a.V + 16383) / 16384) >= 512;
    if (a.fp32)
        wide ? launch_w<float, 1024>(a, st) : launch_w<float, 256>(a, st);
    else
        wide ? launch_w<uint16_t, 1024>(a, st) : launch_w<uint16_t, 256>(a, st);
    return hipGetLastError();
}

}  // namespace flint
