// logits.hip -- penalties for repeated tokens, biases and grammar masks on logits.
//
//   x = l;  seen: x > 0 ? x / r : x r;  x -= f c + p [c > 0];  x += bias;  not allowed: -inf
//
// A workgroup takes a range of one row's vocabulary, whose logits are on their way to registers while it
// counts the row's history in LDS, a word per token of the range.  The few tokens whose words are not
// zero are taken out of their piece, computed and put back; all others pass as bits, -inf where the
// mask says so.  A word is a bit for a token of the prompt, above the row's bias entries (the highest of
// a token stays, by an atomic maximum before anything is counted), above a count of the row's own;
// sums of whole numbers and maxima, so their order does not matter.  Where a row has too many entries for the
// bits that its history leaves, a thread keeps its words in registers and the entries take them after that.
// Every workgroup of a row reads the whole history, from L2, eight tokens per thread on their way at a time.
//
// Bound by the logits' bytes, read and written once, and by what comes before them: 128 rows of 131072 are two
// rounds of two workgroups to a CU, each of which clears and counts first (20 us, 3.4 TB/s).  In place only
// pieces of 16 bytes that something changes are touched (17 us).  (The copy first and the tokens after it in a
// turn of their own took 24 us for them: a workgroup then waits for its stores.)
#include "serve.h"

#include <type_traits>

namespace flint {

namespace {

constexpr int kAhead = 8;  // tokens of the history that a thread has on their way
constexpr uint32_t kPrompt = 0x80000000u;

// The rules of a row.  Histories and bias entries end at 2^31 - 1 at most; numbers that run past their ends
// by a turn of the workgroup are unsigned.
struct Row {
    uint32_t total, prompt;
    float rep, freq, pres;
    uint32_t b0, b1;          // its bias entries, b0 <= b1
    const uint32_t *mask;     // or null
};
__device__ __forceinline__ Row row_of(const LogitsArgs &a, int t)
{
    Row r;
    r.total = r.prompt = 0;
    if (a.history) {
        const int64_t n = a.total_len ? min((int64_t)max(a.total_len[t], 0), a.ldh) : a.ldh;
        r.total = (uint32_t)n;
        r.prompt = a.prompt_len ? min((uint32_t)max(a.prompt_len[t], 0), r.total) : 0u;
    }
    r.rep = a.repetition ? a.repetition[t] : 1.f;
    r.freq = a.frequency ? a.frequency[t] : 0.f;
    r.pres = a.presence ? a.presence[t] : 0.f;
    r.b0 = r.b1 = 0;
    if (a.bias_start) {
        r.b0 = (uint32_t)max(a.bias_start[t], 0);
        r.b1 = max(r.b0, (uint32_t)min((int64_t)max(a.bias_start[t + 1], 0), a.n_bias));
    }
    r.mask = nullptr;
    if (a.masks) {
        const int64_t m = a.mask_rows ? a.mask_rows[t] : t;
        if (m >= 0 && m < a.n_masks) r.mask = a.masks + m * a.ldm;
    }
    return r;
}

// Element b of a piece of 16 bytes, as its bits; and the piece with it replaced.
template <int BITS>
__device__ __forceinline__ uint32_t take(u32x4 x, int b)
{
    const int d = BITS == 32 ? b : b >> 1;
    const uint32_t lo = d & 1 ? x[1] : x[0], hi = d & 1 ? x[3] : x[2], v = d & 2 ? hi : lo;
    return BITS == 32 ? v : b & 1 ? v >> 16 : v & 0xffffu;
}
template <int BITS>
__device__ __forceinline__ u32x4 put(u32x4 x, int b, uint32_t v)
{
    const int d = BITS == 32 ? b : b >> 1;
    const uint32_t keep = BITS == 32 ? 0u : b & 1 ? 0xffffu : 0xffff0000u, w = BITS == 32 ? v : b & 1 ? v << 16 : v;
#pragma unroll
    for (int i = 0; i < 4; i++) x[i] = i == d ? (x[i] & keep) | w : x[i];
    return x;
}

// Bits of a count of up to n tokens.
__host__ __device__ inline int count_bits_of(int n) { return 32 - __builtin_clz(n | 1); }

// Ranges of N elements, from `head` on where pieces of 16 bytes are aligned (VEC; the first range takes
// the elements before them too) or from 0.  SAME: out is logits.  SPLIT: there may be rows whose words do
// not hold both a count and an entry's number.
template <typename E, int W, int N, bool VEC, bool SAME, bool SPLIT>
__global__ __launch_bounds__(W) void logits_kernel(LogitsArgs a, int ranges)
{
    // Pieces of 16 bytes, or of one element that is moved alone; EPC elements.
    constexpr int BITS = 8 * sizeof(E), EPC = VEC ? 128 / BITS : 1, NP = N / (W * EPC);
    constexpr uint32_t kNegInf = BITS == 32 ? 0xff800000u : 0xff80u, kAll = (1u << EPC) - 1;
    typedef typename std::conditional<BITS == 32, uint32_t, uint16_t>::type bits_t;
    // a word per element: the pieces' from 0 on, then those of the elements before them
    __shared__ __attribute__((aligned(16))) uint32_t word[N + 8];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), t = blockIdx.x / ranges, c = blockIdx.x % ranges;
    const bits_t *in = (const bits_t *)a.logits + t * a.ld;
    bits_t *out = (bits_t *)a.out + t * a.ldo;
    const int head = VEC ? min((int)((16 - ((uintptr_t)in & 15)) & 15) / (int)sizeof(E), a.V) : 0;
    const int first = head + c * N, hi = min(first + N, a.V), edges = c == 0 ? head : 0;
    if (first >= hi && !edges) return;
    // on their way before the row's rules are known: the history's first tokens and the range's logits
    const int32_t *history = a.history + t * a.ldh;
    int32_t id[kAhead], next[kAhead];
    if (a.history && a.ldh)
#pragma unroll
        for (int u = 0; u < kAhead; u++) id[u] = history[min((int64_t)tid + u * W, a.ldh - 1)];
    auto at = [&](int q) { return first + (tid + W * q) * EPC; };
    u32x4 x[NP];
    uint32_t edge = 0;  // and one element before the pieces
    auto load = [&](int q) {
        const int e = at(q);
        if (EPC > 1 && e + EPC <= hi) {
            x[q] = *reinterpret_cast<const u32x4 *>(in + e);
        } else {
            x[q] = u32x4{0u, 0u, 0u, 0u};
            for (int i = 0; i < EPC; i++)
                if (e + i < hi) x[q] = put<BITS>(x[q], i, in[e + i]);
        }
    };
    if (!SAME) {
#pragma unroll
        for (int q = 0; q < NP; q++) load(q);
        if (tid < edges) edge = in[tid];
    }
    auto clear = [&] {
        for (int i = tid; i < N / 4 + 2; i += W) *reinterpret_cast<u32x4 *>(word + 4 * i) = u32x4{0u, 0u, 0u, 0u};
        __syncthreads();
    };
    const Row r = row_of(a, t);
    uint32_t keep[NP];  // a bit per element that is allowed
#pragma unroll
    for (int q = 0; q < NP; q++) {
        keep[q] = kAll;
        const int e = at(q), last = min(e + EPC, hi) - 1;
        if (r.mask && e < hi) {
            const uint32_t w0 = r.mask[e >> 5], w1 = r.mask[last >> 5];  // the same word, or two
            keep[q] &= (e >> 5) == (last >> 5) ? w0 >> (e & 31) : (uint32_t)(((uint64_t)w1 << 32 | w0) >> (e & 31));
        }
    }
    const bool keep_edge = !(r.mask && tid < edges) || (r.mask[tid >> 5] >> (tid & 31)) & 1;
    uint32_t have = SAME ? 0u : 0xffffffffu, changed = 0;  // pieces that are loaded, that differ; the highest bit: the edge
    // the place of a token in this range, N + 8: none
    auto place = [&](int32_t v) {
        const uint32_t i = (uint32_t)v - (uint32_t)first;
        return i < (uint32_t)(hi - first) ? (int)i : (uint32_t)v < (uint32_t)edges ? N + v : N + 8;
    };
    const uint32_t entries = r.b1 - r.b0;
    const int least_bits = count_bits_of((int)r.total);
    const bool apart = SPLIT && entries >= 1u << (31 - least_bits);  // the entries' numbers come after the counts
    const int count_bits = apart ? 31 : least_bits;
    auto enter = [&](int shift) {
        for (uint32_t i = r.b0 + tid; i < r.b1; i += W) {
            const int p = place(a.bias_ids[i]);
            if (p < N + 8) atomicMax(&word[p], (i - r.b0 + 1) << shift);
        }
        __syncthreads();
    };
    if (r.total > 0 || entries) {
        clear();
        if (entries && !apart) enter(count_bits);
        for (uint32_t i0 = 0; i0 < r.total; i0 += kAhead * W) {
            if (i0 + kAhead * W < r.total)
#pragma unroll
                for (int u = 0; u < kAhead; u++) next[u] = history[min(i0 + (kAhead + u) * W + tid, r.total - 1)];
#pragma unroll
            for (int u = 0; u < kAhead; u++) {
                const uint32_t at0 = i0 + u * W, i = at0 + tid;
                if (at0 >= r.total) break;
                const int p = i < r.total ? place(id[u]) : N + 8;
                if (at0 + 64 * wave >= r.prompt) {  // the wave's are all the row's own
                    if (p < N + 8) atomicAdd(&word[p], 1u);
                } else if (p < N + 8) {
                    if (i < r.prompt)
                        atomicOr(&word[p], kPrompt);
                    else
                        atomicAdd(&word[p], 1u);
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; u++) id[u] = next[u];
        }
        __syncthreads();
        uint32_t said[SPLIT ? NP * EPC : 1] = {}, said_edge = 0;
        if (apart) {
#pragma unroll
            for (int i = 0; i < (SPLIT ? NP * EPC : 0); i++) said[i] = word[(tid + W * (i / EPC)) * EPC + i % EPC];
            if (tid < edges) said_edge = word[N + tid];
            __syncthreads();
            clear();
            enter(0);
        }
        // an element's value, with its word (and its counts, where they are not in that)
        auto one = [&](uint32_t bits, uint32_t w, uint32_t counts) {
            float y = BITS == 32 ? __uint_as_float(bits) : bf2f(bits);
            const uint32_t c = apart ? counts : w, own = c & ((1u << count_bits) - 1);
            if (own || c & kPrompt) y = y > 0.f ? y / r.rep : y * r.rep;
            if (own) y = y - r.freq * (float)own - r.pres;
            const uint32_t k = apart ? w : (w & ~kPrompt) >> count_bits;
            if (k) y += a.bias[r.b0 + k - 1];
            return BITS == 32 ? __float_as_uint(y) : pack_bf16(y, 0.f);
        };
#pragma unroll
        for (int q = 0; q < NP; q++) {
            const uint32_t *w = word + (tid + W * q) * EPC;
            uint32_t found = 0;
            if constexpr (EPC >= 4) {
#pragma unroll
                for (int k = 0; k < EPC / 4; k++) {
                    const u32x4 v = *reinterpret_cast<const u32x4 *>(w + 4 * k);
#pragma unroll
                    for (int e = 0; e < 4; e++) found |= (uint32_t)(v[e] != 0) << (4 * k + e);
                }
            } else {
                found = w[0] != 0;
            }
            if (apart)
#pragma unroll
                for (int e = 0; e < (SPLIT ? EPC : 0); e++) found |= (uint32_t)(said[q * EPC + e] != 0) << e;
            found &= keep[q];
            if (!found) continue;
            if (SAME && !((have >> q) & 1)) load(q);
            have |= 1u << q;
            changed |= 1u << q;
            while (found) {
                const int b = __builtin_ctz(found);
                found &= found - 1;
                uint32_t counts = 0;
                if (apart)
#pragma unroll
                    for (int e = 0; e < (SPLIT ? EPC : 0); e++) counts = e == b ? said[q * EPC + e] : counts;
                x[q] = put<BITS>(x[q], b, one(take<BITS>(x[q], b), w[b], counts));
            }
        }
        if (tid < edges && (word[N + tid] | said_edge) && keep_edge) {
            if (SAME && !(have >> 31)) edge = in[tid];
            have |= 1u << 31;
            changed |= 1u << 31;
            edge = one(edge, word[N + tid], said_edge);
        }
    }
#pragma unroll
    for (int q = 0; q < NP; q++) {
        const int e = at(q);
        if (e >= hi) continue;
        if (keep[q] != kAll) {
            if (SAME && keep[q] && !((have >> q) & 1)) load(q);
            changed |= 1u << q;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                if constexpr (EPC == 1) {
                    x[q][i] = kNegInf;
                } else if constexpr (BITS == 32) {
                    x[q][i] = (keep[q] >> i) & 1 ? x[q][i] : kNegInf;
                } else {
                    const uint32_t m = ((keep[q] >> (2 * i)) & 1 ? 0xffffu : 0u) | ((keep[q] >> (2 * i + 1)) & 1 ? 0xffff0000u : 0u);
                    x[q][i] = (x[q][i] & m) | (kNegInf * 0x10001u & ~m);
                }
            }
        }
        if (SAME && !((changed >> q) & 1)) continue;
        if (EPC > 1 && e + EPC <= hi) {
            *reinterpret_cast<u32x4 *>(out + e) = x[q];
        } else {
            for (int i = 0; i < EPC; i++)
                if (e + i < hi) out[e + i] = (bits_t)take<BITS>(x[q], i);
        }
    }
    if (tid < edges && (!SAME || !keep_edge || changed >> 31)) out[tid] = keep_edge ? (bits_t)edge : (bits_t)kNegInf;
}

template <typename E, int W, int N, bool SPLIT>
void launch_n(const LogitsArgs &a, hipStream_t st)
{
    const bool same = a.logits == a.out;
    // pieces of 16 bytes: rows of logits and out lie alike
    const bool vec = (((uintptr_t)a.logits ^ (uintptr_t)a.out) & 15) == 0 && ((a.ld - a.ldo) * sizeof(E)) % 16 == 0;
    const int ranges = (a.V + N - 1) / N;
    const unsigned grid = (unsigned)(a.T * (int64_t)ranges);
    if (vec && same)
        logits_kernel<E, W, N, true, true, SPLIT><<<grid, W, 0, st>>>(a, ranges);
    else if (vec)
        logits_kernel<E, W, N, true, false, SPLIT><<<grid, W, 0, st>>>(a, ranges);
    else
        logits_kernel<E, W, N, false, false, SPLIT><<<grid, W, 0, st>>>(a, ranges);
}

template <typename E>
void launch_e(const LogitsArgs &a, hipStream_t st)
{
    // The longest history and all entries in one row: the prompt's bit, a count and an entry's number have to
    // fit a word (a history of 16384 leaves room for 65535 entries).  Code for rows where they do not costs the
    // others a little (128 rows of 131072 with 1000 entries each: bf16 25.6 us, 25.3 without it; fp32 43.9, 42.8).
    const int count_bits = count_bits_of(a.history ? (int)a.ldh : 0);
    const bool split = a.bias_start && a.n_bias >= (int64_t)1 << (31 - count_bits);
    // Where ranges of 16384 are two workgroups to a CU, they spare half of the readings of the history (128
    // rows of 131072: 20.5 us, of 8192 25.2); with fewer rows more workgroups are better (32 rows 12.9 of 8192,
    // 13.8; one row 8.7 and 10.4, and 12 with 512 threads, whose share of a history of 20000 is twice as long).
    const bool large = a.T * (int64_t)((a.V + 16383) / 16384) >= 512;
    if (split)
        large ? launch_n<E, 1024, 16384, true>(a, st) : launch_n<E, 1024, 8192, true>(a, st);
    else
        large ? launch_n<E, 1024, 16384, false>(a, st) : launch_n<E, 1024, 8192, false>(a, st);
}

}  // namespace

hipError_t launch_logits_adjust(const LogitsArgs &a, hipStream_t st)
{
    a.fp32 ? launch_e<float>(a, st) : launch_e<uint16_t>(a, st);
    return hipGetLastError();
}

}  // namespace flint
