// kv_pages.hip -- the pages of a cache: the next step's tables (fork, free, reorder, grow, copy
// on write) and the move of live pages to the front of their pool.
//
// Both calls read one state and write another, in two launches.  kv_advance: first every workgroup
// takes a range of pages, counts in LDS what the rows that are forked or ended change of their
// holders, and lists those that became free in ascending order; then a workgroup per new row finds
// its place in the rows' sum of needs, takes its pages and copies the one it may not share.  Counting
// a range in LDS (every workgroup reads all tables for it) needs no cleared memory and leaves no order
// of atomics in the result.  kv_compact: first every workgroup ranks a range of pages among the live
// ones and the free places; then the moves are dealt out in pieces of 16 KB.
//
// Bound by launches and dependent reads where little is copied: eight beams of 2000 tokens in 1024 pages
// 5.6 + 8 us, 256 sequences of 4000 tokens in 16384 pages 8 + 8.5; by the copied bytes otherwise: 4096
// pages, about 940 of them moved (490 MB read and written): 6 + 108 us, 4.3 TB/s; 512 pages 4 + 10 us.
#include "serve.h"

#include <algorithm>

namespace flint {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kScan = 1024;        // threads of a workgroup that takes a range of pages
constexpr int kRowThreads = 256;
constexpr int kCopy = 16384;       // bytes of a copied piece: 64 for each of 256 threads
constexpr int kMaxChunks = 1024;   // ranges of pages
constexpr int kPerLaunch = 128;    // arrays that a launch's arguments hold

struct Arrays {
    int n;
    PageArray a[kPerLaunch];
};

// Pages of a range: one to a thread, or more where every range's reading of all tables or references
// would add up to more than it saves.
__host__ __device__ inline int chunk_pages(int n_pages) { return n_pages <= 256 * kScan ? kScan : n_pages <= 1024 * kScan ? 4 * kScan : 16 * kScan; }
__host__ __device__ inline int chunks_of(int n_pages)
{
    const int c = chunk_pages(n_pages);
    return (n_pages + c - 1) / c;
}

// A growing row and its last page: nobody else's; copied; kept because the rows ahead copy it.  The
// last must not grow unless those do: one of them may have more tokens on that page.
enum { kAlone = 0, kCopies = 1, kKeeps = 2 };

// kv_advance's workspace: free pages found in each range and how many; for each row its parent's
// tokens, the page that it grows into and what becomes of that.
struct AdvanceWs {
    int *freed, *count, *tokens, *into, *copy;
    __host__ __device__ AdvanceWs(const PagesArgs &a)
    {
        freed = a.ws;
        count = freed + a.n_pages;
        tokens = count + kMaxChunks;
        into = tokens + a.rows;
        copy = into + a.rows;
    }
};
// kv_compact's: free places below the live pages' number, the pages that move there, each such
// page's rank among them, how many.
struct CompactWs {
    int *hole, *mover, *rank, *n;
    __host__ __device__ CompactWs(const PagesArgs &a)
    {
        hole = a.ws;
        mover = hole + a.n_pages;
        rank = mover + a.n_pages;
        n = rank + a.n_pages;
    }
};

__device__ __forceinline__ int row_tokens(const PagesArgs &a, const PageState &s, int row)
{
    const int64_t most = a.ldt << a.page_shift;
    return (int)min((int64_t)max(s.kv_len[row], 0), most);
}
__device__ __forceinline__ int pages_for(const PagesArgs &a, int64_t tokens) { return (int)((tokens + a.page - 1) >> a.page_shift); }
__device__ __forceinline__ bool is_page(const PagesArgs &a, int p) { return (uint32_t)p < (uint32_t)a.n_pages; }
__device__ __forceinline__ int parent_of(const PagesArgs &a, int r)
{
    const int p = a.parent[r];
    return p >= 0 && p < a.rows_old ? p : -1;
}

// The sum of the workgroup's values, and of those of the threads before this one.  sh: a word per
// wave and one more.
template <int N, typename I>
__device__ __forceinline__ I block_sum(I v, I *sh, I &before)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    I s = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const I o = __shfl_up(s, d);
        if (lane >= d) s += o;
    }
    __syncthreads();
    if (lane == 63) sh[wave] = s;
    __syncthreads();
    I base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < N / 64; w++) {
        const I x = sh[w];
        if (w < wave) base += x;
        all += x;
    }
    before = base + s - v;
    return all;
}

// ---- kv_advance --------------------------------------------------------------------------
__global__ __launch_bounds__(kScan) void pages_refs_kernel(PagesArgs a)
{
    extern __shared__ int refs[];  // of this range's pages
    __shared__ int more[kPagesMaxRows], len[kPagesMaxRows], start[kPagesMaxRows], sh[kScan / 64];
    __shared__ __attribute__((aligned(16))) int last[kPagesMaxRows];
    const AdvanceWs w(a);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int size = chunk_pages(a.n_pages), lo = blockIdx.x * size, n = min(size, a.n_pages - lo);
    const int by = tid < a.rows ? a.grow[tid] : 0, p = tid < a.rows ? parent_of(a, tid) : -1;
    if (tid < a.rows_old) {
        more[tid] = -1;
        len[tid] = row_tokens(a, a.old, tid);
    }
    for (int i = tid; i < n; i += kScan) refs[i] = a.old.refs[lo + i];
    __syncthreads();
    int into = -1;  // the page that the row grows into beside what it holds
    if (p >= 0) {
        atomicAdd(&more[p], 1);
        if (by > 0 && (len[p] & (a.page - 1)) && (int64_t)len[p] + by <= a.ldt << a.page_shift) {
            const int e = a.old.table[p * a.ldt + (len[p] >> a.page_shift)];
            if (is_page(a, e)) into = e;
        }
    }
    if (blockIdx.x == 0 && tid < a.rows) {
        w.tokens[tid] = p >= 0 ? len[p] : 0;
        w.into[tid] = into;
    }
    __syncthreads();
    // the entries of the rows whose pages' holders change, in blocks of 64 and kAt blocks of a wave at once
    constexpr int kAt = 8;
    const int mine_blocks = tid < a.rows_old && more[tid] ? (pages_for(a, len[tid]) + 63) / 64 : 0;
    int at;
    const int blocks = block_sum<kScan>(mine_blocks, sh, at);
    start[tid] = at;
    last[tid] = into;
    __syncthreads();
    for (int b0 = wave * kAt; b0 < blocks; b0 += kAt * (kScan / 64)) {
        const int b = min(b0 + (lane & (kAt - 1)), blocks - 1);
        int row = 0;  // the last one that starts at b or before
#pragma unroll
        for (int d = kPagesMaxRows / 2; d; d /= 2)
            if (start[row + d] <= b) row += d;
        const int j0 = 64 * (b - start[row]), used = b0 + (lane & (kAt - 1)) < blocks ? pages_for(a, len[row]) : 0, add = more[row];
        int e[kAt];
#pragma unroll
        for (int k = 0; k < kAt; k++) {
            const int j = __builtin_amdgcn_readlane(j0, k) + lane;
            e[k] = j < __builtin_amdgcn_readlane(used, k) ? a.old.table[__builtin_amdgcn_readlane(row, k) * a.ldt + j] : -1;
        }
#pragma unroll
        for (int k = 0; k < kAt; k++)
            if (e[k] >= lo && e[k] < lo + n) atomicAdd(&refs[e[k] - lo], __builtin_amdgcn_readlane(add, k));
    }
    __syncthreads();
    // Of the growing rows with one last page, in order, each copies while more holders are left.  Lane l
    // of a wave has row wave + 16 l, and all rows' pages, 64 to a register, to count those ahead of it in
    // (256 rows in groups of four: 8 us, each thread reading the rows ahead of its own 14).
    const int row = wave + lane * (kScan / 64), page = last[row];
    const bool here = page >= lo && page < lo + n;
    const int holders = here ? refs[page - lo] : 0;
    int pages[kPagesMaxRows / 64], ahead = 0;
#pragma unroll
    for (int k = 0; k < kPagesMaxRows / 64; k++) pages[k] = last[64 * k + lane];
    for (uint64_t todo = __ballot(holders > 1); todo; todo &= todo - 1) {
        const int l = __builtin_ctzll(todo), x = __builtin_amdgcn_readlane(page, l), r = wave + l * (kScan / 64);
        int c = 0;
#pragma unroll
        for (int k = 0; k < kPagesMaxRows / 64; k++) {
            if (64 * k >= r) break;
            const uint64_t same = __ballot(pages[k] == x);
            c += __popcll(r - 64 * k >= 64 ? same : same & ((1ull << (r - 64 * k)) - 1));
        }
        if (lane == l) ahead = c;
    }
    if (row < a.rows && (here || (page < 0 && blockIdx.x == 0)))
        w.copy[row] = holders - ahead > 1 ? kCopies : ahead ? kKeeps : kAlone;
    // free pages in ascending order: a thread takes consecutive ones
    const int per = size / kScan, i0 = tid * per;
    int mine = 0;
    for (int i = i0; i < min(i0 + per, n); i++) {
        const int now = max(refs[i], 0);
        mine += now == 0 && a.old.refs[lo + i] > 0;
        a.state.refs[lo + i] = now;
    }
    const int all = block_sum<kScan>(mine, sh, at);
    if (mine)
        for (int i = i0; i < min(i0 + per, n); i++)
            if (refs[i] <= 0 && a.old.refs[lo + i] > 0) w.freed[lo + at++] = lo + i;
    if (tid == 0) w.count[blockIdx.x] = all;
}

// The k-th free page that the first launch found, in ascending order; first: free pages before each range.
__device__ __forceinline__ int freed_page(const PagesArgs &a, const AdvanceWs &w, const int *first, int chunks, int k)
{
    int lo = 0, hi = chunks - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (first[mid] <= k)
            lo = mid;
        else
            hi = mid - 1;
    }
    return w.freed[lo * chunk_pages(a.n_pages) + k - first[lo]];
}

// A page's share `part` of `parts` of the pieces of every array.
__device__ __forceinline__ void copy_page(const Arrays &arr, int src, int dst, int part, int parts)
{
    int unit = 0;
    for (int i = 0; i < arr.n; i++) {
        const PageArray &x = arr.a[i];
        const uint8_t *from = x.base + src * x.stride;
        uint8_t *to = x.base + dst * x.stride;
        const int pieces = (int)((x.bytes + kCopy - 1) / kCopy);
        for (int c = 0; c < pieces; c++, unit++) {
            if (unit % parts != part) continue;
            const int64_t at = (int64_t)c * kCopy + 16 * threadIdx.x;
            u32x4 v[4];
#pragma unroll
            for (int j = 0; j < 4; j++)
                if (at + 4096 * j < x.bytes) v[j] = *reinterpret_cast<const u32x4 *>(from + at + 4096 * j);
#pragma unroll
            for (int j = 0; j < 4; j++)
                if (at + 4096 * j < x.bytes) *reinterpret_cast<u32x4 *>(to + at + 4096 * j) = v[j];
        }
    }
}

// Workgroup (row, part): part 0 writes the row's share of the state, every part its share of the
// row's copied page.
__global__ __launch_bounds__(kRowThreads) void pages_rows_kernel(PagesArgs a, Arrays arr, int parts, int tables)
{
    __shared__ int first[kMaxChunks], s_want, s_tokens, s_ok, s_copy;
    __shared__ uint32_t s_end, sh[kRowThreads / 64];
    const AdvanceWs w(a);
    const int tid = threadIdx.x, row = blockIdx.x / parts, part = blockIdx.x % parts;
    const bool writes = tables && part == 0;
    if (!writes && (row >= a.rows || w.copy[row] != kCopies)) return;
    const int parent = row < a.rows ? parent_of(a, row) : -1, into = row < a.rows ? w.into[row] : -1;
    // free pages of the ranges
    const int chunks = chunks_of(a.n_pages);
    constexpr int CPT = kMaxChunks / kRowThreads;
    int c[CPT];
    uint32_t sum = 0, before;
#pragma unroll
    for (int i = 0; i < CPT; i++) {
        c[i] = CPT * tid + i < chunks ? w.count[CPT * tid + i] : 0;
        sum += c[i];
    }
    const int freed = (int)block_sum<kRowThreads>(sum, sh, before);
#pragma unroll
    for (int i = 0; i < CPT; i++) {
        first[CPT * tid + i] = (int)before;
        before += c[i];
    }
    const int old_free = min(max(*a.old.n_free, 0), a.n_pages), avail = old_free + freed;
    // the rows' needs, four to a thread: 1024 rows of up to 2^21 pages, so that their sum needs all 32 bits
    constexpr int RPT = kPagesMaxRows / kRowThreads;
    int want[RPT], tokens[RPT], own[RPT];
    bool fits[RPT];
    sum = 0;
#pragma unroll
    for (int i = 0; i < RPT; i++) {
        const int r = RPT * tid + i;
        want[i] = tokens[i] = own[i] = 0;
        fits[i] = false;
        if (r < a.rows) {
            tokens[i] = w.tokens[r];
            const int64_t then = tokens[i] + (int64_t)max(a.grow[r], 0);
            fits[i] = then <= a.ldt << a.page_shift;
            own[i] = w.copy[r];
            if (fits[i]) want[i] = pages_for(a, then) - pages_for(a, tokens[i]) + (own[i] == kCopies);
        }
        sum += want[i];
    }
    block_sum<kRowThreads>(sum, sh, before);
    int taken = 0;  // pages that are taken in all: the last served row's end
    {
        uint32_t end = before;
#pragma unroll
        for (int i = 0; i < RPT; i++) {
            end += want[i];
            const bool ok = fits[i] && ((want[i] == 0 && own[i] != kKeeps) || end <= (uint32_t)avail);
            if (ok && want[i]) taken = (int)end;
            if (RPT * tid + i == row) {
                s_want = ok ? want[i] : 0;
                s_end = end;
                s_tokens = tokens[i];
                s_ok = ok;
                s_copy = own[i] == kCopies;
            }
        }
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) taken = max(taken, __shfl_xor(taken, d));
    __syncthreads();
    if ((tid & 63) == 0) sh[tid >> 6] = taken;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRowThreads / 64; i++) taken = max(taken, (int)sh[i]);
    // the stack's k-th page from the top
    auto pop = [&](int k) { return k < freed ? freed_page(a, w, first, chunks, freed - 1 - k) : a.old.free_list[old_free - 1 - (k - freed)]; };

    if (row < a.rows) {
        const bool ok = s_ok;
        const int got = s_want, k0 = (int)s_end - got, len = s_tokens;  // k0: of a served row
        const bool copy = ok && s_copy;
        const int used = pages_for(a, len), e0 = used - copy;  // the first new entry
        const int32_t *from = a.old.table + max(parent, 0) * a.ldt;
        if (copy) {
            const int dst = pop(k0);
            if (is_page(a, dst)) copy_page(arr, into, dst, part, parts);
            if (writes && tid == 0) atomicSub(&a.state.refs[into], 1);
        }
        if (writes) {
            for (int64_t j = tid; j < a.ldt; j += kRowThreads) {
                int e = -1;
                if (j >= e0 && j < e0 + got) {
                    e = pop(k0 + (int)j - e0);
                    if (is_page(a, e)) a.state.refs[e] = 1;
                } else if (j < used) {
                    e = from[j];
                }
                a.state.table[row * a.ldt + j] = e;
            }
            const int add = ok ? max(a.grow[row], 0) : 0;
            if (tid == 0) a.state.kv_len[row] = len + add;
            if (a.slots) {
                for (int64_t i = tid; i < a.lds; i += kRowThreads) {
                    int64_t slot = -1;
                    if (i < add) {
                        const int64_t at = len + i;
                        const int j = (int)(at >> a.page_shift);
                        const int e = j >= e0 && j < e0 + got ? pop(k0 + j - e0) : from[j];
                        if (is_page(a, e)) slot = ((int64_t)e << a.page_shift) + (at & (a.page - 1));
                    }
                    a.slots[row * a.lds + i] = slot;
                }
            }
        }
    }
    if (!writes) return;
    // what is left of the stack, shared out over the rows' workgroups
    const int left = min(avail - taken, a.n_pages), stride = (gridDim.x / parts) * kRowThreads;
    if (row == 0 && tid == 0) *a.state.n_free = left;
    for (int i = row * kRowThreads + tid; i < a.n_pages; i += stride)
        a.state.free_list[i] = i >= left ? -1 : i < old_free ? a.old.free_list[i] : freed_page(a, w, first, chunks, i - old_free);
}

// ---- kv_compact ----------------------------------------------------------------------------
__global__ __launch_bounds__(kScan) void compact_scan_kernel(PagesArgs a)
{
    __shared__ int sh[kScan / 64];
    const CompactWs w(a);
    const int tid = threadIdx.x, size = chunk_pages(a.n_pages), lo = blockIdx.x * size, hi = min(lo + size, a.n_pages);
    constexpr int kAt = 8;  // references of a thread on their way
    int all = 0, ahead = 0, at;
    for (int i0 = tid; i0 < a.n_pages; i0 += kAt * kScan) {
        int v[kAt];
#pragma unroll
        for (int k = 0; k < kAt; k++) v[k] = a.old.refs[min(i0 + k * kScan, a.n_pages - 1)];
#pragma unroll
        for (int k = 0; k < kAt; k++) {
            const int i = i0 + k * kScan, live = v[k] > 0 && i < a.n_pages;
            all += live;
            ahead += live && i < lo;
        }
    }
    const int n = block_sum<kScan>(all, sh, at);  // live pages
    int below = 0;
    for (int i0 = tid; i0 < n; i0 += kAt * kScan) {
        int v[kAt];
#pragma unroll
        for (int k = 0; k < kAt; k++) v[k] = a.old.refs[min(i0 + k * kScan, n - 1)];
#pragma unroll
        for (int k = 0; k < kAt; k++) below += v[k] > 0 && i0 + k * kScan < n;
    }
    below = block_sum<kScan>(below, sh, at);  // those that stay
    ahead = block_sum<kScan>(ahead, sh, at);
    const int per = size / kScan, i0 = lo + tid * per;
    int mine = 0;
    for (int i = i0; i < min(i0 + per, hi); i++) mine += a.old.refs[i] > 0;
    block_sum<kScan>(mine, sh, at);
    int before = ahead + at;  // live pages before page i
    for (int i = i0; i < min(i0 + per, hi); i++) {
        const int r = a.old.refs[i];
        const bool live = r > 0;
        if (i < n) {
            if (live)
                a.state.refs[i] = r;
            else
                w.hole[i - before] = i;
            a.moved[i] = live ? i : -1;
        } else {
            a.state.refs[i] = 0;
            if (live) {
                w.mover[before - below] = i;
                w.rank[i] = before - below;
            } else {
                a.moved[i] = -1;
            }
        }
        a.state.free_list[i] = i < a.n_pages - n ? a.n_pages - 1 - i : -1;
        before += live;
    }
    if (blockIdx.x == 0 && tid == 0) {
        *w.n = n - below;
        *a.state.n_free = a.n_pages - n;
    }
}

__global__ __launch_bounds__(kRowThreads) void compact_move_kernel(PagesArgs a, Arrays arr, int pieces, int tables)
{
    const CompactWs w(a);
    const int moves = *w.n, tid = threadIdx.x;
    if (tables) {
        const int64_t total = a.rows * a.ldt, stride = (int64_t)gridDim.x * kRowThreads, me = (int64_t)blockIdx.x * kRowThreads + tid;
        for (int64_t i = me; i < moves; i += stride) {
            const int src = w.mover[i], dst = w.hole[i];
            a.moved[src] = dst;
            a.state.refs[dst] = a.old.refs[src];
        }
        const int n = a.n_pages - *a.state.n_free;
        for (int64_t i = me; i < total; i += stride) {
            const int row = (int)(i / a.ldt), j = (int)(i % a.ldt);
            int e = -1;
            if (j < pages_for(a, row_tokens(a, a.old, row))) {
                e = a.old.table[i];
                if (is_page(a, e)) e = a.old.refs[e] <= 0 ? -1 : e < n ? e : w.hole[w.rank[e]];
            }
            a.state.table[i] = e;
        }
        for (int64_t r = me; r < a.rows; r += stride) a.state.kv_len[r] = row_tokens(a, a.old, (int)r);
    }
    // move m, array i, piece c
    const int64_t units = (int64_t)moves * arr.n * pieces;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int c = (int)(u % pieces), i = (int)(u / pieces % arr.n), m = (int)(u / ((int64_t)pieces * arr.n));
        const PageArray &x = arr.a[i];
        const int64_t at = (int64_t)c * kCopy + 16 * tid;
        if (at >= x.bytes) continue;
        const uint8_t *from = x.base + w.mover[m] * x.stride;
        uint8_t *to = x.base + w.hole[m] * x.stride;
        u32x4 v[4];
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (at + 4096 * j < x.bytes) v[j] = *reinterpret_cast<const u32x4 *>(from + at + 4096 * j);
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (at + 4096 * j < x.bytes) *reinterpret_cast<u32x4 *>(to + at + 4096 * j) = v[j];
    }
}

// Arrays first .. first + kPerLaunch, and the most pieces of one of them and of all.
Arrays arrays_of(const PagesArgs &a, int first, int &most, int64_t &all)
{
    Arrays r;
    r.n = std::min(a.n_arrays - first, kPerLaunch);
    most = 1;
    all = 0;
    for (int i = 0; i < r.n; i++) {
        r.a[i] = a.arrays[first + i];
        const int64_t pieces = (r.a[i].bytes + kCopy - 1) / kCopy;
        most = (int)std::max<int64_t>(most, pieces);
        all += pieces;
    }
    return r;
}

}  // namespace

size_t kv_pages_ws_bytes(int64_t n_pages, int64_t rows)
{
    const size_t advance = (size_t)n_pages + kMaxChunks + 3 * (size_t)rows, compact = 3 * (size_t)n_pages + 4;
    return 4 * std::max(advance, compact);
}

hipError_t launch_kv_advance(const PagesArgs &a, hipStream_t st)
{
    pages_refs_kernel<<<(unsigned)chunks_of(a.n_pages), kScan, 4 * (size_t)chunk_pages(a.n_pages), st>>>(a);
    hipError_t e = hipGetLastError();
    const int rows = std::max(a.rows, 1);
    for (int first = 0; e == hipSuccess && (first == 0 || first < a.n_arrays); first += kPerLaunch) {
        int most;
        int64_t all;
        const Arrays arr = arrays_of(a, first, most, all);
        // as many workgroups to a row as its copy has pieces, 2048 in all
        const int parts = (int)std::max<int64_t>(1, std::min<int64_t>(all, 2048 / rows));
        pages_rows_kernel<<<(unsigned)(rows * parts), kRowThreads, 0, st>>>(a, arr, parts, first == 0);
        e = hipGetLastError();
    }
    return e;
}

hipError_t launch_kv_compact(const PagesArgs &a, hipStream_t st)
{
    compact_scan_kernel<<<(unsigned)chunks_of(a.n_pages), kScan, 0, st>>>(a);
    hipError_t e = hipGetLastError();
    for (int first = 0; e == hipSuccess && (first == 0 || first < a.n_arrays); first += kPerLaunch) {
        int most;
        int64_t all;
        const Arrays arr = arrays_of(a, first, most, all);
        compact_move_kernel<<<2048, kRowThreads, 0, st>>>(a, arr, most, first == 0);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace flint
