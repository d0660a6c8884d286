// gdn_pages.hip -- the pages of a cache on gfx950: tables of pages and reference counts in
// whole numbers, and the copies of pages that follow from them.
//
// Tables and counts are small (a few thousand requests and pages): one workgroup keeps
// them, whose requests and pages are ordered by prefix sums over its threads, so that the
// outcome does not depend on the order in which threads run. Where pages move, it leaves a list
// in the workspace, and a second launch over the whole card copies them, plane after plane:
// bound by the bytes of the copied pages, each read and written once. 477 pages on 24 planes of 16 KB: 7 us of tables and
// 71 of copies (5.3 TB/s); a fork of 32 samples 13 us, bound by the latency of a few dependent loads and 2400 atomics.

#include "gdn_device.h"
#include "gdn_attn.h"

namespace gdn {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
static_assert(kPageRequests == kThreads, "one thread for each request");

// Workspace: the number of copies, then their (from, to) pairs (at most half of the pages are
// free, or as many as requests), then the free pages
struct Copies {
    int32_t *count;
    int2 *pages;
};
__host__ __device__ __forceinline__ Copies copies_of(int32_t *workspace)
{
    return Copies{workspace, reinterpret_cast<int2 *>(workspace + 64)};
}

// Exclusive sum over the workgroup's threads, and the total.
__device__ __forceinline__ int scan(int x, int *sums, int &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int in = x;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int y = __shfl_up(in, d, 64);
        in += lane >= d ? y : 0;
    }
    __syncthreads();  // sums may still be read from a call before
    if (lane == 63)
        sums[wave] = in;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < kWaves; ++w) {
        before += w < wave ? sums[w] : 0;
        total += sums[w];
    }
    return before + in - x;
}

__device__ __forceinline__ bool is_page(const PageParams &p, int page) { return page >= 0 && page < p.num_pages; }

constexpr int kEach = 8, kStep = kEach * kThreads;  // pages a thread looks at, and the workgroup, at a time

// The pages that a thread looks at from page `base` on: bit j, whether the j-th is free
__device__ __forceinline__ uint32_t free_pages(const PageParams &p, int base)
{
    const int at = base + kEach * threadIdx.x;
    int refs[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        refs[j] = p.refs[min(at + j, p.num_pages - 1)];
    uint32_t open = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        open |= at + j < p.num_pages && refs[j] <= 0 ? 1u << j : 0u;
    return open;
}

// Hands free pages, lowest first, to give(rank, page) for the ranks below `want`; returns how many it has. `open`: what the
// thread found from page 0 on.
template <class F>
__device__ __forceinline__ int lowest_free(const PageParams &p, int want, uint32_t open, int *sums, F give)
{
    int found = 0;
    for (int base = 0; base < p.num_pages && found < want; base += kStep) {
        if (base > 0)
            open = free_pages(p, base);
        int total;
        int rank = found + scan(__popc(open), sums, total);
        for (uint32_t left = open; left && rank < want; left &= left - 1, ++rank)
            give(rank, base + kEach * (int)threadIdx.x + __ffs(left) - 1);
        found += total;
    }
    return min(found, want);
}

// ---- free ---------------------------------------------------------------------

__global__ __launch_bounds__(256) void free_kernel(const PageParams p)
{
    const int row = p.row[blockIdx.x];
    if (row < 0 || row >= p.rows)
        return;
    const int keep = p.len ? max(p.len[blockIdx.x], 0) : 0;
    int32_t *entries = p.table + row * p.table_stride;
    for (int64_t e = (int64_t)keep + threadIdx.x; e < p.width; e += 256) {
        // taken out once, whoever else names the row
        const int page = atomicExch(entries + e, -1);
        if (is_page(p, page))
            atomicSub(p.refs + page, 1);
    }
}

// ---- reserve and fork ---------------------------------------------------------

// Whether x is among list[0 .. n); the list is readable up to a multiple of 8
__device__ __forceinline__ bool among(const int *list, int n, int x)
{
    bool found = false;
    for (int i = 0; i < n; i += 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            found |= list[i + j] == x && i + j < n;
    }
    return found;
}

// Requests are looked after by half waves: most calls name no more of them, and rows of hundreds of entries are few loads.
constexpr int kHalf = 32, kHalves = kThreads / kHalf;

// Which lanes of the half wave have x
__device__ __forceinline__ uint32_t half_ballot(bool x) { return (uint32_t)(__ballot(x) >> (threadIdx.x & kHalf)); }

// Calls f(entry, page, in range) for a half wave's entries of a row below n, four loads at a time in flight
template <class F>
__device__ __forceinline__ void each_entry(const int32_t *row, int n, F f)
{
    const int lane = threadIdx.x & (kHalf - 1);
    for (int e0 = 0; e0 < n; e0 += 4 * kHalf) {
        int v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = row[min(e0 + kHalf * j + lane, n - 1)];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (e0 + kHalf * j < n)
                f(e0 + kHalf * j + lane, v[j], e0 + kHalf * j + lane < n);
    }
}

// Entries that `tokens` tokens take; -1: not a length of a row
__device__ __forceinline__ int entries_of(const PageParams &p, int tokens)
{
    const int64_t n = ((int64_t)tokens + p.page_size - 1) / p.page_size;
    return tokens < 0 || n > p.width ? -1 : (int)n;
}

constexpr int kList = 4096;  // pages handed out at a time

__global__ __launch_bounds__(kThreads) void reserve_kernel(const PageParams p)
{
    __shared__ int sums[kWaves], rows[kPageRequests], need[kPageRequests], first[kPageRequests], list[kList];
    const int tid = threadIdx.x, lane = tid & (kHalf - 1);
    const int entries = tid < p.n ? entries_of(p, p.len[tid]) : 0;
    int state = 0;
    rows[tid] = tid < p.n ? p.row[tid] : -1;
    const uint32_t open = p.num_pages > 0 ? free_pages(p, 0) : 0;
    __syncthreads();
    if (tid < p.n)
        state = rows[tid] < 0 || rows[tid] >= p.rows || entries < 0 || among(rows, tid, rows[tid]) ? 2 : 0;
    need[tid] = state == 0 ? entries : 0;
    first[tid] = 0;
    __syncthreads();
    // the entries that a request misses
    for (int i = tid / kHalf; i < p.n; i += kHalves) {
        const int32_t *row = p.table + (int64_t)rows[i] * p.table_stride;
        int missing = 0;
        each_entry(row, need[i], [&](int, int page, bool in) { missing += __popc(half_ballot(in && !is_page(p, page))); });
        if (lane == 0)
            first[i] = missing;
    }
    __syncthreads();
    const int wants = first[tid];
    int all;
    const int before = scan(wants, sums, all);
    const int have = lowest_free(p, all, open, sums, [&](int rank, int page) {
        if (rank < kList)
            list[rank] = page;
    });
    if (wants > 0 && before + wants > have) {
        state = 1;
        need[tid] = 0;
    }
    if (tid < p.n)
        p.status[tid] = state;
    first[tid] = before;
    int given;
    scan(state == 0 ? wants : 0, sums, given);
    for (int from = 0; from < given; from += kList) {
        const int count = min(kList, given - from);
        if (from > 0)  // the lowest pages that are free now: those handed out in a turn before are in use
            lowest_free(p, count, free_pages(p, 0), sums, [&](int rank, int page) { list[rank] = page; });
        __syncthreads();
        for (int i = tid / kHalf; i < p.n; i += kHalves) {
            int32_t *row = p.table + (int64_t)rows[i] * p.table_stride;
            int rank = max(first[i] - from, 0);  // of the first entry that the row still misses
            if (first[i] >= from + count)
                continue;
            each_entry(row, need[i], [&](int e, int page, bool in) {
                const bool miss = in && !is_page(p, page);
                const uint32_t all_miss = half_ballot(miss);
                const int mine = rank + __popc(all_miss & ((1u << lane) - 1));
                if (miss && mine < count) {
                    row[e] = list[mine];
                    p.refs[list[mine]] = 1;
                }
                rank += __popc(all_miss);
            });
        }
        __syncthreads();
    }
}

__global__ __launch_bounds__(kThreads) void fork_kernel(const PageParams p)
{
    __shared__ int sums[kWaves], srcs[kPageRequests], dsts[kPageRequests], full[kPageRequests], states[kPageRequests],
        ranks[kPageRequests], list[kPageRequests];
    const int tid = threadIdx.x, lane = tid & (kHalf - 1);
    const int tokens = tid < p.n ? p.len[tid] : 0, entries = entries_of(p, tokens);
    srcs[tid] = tid < p.n ? p.src[tid] : -1;
    dsts[tid] = tid < p.n ? p.row[tid] : -1;
    const uint32_t open = p.num_pages > 0 ? free_pages(p, 0) : 0;
    __syncthreads();
    int state = 2;
    if (tid < p.n && entries >= 0 && srcs[tid] >= 0 && srcs[tid] < p.rows && dsts[tid] >= 0 && dsts[tid] < p.rows)
        state = among(dsts, tid, dsts[tid]) || among(dsts, p.n, srcs[tid]) ? 2 : 0;
    states[tid] = state;
    full[tid] = entries;
    __syncthreads();
    // both rows of a request, loads of either in flight together
    for (int i = tid / kHalf; i < p.n; i += kHalves) {
        if (states[i] != 0)
            continue;
        const int32_t *src = p.table + (int64_t)srcs[i] * p.table_stride, *dst = p.table + (int64_t)dsts[i] * p.table_stride;
        bool bad = false;
        for (int e0 = 0; e0 < p.width; e0 += 4 * kHalf) {
            int from[4], to[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int e = min(e0 + kHalf * j + lane, p.width - 1);
                from[j] = src[e];
                to[j] = dst[e];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                bad |= is_page(p, to[j]) || (e0 + kHalf * j + lane < full[i] && !is_page(p, from[j]));
        }
        if (half_ballot(bad) != 0 && lane == 0)
            states[i] = 2;
    }
    __syncthreads();
    state = states[tid];
    const bool part = state == 0 && tokens % p.page_size != 0;
    int all;
    const int rank = scan(part, sums, all);
    const int have = lowest_free(p, all, open, sums, [&](int r, int page) { list[r] = page; });
    if (part && rank >= have)
        state = 1;
    states[tid] = state;
    ranks[tid] = part ? rank : -1;
    if (part)
        full[tid] = entries - 1;
    if (tid < p.n)
        p.status[tid] = state;
    const Copies copies = copies_of(p.workspace);
    if (tid == 0)
        *copies.count = have;
    __syncthreads();
    for (int i = tid / kHalf; i < p.n; i += kHalves) {
        if (states[i] != 0)
            continue;
        const int32_t *src = p.table + (int64_t)srcs[i] * p.table_stride;
        int32_t *dst = p.table + (int64_t)dsts[i] * p.table_stride;
        each_entry(src, full[i], [&](int e, int page, bool in) {
            if (in) {
                dst[e] = page;
                atomicAdd(p.refs + page, 1);
            }
        });
        if (lane == 0 && ranks[i] >= 0) {
            const int page = list[ranks[i]];
            dst[full[i]] = page;
            p.refs[page] = 1;
            copies.pages[ranks[i]] = make_int2(src[full[i]], page);
        }
    }
}

// ---- compact ------------------------------------------------------------------

__global__ __launch_bounds__(kThreads) void compact_kernel(const PageParams p)
{
    __shared__ int sums[kWaves];
    int mine = 0;
    for (int page = threadIdx.x; page < p.num_pages; page += kThreads)
        mine += p.refs[page] > 0;
    int used;
    scan(mine, sums, used);
    const Copies copies = copies_of(p.workspace);
    // free pages before `used` and pages in use from there on: as many of the one as of the other
    int holes = 0, movers = 0;
    for (int base = 0; base < p.num_pages; base += kStep) {
        const int at = base + kEach * threadIdx.x;
        int refs[kEach], n = 0, m = 0;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            refs[j] = at + j < p.num_pages ? p.refs[at + j] : 0;
            n += refs[j] <= 0 && at + j < used;
            m += refs[j] > 0 && at + j >= used;
        }
        int all_n, all_m;
        int hole = holes + scan(n, sums, all_n), mover = movers + scan(m, sums, all_m);
#pragma unroll
        for (int j = 0; j < kEach; ++j)
            if (at + j < p.num_pages) {
                if (refs[j] <= 0 && at + j < used)
                    copies.pages[hole++].y = at + j;
                if (refs[j] > 0 && at + j >= used)
                    copies.pages[mover++].x = at + j;
                p.page_map[at + j] = at + j;
            }
        holes += all_n;
        movers += all_m;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < movers; i += kThreads) {
        const int2 c = copies.pages[i];
        p.page_map[c.x] = c.y;
        p.refs[c.y] = p.refs[c.x];
        p.refs[c.x] = 0;
    }
    if (threadIdx.x == 0) {
        *copies.count = movers;
        *p.used = used;
    }
}

// ---- the copies ---------------------------------------------------------------

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
constexpr int kCopyThreads = 256, kCopyEach = 4, kCopyBytes = kCopyThreads * kCopyEach * 16;

// Pages of the list, plane after plane, in pieces of kCopyBytes. No page is both a source and a destination, and none
// is a destination twice. MAP: table entries to where their pages went.
template <bool MAP>
__global__ __launch_bounds__(kCopyThreads) void copy_kernel(const PageParams p)
{
    const Copies copies = copies_of(p.workspace);
    const int count = *copies.count;
    const int64_t pieces = (p.page_bytes + kCopyBytes - 1) / kCopyBytes, items = pieces * p.num_planes * count;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t rest = item / pieces;
        const int plane = (int)(rest / count);
        const int2 c = copies.pages[rest % count];
        const unsigned char *from = p.data + plane * p.plane_stride + c.x * p.page_stride;
        unsigned char *to = p.data + plane * p.plane_stride + c.y * p.page_stride;
        const int64_t at = item % pieces * kCopyBytes + 16 * threadIdx.x;
        u32x4 w[kCopyEach];
#pragma unroll
        for (int i = 0; i < kCopyEach; ++i)
            if (at + i * kCopyThreads * 16 < p.page_bytes)
                w[i] = *reinterpret_cast<const u32x4 *>(from + at + i * kCopyThreads * 16);
#pragma unroll
        for (int i = 0; i < kCopyEach; ++i)
            if (at + i * kCopyThreads * 16 < p.page_bytes)
                *reinterpret_cast<u32x4 *>(to + at + i * kCopyThreads * 16) = w[i];
    }
    if constexpr (MAP) {
        const int64_t entries = (int64_t)p.rows * p.width;
        for (int64_t i = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; i < entries; i += (int64_t)gridDim.x * kCopyThreads) {
            int32_t *entry = p.table + i / p.width * p.table_stride + i % p.width;
            if (is_page(p, *entry))
                *entry = p.page_map[*entry];
        }
    }
}

constexpr int kCopyGrid = 2048;  // eight workgroups for each CU

}  // namespace

size_t pages_workspace_bytes(int num_pages)
{
    const size_t most = (size_t)(num_pages / 2 + 1 > kPageRequests ? num_pages / 2 + 1 : kPageRequests);
    return 256 + most * sizeof(int2);
}

hipError_t launch_pages_free(const PageParams &p, hipStream_t s)
{
    free_kernel<<<p.n, 256, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_pages_reserve(const PageParams &p, hipStream_t s)
{
    reserve_kernel<<<1, kThreads, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_pages_fork(const PageParams &p, hipStream_t s)
{
    fork_kernel<<<1, kThreads, 0, s>>>(p);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    copy_kernel<false><<<kCopyGrid, kCopyThreads, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_pages_compact(const PageParams &p, hipStream_t s)
{
    compact_kernel<<<1, kThreads, 0, s>>>(p);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    copy_kernel<true><<<kCopyGrid, kCopyThreads, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace gdn
