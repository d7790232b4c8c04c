// kvc_pages.cu -- pages of a cache handed out, shared, given back and closed up on the device.
//
// page_refs[p] counts the table rows that list page p; 0 is a free page.  Everything here is integer
// work with one right answer (the lowest free pages first, rows in order), so results do not depend on
// the order in which blocks run: counts change by atomic adds, and every other value has one writer.
//
//   truncate  a block a row: the entries past the new length lose a reference.
//   fork      a block a new row: copies the parent's entries and adds a reference for each.
//   reserve   count: blocks over the pool count its free pages, kSegment pages each, while one more block
//             goes over the rows: how many pages each needs (its start in the order is a prefix sum), and
//             which copy a shared last page.  Sequentially, a row that grows into a page copies it if
//             more than one reference is left when its turn comes, each earlier copier having dropped
//             one; so of the rows that grow into one page all copy, but the last of them does not if
//             nobody else holds the page (their number equals its count).
//             assign: each block knows the free pages before its segment, so page p is the r-th free one;
//             the row whose start is the last at or below r gets it, and writes its table entry.
//             finish: the rows' lengths, and the copied pages of every array.
//   compact   count the pages in use per segment; map: the i-th used page at or past the number in use goes
//             to the i-th free one below it; finish: tables, counts and the map follow, and the copies.
// Up to kRowThreads rows and kOneBlockPages pages one block makes the decision of either, in one launch with the
// copies where these are small: no count and assignment to meet between launches.
// 256 branches of 64 sequences in 8 arrays, with truncate and fork, 40 -> 33 us, 8 of 4 short ones 26 -> 20.
// Past either (one call between events, which are some 10 us of each figure): a token each for 64 rows 22 us over
// 16,384 pages and 25 over 100,000, 2,000 rows 32; these with 1,866 pages to copy in 8 arrays of 32 KB 193 (5.1 TB/s),
// in 64 of 4 KB 268 (3.7); closing up 17,771 pages in use of 100,000, 8,892 of them moved, 768 and 1,088 (6.1 and 4.3
// TB/s), without arrays 23.
// Bytes: the pool's counts once or twice (4 bytes a page), the rows' entries, and each copied page read and
// written once in every array: HBM-bound from some tens of pages on (4,400 pages of 4 x 32 KB: 178 us, 6.4
// TB/s), launches and chains of dependent loads before (truncate and fork 4 us each, a decision 6 to 10).
#include <algorithm>

#include "kvc_device.cuh"
#include "kvc_launch.h"

namespace kvc {

namespace {

__device__ uint32_t g_pages_errors;

constexpr int kThreads = 256;
constexpr int kRowThreads = 1024;
constexpr int kClusterBlocks = 8;

// All threads of the cluster; what they wrote before is seen after.
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

constexpr int kPageSegment = 4096;   // pages that a block looks at
constexpr int kMaxCopyArrays = 128;  // arrays of one launch (its parameters are limited)
constexpr int kPieceChunks = 1024;   // 16-byte chunks of a page that a block copies at a time

struct CopyArrays {
    int num;
    uint32_t pieces;                 // of the largest page
    uint8_t *data[kMaxCopyArrays];
    uint32_t chunks[kMaxCopyArrays]; // of a page
};

struct ReserveSpace {
    long long *totals;               // pages needed, pages copied
    int32_t *copies;                 // pages that are copied
    int32_t *seg_counts;
    int32_t *start, *grow, *copy_at; // of each row
    int32_t *copy_src, *copy_dst;
    int2 *sharers;                   // of each page: rows that grow into it, the last of them
};

struct CompactSpace {
    int32_t *copies, *seg_counts, *copy_src, *copy_dst;
};

struct Table {
    int32_t *rows;
    int stride;
    int32_t *lens;
    int num_seqs;
    int32_t *refs;
    int num_pages, page_size;
};

__device__ __forceinline__ int pages_of(int positions, int page_size)
{
    return static_cast<int>((static_cast<unsigned>(positions) + page_size - 1) / page_size);
}

// A row's length, held inside the row (one that is not is flagged by the thread that says so).
__device__ __forceinline__ int row_len(const int32_t *lens, int s, int stride, int page_size, bool flag,
                                       uint32_t *err)
{
    const int n = lens[s];
    const int cap = stride * page_size;
    if (n > cap && flag)
        atomicOr(err, kErrContextRange);
    return min(max(n, 0), cap);
}

// One reference fewer; a page that had none is flagged and left at that.
__device__ __forceinline__ void drop_ref(int32_t *refs, int page, int num_pages, uint32_t *err)
{
    if (page < 0 || page >= num_pages) {
        atomicOr(err, kErrPageRange);
    } else if (atomicSub(refs + page, 1) <= 0) {
        atomicAdd(refs + page, 1);
        atomicOr(err, kErrPageRefs);
    }
}

__global__ void __launch_bounds__(kThreads) truncate_kernel(const Table t, const int32_t *new_lens,
                                                            uint32_t *word)
{
    pdl_wait();
    pdl_trigger();
    uint32_t *err = word ? word : &g_pages_errors;
    const int s = blockIdx.x;
    const int had = row_len(t.lens, s, t.stride, t.page_size, threadIdx.x == 0, err);
    const int want = new_lens ? new_lens[s] : 0;
    const int n = min(had, max(want, 0));
    __syncthreads();
    if (threadIdx.x == 0)
        t.lens[s] = n;
    const int32_t *row = t.rows + static_cast<size_t>(s) * t.stride;
    const int end = pages_of(had, t.page_size);
    for (int i = pages_of(n, t.page_size) + threadIdx.x; i < end; i += kThreads)
        drop_ref(t.refs, row[i], t.num_pages, err);
}

__global__ void __launch_bounds__(kThreads) fork_kernel(const Table t, int32_t *out_rows, int out_stride,
                                                        int32_t *out_lens, const int32_t *parents,
                                                        const int32_t *share_lens, uint32_t *word)
{
    pdl_wait();
    pdl_trigger();
    uint32_t *err = word ? word : &g_pages_errors;
    const int s = blockIdx.x;
    const int p = parents[s];
    int n = 0;
    if (p >= t.num_seqs) {
        if (threadIdx.x == 0)
            atomicOr(err, kErrRowRange);
    } else if (p >= 0) {
        n = row_len(t.lens, p, t.stride, t.page_size, threadIdx.x == 0, err);
        if (share_lens)
            n = min(n, max(share_lens[s], 0));
        if (pages_of(n, t.page_size) > out_stride) {   // the new row is too short
            if (threadIdx.x == 0)
                atomicOr(err, kErrContextRange);
            n = out_stride * t.page_size;
        }
        const int32_t *from = t.rows + static_cast<size_t>(p) * t.stride;
        int32_t *to = out_rows + static_cast<size_t>(s) * out_stride;
        const int end = pages_of(n, t.page_size);
        for (int i = threadIdx.x; i < end; i += kThreads) {
            const int page = from[i];
            to[i] = page;
            if (page < 0 || page >= t.num_pages)
                atomicOr(err, kErrPageRange);
            else
                atomicAdd(t.refs + page, 1);
        }
    }
    if (threadIdx.x == 0)
        out_lens[s] = n;
}

// Pages src[i] -> dst[i] of every array, i < n, by all blocks of N threads.  No page is both a source and a
// destination.
template <int N>
__device__ __forceinline__ void copy_listed(const CopyArrays &arrays, const int32_t *src, const int32_t *dst,
                                            int n)
{
    constexpr int kLoads = kPieceChunks / N;
    const long long per_page = static_cast<long long>(arrays.num) * arrays.pieces;
    for (long long u = blockIdx.x; u < n * per_page; u += gridDim.x) {
        const int i = static_cast<int>(u / per_page);
        const unsigned rest = static_cast<unsigned>(u - i * per_page);
        const unsigned array = rest / arrays.pieces;
        const unsigned c0 = (rest - array * arrays.pieces) * kPieceChunks + threadIdx.x;
        const size_t chunks = arrays.chunks[array];
        uint4 *data = reinterpret_cast<uint4 *>(arrays.data[array]);
        const uint4 *from = data + __ldcg(src + i) * chunks;
        uint4 *to = data + __ldcg(dst + i) * chunks;
        uint4 x[kLoads];
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            if (c0 + j * N < chunks)
                x[j] = __ldcs(from + c0 + j * N);
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            if (c0 + j * N < chunks)
                to[c0 + j * N] = x[j];
    }
}

// ---------------------------------------------------------------------------------------
// Sums over a block
// ---------------------------------------------------------------------------------------
// The sum of the earlier threads' v, and of all (N threads, red: N / 32 values).
template <int N>
__device__ __forceinline__ long long scan_exclusive(long long v, long long *red, long long *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off)
            x += o;
    }
    if (lane == 31)
        red[warp] = x;
    __syncthreads();
    if (warp == 0) {
        long long w = lane < N / 32 ? red[lane] : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, w, off);
            if (lane >= off)
                w += o;
        }
        if (lane < N / 32)
            red[lane] = w;
    }
    __syncthreads();
    *total = red[N / 32 - 1];
    const long long before = x - v + (warp > 0 ? red[warp - 1] : 0);
    __syncthreads();
    return before;
}

// Pages of a segment (a sum of its begin and kPageSegment may not be an int).
__device__ __forceinline__ int segment_pages(int begin, int num_pages)
{
    return min(kPageSegment, num_pages - begin);
}

// Pages in use (or free) of `pages` ones from begin on, by all threads of a block; every thread gets the sum.
template <int N>
__device__ __forceinline__ int count_pages(const int32_t *refs, int begin, int pages, bool used, long long *red)
{
    int n = 0;
    for (int i = threadIdx.x; i < pages; i += N)
        n += (refs[begin + i] > 0) == used;
    long long total;
    scan_exclusive<N>(n, red, &total);
    return static_cast<int>(total);
}

// ---------------------------------------------------------------------------------------
// reserve
// ---------------------------------------------------------------------------------------
// What a row needs, and where it starts among all that are needed.
__device__ __forceinline__ void row_wants(const Table &t, const int32_t *new_tokens, int s, bool flag,
                                          uint32_t *err, int *len, int *grow, int *last)
{
    const int cap = t.stride * t.page_size;
    const int n = row_len(t.lens, s, t.stride, t.page_size, flag, err);
    int g = new_tokens ? max(new_tokens[s], 0) : 1;
    if (t.lens[s] > cap || g > cap - n) {   // no room in the row: it stays as it is
        if (flag)
            atomicOr(err, kErrContextRange);
        g = 0;
    }
    *len = n;
    *grow = g;
    *last = -1;
    if (g > 0 && n % t.page_size != 0) {
        const int page = t.rows[static_cast<size_t>(s) * t.stride + n / t.page_size];
        if (page >= 0 && page < t.num_pages)
            *last = page;
        else if (flag)
            atomicOr(err, kErrPageRange);
    }
}

__global__ void __launch_bounds__(kRowThreads, 1)
    reserve_count_kernel(const Table t, const int32_t *new_tokens, ReserveSpace w, uint32_t *word)
{
    pdl_wait();
    pdl_trigger();
    uint32_t *err = word ? word : &g_pages_errors;
    __shared__ long long red[32];
    if (blockIdx.x > 0) {
        const int seg = blockIdx.x - 1;
        const int begin = seg * kPageSegment;
        const int n =
            count_pages<kRowThreads>(t.refs, begin, segment_pages(begin, t.num_pages), false, red);
        if (threadIdx.x == 0)
            w.seg_counts[seg] = n;
        return;
    }
    int len, grow, last;
    // of every page that rows grow into: how many they are, and the last of them
    for (int s = threadIdx.x; s < t.num_seqs; s += kRowThreads) {
        row_wants(t, new_tokens, s, true, err, &len, &grow, &last);
        if (last >= 0)
            w.sharers[last] = make_int2(0, -1);
    }
    __syncthreads();
    for (int s = threadIdx.x; s < t.num_seqs; s += kRowThreads) {
        row_wants(t, new_tokens, s, false, err, &len, &grow, &last);
        if (last >= 0) {
            atomicAdd(&w.sharers[last].x, 1);
            atomicMax(&w.sharers[last].y, s);
        }
    }
    __syncthreads();
    long long needed = 0, copied = 0;
    for (int s0 = 0; s0 < t.num_seqs; s0 += kRowThreads) {
        const int s = s0 + threadIdx.x;
        int need = 0, copy = 0, page = -1;
        if (s < t.num_seqs) {
            row_wants(t, new_tokens, s, false, err, &len, &grow, &page);
            if (page >= 0) {
                const int2 sh = __ldcg(&w.sharers[page]);
                const int refs = t.refs[page];
                if (sh.x > refs)   // more rows list the page than are counted
                    atomicOr(err, kErrPageRefs);
                copy = !(sh.x >= refs && sh.y == s);
            }
            need = copy + pages_of(len + grow, t.page_size) - pages_of(len, t.page_size);
        }
        long long total, copies;
        const long long start = needed + scan_exclusive<kRowThreads>(need, red, &total);
        const long long at = copied + scan_exclusive<kRowThreads>(copy, red, &copies);
        if (s < t.num_seqs) {
            w.start[s] = static_cast<int>(min(start, static_cast<long long>(0x7FFFFFFF)));
            w.grow[s] = grow;
            w.copy_at[s] = copy ? static_cast<int>(at) : -1;
        }
        needed += total;
        copied += copies;
    }
    if (threadIdx.x == 0) {
        w.totals[0] = needed;
        w.totals[1] = copied;
    }
}

__global__ void __launch_bounds__(kRowThreads, 1)
    reserve_assign_kernel(const Table t, ReserveSpace w, int segments, int32_t *missing)
{
    pdl_wait();
    pdl_trigger();
    __shared__ long long red[32];
    const int seg = blockIdx.x;
    long long before = 0, free_pages = 0;
    {
        long long b = 0, f = 0;
        for (int i = threadIdx.x; i < segments; i += kRowThreads) {
            const int n = w.seg_counts[i];
            f += n;
            b += i < seg ? n : 0;
        }
        scan_exclusive<kRowThreads>(b, red, &before);
        scan_exclusive<kRowThreads>(f, red, &free_pages);
    }
    const long long needed = w.totals[0];
    const bool fits = needed <= free_pages;
    if (seg == 0 && threadIdx.x == 0) {
        *missing = static_cast<int>(min(max(needed - free_pages, 0LL), static_cast<long long>(0x7FFFFFFF)));
        *w.copies = fits ? static_cast<int>(w.totals[1]) : 0;
    }
    if (!fits)
        return;
    const int begin = seg * kPageSegment, pages = segment_pages(begin, t.num_pages);
    for (int i0 = 0; i0 < pages && before < needed; i0 += kRowThreads) {
        const int i = i0 + threadIdx.x, p = begin + i;
        const bool free_page = i < pages && t.refs[p] <= 0;
        long long total;
        const long long r = before + scan_exclusive<kRowThreads>(free_page, red, &total);
        before += total;
        if (!free_page || r >= needed)
            continue;
        // the last row that starts at or below r (rows that need nothing start where the next does)
        int lo = 0, hi = t.num_seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (w.start[mid] <= r)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int s = lo;
        const int j = static_cast<int>(r) - w.start[s];
        const int len = max(t.lens[s], 0);   // (a negative length is none)
        const int copy = w.copy_at[s];
        int32_t *row = t.rows + static_cast<size_t>(s) * t.stride;
        int entry = pages_of(len, t.page_size) + j - (copy >= 0);
        if (copy >= 0 && j == 0) {
            entry = len / t.page_size;
            w.copy_src[copy] = row[entry];
            w.copy_dst[copy] = p;
        }
        row[entry] = p;
        t.refs[p] = 1;
    }
}

// Up to kOneBlockPages pages looked at by one block at once, a bit for each: all loads are on their way
// together, and one scan gives every word the number of set bits before it.
constexpr int kOneBlockPages = 16384;
constexpr int kPageWords = kOneBlockPages / 32;

struct PageBits {
    unsigned word[kPageWords];
    int before[kPageWords];

    // Bits of the pages that are used (or free); by all threads, which need a barrier before count().
    __device__ __forceinline__ void load(const int32_t *refs, int num_pages, bool used)
    {
        constexpr int kEach = kOneBlockPages / kRowThreads;
        int32_t n[kEach];
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int p = j * kRowThreads + threadIdx.x;
            n[j] = p < num_pages ? refs[p] : (used ? 0 : 1);
        }
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const unsigned bits = __ballot_sync(0xffffffffu, (n[j] > 0) == used);
            if ((threadIdx.x & 31) == 0)
                word[(j * kRowThreads + threadIdx.x) / 32] = bits;
        }
    }
    // Of all pages, and the numbers before each word.
    __device__ __forceinline__ int count(long long *red)
    {
        const int i = threadIdx.x;
        long long total;
        const long long n = scan_exclusive<kRowThreads>(i < kPageWords ? __popc(word[i]) : 0, red, &total);
        if (i < kPageWords)
            before[i] = static_cast<int>(n);
        __syncthreads();
        return static_cast<int>(total);
    }
    __device__ __forceinline__ bool has(int p) const { return (word[p >> 5] >> (p & 31) & 1) != 0; }
    // How many are below page p.
    __device__ __forceinline__ int below(int p) const
    {
        return p >= kOneBlockPages ? before[kPageWords - 1] + __popc(word[kPageWords - 1])
                                   : before[p >> 5] + __popc(word[p >> 5] & ((1u << (p & 31)) - 1));
    }
};

// The whole of it but the copies by one block, for at most kRowThreads rows and kOneBlockPages pages: a thread a
// row, the sharers of a page counted in a hash table in shared memory.
constexpr int kHashSlots = 2 * kRowThreads;

struct DecideShared {
    long long red[32];
    int start[kRowThreads], len[kRowThreads], copy_at[kRowThreads];
    PageBits free_pages;
    union {
        struct {
            int key[kHashSlots], sharers[kHashSlots], last_row[kHashSlots];
        };
        uint16_t page[kHashSlots * 6];   // the free pages in order, up to as many (the hash table is done with)
    };
};
static_assert(sizeof(DecideShared) <= 48 * 1024, "shared memory");
constexpr int kListed = kHashSlots * 6;

__device__ void reserve_decide(const Table &t, const int32_t *new_tokens, const ReserveSpace &w,
                               int32_t *missing, uint32_t *err, DecideShared &sh)
{
    const int s = threadIdx.x;
    const bool row = s < t.num_seqs;
    for (int i = s; i < kHashSlots; i += kRowThreads) {
        sh.key[i] = -1;
        sh.sharers[i] = 0;
        sh.last_row[i] = -1;
    }
    sh.free_pages.load(t.refs, t.num_pages, false);
    int len = 0, grow = 0, last = -1, refs = 0;
    if (row) {
        row_wants(t, new_tokens, s, true, err, &len, &grow, &last);
        if (last >= 0)
            refs = t.refs[last];
    }
    __syncthreads();
    int slot = 0;
    if (last >= 0) {
        slot = static_cast<int>((static_cast<unsigned>(last) * 2654435761u) >> 16) % kHashSlots;
        for (;;) {   // ends: half of the slots stay empty
            const int held = atomicCAS(&sh.key[slot], -1, last);
            if (held == -1 || held == last)
                break;
            slot = (slot + 1) % kHashSlots;
        }
        atomicAdd(&sh.sharers[slot], 1);
        atomicMax(&sh.last_row[slot], s);
    }
    __syncthreads();
    int copy = 0;
    if (last >= 0) {
        if (sh.sharers[slot] > refs)   // more rows list the page than are counted
            atomicOr(err, kErrPageRefs);
        copy = !(sh.sharers[slot] >= refs && sh.last_row[slot] == s);
    }
    const int need = row ? copy + pages_of(len + grow, t.page_size) - pages_of(len, t.page_size) : 0;
    // both sums in one: copies above bit 48, pages below (less than 2^10 rows of at most 2^30)
    long long totals;
    const long long both =
        scan_exclusive<kRowThreads>((static_cast<long long>(copy) << 48) + need, sh.red, &totals);
    constexpr long long kLow = (1LL << 48) - 1;
    const long long needed = totals & kLow, start = both & kLow;
    const int at = static_cast<int>(both >> 48);
    const int there = sh.free_pages.count(sh.red);
    const bool fits = needed <= there;
    if (row) {
        sh.start[s] = static_cast<int>(min(start, static_cast<long long>(0x7FFFFFFF)));
        sh.len[s] = len;
        sh.copy_at[s] = copy ? at : -1;
    }
    if (s == 0) {
        *w.copies = fits ? static_cast<int>(totals >> 48) : 0;
        *missing = fits ? 0 : static_cast<int>(min(needed - there, static_cast<long long>(0x7FFFFFFF)));
    }
    __syncthreads();
    if (!fits)
        return;
    for (long long first = 0; first < needed; first += kListed) {
        // pages of rank first .. first + kListed - 1
        for (int p = s; p < t.num_pages; p += kRowThreads) {
            const int r = sh.free_pages.below(p);
            if (sh.free_pages.has(p) && r >= first && r < first + kListed)
                sh.page[r - first] = static_cast<uint16_t>(p);
        }
        __syncthreads();
        const int n = static_cast<int>(min(needed - first, static_cast<long long>(kListed)));
        for (int i = s; i < n; i += kRowThreads) {
            const int r = static_cast<int>(first) + i, p = sh.page[i];
            int lo = 0, hi = t.num_seqs - 1;   // the last row that starts at or below r
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (sh.start[mid] <= r)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int j = r - sh.start[lo];
            const int c = sh.copy_at[lo];
            int entry = pages_of(sh.len[lo], t.page_size) + j - (c >= 0);
            if (c >= 0 && j == 0) {
                entry = sh.len[lo] / t.page_size;
                w.copy_dst[c] = p;
            }
            t.rows[static_cast<size_t>(lo) * t.stride + entry] = p;
            t.refs[p] = 1;
        }
        __syncthreads();
    }
    if (row) {
        if (grow > 0)   // (a negative length is none)
            t.lens[s] = len + grow;
        if (copy) {
            w.copy_src[at] = last;
            atomicSub(t.refs + last, 1);
        }
    }
}

// The decision and the copies in one launch: a cluster, whose first block decides.  For copies that eight SMs
// make as fast as a second launch would start.
__global__ void __cluster_dims__(kClusterBlocks, 1, 1) __launch_bounds__(kRowThreads, 1)
    reserve_cluster_kernel(const Table t, const int32_t *new_tokens, ReserveSpace w, int32_t *missing,
                           const CopyArrays arrays, uint32_t *word)
{
    pdl_wait();
    pdl_trigger();
    __shared__ DecideShared sh;
    if (blockIdx.x == 0)
        reserve_decide(t, new_tokens, w, missing, word ? word : &g_pages_errors, sh);
    cluster_sync();
    copy_listed<kRowThreads>(arrays, w.copy_src, w.copy_dst, __ldcg(w.copies));
}

__global__ void __launch_bounds__(kRowThreads, 1)
    reserve_decide_kernel(const Table t, const int32_t *new_tokens, ReserveSpace w, int32_t *missing,
                          uint32_t *word)
{
    pdl_wait();
    pdl_trigger();
    __shared__ DecideShared sh;
    reserve_decide(t, new_tokens, w, missing, word ? word : &g_pages_errors, sh);
}

// The rows' lengths and the copied pages' counts, once every block of the assignment has read them, and
// the copies.
__global__ void __launch_bounds__(kThreads)
    reserve_finish_kernel(const Table t, ReserveSpace w, const int32_t *missing, const CopyArrays arrays)
{
    pdl_wait();
    pdl_trigger();
    const int copies = *w.copies;
    if (*missing == 0) {
        const int i0 = blockIdx.x * kThreads + threadIdx.x, step = gridDim.x * kThreads;
        for (int s = i0; s < t.num_seqs; s += step)
            if (w.grow[s] > 0)   // (a negative length is none)
                t.lens[s] = max(t.lens[s], 0) + w.grow[s];
        for (int i = i0; i < copies; i += step)
            atomicSub(t.refs + w.copy_src[i], 1);
    }
    copy_listed<kThreads>(arrays, w.copy_src, w.copy_dst, copies);
}

// ---------------------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------------------
__global__ void __launch_bounds__(kRowThreads, 1)
    compact_count_kernel(const int32_t *refs, int num_pages, CompactSpace w)
{
    pdl_wait();
    pdl_trigger();
    __shared__ long long red[32];
    const int begin = blockIdx.x * kPageSegment;
    const int n = count_pages<kRowThreads>(refs, begin, segment_pages(begin, num_pages), true, red);
    if (threadIdx.x == 0)
        w.seg_counts[blockIdx.x] = n;
}

// Where page p goes, `rank` used ones lying below it: those below the border (the number in use) stay, `stay`
// of them in all.  A page that moves is marked -2 - i, i its place in the list of moves.
__device__ __forceinline__ void map_page(int p, bool used, int rank, int border, int stay,
                                         const CompactSpace &w, int32_t *page_map)
{
    int to = used ? p : -1;
    if (used && p >= border) {
        const int i = rank - stay;
        w.copy_src[i] = p;
        to = -2 - i;
    } else if (!used && p < border) {
        w.copy_dst[p - rank] = p;
    }
    page_map[p] = to;
}

// The same for `pages` ones from begin on, `before` used ones lying below them.
__device__ __forceinline__ void map_pages(const int32_t *refs, int begin, int pages, long long before,
                                          int border, int stay, const CompactSpace &w, int32_t *page_map,
                                          long long *red)
{
    for (int i0 = 0; i0 < pages; i0 += kRowThreads) {
        const int i = i0 + threadIdx.x, p = begin + i;
        const bool used = i < pages && refs[p] > 0;
        long long total;
        const int rank = static_cast<int>(before + scan_exclusive<kRowThreads>(used, red, &total));
        before += total;
        if (i < pages)
            map_page(p, used, rank, border, stay, w, page_map);
    }
}

__global__ void __launch_bounds__(kRowThreads, 1)
    compact_map_kernel(const int32_t *refs, int num_pages, CompactSpace w, int segments, int32_t *page_map,
                       int32_t *num_live)
{
    pdl_wait();
    pdl_trigger();
    __shared__ long long red[32];
    const int seg = blockIdx.x;
    long long before, live;
    {
        long long b = 0, f = 0;
        for (int i = threadIdx.x; i < segments; i += kRowThreads) {
            const int n = w.seg_counts[i];
            f += n;
            b += i < seg ? n : 0;
        }
        scan_exclusive<kRowThreads>(b, red, &before);
        scan_exclusive<kRowThreads>(f, red, &live);
    }
    // used pages below the number in use: they stay
    const int border = static_cast<int>(live);
    long long stay;
    {
        long long b = 0;
        const int whole = border / kPageSegment;
        for (int i = threadIdx.x; i < whole; i += kRowThreads)
            b += w.seg_counts[i];
        scan_exclusive<kRowThreads>(b, red, &stay);
        stay += count_pages<kRowThreads>(refs, whole * kPageSegment, border % kPageSegment, true, red);
    }
    if (seg == 0 && threadIdx.x == 0) {
        *num_live = border;
        *w.copies = static_cast<int>(live - stay);
    }
    const int begin = seg * kPageSegment;
    map_pages(refs, begin, segment_pages(begin, num_pages), before, border, static_cast<int>(stay), w,
              page_map, red);
}

// The map by one block, for at most kOneBlockPages pages.
__device__ void compact_decide(const int32_t *refs, int num_pages, const CompactSpace &w, int32_t *page_map,
                               int32_t *num_live, long long *red, PageBits &used)
{
    used.load(refs, num_pages, true);
    __syncthreads();
    const int border = used.count(red);
    const int stay = used.below(border);
    if (threadIdx.x == 0) {
        *num_live = border;
        *w.copies = border - stay;
    }
    for (int p = threadIdx.x; p < num_pages; p += kRowThreads)
        map_page(p, used.has(p), used.below(p), border, stay, w, page_map);
}

// The tables, the counts and the map follow the moves, and the copies, by all blocks of N threads.  A table
// entry reads a mark or what has already replaced it: the same page either way.
template <int N>
__device__ __forceinline__ void compact_finish(const Table &t, const CompactSpace &w, int32_t *page_map,
                                               const CopyArrays &arrays, uint32_t *err)
{
    const int moves = __ldcg(w.copies);
    for (int s = blockIdx.x; s < t.num_seqs; s += gridDim.x) {
        const int n = row_len(t.lens, s, t.stride, t.page_size, threadIdx.x == 0, err);
        int32_t *row = t.rows + static_cast<size_t>(s) * t.stride;
        const int end = pages_of(n, t.page_size);
        for (int i = threadIdx.x; i < end; i += N) {
            const int page = row[i];
            if (page < 0 || page >= t.num_pages) {
                atomicOr(err, kErrPageRange);
                continue;
            }
            const int to = __ldcg(page_map + page);
            if (to == -1)
                atomicOr(err, kErrPageRefs);   // a page that nothing counts: left as it is
            else if (to != page)
                row[i] = to >= 0 ? to : __ldcg(w.copy_dst + (-2 - to));
        }
    }
    for (int i = blockIdx.x * N + threadIdx.x; i < moves; i += gridDim.x * N) {
        const int src = __ldcg(w.copy_src + i), dst = __ldcg(w.copy_dst + i);
        t.refs[dst] = t.refs[src];
        t.refs[src] = 0;
        page_map[src] = dst;
    }
    copy_listed<N>(arrays, w.copy_src, w.copy_dst, moves);
}

__global__ void __launch_bounds__(kThreads)
    compact_finish_kernel(const Table t, CompactSpace w, int32_t *page_map, const CopyArrays arrays,
                          uint32_t *word)
{
    pdl_wait();
    pdl_trigger();
    compact_finish<kThreads>(t, w, page_map, arrays, word ? word : &g_pages_errors);
}

__global__ void __launch_bounds__(kRowThreads, 1)
    compact_decide_kernel(const int32_t *refs, int num_pages, CompactSpace w, int32_t *page_map,
                          int32_t *num_live)
{
    pdl_wait();
    pdl_trigger();
    __shared__ long long red[32];
    __shared__ PageBits used;
    compact_decide(refs, num_pages, w, page_map, num_live, red, used);
}

__global__ void __cluster_dims__(kClusterBlocks, 1, 1) __launch_bounds__(kRowThreads, 1)
    compact_cluster_kernel(const Table t, CompactSpace w, int32_t *page_map, int32_t *num_live,
                           const CopyArrays arrays, uint32_t *word)
{
    pdl_wait();
    pdl_trigger();
    __shared__ long long red[32];
    __shared__ PageBits used;
    if (blockIdx.x == 0)
        compact_decide(t.refs, t.num_pages, w, page_map, num_live, red, used);
    cluster_sync();
    compact_finish<kRowThreads>(t, w, page_map, arrays, word ? word : &g_pages_errors);
}

// More arrays than one launch takes.
__global__ void __launch_bounds__(kThreads)
    copy_listed_kernel(const CopyArrays arrays, const int32_t *src, const int32_t *dst, const int32_t *count)
{
    pdl_wait();
    pdl_trigger();
    copy_listed<kThreads>(arrays, src, dst, *count);
}

int segments_of(int num_pages) { return (num_pages - 1) / kPageSegment + 1; }

// Arrays first .. first + kMaxCopyArrays - 1.
CopyArrays some_arrays(const PagesLaunch &l, int first)
{
    CopyArrays c;
    c.num = 0;
    c.pieces = 0;
    for (int i = first; i < l.num_arrays && c.num < kMaxCopyArrays; ++i, ++c.num) {
        c.data[c.num] = static_cast<uint8_t *>(l.arrays[i].data);
        c.chunks[c.num] = static_cast<uint32_t>(l.arrays[i].page_bytes / 16);
        const uint32_t pieces = (c.chunks[c.num] + kPieceChunks - 1) / kPieceChunks;
        c.pieces = pieces > c.pieces ? pieces : c.pieces;
    }
    return c;
}

Table table_of(const PagesLaunch &l)
{
    Table t;
    t.rows = l.block_table;
    t.stride = l.bt_stride;
    t.lens = l.context_lens;
    t.num_seqs = l.num_seqs;
    t.refs = l.page_refs;
    t.num_pages = l.num_pages;
    t.page_size = l.page_size;
    return t;
}

// Blocks of a launch that copies up to `most` pages of the arrays, and does `other` blocks' worth else.
unsigned copy_blocks(const CopyArrays &c, long long most, long long other)
{
    const long long work = std::max(most * c.num * c.pieces, other);
    const long long cap = static_cast<long long>(current_sm_count()) * 8;
    return static_cast<unsigned>(std::max<long long>(1, std::min(work, cap)));
}

// Bytes of a page in all arrays.
long long page_bytes(const PagesLaunch &l)
{
    long long n = 0;
    for (int i = 0; i < l.num_arrays; ++i)
        n += l.arrays[i].page_bytes;
    return n;
}

// Copies of at most this much are left to a cluster of eight SMs (which move about 1 TB/s).
constexpr long long kClusterBytes = 4LL << 20;

cudaError_t copy_the_rest(const PagesLaunch &l, const int32_t *src, const int32_t *dst,
                          const int32_t *count, long long most, cudaStream_t stream)
{
    for (int first = kMaxCopyArrays; first < l.num_arrays; first += kMaxCopyArrays) {
        const CopyArrays c = some_arrays(l, first);
        const cudaError_t err = launch_pdl(copy_listed_kernel, dim3(copy_blocks(c, most, 1)),
                                           dim3(kThreads), 0, stream, c, src, dst, count);
        if (err != cudaSuccess)
            return err;
    }
    return cudaSuccess;
}

// Carves arrays out of a workspace; without one it only adds up.
struct Carver {
    uint8_t *base;
    size_t used = 0;
    template <class T>
    T *take(size_t n)
    {
        T *p = base ? reinterpret_cast<T *>(base + used) : nullptr;
        used += (n * sizeof(T) + 255) / 256 * 256;
        return p;
    }
};

ReserveSpace reserve_space(void *base, int num_seqs, int num_pages, size_t *bytes)
{
    Carver c{static_cast<uint8_t *>(base)};
    ReserveSpace w;
    w.totals = c.take<long long>(2);
    w.copies = c.take<int32_t>(1);
    w.seg_counts = c.take<int32_t>(segments_of(num_pages));
    w.start = c.take<int32_t>(num_seqs);
    w.grow = c.take<int32_t>(num_seqs);
    w.copy_at = c.take<int32_t>(num_seqs);
    w.copy_src = c.take<int32_t>(num_seqs);
    w.copy_dst = c.take<int32_t>(num_seqs);
    w.sharers = c.take<int2>(num_pages);
    *bytes = c.used;
    return w;
}

CompactSpace compact_space(void *base, int num_pages, size_t *bytes)
{
    Carver c{static_cast<uint8_t *>(base)};
    CompactSpace w;
    w.copies = c.take<int32_t>(1);
    w.seg_counts = c.take<int32_t>(segments_of(num_pages));
    w.copy_src = c.take<int32_t>(num_pages / 2 + 1);   // as many moves as holes, at most half
    w.copy_dst = c.take<int32_t>(num_pages / 2 + 1);
    *bytes = c.used;
    return w;
}

}  // namespace

size_t reserve_workspace_bytes(int num_seqs, int num_pages)
{
    size_t bytes;
    reserve_space(nullptr, num_seqs, num_pages, &bytes);
    return bytes;
}

size_t compact_workspace_bytes(int num_pages)
{
    size_t bytes;
    compact_space(nullptr, num_pages, &bytes);
    return bytes;
}

cudaError_t launch_truncate(const PagesLaunch &l, const int32_t *new_lens, cudaStream_t stream)
{
    if (l.num_seqs == 0)
        return cudaSuccess;
    return launch_pdl(truncate_kernel, dim3(l.num_seqs), dim3(kThreads), 0, stream, table_of(l), new_lens,
                      current_error_word());
}

cudaError_t launch_fork(const PagesLaunch &l, int32_t *out_rows, int out_stride, int32_t *out_lens,
                        const int32_t *parents, const int32_t *share_lens, int num_out, cudaStream_t stream)
{
    if (num_out == 0)
        return cudaSuccess;
    return launch_pdl(fork_kernel, dim3(num_out), dim3(kThreads), 0, stream, table_of(l), out_rows,
                      out_stride, out_lens, parents, share_lens, current_error_word());
}

cudaError_t launch_reserve(const PagesLaunch &l, const int32_t *new_tokens, int32_t *missing,
                           void *workspace, cudaStream_t stream)
{
    size_t bytes;
    const ReserveSpace w = reserve_space(workspace, l.num_seqs, l.num_pages, &bytes);
    const Table t = table_of(l);
    const CopyArrays c = some_arrays(l, 0);
    const bool one_block = l.num_seqs <= kRowThreads && l.num_pages <= kOneBlockPages;
    if (one_block && page_bytes(l) * l.num_seqs <= kClusterBytes && l.num_arrays <= kMaxCopyArrays)
        return launch_pdl(reserve_cluster_kernel, dim3(kClusterBlocks), dim3(kRowThreads), 0, stream, t,
                          new_tokens, w, missing, c, current_error_word());
    cudaError_t err;
    if (one_block) {
        err = launch_pdl(reserve_decide_kernel, dim3(1), dim3(kRowThreads), 0, stream, t, new_tokens, w,
                         missing, current_error_word());
        if (err == cudaSuccess && l.num_arrays > 0)
            err = launch_pdl(copy_listed_kernel, dim3(copy_blocks(c, l.num_seqs, 1)), dim3(kThreads), 0,
                             stream, c, static_cast<const int32_t *>(w.copy_src),
                             static_cast<const int32_t *>(w.copy_dst),
                             static_cast<const int32_t *>(w.copies));
    } else {
        const int segments = segments_of(l.num_pages);
        err = launch_pdl(reserve_count_kernel, dim3(segments + 1), dim3(kRowThreads), 0, stream, t,
                         new_tokens, w, current_error_word());
        if (err != cudaSuccess)
            return err;
        err = launch_pdl(reserve_assign_kernel, dim3(segments), dim3(kRowThreads), 0, stream, t, w,
                         segments, missing);
        if (err != cudaSuccess)
            return err;
        err = launch_pdl(reserve_finish_kernel,
                         dim3(copy_blocks(c, l.num_seqs, (l.num_seqs + kThreads - 1) / kThreads)),
                         dim3(kThreads), 0, stream, t, w, static_cast<const int32_t *>(missing), c);
    }
    return err != cudaSuccess ? err : copy_the_rest(l, w.copy_src, w.copy_dst, w.copies, l.num_seqs, stream);
}

cudaError_t launch_compact(const PagesLaunch &l, int32_t *page_map, int32_t *num_live, void *workspace,
                           cudaStream_t stream)
{
    size_t bytes;
    const CompactSpace w = compact_space(workspace, l.num_pages, &bytes);
    const Table t = table_of(l);
    const CopyArrays c = some_arrays(l, 0);
    const bool one_block = l.num_pages <= kOneBlockPages;
    if (one_block && page_bytes(l) * (l.num_pages / 2) <= kClusterBytes && l.num_arrays <= kMaxCopyArrays &&
        l.num_seqs <= kRowThreads)
        return launch_pdl(compact_cluster_kernel, dim3(kClusterBlocks), dim3(kRowThreads), 0, stream, t, w,
                          page_map, num_live, c, current_error_word());
    cudaError_t err;
    if (one_block) {
        err = launch_pdl(compact_decide_kernel, dim3(1), dim3(kRowThreads), 0, stream,
                         static_cast<const int32_t *>(t.refs), t.num_pages, w, page_map, num_live);
    } else {
        const int segments = segments_of(l.num_pages);
        err = launch_pdl(compact_count_kernel, dim3(segments), dim3(kRowThreads), 0, stream,
                         static_cast<const int32_t *>(t.refs), t.num_pages, w);
        if (err != cudaSuccess)
            return err;
        err = launch_pdl(compact_map_kernel, dim3(segments), dim3(kRowThreads), 0, stream,
                         static_cast<const int32_t *>(t.refs), t.num_pages, w, segments, page_map, num_live);
    }
    if (err != cudaSuccess)
        return err;
    err = launch_pdl(compact_finish_kernel, dim3(copy_blocks(c, l.num_pages / 2, l.num_seqs)),
                     dim3(kThreads), 0, stream, t, w, page_map, c, current_error_word());
    return err != cudaSuccess ? err
                              : copy_the_rest(l, w.copy_src, w.copy_dst, w.copies, l.num_pages / 2, stream);
}

cudaError_t read_and_clear_pages_errors(uint32_t *flags)
{
    uint32_t zero = 0;
    cudaError_t err = cudaMemcpyFromSymbol(flags, g_pages_errors, sizeof(uint32_t));
    if (err != cudaSuccess)
        return err;
    return cudaMemcpyToSymbol(g_pages_errors, &zero, sizeof(uint32_t));
}

}  // namespace kvc
