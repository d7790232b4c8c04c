// kvc_evict.cu -- eviction from the paged cache by accumulated attention weight.
//
// What it computes, for every sequence s and kv head h on its own: of the N = context_lens[s] slots
// keep n = min(N, budget): first those whose original position is among the newest `recent`, then
// the ones with the largest accumulated weight, equal weights in slot order.  The kept slots at n and
// above move into the evicted slots below n, both in ascending order, so the kept ones end up in
// slots 0 .. n - 1.  Attention does not ask for an order (keys carry their positions), and moving
// only what has to move leaves every slot either a source or a destination, never both: all moves
// run at once, in place, at the least traffic (closing the gaps in order would move nearly every
// row after the first gap).  `positions` keeps each slot's original position, which is what the
// newest are told by.
//
// Selection.  A weight becomes a 32-bit key of the same order (NaN as the lowest, -0 as 0, the newest
// slots above every weight), and the n-th largest key is found digit by digit: four histograms of
// 8 bits, then the slots equal to it are kept in slot order until n is full.  One cluster of 1 to 8
// CTAs per (sequence, kv head): the histograms meet through distributed shared memory, one
// cluster barrier each.  The keys stay in shared memory between the passes (beyond kMaxCached slots a
// CTA makes them anew from weights and positions).  Every warp owns consecutive slots, so ranks in
// slot order are ballots and one prefix over warps and CTAs; nothing depends on the order of
// atomics (the histograms only count).
//
// Bound: the moved rows (4 D bytes read and written each) by HBM when there are many, else the chain of
// barriers; the selection reads 8 and writes 8 bytes a slot.
#include <cooperative_groups.h>

#include "kvc_device.cuh"
#include "kvc_launch.h"

namespace kvc {

namespace {

namespace cg = cooperative_groups;

__device__ uint32_t g_evict_errors;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 256;
constexpr uint32_t kNewest = 0xFFFFFFFFu;

struct Args {
    uint4 *k_pool, *v_pool;
    const int32_t *block_table;
    int bt_stride;
    const int32_t *context_lens;
    int num_seqs, max_ctx;
    const float *weights;
    const int32_t *positions;
    float *weights_out;
    int32_t *positions_out;
    const int32_t *rows;
    int num_rows, stride;
    int budget, recent;
    int32_t *new_lens;
    int32_t *lists;      // [S][Hkv][2][list_cap]: destinations, sources
    int list_cap;
    int kv_heads, log2_page, num_pages, hnd;
    int cached;          // keys that fit a CTA's shared memory
    uint32_t *err;
};

// Sums over the CTA's warps, and the ranks before each.
struct Shared {
    uint32_t hist[2][kBins];
    uint32_t warp_sum[2][kWarps];
    uint32_t total[2];        // this CTA's counts, read by the cluster
    uint32_t digit, above;    // the digit of the threshold and the keys above it in this pass
};

// The order of floats as unsigned integers: NaN is taken as -infinity, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (w != w)
        w = -__int_as_float(0x7F800000);
    const uint32_t b = __float_as_uint(w + 0.0f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

template <int D>
__global__ void __launch_bounds__(kThreads) evict_kernel(const Args a)
{
    pdl_wait();
    pdl_trigger();
    extern __shared__ __align__(16) uint32_t keys[];   // [cached], then Shared
    Shared &sh = *reinterpret_cast<Shared *>(keys + a.cached);
    const cg::cluster_group cluster = cg::this_cluster();
    const int cta = static_cast<int>(cluster.block_rank());
    const int ctas = static_cast<int>(cluster.num_blocks());
    const int unit = blockIdx.x / ctas;
    const int kvh = unit % a.kv_heads;
    const int s = unit / a.kv_heads;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    uint32_t *err = a.err ? a.err : &g_evict_errors;

    const int raw = a.context_lens[s];
    const long long cap = min(static_cast<long long>(a.bt_stride) << a.log2_page,
                              static_cast<long long>(min(a.max_ctx, a.stride)));
    const int N = static_cast<int>(max(0LL, min(static_cast<long long>(raw), cap)));
    const int row = a.rows ? a.rows[s] : s;
    const bool first = kvh == 0 && cta == 0 && threadIdx.x == 0;
    if (first) {
        if (raw > cap)
            atomicOr(err, kErrContextRange);
        if (row >= a.num_rows)
            atomicOr(err, kErrSlotRange);
    }
    if (row < 0 || row >= a.num_rows) {   // a sequence without a row keeps everything
        if (first)
            a.new_lens[s] = raw;
        return;
    }
    const int n = min(N, a.budget);
    const size_t base = (static_cast<size_t>(row) * a.kv_heads + kvh) * a.stride;
    const float *w_in = a.weights + base;
    const int32_t *p_in = a.positions + base;
    float *w_out = a.weights_out + base;
    int32_t *p_out = a.positions_out + base;
    const int last = N > 0 ? p_in[N - 1] : -1;   // the newest token's original position
    if (first)
        a.new_lens[s] = n;

    // this warp's slots [lo, hi); the CTA's begin at cta_lo
    const int per_warp = static_cast<int>(
        (static_cast<long long>(N) + 32LL * kWarps * ctas - 1) / (32LL * kWarps * ctas)) * 32;
    const int cta_lo = static_cast<int>(
        min(static_cast<long long>(N), static_cast<long long>(per_warp) * kWarps * cta));
    const int lo = static_cast<int>(min(static_cast<long long>(N),
                                        cta_lo + static_cast<long long>(per_warp) * warp));
    const int hi = static_cast<int>(min(static_cast<long long>(N),
                                        lo + static_cast<long long>(per_warp)));

    if (N <= a.budget) {   // nothing to evict
        for (int i = lo + lane; i < hi; i += 32) {
            w_out[i] = w_in[i];
            p_out[i] = p_in[i];
        }
        for (long long i = static_cast<long long>(N) + cta * kThreads + threadIdx.x; i < a.stride;
             i += ctas * kThreads)
            p_out[i] = static_cast<int32_t>(last + 1 + (i - n));
        return;
    }

    const long long newest = static_cast<long long>(last) - a.recent;   // positions above it
    auto make_key = [&](int i) -> uint32_t {
        const float w = w_in[i];
        return p_in[i] > newest ? kNewest : weight_key(w);
    };
    auto key_at = [&](int i) -> uint32_t {
        const int c = i - cta_lo;
        return c < a.cached ? keys[c] : make_key(i);
    };
#pragma unroll 4
    for (int i = lo + lane; i < hi; i += 32) {
        const uint32_t k = make_key(i);
        if (i - cta_lo < a.cached)
            keys[i - cta_lo] = k;
    }

    // ---- the n-th largest key, and how many equal to it are kept ----
    uint32_t prefix = 0;
    uint32_t need = n;   // keys still wanted among those that share the prefix
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        uint32_t *hist = sh.hist[pass & 1];
        if (threadIdx.x < kBins)
            hist[threadIdx.x] = 0;
        __syncthreads();
        for (int i0 = lo; i0 < hi; i0 += 32) {
            const int i = i0 + lane;
            const uint32_t k = i < hi ? key_at(i) : 0u;
            const bool in = i < hi && (pass == 0 || (k >> (shift + 8)) == prefix);
            const uint32_t bin = in ? (k >> shift) & 0xFFu : kBins;
            // slots of one value (zeros, the newest) would queue up on one counter
            int same;
            __match_all_sync(0xffffffffu, bin, &same);
            if (same) {
                if (lane == 0 && in)
                    atomicAdd(&hist[bin], 32u);
            } else if (in) {
                atomicAdd(&hist[bin], 1u);
            }
        }
        cluster.sync();
        if (threadIdx.x < kBins) {
            // bin b of the whole cluster to thread 255 - b: a prefix sum counts from the top
            const int b = kBins - 1 - threadIdx.x;
            uint32_t count = 0;
            for (int c = 0; c < ctas; ++c)
                count += *cluster.map_shared_rank(&hist[b], c);
            uint32_t incl = count;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off)
                    incl += v;
            }
            if (lane == 31)
                sh.warp_sum[0][warp] = incl;
            named_barrier(1, kBins);
            uint32_t before = incl - count;
            for (int v = 0; v < warp; ++v)
                before += sh.warp_sum[0][v];
            if (before < need && need <= before + count) {
                sh.digit = b;
                sh.above = before;
            }
        }
        __syncthreads();
        prefix = (prefix << 8) | sh.digit;
        need -= sh.above;
    }
    // The last pass counted the keys equal to the threshold (its own digit's bin): those of the
    // CTAs before this one come first.
    const uint32_t threshold = prefix;
    uint32_t eq_before = 0;
    for (int c = 0; c < cta; ++c)
        eq_before += *cluster.map_shared_rank(&sh.hist[1][threshold & 0xFFu], c);

    // ---- ranks in slot order: equal keys, then gaps below n and kept slots from n on ----
    uint32_t eq = 0;
    for (int i0 = lo; i0 < hi; i0 += 32) {
        const int i = i0 + lane;
        eq += __popc(__ballot_sync(0xffffffffu, i < hi && key_at(i) == threshold));
    }
    if (lane == 0)
        sh.warp_sum[1][warp] = eq;
    __syncthreads();
    for (int v = 0; v < warp; ++v)
        eq_before += sh.warp_sum[1][v];
    auto kept_lanes = [&](int i0, uint32_t &eq_rank) -> uint32_t {
        const int i = i0 + lane;
        const uint32_t k = i < hi ? key_at(i) : 0u;
        const bool is_eq = i < hi && k == threshold;
        const uint32_t eqs = __ballot_sync(0xffffffffu, is_eq);
        const uint32_t rank = eq_rank + __popc(eqs & ((1u << lane) - 1u));
        eq_rank += __popc(eqs);
        return __ballot_sync(0xffffffffu,
                             i < hi && (k > threshold || (is_eq && rank < need)));
    };
    uint32_t gaps = 0, tails = 0;
    {
        uint32_t rank = eq_before;
        for (int i0 = lo; i0 < hi; i0 += 32) {
            const uint32_t kept = kept_lanes(i0, rank);
            const int i = i0 + lane;
            const bool keep = (kept >> lane) & 1u;
            gaps += __popc(__ballot_sync(0xffffffffu, i < n && !keep));
            tails += __popc(__ballot_sync(0xffffffffu, i >= n && keep));
        }
    }
    __syncthreads();   // every warp has read the counts of equal keys
    if (lane == 0) {
        sh.warp_sum[0][warp] = gaps;
        sh.warp_sum[1][warp] = tails;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        uint32_t t = 0;
        for (int v = 0; v < kWarps; ++v)
            t += sh.warp_sum[threadIdx.x][v];
        sh.total[threadIdx.x] = t;
    }
    cluster.sync();
    uint32_t gap_at = 0, tail_at = 0, moves = 0;
    for (int c = 0; c < ctas; ++c) {
        const uint32_t *t = cluster.map_shared_rank(sh.total, c);
        if (c < cta) {
            gap_at += t[0];
            tail_at += t[1];
        }
        moves += t[0];
    }
    for (int v = 0; v < warp; ++v) {
        gap_at += sh.warp_sum[0][v];
        tail_at += sh.warp_sum[1][v];
    }
    int32_t *dst_list = a.lists + static_cast<size_t>(unit) * 2 * a.list_cap;
    int32_t *src_list = dst_list + a.list_cap;
    {
        uint32_t rank = eq_before;
        for (int i0 = lo; i0 < hi; i0 += 32) {
            const uint32_t kept = kept_lanes(i0, rank);
            const int i = i0 + lane;
            const bool keep = (kept >> lane) & 1u;
            const uint32_t g = __ballot_sync(0xffffffffu, i < n && !keep);
            const uint32_t t = __ballot_sync(0xffffffffu, i >= n && keep);
            const uint32_t below = (1u << lane) - 1u;
            if ((g >> lane) & 1u)
                dst_list[gap_at + __popc(g & below)] = i;
            if ((t >> lane) & 1u)
                src_list[tail_at + __popc(t & below)] = i;
            if (keep && i < n) {   // stays where it is
                w_out[i] = w_in[i];
                p_out[i] = p_in[i];
            }
            gap_at += __popc(g);
            tail_at += __popc(t);
        }
    }
    __threadfence();
    cluster.sync();

    // ---- the moves ----
    constexpr int kVec = D / 8;                 // 16-byte chunks of a vector
    constexpr int kMoveLanes = 2 * kVec;        // K and V
    constexpr int kPerWarp = 32 / kMoveLanes;   // moves that a warp makes at a time
    constexpr int kUnroll = 4;
    const int sub = lane / kMoveLanes;
    const int in_move = lane % kMoveLanes;
    uint4 *pool = in_move < kVec ? a.k_pool : a.v_pool;
    const int chunk = in_move % kVec;
    const int32_t *bt = a.block_table + static_cast<size_t>(s) * a.bt_stride;
    const int P1 = (1 << a.log2_page) - 1;
    auto place = [&](int slot, bool &ok) -> size_t {
        const int page = bt[slot >> a.log2_page];
        ok = ok && page >= 0 && page < a.num_pages;
        const size_t off = slot & P1;
        const size_t vec =
            a.hnd ? ((static_cast<size_t>(page) * a.kv_heads + kvh) << a.log2_page) + off
                  : ((static_cast<size_t>(page) << a.log2_page) + off) * a.kv_heads + kvh;
        return vec * kVec + chunk;
    };
    const int movers = ctas * kWarps * kPerWarp;
    for (int j0 = (cta * kWarps + warp) * kPerWarp + sub; j0 - sub < static_cast<int>(moves);
         j0 += movers * kUnroll) {
        size_t to[kUnroll];
        uint4 x[kUnroll];
        bool go[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int j = j0 + u * movers;
            const bool in = j < static_cast<int>(moves);
            go[u] = in;
            if (in) {
                const int src = __ldcg(src_list + j), dst = __ldcg(dst_list + j);
                if (in_move == 0) {
                    w_out[dst] = w_in[src];
                    p_out[dst] = p_in[src];
                }
                const size_t from = place(src, go[u]);
                to[u] = place(dst, go[u]);
                if (go[u])
                    x[u] = pool[from];
                else if (in_move == 0)
                    atomicOr(err, kErrPageRange);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (go[u])
                pool[to[u]] = x[u];
    }
    cluster.sync();   // the moved slots' weights and positions are read: the tail may be written

    // ---- the slots from n on are free: weight 0, and the positions that tokens to come will have ----
    for (long long i = static_cast<long long>(n) + cta * kThreads + threadIdx.x; i < a.stride;
         i += ctas * kThreads) {
        if (i < N)
            w_out[i] = 0.0f;
        p_out[i] = static_cast<int32_t>(last + 1 + (i - n));
    }
}

template <int D>
cudaError_t launch_t(const EvictLaunch &l, const Args &args, cudaStream_t stream)
{
    Args a = args;
    const long long units = static_cast<long long>(l.num_seqs) * l.kv_heads;
    // Clusters only where (sequence, kv head) units alone leave SMs idle and rows are long
    // enough to share: a cluster barrier costs more than a CTA's.
    int ctas = 1;
    while (ctas < 8 && units * ctas * 2 <= 4LL * current_sm_count() &&
           l.max_ctx / (ctas * 2) >= 1024)
        ctas *= 2;
    const long long per_cta =
        (static_cast<long long>(l.max_ctx) + 32LL * kWarps * ctas - 1) / (32LL * kWarps * ctas) *
        32 * kWarps;
    a.cached = static_cast<int>(per_cta < kMaxCached ? per_cta : kMaxCached);
    const size_t smem = static_cast<size_t>(a.cached) * 4 + sizeof(Shared);
    auto kernel = evict_kernel<D>;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           kMaxCached * 4 + static_cast<int>(sizeof(Shared)));
    if (err != cudaSuccess)
        return err;
    if (units * ctas > 0x7FFFFFFFLL)
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(units * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_evict(const EvictLaunch &l, cudaStream_t stream)
{
    if (l.num_seqs == 0)
        return cudaSuccess;
    Args a;
    a.k_pool = static_cast<uint4 *>(l.k_pool);
    a.v_pool = static_cast<uint4 *>(l.v_pool);
    a.block_table = l.block_table;
    a.bt_stride = l.bt_stride;
    a.context_lens = l.context_lens;
    a.num_seqs = l.num_seqs;
    a.max_ctx = l.max_ctx;
    a.weights = l.weights;
    a.positions = l.positions;
    a.weights_out = l.weights_out;
    a.positions_out = l.positions_out;
    a.rows = l.rows;
    a.num_rows = l.num_rows;
    a.stride = l.stride;
    a.budget = l.budget;
    a.recent = l.recent;
    a.new_lens = l.new_lens;
    a.lists = static_cast<int32_t *>(l.lists);
    a.list_cap = l.list_cap;
    a.kv_heads = l.kv_heads;
    a.log2_page = l.page_size == 16 ? 4 : l.page_size == 32 ? 5 : 6;
    a.num_pages = l.num_pages;
    a.hnd = l.hnd ? 1 : 0;
    a.err = current_error_word();
    return l.head_dim == 128 ? launch_t<128>(l, a, stream) : launch_t<64>(l, a, stream);
}

cudaError_t read_and_clear_evict_errors(uint32_t *flags)
{
    uint32_t zero = 0;
    cudaError_t err = cudaMemcpyFromSymbol(flags, g_evict_errors, sizeof(uint32_t));
    if (err != cudaSuccess)
        return err;
    return cudaMemcpyToSymbol(g_evict_errors, &zero, sizeof(uint32_t));
}

}  // namespace kvc
