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
// newest are told by; the newest one itself is what the first free slot's position follows, because
// after a cut the last slot may hold any token, and a sequence may pause before its next one.
//
// Selection (select_kernel).  A weight becomes a 32-bit key of the same order (NaN as the lowest, -0
// as 0, the newest slots above every weight), and the n-th largest key is found digit by digit:
// histograms of 11, 11 and 10 bits.  (Digits of 8 bits would be four passes, and the first one, sign
// and seven exponent bits, would put all weights into a handful of counters that queue up.)  After the
// first digit a slot is kept, evicted or one of a few per cent still open: two bits a slot and a list of
// the open ones with their keys, so the weights and positions are read twice at most, and the other
// digits and the ranks work on those.  (With every step going over the keys again the selection of
// 64 rows of up to 131,072 slots took 74 us, now 58.)  Only a list that runs over sends the digits over
// all keys again.  One cluster of 1 to 8 CTAs per (sequence, kv head): the histograms meet through
// distributed shared memory, one cluster barrier each.  As many keys as fit stay in shared memory: with
// four CTAs an SM 6,528 a CTA, so a row of 131,072 slots over 8 CTAs has 60% of its slots read and made
// into keys twice, and shorter rows of the launch are spread over as many CTAs (of its 58 us, 15 are
// the bytes).
// Every warp owns consecutive slots and every lane four at a time, so ranks in slot order are one warp
// scan per 128 slots and a prefix over warps and CTAs; nothing depends on the order of atomics (the
// histograms only count, the list is read as a set).  The kernel leaves the moves as two lists.
//
// Moves (move_kernel).  One launch over all lists, 64 moves a CTA: rows differ in how much they
// move (a batch's longest several times its average), so the copies are spread over the SMs
// apart from the selection.  A warp looks up 16 moves and their pages at once and then keeps 3 rows
// in flight.  What bounds it is how HBM takes 256-byte rows at random places, read and written at
// once: 5.0 to 5.6 TB/s here, and more in flight makes it worse (64 sequences of up to 4,096 slots
// cut to 2,048, selection and moves: 57.6 us with 3 rows of 16 moves, 58.1 with 4, 71 with 8, 70 with 8
// moves looked up at once; the moves cut into equal ranges over one wave of CTAs 68).
//
// Bound: the moved rows (4 D bytes read and written each) by HBM when there are many, else the chain of
// barriers; the selection reads 8 and writes 8 bytes a slot.
#include <cooperative_groups.h>

#include <algorithm>

#include "kvc_device.cuh"
#include "kvc_launch.h"

namespace kvc {

namespace {

namespace cg = cooperative_groups;

__device__ uint32_t g_evict_errors;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kWarpSlots = 128;   // slots of one step of a warp, four consecutive ones a lane
constexpr int kListed = 1024;     // slots of a CTA in the first digit's bin that are kept apart
constexpr int kAhead = 2;         // steps of loads that a thread has in flight
constexpr int kMaxCtas = 8;       // of a cluster
static_assert(kEvictMaxCtx <= kMaxCtas * kEvictCtaSlots, "the masks of a row");
constexpr uint32_t kNewest = 0xFFFFFFFFu;
constexpr long long kSmemPerSm = 228 * 1024;
constexpr long long kSmemPerCta = 227 * 1024;
constexpr int kMoveThreads = 128;
constexpr int kMoveCtas = 80;     // of the moves' launch, per SM (most of them find no move)
constexpr int kWarpMoves = 16;    // moves that a warp looks up at once
constexpr int kInlineMoves = 256;
constexpr int kInlineUnits = 8;   // units per SM up to which rows make their own moves
constexpr int kMovesPerCta = kMoveThreads / 32 * kWarpMoves;

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
    int2 *counts;        // [S][Hkv]: moves, and the position of a free slot i less i
    int list_cap;
    int kv_heads, log2_page, num_pages, hnd;
    int cached;          // keys that fit a CTA's shared memory
    int vec;             // rows of weights and positions start on 16 bytes
    int inline_moves;    // one CTA per row, few moves: no second launch
    uint32_t *err;
};

struct __align__(16) Shared {
    uint32_t hist[2][kBins];
    uint32_t listed[kListed];    // keys that share the first digit, and their slots in the CTA
    int listed_slot[kListed];
    uint32_t list_size;
    // Sums of the histogram's bins, eight each, top first.  The passes alternate: a CTA may be in the
    // next pass while another one still reads this pass's sums, but not in the next but one.
    uint32_t coarse[2][kThreads];
    uint32_t warp_sum[2][kWarps];
    uint32_t equal_here, gaps, tails;   // this CTA's, read by the cluster
    uint32_t digit, above, equal;       // the digit found, the keys above it and those in it
};

// The order of floats as unsigned integers: NaN is taken as -infinity, -0 as 0.  Never 0, which
// stands for no slot.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    const int b = __float_as_int(w + 0.0f);
    const uint32_t key = static_cast<uint32_t>(b) ^ (static_cast<uint32_t>(b >> 31) | 0x80000000u);
    return w != w ? 0x007FFFFFu : key;
}

__device__ __forceinline__ uint32_t warp_scan(uint32_t x, int lane)
{
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off)
            x += v;
    }
    return x;
}

// Carries out moves j0 .. j0 + n - 1 (n at most kWarpMoves) of a unit's lists, K and V, weight and
// position, by one warp.
template <int D>
__device__ __forceinline__ void move_rows(const Args &a, int unit, int j0, int n, int free_pos)
{
    const int lane = threadIdx.x & 31;
    constexpr int kVec = D / 8;                 // 16-byte chunks of a vector
    constexpr int kMoveLanes = 2 * kVec;        // K and V of one move
    constexpr int kAtOnce = 32 / kMoveLanes;    // moves that a warp copies with one load
    constexpr int kFly = 3;                     // loads in flight
    const int kvh = unit % a.kv_heads;
    const int s = unit / a.kv_heads;
    const int32_t *dst_list = a.lists + static_cast<size_t>(unit) * 2 * a.list_cap;
    const int32_t *bt = a.block_table + static_cast<size_t>(s) * a.bt_stride;
    long long from = -1, to = -1;   // 16-byte chunks; below 0: no copy
    int dst = -1, src = -1;
    if (lane < n) {
        dst = __ldcg(dst_list + j0 + lane);
        src = __ldcg(dst_list + a.list_cap + j0 + lane);
    }
    // (an entry that no slot was written to: the weights changed under the selection)
    if (static_cast<uint32_t>(dst) < static_cast<uint32_t>(a.max_ctx) &&
        static_cast<uint32_t>(src) < static_cast<uint32_t>(a.max_ctx)) {
        const int dp = bt[dst >> a.log2_page], sp = bt[src >> a.log2_page];
        if (dp >= 0 && dp < a.num_pages && sp >= 0 && sp < a.num_pages) {
            const int mask = (1 << a.log2_page) - 1;
            auto place = [&](int page, int off) -> long long {
                const long long vec =
                    a.hnd ? ((static_cast<long long>(page) * a.kv_heads + kvh) << a.log2_page) + off
                          : ((static_cast<long long>(page) << a.log2_page) + off) * a.kv_heads + kvh;
                return vec * kVec;
            };
            from = place(sp, src & mask);
            to = place(dp, dst & mask);
        } else {
            atomicOr(a.err ? a.err : &g_evict_errors, kErrPageRange);
        }
        const int row = a.rows ? a.rows[s] : s;
        const size_t base = (static_cast<size_t>(row) * a.kv_heads + kvh) * a.stride;
        const float w = a.weights[base + src];
        const int32_t p = a.positions[base + src];
        a.weights_out[base + dst] = w;
        a.positions_out[base + dst] = p;
        a.weights_out[base + src] = 0.0f;
        a.positions_out[base + src] = free_pos + src;
    }
    const int sub = lane / kMoveLanes;
    const int in_move = lane % kMoveLanes;
    uint4 *pool = (in_move < kVec ? a.k_pool : a.v_pool) + in_move % kVec;
    for (int u0 = 0; u0 < n; u0 += kFly * kAtOnce) {
        uint4 x[kFly];
        long long dst[kFly];
#pragma unroll
        for (int u = 0; u < kFly; ++u) {
            const int m = u0 + u * kAtOnce + sub;   // below 64; past n the lane's places are -1
            const long long f = __shfl_sync(0xffffffffu, from, m & 31);
            dst[u] = __shfl_sync(0xffffffffu, to, m & 31);
            if (m >= n)
                dst[u] = -1;
            if (dst[u] >= 0)
                x[u] = __ldcg(pool + f);
        }
#pragma unroll
        for (int u = 0; u < kFly; ++u)
            if (dst[u] >= 0)
                pool[dst[u]] = x[u];
    }
}

// (four CTAs an SM hold a thread to 64 registers, and 20 bytes of it are spilled)
template <int D>
__global__ void __launch_bounds__(kThreads, 4) select_kernel(const Args a)
{
    pdl_wait();
    pdl_trigger();
    extern __shared__ __align__(16) uint32_t keys[];   // [cached], then Shared and the masks
    Shared &sh = *reinterpret_cast<Shared *>(keys + a.cached);
    // A byte per four slots: bit e says that slot e of them is above the threshold, bit 4 + e that it
    // is equal to it.
    uint8_t *masks = reinterpret_cast<uint8_t *>(&sh + 1);
    const cg::cluster_group cluster = cg::this_cluster();
    const int cta = static_cast<int>(cluster.block_rank());
    const int ctas = static_cast<int>(cluster.num_blocks());
    auto cluster_sync = [&] {   // a cluster barrier costs more, even for one CTA
        if (ctas == 1)
            __syncthreads();
        else
            cluster.sync();
    };
    const int unit = blockIdx.x / ctas;
    const int kvh = unit % a.kv_heads;
    const int s = unit / a.kv_heads;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    uint32_t *err = a.err ? a.err : &g_evict_errors;

    for (int i = threadIdx.x; i < 2 * kBins; i += kThreads)
        sh.hist[0][i] = 0;
    if (threadIdx.x == 0)
        sh.list_size = 0;
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
    const bool none = row < 0 || row >= a.num_rows;   // a sequence without a row keeps everything
    const int n = min(N, a.budget);
    if (first)
        a.new_lens[s] = none ? raw : n;
    if (a.counts != nullptr && cta == 0 && threadIdx.x == 0 && (none || N <= a.budget))
        a.counts[unit] = make_int2(0, 0);
    if (none)
        return;
    const size_t base = (static_cast<size_t>(row) * a.kv_heads + kvh) * a.stride;
    const float *w_in = a.weights + base;
    const int32_t *p_in = a.positions + base;
    float *w_out = a.weights_out + base;
    int32_t *p_out = a.positions_out + base;
    // The newest token's original position.  In place one thread writes p_in[N] again: behind the
    // cluster's barriers, or (nothing to evict) with a value from which the same `last` follows.
    const int held = N > 0 ? p_in[N - 1] : -1;
    const bool has_next = N > 0 && N < a.stride;
    const int next = has_next ? p_in[N] : 0;
    const int last = has_next && next > held ? next - 1 : held;

    // this warp's slots [lo, hi); the CTA's begin at cta_lo
    const long long per_warp = (N + static_cast<long long>(kWarpSlots) * kWarps * ctas - 1) /
                               (kWarpSlots * kWarps * ctas) * kWarpSlots;
    const int cta_lo = static_cast<int>(min(static_cast<long long>(N), per_warp * kWarps * cta));
    const int lo = static_cast<int>(min(static_cast<long long>(N), cta_lo + per_warp * warp));
    const int hi = static_cast<int>(min(static_cast<long long>(N), lo + per_warp));

    if (N <= a.budget) {   // nothing to evict
        if (cta == 0 && threadIdx.x == 0 && has_next && next <= held)
            atomicOr(err, kErrPositionOrder);
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
    // Below n a slot keeps its weight and position (the moves write over the gaps); a free slot gets
    // weight 0 and the position that a token to come will have there.  Arrays apart from those that are
    // read get this with the first pass; in place, the slots that rows move out of become free with
    // the move.
    const int32_t free_pos = static_cast<int32_t>(static_cast<long long>(last) + 1 - n);
    const bool w_apart = w_out != w_in, p_apart = p_out != p_in;
    auto hand_on = [&](int i, const float (&w)[4], const int (&p)[4]) {
        if (a.vec && i + 3 < hi && (i >= n || i + 4 <= n)) {
            if (w_apart)
                *reinterpret_cast<float4 *>(w_out + i) =
                    i < n ? make_float4(w[0], w[1], w[2], w[3]) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (p_apart)
                *reinterpret_cast<int4 *>(p_out + i) =
                    i < n ? make_int4(p[0], p[1], p[2], p[3])
                          : make_int4(free_pos + i, free_pos + i + 1, free_pos + i + 2,
                                      free_pos + i + 3);
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e < hi) {
                if (w_apart)
                    w_out[i + e] = i + e < n ? w[e] : 0.0f;
                if (p_apart)
                    p_out[i + e] = i + e < n ? p[e] : free_pos + i + e;
            }
    };
    auto key_of = [&](float w, int p) { return p > newest ? kNewest : weight_key(w); };
    // Calls f(i, keys of slots i .. i + 3) for the warp's slots in order, i = 4 lane past each step's
    // first slot; all lanes go together, with keys 0 from hi on.  The slots below `from` come from
    // shared memory, the others from memory, kAhead steps' loads in flight; the first sweep also
    // hands weights and positions on.
    auto sweep = [&](int from, auto &&f, bool first = false) {
#pragma unroll 1
        for (int i0 = lo; i0 < hi; i0 += kAhead * kWarpSlots) {
            float w[kAhead][4];   // of cached slots the keys
            int p[kAhead][4];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = i0 + u * kWarpSlots + 4 * lane;
                if (!first && i0 + u * kWarpSlots - cta_lo < from) {
                    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);   // the bits of no slot
                    if (i < hi)
                        x = *reinterpret_cast<const float4 *>(keys + (i - cta_lo));
                    w[u][0] = x.x, w[u][1] = x.y, w[u][2] = x.z, w[u][3] = x.w;
                } else if (a.vec && i + 3 < hi) {
                    const float4 x = *reinterpret_cast<const float4 *>(w_in + i);
                    const int4 y = *reinterpret_cast<const int4 *>(p_in + i);
                    w[u][0] = x.x, w[u][1] = x.y, w[u][2] = x.z, w[u][3] = x.w;
                    p[u][0] = y.x, p[u][1] = y.y, p[u][2] = y.z, p[u][3] = y.w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (i + e < hi) {
                            w[u][e] = w_in[i + e];
                            p[u][e] = p_in[i + e];
                        }
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = i0 + u * kWarpSlots + 4 * lane;
                if (i0 + u * kWarpSlots >= hi)
                    break;
                if (first)
                    hand_on(i, w[u], p[u]);
                uint32_t k[4];
                if (!first && i0 + u * kWarpSlots - cta_lo < from) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        k[e] = __float_as_uint(w[u][e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        k[e] = key_of(w[u][e], p[u][e]);
                    if (i0 + (u + 1) * kWarpSlots > hi) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            k[e] = i + e < hi ? k[e] : 0u;
                    }
                }
                f(i, make_uint4(k[0], k[1], k[2], k[3]));
            }
        }
    };

    // ---- the n-th largest key, and how many equal to it are kept ----
    __syncthreads();   // the histograms are zero
    if (cta == 0 && threadIdx.x == 0 && has_next && (next <= held || next - 1 != held))
        atomicOr(err, kErrPositionOrder);
    sweep(0, [&](int i, const uint4 k) {
        if (i < hi && i - cta_lo < a.cached)
            *reinterpret_cast<uint4 *>(keys + (i - cta_lo)) = k;
        const uint32_t ks[4] = {k.x, k.y, k.z, k.w};
        // zeros and the newest come in runs, and would queue up on one counter
        int same;
        __match_all_sync(0xffffffffu, k.x, &same);
        if (same && __all_sync(0xffffffffu, k.x == k.y && k.x == k.z && k.x == k.w)) {
            if (lane == 0 && k.x != 0)
                atomicAdd(&sh.hist[0][k.x >> 21], static_cast<uint32_t>(kWarpSlots));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (ks[e] != 0)
                    atomicAdd(&sh.hist[0][ks[e] >> 21], 1u);
        }
    }, true);
    uint32_t prefix = 0;   // the digits found so far
    uint32_t need = n;     // keys still wanted among those that begin with them
    uint32_t equal = 0;    // how many these are
#pragma unroll 1
    for (int pass = 0;; ++pass) {
        uint32_t *hist = sh.hist[pass & 1];
        const int skip = pass == 1 ? 21 : pass == 2 ? 10 : 0;    // bits below the digits found
        const int shift = pass == 1 ? 10 : 0;
        const uint32_t mask = pass == 1 ? 0x7FFu : 0x3FFu;
        if (pass >= 2 && sh.list_size <= kListed) {
            for (int j = threadIdx.x; j < static_cast<int>(sh.list_size); j += kThreads) {
                const uint32_t key = sh.listed[j];
                const int slot = sh.listed_slot[j];
                if (pass == 2) {
                    if ((key >> skip) == prefix)
                        atomicAdd(&hist[key & mask], 1u);
                } else if (key >= prefix) {
                    atomicOr(reinterpret_cast<uint32_t *>(masks) + slot / 16,
                             1u << (slot / 4 % 4 * 8 + (key > prefix ? 0 : 4) + slot % 4));
                }
            }
        } else if (pass > 0) {
            // what the first digit decides goes to the masks and the rest to the list; without a
            // whole list the masks are made at the end
            const uint32_t least = max(prefix << skip, 1u);   // of the keys that begin with them
            const uint32_t most = prefix << skip | ((1u << skip) - 1u);
            sweep(a.cached, [&](int i, const uint4 k) {
                const uint32_t ks[4] = {k.x, k.y, k.z, k.w};
                uint32_t over = 0, in = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    over |= ks[e] > most ? 1u << e : 0u;
                    in |= ks[e] >= least ? 1u << e : 0u;
                }
                in &= ~over;
                if (pass != 2)
                    masks[(i - cta_lo) / 4] = static_cast<uint8_t>(pass == 3 ? over | in << 4 : over);
                if (pass == 3 || in == 0)
                    return;
                uint32_t at = pass == 1 ? atomicAdd(&sh.list_size, static_cast<uint32_t>(__popc(in)))
                                        : static_cast<uint32_t>(kListed);
                for (; in; in &= in - 1, ++at) {
                    const int e = __ffs(in) - 1;
                    const uint32_t key = e < 2 ? e == 0 ? k.x : k.y : e == 2 ? k.z : k.w;
                    atomicAdd(&hist[(key >> shift) & mask], 1u);
                    if (at < kListed) {
                        sh.listed[at] = key;
                        sh.listed_slot[at] = i + e - cta_lo;
                    }
                }
            });
        }
        if (pass == 3)
            break;
        // Every CTA gives away the sums of eight bins each, top first; only the thread whose eight
        // bins hold the wanted key reads these bins of every CTA (all bins of all CTAs would be 64 KB
        // through distributed shared memory).
        __syncthreads();
        const int top_bin = kBins - 1 - 8 * static_cast<int>(threadIdx.x);
        {
            const uint4 *h = reinterpret_cast<const uint4 *>(&hist[top_bin - 7]);
            const uint4 x = h[0], y = h[1];
            sh.coarse[pass & 1][threadIdx.x] = x.x + x.y + x.z + x.w + y.x + y.y + y.z + y.w;
        }
        cluster_sync();
        uint32_t mine = 0;
#pragma unroll
        for (int c = 0; c < kMaxCtas; ++c)
            if (c < ctas)
                mine += *cluster.map_shared_rank(&sh.coarse[pass & 1][threadIdx.x], c);
        const uint32_t incl = warp_scan(mine, lane);
        if (lane == 31)
            sh.warp_sum[0][warp] = incl;
        __syncthreads();
        uint32_t before = incl - mine;
#pragma unroll
        for (int v = 0; v < kWarps; ++v)
            before += v < warp ? sh.warp_sum[0][v] : 0u;
        if (before < need && need <= before + mine) {
            uint32_t c8[8] = {};
#pragma unroll
            for (int c = 0; c < kMaxCtas; ++c)
                if (c < ctas) {
                    const uint4 *h = reinterpret_cast<const uint4 *>(
                        cluster.map_shared_rank(&hist[top_bin - 7], c));
                    const uint4 x = h[0], y = h[1];
                    c8[0] += y.w;
                    c8[1] += y.z;
                    c8[2] += y.y;
                    c8[3] += y.x;
                    c8[4] += x.w;
                    c8[5] += x.z;
                    c8[6] += x.y;
                    c8[7] += x.x;
                }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (before < need && need <= before + c8[e]) {
                    sh.digit = top_bin - e;
                    sh.above = before;
                    sh.equal = c8[e];
                }
                before += c8[e];
            }
        }
        if (pass == 1)   // past this barrier every CTA has read the first pass's bins: free again
            for (int i = threadIdx.x; i < kBins; i += kThreads)
                sh.hist[0][i] = 0;
        __syncthreads();
        prefix = (prefix << (pass == 2 ? 10 : 11)) | sh.digit;
        need -= sh.above;
        equal = sh.equal;
    }
    __syncthreads();   // the masks
    // Calls f(i, above, equal) for the warp's steps in order: slots i .. i + 3 above the threshold
    // and equal to it, as four bits each.
    auto visit = [&](auto &&f) {
#pragma unroll 1
        for (int i0 = lo; i0 < hi; i0 += kWarpSlots) {
            const uint32_t m = masks[(i0 - cta_lo) / 4 + lane];
            f(i0 + 4 * lane, m & 15u, m >> 4);
        }
    };
    // Where only some of the keys equal to the threshold stay, these take their ranks in slot order.
    const bool ties = need < equal;
    uint32_t eq_first = 0;   // equal keys before this warp's
    if (ties) {
        uint32_t here = 0;
        visit([&](int, uint32_t, uint32_t eq) { here += __popc(eq); });
        here = __reduce_add_sync(0xffffffffu, here);
        if (lane == 0)
            sh.warp_sum[1][warp] = here;
        __syncthreads();
        uint32_t all = 0;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) {
            eq_first += v < warp ? sh.warp_sum[1][v] : 0u;
            all += sh.warp_sum[1][v];
        }
        if (threadIdx.x == 0)
            sh.equal_here = all;
        cluster_sync();
        for (int c = 0; c < cta; ++c)
            eq_first += *cluster.map_shared_rank(&sh.equal_here, c);
    }
    // The kept ones of four slots as four bits; the warp goes together.
    auto kept = [&](uint32_t gt, uint32_t eq, uint32_t &eq_rank) -> uint32_t {
        if (!ties)
            return gt | eq;
        const uint32_t cnt = __popc(eq);
        const uint32_t incl = warp_scan(cnt, lane);
        uint32_t rank = eq_rank + incl - cnt;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if ((eq >> e) & 1u) {
                gt |= (rank < need ? 1u : 0u) << e;
                ++rank;
            }
        eq_rank += __shfl_sync(0xffffffffu, incl, 31);
        return gt;
    };
    auto below_n = [&](int i) -> uint32_t {   // the slots of i .. i + 3 below n, as four bits
        const int b = n - i;
        return b >= 4 ? 15u : b <= 0 ? 0u : (1u << b) - 1u;
    };
    {
        uint32_t rank = eq_first, gaps = 0, tails = 0;
        visit([&](int i, uint32_t gt, uint32_t eq) {
            const uint32_t m = kept(gt, eq, rank), in = below_n(i);
            gaps += __popc(in & ~m);
            tails += __popc(m & ~in);
        });
        gaps = __reduce_add_sync(0xffffffffu, gaps);
        tails = __reduce_add_sync(0xffffffffu, tails);
        __syncthreads();   // warp_sum is read
        if (lane == 0) {
            sh.warp_sum[0][warp] = gaps;
            sh.warp_sum[1][warp] = tails;
        }
    }
    __syncthreads();
    uint32_t gap_at = 0, tail_at = 0, moves = 0;
    {
        uint32_t gaps = 0, tails = 0;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) {
            gap_at += v < warp ? sh.warp_sum[0][v] : 0u;
            tail_at += v < warp ? sh.warp_sum[1][v] : 0u;
            gaps += sh.warp_sum[0][v];
            tails += sh.warp_sum[1][v];
        }
        if (threadIdx.x == 0) {
            sh.gaps = gaps;
            sh.tails = tails;
        }
    }
    cluster_sync();
    for (int c = 0; c < ctas; ++c) {
        const uint32_t g = *cluster.map_shared_rank(&sh.gaps, c);
        const uint32_t t = *cluster.map_shared_rank(&sh.tails, c);
        gap_at += c < cta ? g : 0u;
        tail_at += c < cta ? t : 0u;
        moves += g;
    }
    int32_t *dst_list = a.lists + static_cast<size_t>(unit) * 2 * a.list_cap;
    int32_t *src_list = dst_list + a.list_cap;
    if (cta == 0 && threadIdx.x == 0)
        a.counts[unit] = make_int2(min(static_cast<int>(moves), a.list_cap), free_pos);
    {
        uint32_t rank = eq_first;
        visit([&](int i, uint32_t gt, uint32_t eq) {
            const uint32_t m = kept(gt, eq, rank), in = below_n(i);
            uint32_t g = in & ~m, t = m & ~in;
            const uint32_t both = __popc(g) | (__popc(t) << 16);
            const uint32_t incl = warp_scan(both, lane);
            const uint32_t at = incl - both, all = __shfl_sync(0xffffffffu, incl, 31);
            // (both ranks are below list_cap unless the weights changed under the launch)
            uint32_t d = gap_at + (at & 0xFFFFu), f = tail_at + (at >> 16);
            for (; g; g &= g - 1, ++d)
                if (d < static_cast<uint32_t>(a.list_cap))
                    dst_list[d] = i + __ffs(g) - 1;
            for (; t; t &= t - 1, ++f)
                if (f < static_cast<uint32_t>(a.list_cap))
                    src_list[f] = i + __ffs(t) - 1;
            gap_at += all & 0xFFFFu;
            tail_at += all >> 16;
            // in place the kept slots behind n are read by the moves first
            if (!(w_apart && p_apart))
                for (int e = 0; e < 4; ++e)
                    if (i + e < hi && !(((m | in) >> e) & 1u)) {
                        w_out[i + e] = 0.0f;
                        p_out[i + e] = free_pos + i + e;
                    }
        });
    }
    for (long long i = static_cast<long long>(N) + cta * kThreads + threadIdx.x; i < a.stride;
         i += ctas * kThreads)
        p_out[i] = free_pos + static_cast<int32_t>(i);
    cluster_sync();   // the others' counts are read: shared memory may go; the lists are written
    if (a.inline_moves) {
        const int n_moves = min(static_cast<int>(moves), a.list_cap);
        for (int j0 = warp * kWarpMoves; j0 < n_moves; j0 += kWarps * kWarpMoves)
            move_rows<D>(a, unit, j0, min(kWarpMoves, n_moves - j0), free_pos);
    }
}

// CTA = (chunk of kMovesPerCta moves, unit), unit fastest, and as many chunks on as the grid has.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const Args a, int units)
{
    pdl_wait();
    pdl_trigger();
    const int unit = blockIdx.x % units;
    const int2 count = __ldcg(a.counts + unit);
    // (the grid's chunks are counted where they are needed: before the loop, 61 us instead of 57.6)
    for (int j0 = (blockIdx.x / units) * kMovesPerCta + (threadIdx.x >> 5) * kWarpMoves;
         j0 < count.x; j0 += gridDim.x / units * kMovesPerCta)
        move_rows<D>(a, unit, j0, min(kWarpMoves, count.x - j0), count.y);
}

cudaError_t launch_t(const EvictLaunch &l, const Args &args, cudaStream_t stream)
{
    Args a = args;
    const long long units = static_cast<long long>(l.num_seqs) * l.kv_heads;
    // Clusters only where (sequence, kv head) units alone leave SMs idle and rows are long
    // enough to share: a cluster barrier costs more than a CTA's.
    int ctas = 1;
    while (ctas < kMaxCtas && (l.max_ctx > ctas * kEvictCtaSlots ||
                               (units * ctas * 2 <= 4LL * current_sm_count() &&
                                l.max_ctx / (ctas * 2) >= 1024)))
        ctas *= 2;
    const long long step = static_cast<long long>(kWarpSlots) * kWarps;
    const long long per_cta = (l.max_ctx + step * ctas - 1) / (step * ctas) * step;
    // As many keys in shared memory as leave every CTA of the launch room beside the others (the
    // SM's threads and registers hold 4): on 64 rows of up to 131,072 slots all keys in shared
    // memory mean two waves of clusters.
    const int sms = current_sm_count();
    const long long per_sm = std::min<long long>(4, (units * ctas + sms - 1) / sms);
    const long long rest = static_cast<long long>(sizeof(Shared)) + per_cta / 4;
    const long long room =
        std::max(0LL, kSmemPerSm / per_sm - 1024 - rest) / 4 / kWarpSlots * kWarpSlots;
    a.cached = static_cast<int>(std::min(per_cta, room));
    const size_t smem = static_cast<size_t>(a.cached) * 4 + rest;
    // Few moves a row are made by the row's own CTA, unless the selection's CTAs come in several
    // rounds: 64 sequences (8 kv heads) of 300 slots cut to 256 take 13.3 us against 18.3 with a second
    // launch, of 512 cut to 400 16.4 against 22.6, of 4,096 cut to 3,840 44.0 against 48.5; with 512
    // cut to 256 it is 24.6 against 23.8, with 1,024 cut to 512 43.7 against 40.9, and on 256 sequences
    // of 512 cut to 448 69.6 against 62.4.
    a.inline_moves = ctas == 1 && l.list_cap <= kInlineMoves && units <= 1LL * kInlineUnits * sms;
    auto select = l.head_dim == 128 ? select_kernel<128> : select_kernel<64>;
    auto move = l.head_dim == 128 ? move_kernel<128> : move_kernel<64>;
    cudaError_t err =
        cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemPerCta));
    if (err != cudaSuccess)
        return err;
    const long long chunks =
        std::min((l.list_cap + kMovesPerCta - 1LL) / kMovesPerCta,
                 std::max(1LL, static_cast<long long>(kMoveCtas) * sms / units));
    if (units * ctas > 0x7FFFFFFFLL || units * chunks > 0x7FFFFFFFLL)
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
    err = cudaLaunchKernelEx(&cfg, select, a);
    if (err != cudaSuccess || l.list_cap == 0 || a.inline_moves)
        return err;
    return launch_pdl(move, dim3(static_cast<unsigned>(units * chunks)), dim3(kMoveThreads), 0,
                      stream, a, static_cast<int>(units));
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
    a.lists = l.lists;
    a.counts = reinterpret_cast<int2 *>(l.counts);
    a.list_cap = l.list_cap;
    a.kv_heads = l.kv_heads;
    a.log2_page = l.page_size == 16 ? 4 : l.page_size == 32 ? 5 : 6;
    a.num_pages = l.num_pages;
    a.hnd = l.hnd ? 1 : 0;
    const uintptr_t rows = reinterpret_cast<uintptr_t>(l.weights) |
                           reinterpret_cast<uintptr_t>(l.positions) |
                           reinterpret_cast<uintptr_t>(l.weights_out) |
                           reinterpret_cast<uintptr_t>(l.positions_out);
    a.vec = (rows & 15) == 0 && l.stride % 4 == 0;
    a.err = current_error_word();
    return launch_t(l, a, stream);
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
