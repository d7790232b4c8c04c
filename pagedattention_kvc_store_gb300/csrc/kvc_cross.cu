// kvc_cross.cu -- attention of queries to the states of a source of another length, no causal limit, on the
// 5th-generation tensor cores (tcgen05, accumulators in tensor memory).
//
//   out[t][h] = sum_p softmax_p(q[t][h] . K[p][h / G] * scale) V[p][h / G],   p < source_lens[s],
// for the tokens t of q_indptr[s] .. q_indptr[s + 1] - 1, the source's pages read in place.
//
// Tiling: the rows of one (source, kv head) are its (token, query head of the group) pairs, token-major, in
// tiles of 128 (the tcgen05 M).  A work item is a pair of consecutive tiles over one chunk of the source's
// positions (the whole source where there is one split); both tiles see the same pages, so every K or V
// stage feeds two products.  One CTA per SM goes on from item to item, its roles running ahead across them:
//   warps 0, 2  TMA, K and V: 128-position stages in one ring in the order K(0), K(1), V(0), K(2), V(1), ...; a
//               box per page, issued by parallel lanes, that lands as [8 positions][column half][8 rows]
//               [128 bytes, swizzled], so that a stage is one operand whatever the page size (a box per page and
//               half took twice as many, and 16-position pages 37% more time).  A warp issues a box in some
//               150 cycles: one for both K and V held 16-position pages back (prompts over them 766 us, with
//               two 670)
//   warp 1      allocates TMEM (512 columns) and issues S = Q_w K(b)^T (M 128, N 128, K head_dim) of the tiles w
//               into score slots in turn (two at head dim 128, three at 64) and O_w += P V(b) (N head_dim, K 128,
//               P from the slot); the next S into a slot right behind the product that reads P from it
//   warp 3      the items (cancels blocks of the grid that have not started and hands theirs round), and
//               their query tiles
//   warps 4-11  softmax of tile 0, warps 12-19 of tile 1, 16 rows each: the running maximum (O rescaled only when
//               p of the maximum before add up to more than 2^8) and sum, P as bf16 over S's columns, and O / l
//               at the end
// An item of a single tile puts its blocks in turn on the O of both tiles, so that the softmax of one runs
// beside the products of the other as it does with two tiles, and joins the two at the end.
// 64 sources of 2,048 positions x 512 queries, 32 / 8 heads: 735 us at head dim 128 (1,495 TFLOP/s, 79% of the
// burst rate of a library product), 550 at 64.  Bound by a tile's chain at 128: scores 512 cycles, softmax some
// 1,600 (its loads from TMEM 150, 900-1,100 for the exponentials, vote and hand-over 500), products 512; the
// other tile's products fit into that, the two exposed ends do not.  At 64 not established: the softmax warps issue
// in 58% of their slots, the exponential unit is busy 39%.
// Few rows and many positions: the positions are cut into chunks (splits), partial rows and their
// log-sum-exps go to the workspace and cross_merge_kernel joins them.
// Sums: P is rounded to bf16 for the product (2^-8 of each, the same the append makes), l sums the unrounded
// values in fp32, which the log-sum-exp needs; summing the rounded ones besides took 128 more steps a row.
#include <math.h>

#include "kvc_device.cuh"
#include "kvc_launch.h"

namespace kvc {

namespace {

__device__ uint32_t g_cross_errors;

constexpr int kM = 128;           // rows per tile
constexpr int kBN = kCrossBlock;  // positions per K or V stage (the N of S = Q K^T)
constexpr int kRoleWarps = 4;     // K loads, MMA issue, V loads, items and queries
constexpr int kSoftmaxWarps = 16; // eight for each tile
constexpr int kThreads = (kRoleWarps + kSoftmaxWarps) * 32;
constexpr int kMaxStages = 8;
constexpr int kMaxOrdered = 256;  // sources whose items are ordered
// Registers a thread: the launch's, and after the role warps gave theirs to the softmax warps.  128 * 64 +
// 512 * 104 is 640 * 96: what the block was launched with.
constexpr int kLaunchRegs = 96, kRoleRegs = 64, kSoftmaxRegs = 104;
static_assert(kRoleWarps * kRoleRegs + kSoftmaxWarps * kSoftmaxRegs <=
                  (kRoleWarps + kSoftmaxWarps) * kLaunchRegs, "registers of the launch");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleSum = 256.0f;   // of the p of a thread's 32 columns of a row
// Waits for work are as long as a CTA's items: they may take two seconds and one more for every 2^21 positions of a
// chunk (16,384 blocks, some 30 ms of work).
constexpr int kPatienceLog2 = 21;

template <int D>
struct Geom {
    static constexpr int kHalves = D / 64;
    static constexpr int kQBytes = kHalves * kM * 128;       // one query tile
    static constexpr int kStageBytes = kHalves * kBN * 128;  // K or V of 128 positions
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kOffStages = 2 * kQBytes;           // Q: [tile]
    static constexpr int kOffExchange = kOffStages + kStages * kStageBytes;   // [m, l][tile][row] floats
    static constexpr int kOffBar = kOffExchange + 4 * kM * 4;
    static constexpr int kOffItem = kOffBar + 384;           // after the barriers: the item, an answer
    static constexpr int kOffAnswer = kOffItem + 64;
    static constexpr int kOffOrder = kOffBar + 512;          // sources, the longest first
    static constexpr size_t kSmemBytes = kOffOrder + 2 * kMaxOrdered;   // base is 1024-aligned
    // TMEM: O of tile w at w * D, then as many slots of 128 columns as fit, for the scores of a tile and block
    // each; P, two positions a column, overwrites S's first 64, and S's columns 64 .. 127 stay for a second look.
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kColS = 2 * D;
    static constexpr int kSlots = (kTmemCols - kColS) / kBN;
    static_assert(kSlots == 2 || kSlots == 3, "score slots");
    static_assert(kStages <= kMaxStages, "ring barriers");
    static_assert(kSmemBytes <= 232448, "shared memory");
};

struct Args {
    void *out;
    int out_f32;
    float *lse;                 // [T][q_heads] or null (one split)
    float *part_o, *part_lse;   // [T][q_heads][n_split][D], [T][q_heads][n_split] (more than one)
    const int32_t *block_table;
    int bt_stride;
    const int32_t *q_indptr, *source_lens;
    int kv_heads, q_heads, group, page_size, pairs_per_seq;
    int num_tokens, max_q_len, max_src, chunk, n_split;
    float scale_log2;
    int ordered;   // sources whose items go by their lengths, the longest first; 0: as they come
    int hnd;   // HND pools: half boxes addressed by (offset, page * kv_heads + kv head)
    uint32_t *err;
};

enum BarIndex : int {
    kBarKvFull = 0,                         // [ring slot]
    kBarKvEmpty = kBarKvFull + kMaxStages,  // [ring slot], one MMA commit
    kBarQFull = kBarKvEmpty + kMaxStages,   // [tile]
    kBarQEmpty = kBarQFull + 2,             // [tile], one MMA commit after its last S product
    kBarSFull = kBarQEmpty + 2,             // [tile][its blocks in turn]
    kBarPFull = kBarSFull + 4,              // [tile][its blocks in turn], an arrival of each of its eight warps
    kBarPvDone = kBarPFull + 4,             // [tile][its blocks in turn]; with two slots [tile][0], once per item
    kBarDrain = kBarPvDone + 4,
    kBarItemFull = kBarDrain + 1,           // the item in shared memory is the next one
    kBarItemEmpty = kBarItemFull + 1,       // an arrival of every warp that reads items
    kBarCancel = kBarItemEmpty + 1,         // the answer to a request for a block that has not started
    kBarBoth = kBarCancel + 1,              // the softmax warps of both tiles meet, an arrival of each
    kBarCount = kBarBoth + 1
};
constexpr int kItemReaders = 3 + kSoftmaxWarps;

// Tiles 2 tp and 2 tp + 1 of one (source, kv head) over positions key0 .. key0 + n_keys - 1.
struct __align__(16) Item {
    int s, kvh, split, tok0;
    int rows, row_begin;         // row_begin: first row of tile 2 tp
    int key0, n_keys, n_blocks;  // n_keys 0: nothing to attend to, rows are written all the same
    int has_b;                   // tile 2 tp + 1 exists
    int dual;                    // it does not: the blocks in turn on both halves of TMEM, joined at the end
    int done;                    // no item: the last one was

    // Its units (a tile and a block each, the tile of unit u being u & 1 where there is more than one).  All
    // units of a CTA take the score slots in turn.
    __device__ __forceinline__ int units() const
    {
        return has_b ? 2 * n_blocks : n_blocks;
    }
};

// Item `it` from its source's lengths; false where it has no rows.
__device__ __forceinline__ bool make_item(const Args &a, int it, const uint16_t *order, Item &x,
                                          uint32_t *err)
{
    const int tp = it % a.pairs_per_seq;
    int rest = it / a.pairs_per_seq;
    x.kvh = rest % a.kv_heads;
    rest /= a.kv_heads;
    x.split = rest % a.n_split;
    x.s = rest / a.n_split;
    if (a.ordered > 0)
        x.s = order[x.s];
    x.tok0 = a.q_indptr[x.s];
    bool in_range;
    const int n_tok = source_tokens(x.tok0, a.q_indptr[x.s + 1], a.num_tokens, in_range);
    const int given = a.source_lens[x.s], most = min(a.max_src, a.bt_stride * a.page_size);
    if (given > most || n_tok > a.max_q_len || !in_range)
        atomicOr(err, kErrContextRange);
    const int len = min(max(given, 0), most);   // a negative length is none
    x.rows = min(n_tok, a.max_q_len) * a.group;
    x.row_begin = tp * 2 * kM;
    if (x.row_begin >= x.rows)
        return false;
    x.has_b = x.row_begin + kM < x.rows;
    x.key0 = x.split * a.chunk;
    x.n_keys = min(max(len - x.key0, 0), a.chunk);
    x.n_blocks = (x.n_keys + kBN - 1) / kBN;
    x.dual = !x.has_b && x.n_blocks > 1;
    x.done = 0;
    return true;
}

// A role's view of the items: each is read from shared memory by every warp that works on it.
struct Feed {
    Item x;
    int n = 0;   // items read
    int patience;
    volatile uint32_t *gave_up;
    __device__ __forceinline__ Feed(int times, volatile uint32_t *word) : patience(times), gave_up(word) {}
    __device__ __forceinline__ void read(const Item *slot)
    {
        const int4 *from = reinterpret_cast<const int4 *>(slot);
        int4 *to = reinterpret_cast<int4 *>(&x);
        static_assert(sizeof(Item) == 48, "three words of 16 bytes");
        to[0] = from[0];
        to[1] = from[1];
        to[2] = from[2];
        ++n;
    }
    // Waits for the next item, by a whole warp; false (and ok) if the wait ran out.
    __device__ __forceinline__ bool get(uint64_t *bars, const Item *slot, bool &ok)
    {
        if (!__all_sync(0xffffffffu, mbar_wait_work(&bars[kBarItemFull], n & 1, patience, gave_up))) {
            ok = false;
            return false;
        }
        read(slot);
        return true;
    }
    // And acknowledges it.  False at the end too.
    __device__ __forceinline__ bool next(uint64_t *bars, const Item *slot, bool &ok)
    {
        if (!get(bars, slot, ok))
            return false;
        has_read(bars);
        return !x.done;
    }
    __device__ __forceinline__ void has_read(uint64_t *bars)
    {
        __syncwarp();
        if ((threadIdx.x & 31) == 0)
            mbar_arrive(&bars[kBarItemEmpty]);
    }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    cross_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                 const __grid_constant__ CUtensorMap tmap_v, const Args a)
{
    pdl_wait();
    pdl_trigger();
    uint32_t *const err_word = a.err ? a.err : &g_cross_errors;
    using G_ = Geom<D>;
    constexpr int kHalves = D / 64;
    constexpr int kStages = G_::kStages;

    // The swizzled tiles need a 1024-byte-aligned base, which is checked rather than padded for.
    extern __shared__ __align__(1024) uint8_t smem[];
    if ((smem_addr(smem) & 1023u) != 0) {
        if (threadIdx.x == 0)
            atomicOr(err_word, kErrSmemAlign);
        return;
    }
    uint8_t *sStages = smem + G_::kOffStages;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + G_::kOffBar);
    static_assert(kBarCount * 8 + 8 <= 384, "barriers");
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kBarCount);
    // A wait that ran out: the other waits for work end too, and the rest of the grid's items are let go.
    volatile uint32_t *gave_up = tmem_slot + 1;
    const int patience = 2 + (a.chunk >> kPatienceLog2);
    Item *item = reinterpret_cast<Item *>(smem + G_::kOffItem);
    uint16_t *order = reinterpret_cast<uint16_t *>(smem + G_::kOffOrder);
    auto q_tile = [&](int tile) { return smem + tile * G_::kQBytes; };

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int G = a.group;
    const int P = a.page_size;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kBarCount; ++i)
            mbar_init(&bars[i], (i >= kBarPFull && i < kBarPvDone) ? 8u
                                : i == kBarItemEmpty               ? static_cast<uint32_t>(kItemReaders)
                                : i == kBarBoth                    ? static_cast<uint32_t>(kSoftmaxWarps)
                                                                   : 1u);
        fence_mbar_init();
        *gave_up = 0;
    }
    if (warp == 1)
        tmem_alloc(tmem_slot, G_::kTmemCols);
    if (a.ordered > 0) {
        // The SMs end together if the longest items come first.  64 classes by length, the longest first, and
        // sources as they come in each: a counting sort, [class][warp of sources] counts in shared memory.
        int *counts = reinterpret_cast<int *>(smem + G_::kOffExchange);
        constexpr int kWarps = kMaxOrdered / 32, kClasses = 4 * kM / kWarps;
        const int i = threadIdx.x;
        if (i < kClasses * kWarps)
            counts[i] = 0;
        int cls = 0, ahead = 0;
        __syncthreads();
        if (warp < kWarps) {
            const int len = i < a.ordered ? min(max(a.source_lens[i], 0), a.max_src) : 0;
            cls = kClasses - 1 - static_cast<int>(static_cast<long long>(len) * kClasses / (a.max_src + 1LL));
            const uint32_t same = __match_any_sync(0xffffffffu, i < a.ordered ? cls : -1 - cls);
            ahead = __popc(same & ((1u << lane) - 1));
            if (ahead == 0 && i < a.ordered)
                counts[cls * kWarps + warp] = __popc(same);
        }
        __syncthreads();
        if (warp == 0) {
            constexpr int kEach = kClasses * kWarps / 32;
            int sum = 0, c[kEach];
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                c[j] = counts[lane * kEach + j];
                sum += c[j];
            }
            int upto = sum;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int other = __shfl_up_sync(0xffffffffu, upto, d);
                upto += lane >= d ? other : 0;
            }
            upto -= sum;
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                counts[lane * kEach + j] = upto;
                upto += c[j];
            }
        }
        __syncthreads();
        if (i < a.ordered)
            order[counts[cls * kWarps + warp] + ahead] = static_cast<uint16_t>(i);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;

    if (warp < kRoleWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRoleRegs));
    if (warp == 0 || warp == 2) {
        // ------------------------------ K loads (warp 0), V loads (warp 2) -----------------
        const bool is_k = warp == 0;
        const CUtensorMap *map = is_k ? &tmap_k : &tmap_v;
        if (lane == 0)
            prefetch_tensormap(map);
        // K and V that several tile pairs read stay in L2 like anything else (64 sources of 512 to 4,096
        // positions x 200-400 queries with the L2 cold: 644 us, marked to leave first 669 and 1.7 GB from
        // memory instead of 0.9, marked to leave last 644); what is read once leaves first
        const uint64_t policy = a.pairs_per_seq > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
        Feed w(patience, gave_up);
        int n0 = 0;          // ring index of the item's first slot
        int begun = 0;       // ring index behind the last slot that this warp filled
        for (; w.next(bars, item, ok); n0 += 2 * w.x.n_blocks) {
            const Item &x = w.x;
            if (!ok)
                continue;   // a wait ran out: the rest of the items are only taken note of
            const int32_t *bt_row =
                a.block_table + static_cast<size_t>(x.s) * a.bt_stride + x.key0 / P;
            const int n_pages = (x.n_keys + P - 1) / P;
            int cached_base = 0;
            int cached_page = lane < n_pages ? bt_row[lane] : 0;
            const int nb = x.n_blocks;
            for (int b = 0; b < nb; ++b) {
                const int n = n0 + (is_k ? (b == 0 ? 0 : 2 * b - 1) : (b == nb - 1 ? 2 * nb - 1 : 2 * b + 2));
                const int np = (min(kBN, x.n_keys - b * kBN) + P - 1) / P;
                const int st = n % kStages;
                const int lp0 = b * kBN / P;   // first page of the block
                if (lp0 + np > cached_base + 32) {
                    cached_base = lp0;
                    cached_page = (lp0 + lane < n_pages) ? bt_row[lp0 + lane] : 0;
                }
                // lane i issues the box of page i; NHD maps end in {group, kv head}, HND maps in {group of
                // the block, block}
                const int page =
                    __shfl_sync(0xffffffffu, cached_page, (lp0 - cached_base + lane) & 31);
                uint8_t *dst = sStages + st * G_::kStageBytes + lane * P * (D * 2);
                if (n >= kStages && !__all_sync(0xffffffffu, mbar_wait(&bars[kBarKvEmpty + st],
                                                                       ((n / kStages) - 1) & 1))) {
                    ok = false;
                    break;
                }
                if (lane == 0)
                    mbar_arrive_expect_tx(&bars[kBarKvFull + st], static_cast<uint32_t>(np * P * D * 2));
                __syncwarp();
                if (lane < np)
                    tma_load_5d_hint(dst, map, 0, 0, 0, a.hnd ? 0 : page * (P / 8),
                                     a.hnd ? page * a.kv_heads + x.kvh : x.kvh, &bars[kBarKvFull + st],
                                     policy);
                begun = n + 1;
            }
            if (!ok)
                *gave_up = 1;
        }
        if (!ok && lane == 0) {
            atomicOr(err_word, kErrCrossWait);
            // let every copy in flight land before the CTA can exit: the slots of the other warp too
            for (int m = max(0, begun - kStages); m < begun; ++m)
                if (!mbar_wait(&bars[kBarKvFull + m % kStages], (m / kStages) & 1))
                    atomicOr(err_word, kErrDrainWait);
        }
    } else if (warp == 1) {
        // ------------------------------ MMA issue ----------------------------------------
        // What lies between P and the products that wait for it are this warp's own steps, and registers that
        // spill there cost more than the steps: the whole warp goes through them, so that what they are made of
        // lives in uniform registers (one thread alone took 1,800 cycles for the products of 128 positions of
        // two tiles), ring positions are carried along, and waits are one instruction sequence each without a
        // branch on their result.  A wait that runs out makes the others go through at once, up to the item's end.
        const bool leader = elect_one();
        constexpr uint32_t kIdescPV = umma_idesc_bf16(kM, D, 1), kIdescQK = umma_idesc_bf16(kM, kBN, 0);
        constexpr uint32_t kStageLo = G_::kStageBytes / 16;
        constexpr uint64_t kHighQ = umma_desc_sw128_high(1024), kHighKv = umma_desc_sw128_high(kHalves * 1024);
        const uint32_t ring_k = umma_desc_sw128_low(smem_addr(sStages), 16);
        const uint32_t ring_v = umma_desc_sw128_low(smem_addr(sStages), 1024);
        const uint32_t q_low = umma_desc_sw128_low(smem_addr(smem), 16);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        uint32_t failed = 0;
        auto wait = [&](int bar, uint32_t parity) { mbar_wait_plain(&bars[bar], parity, failed); };
        // S = Q_q K^T into a score slot, K at a stage
        auto issue_qk = [&](int slot, int q, int stage, uint32_t idesc) {
            uint32_t low = q_low + q * (G_::kQBytes / 16), k_low = ring_k + stage * kStageLo;
            asm volatile("" : "+r"(low));   // or all of Q's descriptors are kept in registers, and spill
            const uint32_t d = tm + G_::kColS + slot * kBN;
            if (leader) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    umma_bf16_ss(d, kHighQ | (low + (k >> 2) * (kM * 128 / 16) + (k & 3) * 2),
                                 kHighKv | (k_low + (k >> 2) * (1024 / 16) + (k & 3) * 2), idesc, k > 0 ? 1u : 0u);
            }
        };
        constexpr int kStep = 2 * kHalves * 1024 / 16;   // 16 positions of V
        // O_t (+)= P V over the first 16 k_steps positions of a block
        auto issue_pv = [&](int t, int slot, int stage, int k_steps, uint32_t keep) {
            const uint32_t d = tm + t * D, p = tm + G_::kColS + slot * kBN, v_low = ring_v + stage * kStageLo;
            if (k_steps == kBN / 16) {
                if (leader) {
#pragma unroll
                    for (int k = 0; k < kBN / 16; ++k)
                        umma_bf16_ts(d, p + k * 8, kHighKv | (v_low + k * kStep), kIdescPV,
                                     k > 0 ? 1u : keep);
                }
            } else if (leader) {
                for (int k = 0; k < k_steps; ++k)
                    umma_bf16_ts(d, p + k * 8, kHighKv | (v_low + k * kStep), kIdescPV,
                                 k > 0 ? 1u : keep);
            }
        };
        auto commit = [&](int bar) {
            if (leader)
                umma_commit(&bars[bar]);
        };
        Feed w(patience, gave_up);
        int s_slot = 0, p_slot = 0;   // score slots of the next unit's S and of the next unit's P
        uint32_t s_count[2] = {0, 0}, p_count[2] = {0, 0};   // the tiles' S products and P so far
        uint32_t q_count[2] = {0, 0};                        // and their items
        int kst = 0;        // ring stage of the current K, in the producers' order K(0), K(1), V(0), ...
        uint32_t kph = 0;   // and its phase
        auto advance = [](int &stage, uint32_t &phase, int n) {
            stage += n;
            if (stage >= kStages) {
                stage -= kStages;
                phase ^= 1;
            }
        };
        auto next_slot = [](int slot) { return slot + 1 == G_::kSlots ? 0 : slot + 1; };
        while (w.next(bars, item, ok)) {
            const int nb = __shfl_sync(0xffffffffu, w.x.n_blocks, 0);
            const int two = __shfl_sync(0xffffffffu, w.x.has_b, 0);
            const int dual = __shfl_sync(0xffffffffu, w.x.dual, 0);
            const int last_cols = (__shfl_sync(0xffffffffu, w.x.n_keys, 0) - (nb - 1) * kBN + 15) & ~15;
            if (!ok || nb == 0)
                continue;
            const uint32_t idesc_last = umma_idesc_bf16(kM, last_cols, 0);
            int vst = kst;
            uint32_t vph = kph;
            advance(vst, vph, nb == 1 ? 1 : 2);
            // S of tile t's block b (K at the current stage) into the next slot
            auto scores = [&](int t, int q, int b) {
                tc_fence_after_sync();
                issue_qk(s_slot, q, kst, b + 1 == nb ? idesc_last : kIdescQK);
                commit(kBarSFull + 2 * t + (s_count[t] & 1));
                if (b + 1 == nb)
                    commit(kBarQEmpty + q);
                ++s_count[t];
                s_slot = next_slot(s_slot);
            };
            // PV of tile t's block b (V at the current stage) once its P is there
            auto products = [&](int t, int b, bool first) {
                wait(kBarPFull + 2 * t + (p_count[t] & 1), (p_count[t] >> 1) & 1);
                tc_fence_after_sync();
                issue_pv(t, p_slot, vst, b + 1 == nb ? last_cols / 16 : kBN / 16, first ? 0u : 1u);
                if (G_::kSlots > 2)
                    commit(kBarPvDone + 2 * t + (p_count[t] & 1));
                else if (b + (dual ? 2 : 1) >= nb)
                    commit(kBarPvDone + 2 * t);
                ++p_count[t];
                p_slot = next_slot(p_slot);
            };
            auto next_k = [&](int b) {   // from K(b - 1) to K(b)
                advance(kst, kph, b == 1 ? 1 : 2);
                wait(kBarKvFull + kst, kph);
            };
            wait(kBarQFull, q_count[0] & 1);
            wait(kBarKvFull + kst, kph);
            if (dual) {
                // block b is a unit of tile b % 2, in the order S(0) .. S(kSlots - 1), PV(0), S(kSlots), PV(1), ...
                for (int b = -G_::kSlots; b < nb; ++b) {
                    if (b >= 0) {
                        wait(kBarKvFull + vst, vph);
                        if (b & 1)
                            products(1, b, b < 2);
                        else
                            products(0, b, b < 2);
                        commit(kBarKvEmpty + vst);
                        advance(vst, vph, b + 2 >= nb ? 1 : 2);
                    }
                    const int next = b + G_::kSlots;
                    if (next < nb) {
                        if (next > 0)
                            next_k(next);
                        if (next & 1)
                            scores(1, 0, next);
                        else
                            scores(0, 0, next);
                        commit(kBarKvEmpty + kst);
                    }
                }
            } else {
                // units in the order S(0) .. S(kSlots - 1), PV(0), S(kSlots), PV(1), ..., S right behind the
                // product that has read P from its slot; K is done with after tile 1's S
                scores(0, 0, 0);
                if (two) {
                    wait(kBarQFull + 1, q_count[1] & 1);
                    scores(1, 1, 0);
                }
                commit(kBarKvEmpty + kst);
                if (G_::kSlots == 3 && nb > 1) {
                    next_k(1);
                    scores(0, 0, 1);
                }
                for (int b = 0; b < nb; ++b) {
                    wait(kBarKvFull + vst, vph);
                    products(0, b, b == 0);
                    if (G_::kSlots == 2 && b + 1 < nb) {
                        next_k(b + 1);
                        scores(0, 0, b + 1);
                    } else if (G_::kSlots == 3 && b + 1 < nb) {
                        scores(1, 1, b + 1);
                        commit(kBarKvEmpty + kst);
                    }
                    if (two) {
                        products(1, b, b == 0);
                        if (G_::kSlots == 2 && b + 1 < nb) {
                            scores(1, 1, b + 1);
                            commit(kBarKvEmpty + kst);
                        } else if (G_::kSlots == 3 && b + 2 < nb) {
                            next_k(b + 2);
                            scores(0, 0, b + 2);
                        }
                    }
                    commit(kBarKvEmpty + vst);
                    advance(vst, vph, b + 2 >= nb ? 1 : 2);
                }
                if (two)
                    ++q_count[1];
            }
            ++q_count[0];
            // behind the last V the next item's K(0)
            kst = vst;
            kph = vph;
            ok = !__any_sync(0xffffffffu, failed != 0);
            if (!ok)
                *gave_up = 1;
        }
        if (!ok && lane == 0)
            atomicOr(err_word, kErrCrossWait);
        // every product that was issued must be complete before TMEM is released
        commit(kBarDrain);
        if (!mbar_wait(&bars[kBarDrain], 0) && lane == 0)
            atomicOr(err_word, kErrDrainWait);
        __syncwarp();
    } else if (elect_one()) {
        // ------------------------------ items and query loads ------------------------------
        // The grid has a block for every item.  This one's own is the first; then it asks for blocks that
        // have not started, and takes their items in their place, until none is left: items are of very
        // different lengths (a static deal of them left SMs idle for a fifth of the time), those of the longest
        // sources first.  An item is handed round as soon as all have read the one before, its query tiles follow
        // as each is free.
        prefetch_tensormap(&tmap_q);
        const uint32_t answer = smem_addr(smem + G_::kOffAnswer);
        int it = blockIdx.x;
        int published = 0, asked = 0;
        int qi[2] = {0, 0};   // items whose query tile t was requested
        bool more = true;
        while (more) {
            Item x;
            ok = ok && *gave_up == 0;   // if not, items are asked for and let go
            if (ok && make_item(a, it, order, x, err_word)) {
                if (published > 0)
                    ok = mbar_wait_work(&bars[kBarItemEmpty], (published - 1) & 1, patience, gave_up);
                if (ok) {
                    *item = x;
                    mbar_arrive(&bars[kBarItemFull]);
                    ++published;
                }
                // the tile's 128 / G tokens x G heads, token-major, by column halves
                for (int t = 0; ok && x.n_blocks > 0 && t < (x.has_b ? 2 : 1); ++t) {
                    if (qi[t] > 0 &&
                        !mbar_wait_work(&bars[kBarQEmpty + t], (qi[t] - 1) & 1, patience, gave_up)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&bars[kBarQFull + t], static_cast<uint32_t>(G_::kQBytes));
#pragma unroll
                    for (int h = 0; h < kHalves; ++h)
                        tma_load_4d(q_tile(t) + h * kM * 128, &tmap_q, h * 64, 0, x.kvh,
                                    x.tok0 + (x.row_begin + t * kM) / G, &bars[kBarQFull + t]);
                    ++qi[t];
                }
            }
            more = false;
            mbar_arrive_expect_tx(&bars[kBarCancel], 16);
            try_cancel_block(answer, &bars[kBarCancel]);
            if (!mbar_wait(&bars[kBarCancel], asked & 1)) {
                ok = false;
                *gave_up = 1;
                break;
            }
            ++asked;
            more = cancelled_block(answer, it);
            fence_proxy_async_smem();
        }
        if (published > 0 && !mbar_wait_work(&bars[kBarItemEmpty], (published - 1) & 1, patience, gave_up))
            ok = false;
        item->done = 1;
        mbar_arrive(&bars[kBarItemFull]);
        if (!ok) {
            atomicOr(err_word, kErrCrossWait);
            // the last requests may still be in flight
            for (int t = 0; t < 2; ++t)
                if (qi[t] > 0 && !mbar_wait(&bars[kBarQFull + t], (qi[t] - 1) & 1))
                    atomicOr(err_word, kErrDrainWait);
        }
    }
    } else {
        // ------------------------------ softmax + epilogue -------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // A warp has 16 rows, a thread every fourth pair of columns of two of them (the 16-lane shapes of tensor
        // memory): all of a row is in one warp, which decides by a vote.  (Two warps with 32 rows and half of the
        // columns each met at a barrier for every block; one warp of a scheduler with 32 whole rows took 1,750
        // cycles from S to P, and the tensor pipe waited.)
        const int t = (warp - kRoleWarps) >> 3;      // tile
        const int half = ((warp - kRoleWarps) >> 2) & 1;
        const int quad = warp & 3;                   // TMEM lanes 32 quad + 16 half ..
        const int row0 = quad * 32 + half * 16 + (lane >> 2);   // rows row0 and row0 + 8 of the tile
        const int col = 2 * (lane & 3);              // columns col, col + 1 of every 8
        const uint32_t tmem_w = tmem + (static_cast<uint32_t>(quad * 32 + half * 16) << 16);
        float *exchange = reinterpret_cast<float *>(smem + G_::kOffExchange);   // [m, l][tile][row]
        const float sl2 = a.scale_log2;
        const uint64_t sl2x2 = f2_pack(sl2, sl2);
        // A wait that runs out is the last one: the warp then goes through the rest of its items without
        // waiting.
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok)
                ok = __all_sync(0xffffffffu, mbar_wait(bar, parity));
        };
        // The softmax warps of both tiles meet, twice for every item that they join (hence the parity).  (Not at a
        // named barrier: that has no limit, and one of them may have left.)
        auto meet = [&](uint32_t parity) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bars[kBarBoth]);
            wait(&bars[kBarBoth], parity);
            tc_fence_after_sync();
        };
        Feed w(patience, gave_up);
        int tb = 0;   // blocks of this tile so far
        int ti = 0;   // items of this tile so far
        // The products of the tile's last block before tb, or with two slots of its last one.  (With three S of
        // block b is committed behind the products of block b - 2, no later ones: hence a barrier for every other
        // block, or a wait for those of b - 1 could take the end of b - 2's for theirs.)
        auto pv_wait = [&] {
            if (G_::kSlots > 2)
                wait(&bars[kBarPvDone + 2 * t + ((tb - 1) & 1)], ((tb - 1) >> 1) & 1);
            else
                wait(&bars[kBarPvDone + 2 * t], ti & 1);
        };
        int n0 = 0;   // ring index of the item's first slot
        int u0 = 0;   // units of the CTA before the item
        for (;; n0 += 2 * w.x.n_blocks, u0 += w.x.units()) {
            if (!ok)
                *gave_up = 1;
            if (!w.get(bars, item, ok) || w.x.done)
                break;
            const Item &x = w.x;
            // That it has read the item a warp says behind its first scores: an arrival waits for the warp's
            // stores, and the rows of the item before are still on their way.
            if ((t == 1 && !x.has_b && !x.dual) || x.n_blocks == 0)
                w.has_read(bars);
            if (t == 1 && !x.has_b && !x.dual)
                continue;
            const int gr = x.row_begin + (x.dual ? 0 : t * kM) + row0;
            const bool warp_valid = __any_sync(0xffffffffu, gr < x.rows);
            float m_used[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
            const int b0 = x.dual ? t : 0;
            for (int b = b0; b < x.n_blocks; b += x.dual ? 2 : 1, ++tb) {
                const uint32_t slot = static_cast<uint32_t>(u0 + (x.has_b ? 2 * b + t : b)) % G_::kSlots;
                const uint32_t tmem_s = tmem_w + G_::kColS + slot * kBN;
                // A barrier for every other block of the tile: S of the next may be ready before this one was
                // waited for, S of the one after that comes behind this one's P.
                wait(&bars[kBarSFull + 2 * t + (tb & 1)], (tb >> 1) & 1);
                if (b == b0)
                    w.has_read(bars);
                tc_fence_after_sync();
                const int n_vis = min(x.n_keys - b * kBN, kBN);   // positions of this block
                if ((n_vis & 15) != 0 && half == 0 && (x.dual || t == 0)) {
                    // The last block's V rows n_vis .. up to the next multiple of 16 become zeros before P is
                    // handed over (this PV product is the first to read them), so that NaN in unused slots
                    // never meets a zero probability.  A warp takes every fourth row.
                    const int vn = n0 + 2 * x.n_blocks - 1;
                    wait(&bars[kBarKvFull + vn % kStages], (vn / kStages) & 1);
                    uint8_t *vt = sStages + (vn % kStages) * G_::kStageBytes;
                    for (int r = n_vis + quad; r < ((n_vis + 15) & ~15); r += 4)
                        if (lane < kHalves * 8)
                            *reinterpret_cast<uint4 *>(vt + ((r >> 3) * kHalves + (lane >> 3)) * 1024 +
                                                       (r & 7) * 128 + (lane & 7) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                }
                if (warp_valid) {
                    float xs[2][32];     // columns 64 c + 8 g + col + j of row r: xs[c][4 g + 2 r + j]
                    uint64_t sum2[2];    // of the two rows
                    auto mask = [&](int c) {
                        if (n_vis < kBN) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (64 * c + 8 * (i >> 2) + (i & 1) + col >= n_vis)
                                    xs[c][i] = -INFINITY;
                        }
                    };
                    // p = 2^(s * scale * log2(e) - m) of 64 columns as bf16 pairs over the first of S's columns,
                    // and their sum before the rounding
                    auto probabilities = [&](int c) {
                        uint64_t nm2[2];
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float neg_mu = (m_used[r] == -INFINITY) ? 0.0f : -m_used[r];
                            nm2[r] = f2_pack(neg_mu, neg_mu);
                        }
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float e0, e1;
                            f2_unpack(f2_fma(f2_pack(xs[c][2 * i], xs[c][2 * i + 1]), sl2x2, nm2[i & 1]), e0, e1);
                            e0 = fast_exp2(e0);
                            e1 = fast_exp2(e1);
                            pk[i] = pack_bf16x2(e0, e1);
                            sum2[i & 1] = f2_add(sum2[i & 1], f2_pack(e0, e1));
                        }
                        tmem_st_16x128_x8(tmem_s + 32 * c, pk);
                    };
                    auto sum_of = [&](int r) {
                        float p0, p1;
                        f2_unpack(sum2[r], p0, p1);
                        return p0 + p1;
                    };
                    sum2[0] = sum2[1] = f2_pack(0.0f, 0.0f);
                    // With the maximum of the blocks before, which nearly always still holds; whether it does
                    // (no sum of a thread's 32 is past 2^8, then no p is) is known while P is on its way.  S's
                    // columns 64 .. 127 stay in TMEM and 0 .. 63 in registers for the case that it does not.
                    // The first block has none before it.
                    tmem_ld_16x256_x8(tmem_s, xs[0]);
                    tmem_ld_16x256_x8(tmem_s + 64, xs[1]);
                    tmem_wait_ld();
                    mask(0);
                    mask(1);
                    bool again = true;
                    if (b > b0) {
                        probabilities(1);
                        probabilities(0);
                        again = __any_sync(0xffffffffu, !(sum_of(0) <= kRescaleSum) || !(sum_of(1) <= kRescaleSum) ||
                                                            fminf(m_used[0], m_used[1]) == -INFINITY);
                    }
                    if (again) {
                        tmem_wait_st();
                        tmem_ld_16x256_x8(tmem_s + 64, xs[1]);
                        tmem_wait_ld();
                        mask(1);
                        float alpha[2];
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
                            for (int g = 0; g < 8; ++g) {
                                m0 = fmax3(m0, xs[0][4 * g + 2 * r], xs[0][4 * g + 2 * r + 1]);
                                m1 = fmax3(m1, xs[1][4 * g + 2 * r], xs[1][4 * g + 2 * r + 1]);
                            }
                            m0 = fmaxf(m0, m1);
                            m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, 1));
                            m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, 2)) * sl2;   // base 2
                            alpha[r] = 1.0f;
                            if (m0 > m_used[r]) {
                                alpha[r] = (m_used[r] == -INFINITY) ? 0.0f : fast_exp2(m_used[r] - m0);
                                m_used[r] = m0;
                            }
                            l[r] *= alpha[r];
                        }
                        // O holds every earlier PV product (with two slots S(b) was committed after them): its
                        // rows of this warp are rescaled in place
                        if (b > b0) {
                            if (G_::kSlots > 2) {
                                pv_wait();
                                tc_fence_after_sync();
                            }
#pragma unroll 1
                            for (int c0 = 0; c0 < D; c0 += 32) {
                                float o[16];
                                tmem_ld_16x256_x4(tmem_w + t * D + c0, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    o[j] *= alpha[(j >> 1) & 1];
                                tmem_st_16x256_x4(tmem_w + t * D + c0, o);
                            }
                        }
                        sum2[0] = sum2[1] = f2_pack(0.0f, 0.0f);
                        probabilities(1);
                        probabilities(0);
                    }
                    l[0] += sum_of(0);
                    l[1] += sum_of(1);
                    tmem_wait_st();
                }
                // (rows of padding: whatever P holds stays in rows of O that nobody reads)
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bars[kBarPFull + 2 * t + (tb & 1)]);
            }
            // epilogue: once this tile's last PV is done, O / l -> global
            if (x.n_blocks > 0) {
                pv_wait();
                ++ti;
                tc_fence_after_sync();
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            }
            float f[2][2] = {{1.0f, 1.0f}, {0.0f, 0.0f}};   // weights of the two halves of TMEM, for both rows
            if (x.dual) {
                // (m, l) of both, read by both; each writes half of the columns
                if ((lane & 3) == 0) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        exchange[t * kM + row0 + 8 * r] = m_used[r];
                        exchange[(2 + t) * kM + row0 + 8 * r] = l[r];
                    }
                }
                meet(0);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float *at = exchange + row0 + 8 * r;
                    const float m0 = at[0], m1 = at[kM];
                    m_used[r] = fmaxf(m0, m1);
                    f[0][r] = m0 == -INFINITY && m_used[r] != m0 ? 0.0f : fast_exp2(m0 - m_used[r]);
                    f[1][r] = m1 == -INFINITY && m_used[r] != m1 ? 0.0f : fast_exp2(m1 - m_used[r]);
                    if (m_used[r] == -INFINITY)   // no score above -inf (or NaN alone, which l and O hold)
                        f[0][r] = f[1][r] = 1.0f;
                    l[r] = at[2 * kM] * f[0][r] + at[3 * kM] * f[1][r];
                }
            }
            // rows of the output, or of the splits' results
            const bool parts = a.n_split > 1;
            uint8_t *out = static_cast<uint8_t *>(parts ? a.part_o : a.out);
            const bool out_f32 = parts || a.out_f32;
            float *lse = parts ? a.part_lse : a.lse;
            uint8_t *to[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int at = gr + 8 * r, tok = at / G;
                size_t out_row = static_cast<size_t>(x.tok0 + tok) * a.q_heads + static_cast<size_t>(x.kvh) * G +
                                 (at - tok * G);
                if (parts)
                    out_row = out_row * a.n_split + x.split;
                if (at < x.rows && lse != nullptr && (lane & 3) == 0 && !(x.dual && t == 1))
                    lse[out_row] = l[r] == 0.0f ? -INFINITY : m_used[r] * kLn2 + logf(l[r]);   // no position: -inf
                to[r] = at < x.rows ? out + out_row * (D * (out_f32 ? 4u : 2u)) : nullptr;
                const float inv = (l[r] == 0.0f) ? 0.0f : 1.0f / l[r];
                f[0][r] *= inv;
                f[1][r] *= inv;
            }
            if (x.n_blocks == 0 && parts)
                continue;   // an empty split's row is not read
            const int c_begin = x.dual ? t * (D / 2) : 0, c_end = x.dual ? c_begin + D / 2 : D;
#pragma unroll 1
            for (int c0 = c_begin; c0 < c_end; c0 += 32) {
                float o[16];   // columns c0 + 8 g + col + j of row r: o[4 g + 2 r + j]
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    o[j] = 0.0f;
                if (x.n_blocks > 0) {
                    tmem_ld_16x256_x4(tmem_w + (x.dual ? 0 : t * D) + c0, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        o[j] *= f[0][(j >> 1) & 1];
                }
                if (x.dual) {
                    float o1[16];
                    tmem_ld_16x256_x4(tmem_w + D + c0, o1);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        o[j] = fmaf(o1[j], f[1][(j >> 1) & 1], o[j]);
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    if (out_f32) {
                        if (to[r] != nullptr) {
#pragma unroll
                            for (int g = 0; g < 4; ++g)
                                *reinterpret_cast<float2 *>(to[r] + (c0 + 8 * g + col) * 4) =
                                    make_float2(o[4 * g + 2 * r], o[4 * g + 2 * r + 1]);
                        }
                        continue;
                    }
                    // the four lanes of a row turn their words, one of every group of 8 columns each, into
                    // 16 bytes of one group each: 64 bytes of a row at a time (8 lines a store, not 32, of
                    // which the stores of both tiles took 4,096 cycles)
                    uint32_t v[4];
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        v[g] = pack_bf16x2(o[4 * g + 2 * r], o[4 * g + 2 * r + 1]);
#pragma unroll
                    for (int bit = 1; bit <= 2; bit *= 2) {
                        const bool upper = lane & bit;
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            if (g & bit)
                                continue;
                            const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? v[g] : v[g + bit], bit);
                            if (upper)
                                v[g] = got;
                            else
                                v[g + bit] = got;
                        }
                    }
                    if (to[r] != nullptr)
                        *reinterpret_cast<uint4 *>(to[r] + c0 * 2 + (lane & 3) * 16) =
                            make_uint4(v[0], v[1], v[2], v[3]);
                }
            }
            tc_fence_before_sync();
            if (x.dual)   // nobody overwrites what the other still reads
                meet(1);
        }
        if (!ok)
            atomicOr(err_word, kErrCrossWait);
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, G_::kTmemCols);
    }
}

// Joins the splits of every row of the sources' tokens, a warp a row: with M the largest log-sum-exp,
// out = sum_j e^(lse_j - M) o_j / sum_j e^(lse_j - M).  Splits without a position (-inf) are not read.
template <int D>
__global__ void __launch_bounds__(128)
    cross_merge_kernel(void *out, int out_f32, float *lse_out, const float *part_o, const float *part_lse,
                       const int32_t *q_indptr, int num_sources, int num_tokens, int q_heads, int n_split)
{
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(num_tokens) * q_heads)
        return;
    const int tok = static_cast<int>(row / q_heads);
    if (tok < q_indptr[0] || tok >= q_indptr[num_sources])   // rows of no source: left as they were
        return;
    const float *lse = part_lse + row * n_split;
    constexpr int E = D / 32;
    float acc[E] = {};
    float total = 0.0f, M = -INFINITY;
    bool nan = false;
    const float *o = part_o + row * n_split * D + lane * E;
    // four splits at a time, their rows loaded with their log-sum-exps (an empty one's row is any memory of the
    // workspace, and is not used)
    for (int j0 = 0; j0 < n_split; j0 += 4) {
        float v[4], x[4][E];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = j0 + j < n_split ? lse[j0 + j] : -INFINITY;
#pragma unroll
            for (int e = 0; e < E; ++e)
                x[j][e] = j0 + j < n_split ? o[static_cast<size_t>(j0 + j) * D + e] : 0.0f;
        }
        const float m = fmaxf(fmaxf(M, fmaxf(v[0], v[1])), fmaxf(v[2], v[3]));
        nan |= isnan(v[0]) || isnan(v[1]) || isnan(v[2]) || isnan(v[3]);
        const float keep = M == -INFINITY ? 0.0f : expf(M - m);
        total *= keep;
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] *= keep;
        M = m;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (v[j] == -INFINITY)
                continue;
            const float w = expf(v[j] - M);
            total += w;
#pragma unroll
            for (int e = 0; e < E; ++e)
                acc[e] += w * x[j][e];
        }
    }
    const float inv = nan ? NAN : (total > 0.0f ? 1.0f / total : 0.0f);
    const size_t idx = static_cast<size_t>(row) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        store_out2(out, out_f32, idx + e, make_float2(acc[e] * inv, acc[e + 1] * inv));
    if (lse_out != nullptr && lane == 0)
        lse_out[row] = nan ? NAN : (total > 0.0f ? M + logf(total) : -INFINITY);
}

template <int D>
cudaError_t launch_t(const CrossLaunch &l, const CUtensorMap &tq, const CUtensorMap &tk,
                     const CUtensorMap &tv, cudaStream_t stream)
{
    Args a;
    a.out = l.out;
    a.out_f32 = l.out_f32 ? 1 : 0;
    a.lse = l.lse;
    a.part_o = l.part_o;
    a.part_lse = l.part_lse;
    a.block_table = l.block_table;
    a.bt_stride = l.bt_stride;
    a.q_indptr = l.q_indptr;
    a.source_lens = l.source_lens;
    a.kv_heads = l.kv_heads;
    a.q_heads = l.q_heads;
    a.group = l.q_heads / l.kv_heads;
    a.page_size = l.page_size;
    a.num_tokens = l.num_tokens;
    a.max_q_len = l.max_q_len;
    a.max_src = l.max_src;
    a.chunk = l.chunk;
    a.n_split = l.n_split;
    a.hnd = l.hnd ? 1 : 0;
    a.err = current_error_word();
    a.scale_log2 = l.scale * kLog2e;
    const int tiles = (l.max_q_len * a.group + kM - 1) / kM;
    a.pairs_per_seq = (tiles + 1) / 2;
    const long long items =
        static_cast<long long>(a.pairs_per_seq) * l.kv_heads * l.n_split * l.num_sources;
    if (items > 0x7FFFFFFFLL)
        return cudaErrorInvalidValue;
    // The longest sources' items first where there are more items than SMs (64 sources of 512 to 4,096 positions x
    // 200-400 queries: 595 us as they come, 583 ordered; 24 of 100 to 4,000 189, 162; 100 of 100 to 2,000 79, 68).  Not
    // where all are short: 250 sources of 10 to 400 went from 61 to 60 at head dim 64, from 98 to 102 at 128.
    a.ordered = items > current_sm_count() && l.max_src > 8 * kBN && l.num_sources > 1 &&
                        l.num_sources <= kMaxOrdered
                    ? l.num_sources
                    : 0;
    auto kernel = cross_kernel<D>;
    // the split of registers draws on what the block is launched with
    cudaFuncAttributes attr;
    cudaError_t err = cudaFuncGetAttributes(&attr, kernel);
    if (err != cudaSuccess)
        return err;
    if (attr.numRegs < kLaunchRegs)
        return cudaErrorLaunchOutOfResources;
    const size_t smem = Geom<D>::kSmemBytes;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(smem));
    if (err != cudaSuccess)
        return err;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(items)), dim3(kThreads), smem, stream, tq, tk, tv,
                      a);
}

}  // namespace

cudaError_t launch_cross(const CrossLaunch &l, const CUtensorMap &tmap_q, const CUtensorMap &tmap_k,
                         const CUtensorMap &tmap_v, cudaStream_t stream)
{
    return l.head_dim == 128 ? launch_t<128>(l, tmap_q, tmap_k, tmap_v, stream)
                             : launch_t<64>(l, tmap_q, tmap_k, tmap_v, stream);
}

cudaError_t launch_cross_merge(const CrossLaunch &l, cudaStream_t stream)
{
    const long long rows = static_cast<long long>(l.num_tokens) * l.q_heads;
    return launch_pdl(l.head_dim == 128 ? cross_merge_kernel<128> : cross_merge_kernel<64>,
                      dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0, stream, l.out,
                      l.out_f32 ? 1 : 0, l.lse, static_cast<const float *>(l.part_o),
                      static_cast<const float *>(l.part_lse), l.q_indptr, l.num_sources, l.num_tokens,
                      l.q_heads, l.n_split);
}

cudaError_t read_and_clear_cross_errors(uint32_t *flags)
{
    uint32_t zero = 0;
    cudaError_t err = cudaMemcpyFromSymbol(flags, g_cross_errors, sizeof(uint32_t));
    if (err != cudaSuccess)
        return err;
    return cudaMemcpyToSymbol(g_cross_errors, &zero, sizeof(uint32_t));
}

}  // namespace kvc
