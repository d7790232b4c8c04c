// kvc_cross.cu -- attention of queries to the states of a source of another length, no causal limit, on the
// 5th-generation tensor cores (tcgen05, accumulators in tensor memory).
//
//   out[t][h] = sum_p softmax_p(q[t][h] . K[p][h / G] * scale) V[p][h / G],   p < source_lens[s],
// for the tokens t of q_indptr[s] .. q_indptr[s + 1] - 1, the source's pages read in place.
//
// Tiling: the rows of one (source, kv head) are its (token, query head of the group) pairs, token-major, in
// tiles of 128 (the tcgen05 M).  A work item is a pair of consecutive tiles over one chunk of the source's
// positions (the whole source where there is one split); both tiles see the same pages, so every K or V
// stage feeds two products.  One persistent CTA per SM walks items c, c + grid, ...; its roles run ahead
// across items:
//   warp 0      TMA, K and V: 128-position stages (a box per page and 64-column half, 128-byte swizzle, issued
//               by parallel lanes) in one ring, filled in the order K(0), K(1), V(0), K(2), V(1), ...
//   warp 1      allocates TMEM (512 columns) and issues S_w = Q_w K(b)^T (M 128, N 128, K head_dim) and
//               O_w += P_w V(b) (N head_dim, K 128, P from TMEM) of the tiles w from one thread; S_w(b + 1)
//               right behind the PV product that reads P_w(b) from the same columns.  The V rows past the
//               source's end, up to the next multiple of 16, are zeroed first, so that NaN in unused slots
//               never meets a zero probability.
//   warp 2      TMA, the item's query tiles
//   warps 3-6   softmax of tile 0, warps 7-10 of tile 1: a thread a row: the running maximum (O rescaled only
//               when it grows by more than 2^8) and sum, P as bf16 over the first half of S's columns, and
//               O / l at the end.
// Few rows and many positions: the positions are cut into chunks (splits), partial rows and their
// log-sum-exps go to the workspace and cross_merge_kernel joins them.
// Sums: P is rounded to bf16 for the product and l sums the rounded values, so that numerator and denominator
// weigh a position alike; a log-sum-exp that is asked for sums the unrounded ones.
#include <math.h>

#include "kvc_device.cuh"
#include "kvc_launch.h"

namespace kvc {

namespace {

__device__ uint32_t g_cross_errors;

constexpr int kM = 128;           // rows per tile
constexpr int kBN = kCrossBlock;  // positions per K or V stage (the N of S = Q K^T)
constexpr int kRoleWarps = 3;     // K/V loads, MMA issue, query loads
constexpr int kSoftmaxWarps = 8;  // two groups of four
constexpr int kThreads = (kRoleWarps + kSoftmaxWarps) * 32;
constexpr int kMaxStages = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.0f;

template <int D>
struct Geom {
    static constexpr int kHalves = D / 64;
    static constexpr int kQBytes = kHalves * kM * 128;       // one query tile
    static constexpr int kStageBytes = kHalves * kBN * 128;  // K or V of 128 positions
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kOffStages = 2 * kQBytes;           // Q: [tile]
    static constexpr int kOffBar = kOffStages + kStages * kStageBytes;
    static constexpr size_t kSmemBytes = kOffBar + 512;      // base is 1024-aligned
    // TMEM, per tile w at w * 256: O [0, D), S [D, D + 128); P overwrites S [D, D + 64).
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kColS = D;
    static_assert(D + kBN <= 256, "TMEM layout");
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
    int kv_heads, q_heads, group, page_size, pairs_per_seq, num_items;
    int max_q_len, max_src, chunk, n_split;
    float scale_log2;
    int hnd;   // HND pools: half boxes addressed by (offset, page * kv_heads + kv head)
    uint32_t *err;
};

enum BarIndex : int {
    kBarKvFull = 0,                         // [ring slot]
    kBarKvEmpty = kBarKvFull + kMaxStages,  // [ring slot], one MMA commit
    kBarQFull = kBarKvEmpty + kMaxStages,   // [tile]
    kBarQEmpty = kBarQFull + 2,             // [tile], one MMA commit after its last S product
    kBarSFull = kBarQEmpty + 2,             // [tile]
    kBarPFull = kBarSFull + 2,              // [tile], 128 arrivals
    kBarPvDone = kBarPFull + 2,             // [tile], once per item
    kBarDrain = kBarPvDone + 2,
    kBarCount = kBarDrain + 1
};

// Tiles 2 tp and 2 tp + 1 of one (source, kv head) over positions key0 .. key0 + n_keys - 1.
struct Item {
    int s, kvh, tp, split;
    int tok0, rows, row_begin;   // row_begin: first row of tile 2 tp
    bool has_b;                  // tile 2 tp + 1 exists
    int key0, n_keys, n_blocks;  // n_keys 0: nothing to attend to, rows are written all the same
};

// Walks this CTA's items, skipping those without rows.  The next item's lengths are requested one item
// ahead: a load under a full memory pipe takes microseconds.
struct Walker {
    int it;
    bool done;
    Item x;
    int pit, p_tok0, p_tok1, p_len;

    __device__ __forceinline__ static int seq_of(const Args &a, int it)
    {
        return it / a.pairs_per_seq / a.kv_heads / a.n_split;
    }
    __device__ __forceinline__ bool make(const Args &a, int tok0, int tok1, int len, uint32_t *err)
    {
        x.tp = it % a.pairs_per_seq;
        int rest = it / a.pairs_per_seq;
        x.kvh = rest % a.kv_heads;
        rest /= a.kv_heads;
        x.split = rest % a.n_split;
        x.s = rest / a.n_split;
        const int most = min(a.max_src, a.bt_stride * a.page_size);
        if (len > most || tok1 - tok0 > a.max_q_len) {
            if (threadIdx.x == 0)
                atomicOr(err, kErrContextRange);
            len = min(len, most);
        }
        x.tok0 = tok0;
        x.rows = min(tok1 - tok0, a.max_q_len) * a.group;
        x.row_begin = x.tp * 2 * kM;
        if (x.row_begin >= x.rows)
            return false;
        x.has_b = x.row_begin + kM < x.rows;
        x.key0 = x.split * a.chunk;
        x.n_keys = min(max(len - x.key0, 0), a.chunk);
        x.n_blocks = (x.n_keys + kBN - 1) / kBN;
        return true;
    }
    __device__ __forceinline__ void prefetch(const Args &a, int idx)
    {
        pit = idx;
        if (idx < a.num_items) {
            const int s = seq_of(a, idx);
            p_tok0 = a.q_indptr[s];
            p_tok1 = a.q_indptr[s + 1];
            p_len = a.source_lens[s];
        }
    }
    __device__ __forceinline__ void next(const Args &a, uint32_t *err)
    {
        for (;;) {
            if (it > a.num_items - 1 - static_cast<int>(gridDim.x)) {
                done = true;
                return;
            }
            it += gridDim.x;
            if (it != pit)
                prefetch(a, it);
            if (make(a, p_tok0, p_tok1, p_len, err))
                break;
        }
        prefetch(a, it < a.num_items - static_cast<int>(gridDim.x) ? it + gridDim.x : a.num_items);
    }
    __device__ __forceinline__ void start(const Args &a, uint32_t *err)
    {
        it = static_cast<int>(blockIdx.x) - static_cast<int>(gridDim.x);
        done = false;
        pit = -1;
        next(a, err);
    }
};

template <int D, bool LSE>
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
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kBarCount);
    auto q_tile = [&](int tile) { return smem + tile * G_::kQBytes; };

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int G = a.group;
    const int P = a.page_size;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kBarCount; ++i)
            mbar_init(&bars[i], (i == kBarPFull || i == kBarPFull + 1) ? 128u : 1u);
        fence_mbar_init();
    }
    if (warp == 1)
        tmem_alloc(tmem_slot, G_::kTmemCols);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;

    if (warp == 0) {
        // ------------------------------ K / V loads --------------------------------------
        if (lane == 0) {
            prefetch_tensormap(&tmap_k);
            prefetch_tensormap(&tmap_v);
        }
        // tiles past the first pair read the pages again: only pages read once may leave L2 early
        const uint64_t policy = a.pairs_per_seq > 1 ? l2_policy_evict_last() : l2_policy_evict_first();
        Walker w;
        int n = 0;   // ring slots filled so far
        for (w.start(a, err_word); ok && !w.done; w.next(a, err_word)) {
            const Item &x = w.x;
            const int32_t *bt_row =
                a.block_table + static_cast<size_t>(x.s) * a.bt_stride + x.key0 / P;
            const int n_pages = (x.n_keys + P - 1) / P;
            int cached_base = 0;
            int cached_page = lane < n_pages ? bt_row[lane] : 0;
            const int nb = x.n_blocks;
            for (int j = 0; j < 2 * nb; ++j, ++n) {
                const bool is_k = j == 0 || (j < 2 * nb - 1 && (j & 1));
                const int b = is_k ? (j + 1) / 2 : (j == 2 * nb - 1 ? nb - 1 : j / 2 - 1);
                const int np = (min(kBN, x.n_keys - b * kBN) + P - 1) / P;
                const int st = n % kStages;
                if (n >= kStages && !__all_sync(0xffffffffu, mbar_wait(&bars[kBarKvEmpty + st],
                                                                       ((n / kStages) - 1) & 1))) {
                    ok = false;
                    break;
                }
                if (lane == 0)
                    mbar_arrive_expect_tx(&bars[kBarKvFull + st], static_cast<uint32_t>(np * P * D * 2));
                __syncwarp();
                uint8_t *dst = sStages + st * G_::kStageBytes;
                const int lp0 = b * kBN / P;   // first page of the block
                if (lp0 < cached_base || lp0 + np > cached_base + 32) {
                    cached_base = lp0;
                    cached_page = (lp0 + lane < n_pages) ? bt_row[lp0 + lane] : 0;
                }
                // lane i * kHalves + h issues the box of page i, column half h
                const int i = lane / kHalves;
                const int h = lane % kHalves;
                const int page =
                    __shfl_sync(0xffffffffu, cached_page, (lp0 - cached_base + i) & 31);
                // NHD maps {head_dim, kv head, slot}; HND maps {head_dim, offset, block}
                if (i < np)
                    tma_load_3d(dst + h * kBN * 128 + i * P * 128, is_k ? &tmap_k : &tmap_v, h * 64,
                                a.hnd ? 0 : x.kvh, a.hnd ? page * a.kv_heads + x.kvh : page * P,
                                &bars[kBarKvFull + st], policy);
            }
            if (!ok)
                break;
        }
        if (!ok && lane == 0) {
            atomicOr(err_word, kErrCrossWait);
            // let every copy in flight land before the CTA can exit
            for (int m = max(0, n - kStages); m < n; ++m)
                if (!mbar_wait(&bars[kBarKvFull + m % kStages], (m / kStages) & 1))
                    atomicOr(err_word, kErrDrainWait);
        }
    } else if (warp == 2) {
        // ------------------------------ query loads --------------------------------------
        if (lane == 0)
            prefetch_tensormap(&tmap_q);
        Walker w;
        int qi[2] = {0, 0};   // items whose query tile t was requested
        for (w.start(a, err_word); ok && !w.done; w.next(a, err_word)) {
            const Item &x = w.x;
            if (x.n_blocks == 0)
                continue;
            // lane h loads column half h of the tile's 128 / G tokens x G heads, token-major
            for (int t = 0; t < (x.has_b ? 2 : 1); ++t) {
                if (qi[t] > 0 &&
                    !__all_sync(0xffffffffu, mbar_wait(&bars[kBarQEmpty + t], (qi[t] - 1) & 1))) {
                    ok = false;
                    break;
                }
                if (lane == 0)
                    mbar_arrive_expect_tx(&bars[kBarQFull + t], static_cast<uint32_t>(G_::kQBytes));
                __syncwarp();
                if (lane < kHalves)
                    tma_load_4d(q_tile(t) + lane * kM * 128, &tmap_q, lane * 64, 0, x.kvh,
                                x.tok0 + (x.row_begin + t * kM) / G, &bars[kBarQFull + t]);
                ++qi[t];
            }
            if (!ok)
                break;
        }
        if (!ok && lane == 0) {
            atomicOr(err_word, kErrCrossWait);
            // the last requests may still be in flight
            for (int t = 0; t < 2; ++t)
                if (qi[t] > 0 && !mbar_wait(&bars[kBarQFull + t], (qi[t] - 1) & 1))
                    atomicOr(err_word, kErrDrainWait);
        }
    } else if (warp == 1) {
        // ------------------------------ MMA issue ----------------------------------------
        constexpr uint32_t kIdescPV = umma_idesc_bf16(kM, D, 1);
        const uint32_t stage_addr = smem_addr(sStages);
        auto stage_of = [&](int n) { return stage_addr + (n % kStages) * G_::kStageBytes; };
        auto wait_slot = [&](int n) {
            return __all_sync(0xffffffffu,
                              mbar_wait(&bars[kBarKvFull + n % kStages], (n / kStages) & 1));
        };
        // S_t = Q_t K^T over n_cols positions (a multiple of 16)
        auto issue_qk = [&](int t, uint32_t k_addr, int n_cols) {
            const uint32_t idesc = umma_idesc_bf16(kM, n_cols, 0);
            const uint32_t q_addr = smem_addr(q_tile(t));
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint64_t da =
                    umma_desc_sw128(q_addr + (k >> 2) * kM * 128 + (k & 3) * 32, 16, 1024);
                const uint64_t db =
                    umma_desc_sw128(k_addr + (k >> 2) * kBN * 128 + (k & 3) * 32, 16, 1024);
                umma_bf16_ss(tmem + t * 256 + G_::kColS, da, db, idesc, k > 0 ? 1u : 0u);
            }
        };
        // O_t (+)= P_t V over k_steps x 16 positions
        auto issue_pv = [&](int t, uint32_t v_addr, int k_steps, bool first) {
            for (int k = 0; k < k_steps; ++k) {
                const uint64_t db = umma_desc_sw128(v_addr + k * 16 * 128, kBN * 128, 1024);
                umma_bf16_ts(tmem + t * 256, tmem + t * 256 + G_::kColS + k * 8, db, kIdescPV,
                             (!first || k > 0) ? 1u : 0u);
            }
        };
        Walker w;
        int n0 = 0;             // ring index of the item's first slot
        int qi[2] = {0, 0};     // items of tile 0 / tile 1
        int tb[2] = {0, 0};     // blocks of tile 0 / tile 1
        for (w.start(a, err_word); ok && !w.done; w.next(a, err_word)) {
            const Item &x = w.x;
            const int nt = x.has_b ? 2 : 1;
            const int nb = x.n_blocks;
            if (nb == 0)
                continue;
            const int last_valid = x.n_keys - (nb - 1) * kBN;   // positions in the last block
            const int last_cols = (last_valid + 15) & ~15;
            // ring indices in the producer's fill order K(0), K(1), V(0), K(2), V(1), ...
            auto k_slot = [&](int b) { return n0 + (b == 0 ? 0 : 2 * b - 1); };
            auto v_slot = [&](int b) { return n0 + (b == nb - 1 ? 2 * nb - 1 : 2 * b + 2); };
            if (!wait_slot(k_slot(0))) {
                ok = false;
                break;
            }
            for (int t = 0; t < nt && ok; ++t) {
                if (!__all_sync(0xffffffffu, mbar_wait(&bars[kBarQFull + t], qi[t] & 1))) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                if (lane == 0) {
                    issue_qk(t, stage_of(k_slot(0)), nb == 1 ? last_cols : kBN);
                    umma_commit(&bars[kBarSFull + t]);
                    if (nb == 1)
                        umma_commit(&bars[kBarQEmpty + t]);
                }
                __syncwarp();
            }
            if (!ok)
                break;
            if (lane == 0)
                umma_commit(&bars[kBarKvEmpty + k_slot(0) % kStages]);
            __syncwarp();
            for (int b = 0; b < nb && ok; ++b) {
                const bool last = b + 1 == nb;
                const int vn = v_slot(b);
                if (!wait_slot(vn)) {
                    ok = false;
                    break;
                }
                if (last && last_valid < last_cols) {
                    // V rows last_valid .. last_cols - 1 of every column half
                    uint8_t *vt = sStages + (vn % kStages) * G_::kStageBytes;
                    const int rows_to_zero = last_cols - last_valid;
                    for (int idx = lane; idx < rows_to_zero * kHalves * 8; idx += 32) {
                        const int chunk = idx & 7;
                        const int rest = idx >> 3;
                        const int h = rest % kHalves;
                        const int r = last_valid + rest / kHalves;
                        *reinterpret_cast<uint4 *>(vt + h * kBN * 128 + r * 128 + chunk * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                const int kn = last ? 0 : k_slot(b + 1);
                for (int t = 0; t < nt; ++t) {
                    if (!__all_sync(0xffffffffu, mbar_wait(&bars[kBarPFull + t], tb[t] & 1))) {
                        ok = false;
                        break;
                    }
                    ++tb[t];
                    tc_fence_after_sync();
                    if (lane == 0) {
                        issue_pv(t, stage_of(vn), last ? last_cols / 16 : kBN / 16, b == 0);
                        if (last)
                            umma_commit(&bars[kBarPvDone + t]);
                    }
                    __syncwarp();
                    if (last)
                        continue;
                    // K(b + 1) is waited for only once PV(b) of tile 0 is on its way
                    if (t == 0 && !wait_slot(kn)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    if (lane == 0) {
                        issue_qk(t, stage_of(kn), b + 2 == nb ? last_cols : kBN);
                        umma_commit(&bars[kBarSFull + t]);
                        if (b + 2 == nb)
                            umma_commit(&bars[kBarQEmpty + t]);
                    }
                    __syncwarp();
                }
                if (!ok)
                    break;
                if (lane == 0) {
                    umma_commit(&bars[kBarKvEmpty + vn % kStages]);
                    if (!last)
                        umma_commit(&bars[kBarKvEmpty + kn % kStages]);
                }
                __syncwarp();
            }
            if (!ok)
                break;
            for (int t = 0; t < nt; ++t)
                ++qi[t];
            n0 += 2 * nb;
        }
        if (!ok && lane == 0)
            atomicOr(err_word, kErrCrossWait);
        // every product that this thread issued must be complete before TMEM is released
        if (lane == 0) {
            umma_commit(&bars[kBarDrain]);
            if (!mbar_wait(&bars[kBarDrain], 0))
                atomicOr(err_word, kErrDrainWait);
        }
        __syncwarp();
    } else {
        // ------------------------------ softmax + epilogue -------------------------------
        const int t = (warp - kRoleWarps) >> 2;      // tile
        const int quad = warp & 3;                   // TMEM lanes 32 quad ..
        const int row = quad * 32 + lane;            // row of the tile = TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t tmem_o = tmem + t * 256 + lane_off;
        const uint32_t tmem_s = tmem + t * 256 + G_::kColS + lane_off;
        const float sl2 = a.scale_log2;
        Walker w;
        int tb = 0;   // blocks of this tile so far
        int ti = 0;   // items of this tile so far
        for (w.start(a, err_word); ok && !w.done; w.next(a, err_word)) {
            const Item &x = w.x;
            if (t == 1 && !x.has_b)
                continue;
            const int gr = x.row_begin + t * kM + row;
            const bool valid = gr < x.rows;
            const int tok = gr / G;
            const bool warp_valid = __any_sync(0xffffffffu, valid);
            float m_used = -INFINITY;
            float l_sum = 0.0f, l_exact = 0.0f;
            for (int b = 0; b < x.n_blocks; ++b, ++tb) {
                if (!__all_sync(0xffffffffu, mbar_wait(&bars[kBarSFull + t], tb & 1))) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const int n_vis = min(x.n_keys - b * kBN, kBN);   // positions of this block
                float alpha = 1.0f;
                bool moved = false;
                if (warp_valid) {
                    // pass 1: the row maximum; masked columns become -inf in TMEM as well
                    float xs[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        tmem_ld32(tmem_s + 32 * c, xs[c]);
                    tmem_wait_ld();
                    float mx = -INFINITY;
                    if (n_vis == kBN) {
#pragma unroll
                        for (int j = 0; j < kBN; j += 2)
                            mx = fmax3(mx, xs[j >> 5][j & 31], xs[j >> 5][(j & 31) + 1]);
                    } else {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (32 * c + j >= n_vis)
                                    xs[c][j] = -INFINITY;
#pragma unroll
                            for (int j = 0; j < 32; j += 2)
                                mx = fmax3(mx, xs[c][j], xs[c][j + 1]);
                            tmem_st32(tmem_s + 32 * c, xs[c]);
                        }
                        tmem_wait_st();
                    }
                    const float mb = mx * sl2;   // base-2 scaled maximum of this block
                    if (mb > m_used + kRescaleLog2) {
                        alpha = (m_used == -INFINITY) ? 0.0f : fast_exp2(m_used - mb);
                        m_used = mb;
                        moved = true;
                    }
                }
                // O holds every earlier PV product (S(b) was committed after them): rescale
                // it in place when the maximum moved.
                if (b > 0 && __any_sync(0xffffffffu, moved)) {
                    const float f = moved ? alpha : 1.0f;
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        float o[32];
                        tmem_ld32(tmem_o + c0, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            o[j] *= f;
                        tmem_st32(tmem_o + c0, o);
                    }
                }
                // pass 2, 32 columns at a time: p = 2^(s * scale * log2(e) - m); the bf16 pairs of
                // chunk c go to S columns [16 c, 16 c + 16), which hold only chunks already read
                const float neg_mu = (m_used == -INFINITY) ? 0.0f : -m_used;
                const uint64_t sl2x2 = f2_pack(sl2, sl2);
                const uint64_t nm2 = f2_pack(neg_mu, neg_mu);
                uint64_t psum2 = f2_pack(0.0f, 0.0f), pexact2 = f2_pack(0.0f, 0.0f);
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t pk[16];
                    if (warp_valid) {
                        float v[32];
                        tmem_ld32(tmem_s + 32 * c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float e0, e1;
                            f2_unpack(f2_fma(f2_pack(v[2 * j], v[2 * j + 1]), sl2x2, nm2), e0, e1);
                            e0 = fast_exp2(e0);
                            e1 = fast_exp2(e1);
                            pk[j] = pack_bf16x2(e0, e1);
                            psum2 = f2_add(psum2, f2_pack(__uint_as_float(pk[j] << 16),
                                                          __uint_as_float(pk[j] & 0xFFFF0000u)));
                            if (LSE)
                                pexact2 = f2_add(pexact2, f2_pack(e0, e1));
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j)   // a warp of padding rows: P = 0
                            pk[j] = 0u;
                    }
                    tmem_st16u(tmem_s + 16 * c, pk);
                }
                float p0, p1;
                f2_unpack(psum2, p0, p1);
                l_sum = l_sum * alpha + (p0 + p1);
                if (LSE) {
                    f2_unpack(pexact2, p0, p1);
                    l_exact = l_exact * alpha + (p0 + p1);
                }
                tmem_wait_st();
                tc_fence_before_sync();
                mbar_arrive(&bars[kBarPFull + t]);
            }
            if (!ok)
                break;
            // epilogue: once this tile's last PV is done, O / l -> global
            if (x.n_blocks > 0) {
                if (!__all_sync(0xffffffffu, mbar_wait(&bars[kBarPvDone + t], ti & 1))) {
                    ok = false;
                    break;
                }
                ++ti;
                tc_fence_after_sync();
            }
            const float inv = (l_sum > 0.0f) ? 1.0f / l_sum : 0.0f;
            const int g = gr - tok * G;
            size_t out_row = static_cast<size_t>(x.tok0 + tok) * a.q_heads +
                             static_cast<size_t>(x.kvh) * G + g;
            void *out = a.out;
            int out_f32 = a.out_f32;
            float *lse = a.lse;
            if (a.n_split > 1) {
                out_row = out_row * a.n_split + x.split;
                out = a.part_o;
                out_f32 = 1;
                lse = a.part_lse;
            }
            if (valid && lse != nullptr) {
                const float l = LSE ? l_exact : l_sum;
                // no position: -inf; a NaN sum stays one
                lse[out_row] = l == 0.0f ? -INFINITY : m_used * kLn2 + logf(l);
            }
            if (x.n_blocks == 0 && a.n_split > 1)
                continue;   // an empty split's row is not read
            out_row *= D;
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += 32) {
                float o[32];
                if (x.n_blocks > 0) {
                    tmem_ld32(tmem_o + c0, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        o[j] = 0.0f;
                }
                if (valid) {
                    if (out_f32) {
                        float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(out) +
                                                                 out_row + c0);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            dst[j] = make_float4(o[4 * j] * inv, o[4 * j + 1] * inv,
                                                 o[4 * j + 2] * inv, o[4 * j + 3] * inv);
                    } else {
                        uint4 *dst = reinterpret_cast<uint4 *>(
                            static_cast<__nv_bfloat16 *>(out) + out_row + c0);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            dst[c] = make_uint4(pack_bf16x2(o[8 * c] * inv, o[8 * c + 1] * inv),
                                                pack_bf16x2(o[8 * c + 2] * inv, o[8 * c + 3] * inv),
                                                pack_bf16x2(o[8 * c + 4] * inv, o[8 * c + 5] * inv),
                                                pack_bf16x2(o[8 * c + 6] * inv, o[8 * c + 7] * inv));
                    }
                }
                __syncwarp();
            }
            tc_fence_before_sync();
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
    float M = -INFINITY;
    bool nan = false;
    for (int j = lane; j < n_split; j += 32) {
        const float v = lse[j];
        nan |= isnan(v);
        M = fmaxf(M, v);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    nan = __any_sync(0xffffffffu, nan);
    constexpr int E = D / 32;
    float acc[E] = {};
    float total = 0.0f;
    const float *o = part_o + row * n_split * D + lane * E;
    for (int j = 0; j < n_split; ++j) {
        const float v = lse[j];
        if (v == -INFINITY)
            continue;
        const float w = expf(v - M);
        total += w;
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] += w * o[static_cast<size_t>(j) * D + e];
    }
    const float inv = nan ? NAN : (total > 0.0f ? 1.0f / total : 0.0f);
    const size_t idx = static_cast<size_t>(row) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        store_out2(out, out_f32, idx + e, make_float2(acc[e] * inv, acc[e + 1] * inv));
    if (lse_out != nullptr && lane == 0)
        lse_out[row] = nan ? NAN : (total > 0.0f ? M + logf(total) : -INFINITY);
}

template <int D, bool LSE>
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
    a.num_items = static_cast<int>(items);
    auto kernel = cross_kernel<D, LSE>;
    const size_t smem = Geom<D>::kSmemBytes;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(smem));
    if (err != cudaSuccess)
        return err;
    const int sms = current_sm_count();
    err = launch_pdl(kernel, dim3(static_cast<unsigned>(items < sms ? items : sms)), dim3(kThreads), smem,
                     stream, tq, tk, tv, a);
    if (err != cudaSuccess || l.n_split == 1)
        return err;
    const long long rows = static_cast<long long>(l.num_tokens) * l.q_heads;
    return launch_pdl(cross_merge_kernel<D>, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0,
                      stream, l.out, l.out_f32 ? 1 : 0, l.lse, static_cast<const float *>(l.part_o),
                      static_cast<const float *>(l.part_lse), l.q_indptr, l.num_sources, l.num_tokens,
                      l.q_heads, l.n_split);
}

}  // namespace

cudaError_t launch_cross(const CrossLaunch &l, const CUtensorMap &tmap_q, const CUtensorMap &tmap_k,
                         const CUtensorMap &tmap_v, cudaStream_t stream)
{
    if (l.head_dim == 128)
        return l.lse ? launch_t<128, true>(l, tmap_q, tmap_k, tmap_v, stream)
                     : launch_t<128, false>(l, tmap_q, tmap_k, tmap_v, stream);
    return l.lse ? launch_t<64, true>(l, tmap_q, tmap_k, tmap_v, stream)
                 : launch_t<64, false>(l, tmap_q, tmap_k, tmap_v, stream);
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
