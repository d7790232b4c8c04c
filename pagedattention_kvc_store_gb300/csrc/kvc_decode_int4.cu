// kvc_decode_int4.cu -- paged decode attention over 4-bit pages.
//
// What it computes: kvc_decode's attention over pages whose vectors are held as groups of 64
// 4-bit codes with a scale and a minimum (kvc_store_int4.cu): K[p] = s u + lo per group.  Nothing
// is dequantised.  With u the codes,
//   score = sum_g s_g (q_g . u_g) + lo_g sum(q_g),   out = sum_p (p s_g) u + sum_p p lo_g,
// so the tensor cores multiply codes, and scale and minimum enter once per (position, group).
//
// Codes as operands.  A word's eight nibbles become four fp16 pairs with one AND each (and one
// shift): the bits of a nibble alone are the fp16 subnormal u 2^-24 (u 2^-20 for the high nibble
// of a byte), which the tensor cores take exactly; no bias has to be added or taken out.  For
// K the two weights are evened out in the query (the dims in low nibbles carry 16 q); V's rows
// accumulate whole bytes (low + 16 high, also an exact subnormal) and high nibbles, and the low
// ones are their difference at the end.  Putting the nibble under an exponent and subtracting
// the bias would double the conversion.  Query rows
// enter as fp16 scaled by a power of two of their own (largest |q| in [2^9, 2^10), so bf16's
// eight bits are exact wherever they matter); probabilities times value scales as fp16 scaled by a
// power of two that follows the largest value scale seen (vnorm), because a scale may have any
// exponent of bf16: rounding errors stay at 2^-11 of each product.  Sums, maxima, the minimum's
// part of both products and the accumulators are fp32.
//
// Work.  Every warp works alone: for each kv head the positions of all sequences, in 32-position
// blocks (sequence-major), are cut into runs of equal cost, one per warp (kv head fastest, so the
// warps of a CTA read the kv heads of the same positions, whose rows are neighbours in NHD pages).
// A warp streams its run through a ring of its own in shared memory, filled with 16-byte cp.async
// two blocks ahead, across the ends of sequences; there is no barrier wider than a warp after
// the set-up.  TMA boxes were not taken: with rows of 64 bytes a box moves half of what it
// moves with 128 and the per-page boxes (1 KB) would be its limit.  A piece (the blocks of one
// sequence in a run) that is all of its sequence writes the output rows, the others a partial,
// merged by a second launch.
//
// Products.  S^T = K Q^T and O^T += V^T P'^T on mma.sync m16n8k16 (16 positions, or dims, by the
// query heads of the group padded to 8: too thin for tcgen05's 128-row tiles).  The contraction
// order is free in both: thread (r, t) = (lane / 4, lane % 4) takes 8 t .. 8 t + 7 of each half of
// K's row bytes, and V's transposing 8-bit ldmatrix hands thread (r, t) the bytes of positions
// 4 t .. 4 t + 3, so contraction index k is position 4 ((k % 8) / 2) + 2 (k % 2) + k / 8 and score
// rows r and r + 8 are positions 2 r and 2 r + 1.
#include <math.h>

#include "kvc_device.cuh"
#include "kvc_launch.h"

namespace kvc {

namespace {

__device__ uint32_t g_decode_int4_errors;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kBlock = kInt4Block;   // positions of one ring stage
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
// The running maximum may lag the true one by this much (log2): probabilities reach 2^4, and
// most blocks skip the reduction over the warp and the rescale.
constexpr float kLagLog2 = 4.0f;
constexpr float kMaxScaled = 2048.0f;   // largest value scale times vnorm: 2^4 * 2^11 < 65504

// Cost of a block and of a piece's start in the cut of the runs.
constexpr long long kBlockCost = 16;
constexpr long long kPieceCost = 16;

// Scratch of the cut (64-bit words): the warps' block sums, four arrays of up to kWarps + 1 bounds,
// and the total cost and run count.
constexpr int kScratchCost = kWarps + 4 * (kWarps + 1);
constexpr int kScratchWords = kScratchCost + 2 + (kScratchCost & 1);

template <int D>
struct I4Geom {
    static constexpr int kRow = D / 2;            // code bytes of a vector
    static constexpr int kChunks = kRow / 16;     // 16-byte chunks of a row
    static constexpr int kGroups = D / 64;
    static constexpr int kStages = D == 128 ? 3 : 4;
    static constexpr int kHalfCodes = 16 * kRow;  // codes of 16 positions
    static constexpr int kOffV = 2 * kHalfCodes;
    static constexpr int kOffKp = 2 * kOffV;      // parameters: 4 bytes a position and group
    static constexpr int kParBytes = kBlock * kGroups * 4;
    static constexpr int kOffVp = kOffKp + kParBytes;
    static constexpr int kStageBytes = kOffVp + kParBytes;
    static constexpr int kWarpBytes = kStages * kStageBytes;
    static constexpr int kMetaBytes = kWarps * kStages * 16;
    static constexpr int kScratchBytes = kScratchWords * 8;
    static constexpr size_t kSmemBytes = kWarps * kWarpBytes + kMetaBytes + kScratchBytes;
    static_assert(kStageBytes % 128 == 0, "stages keep the bank phase of their rows");
};

struct Args {
    const __nv_bfloat16 *q;
    const uint8_t *k_codes, *v_codes, *k_params, *v_params;
    void *out;
    int out_f32;
    float *part_o;      // [slots][G][D], rows normalised by their own sum
    float *part_lse;    // [slots][G], natural log
    int2 *unit_info;    // [S][Hkv]: first slot and piece count of each non-empty unit
    int runs;           // runs per kv head
    const int32_t *block_table;
    int bt_stride;
    const int32_t *context_lens;
    int num_seqs, q_heads, kv_heads, group, log2_page, num_pages;
    int per_unit;       // 1: run = sequence, no partials
    int hnd;
    float scale_log2;
    uint32_t *err;
};

__device__ __forceinline__ uint32_t *err_word(const Args &a)
{
    return a.err ? a.err : &g_decode_int4_errors;
}

// A sequence's context, held to [0, bt_stride * P] (a longer one is flagged where the runs are
// cut and attends over the positions its block-table row holds).
__device__ __forceinline__ int clamped_ctx(const Args &a, int s, bool *over = nullptr)
{
    const int raw = a.context_lens[s];
    const long long cap = static_cast<long long>(a.bt_stride) << a.log2_page;
    if (over)
        *over = raw > cap;
    return raw > cap ? static_cast<int>(cap) : max(raw, 0);
}

__device__ __forceinline__ int blocks_of(int ctx) { return (ctx + kBlock - 1) / kBlock; }

// floor((x y + add) / d), add in {0, -1}, for quotients below 2^63: 64-bit where the product fits
// (every practical size), else 128-bit (a long software routine).
__device__ __forceinline__ long long mul_div(unsigned long long x, unsigned long long y, int add,
                                             unsigned long long d)
{
    if (__umul64hi(x, y) == 0 && x * y >= static_cast<unsigned long long>(-add))
        return static_cast<long long>((x * y + add) / d);
    const unsigned __int128 num = static_cast<unsigned __int128>(x) * y + add;
    return static_cast<long long>(static_cast<unsigned __int128>(num / d));
}

// Block g of sequence s sits at cost kBlockCost g + kPieceCost (s + 1), increasing along a kv
// head's block order; run c of n holds the blocks at costs [floor(c C / n), floor((c + 1) C / n))
// of the total C.
__device__ __forceinline__ long long block_cost(long long g, int s)
{
    return kBlockCost * g + kPieceCost * (s + 1);
}

__device__ __forceinline__ long long run_start(long long c, long long cost, long long n)
{
    return mul_div(c, cost, 0, n);
}

// The run that holds cost position x: the largest c with run_start(c) <= x.
__device__ __forceinline__ long long run_of(long long x, long long cost, long long n)
{
    return mul_div(x + 1, n, -1, cost);
}

// Where 16-byte chunk c of a 16-position half's row (position) `row` lies: even positions in slots
// 0 .. 7, odd ones in 8 .. 15, chunks turned so that both the K reads (8 bytes of rows 2 r for
// eight consecutive r) and ldmatrix (one chunk of 8 consecutive rows) touch every bank once.
template <int D>
__device__ __forceinline__ int half_offset(int row, int c)
{
    const int slot = (row >> 1) + ((row & 1) << 3);
    if (D == 128) {
        const int line = slot >> 1;
        return slot * 64 + ((c ^ (((line & 1) << 1) | (line >> 2))) << 4);
    }
    return slot * 32 + ((c ^ (slot >> 3)) << 4);
}

// 16 bytes global -> shared, of which the first `bytes` are read and the rest become zero.
__device__ __forceinline__ void copy_async16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// What the issuing side of a warp leaves for the computing side, per stage.
constexpr int kFirst = 1, kLast = 2, kWhole = 4;
struct __align__(16) Meta {
    int s, n_valid, flags, unused;
};

// Where a warp fetches next in its kv head's block order.
struct Cursor {
    int s, blk, nb, ctx;
    int left;              // blocks of the run not yet fetched
    int pbase;             // first page (index in the sequence) of the window below
    int page, page_next;   // this lane's page ids of the window and of the one after it
    bool fresh;            // the next block starts a piece
    bool from_start;       // the piece began at the sequence's first block
};

// What a lane's copies have in common, block after block.
struct LaneCopies {
    const uint8_t *k_row;      // K codes of its first row in page 0 (V: v_delta bytes on)
    long long v_delta;
    uint32_t row_bytes, page_bytes;   // from a position to the next, from a page to the next
    const uint8_t *par;        // its parameters in page 0 (K for low lanes, V for high ones)
    uint32_t par_page_bytes;
    uint32_t dst0, dst1, dst_par;     // places in a stage (dst1: the row after, D = 128)
    int row, par_half, par_pos;       // its first row and its parameters' half and first position
};

// Loads sequence c.s (passing by empty ones) and the page ids from block c.blk on; false when no
// sequence is left (the contexts changed under the launch).
__device__ __forceinline__ bool open_sequence(Cursor &c, const Args &a, int lane)
{
    for (; c.s < a.num_seqs; ++c.s) {
        c.ctx = clamped_ctx(a, c.s);
        c.nb = blocks_of(c.ctx);
        if (c.blk < c.nb)
            break;
        c.blk = 0;
    }
    if (c.s >= a.num_seqs)
        return false;
    const int32_t *row = a.block_table + static_cast<size_t>(c.s) * a.bt_stride;
    const int pages = (c.ctx + (1 << a.log2_page) - 1) >> a.log2_page;
    c.pbase = (c.blk * kBlock) >> a.log2_page;
    c.page = c.pbase + lane < pages ? row[c.pbase + lane] : 0;
    c.page_next = c.pbase + 32 + lane < pages ? row[c.pbase + 32 + lane] : 0;
    c.fresh = true;
    c.from_start = c.blk == 0;
    return true;
}

// Fetches the cursor's block into a stage and moves the cursor on.  Rows past the context become
// zeros (read from no memory); a page id outside the pool is flagged and reads as zeros.
template <int D>
__device__ __forceinline__ void fetch_block(Cursor &c, const Args &a, const LaneCopies &l,
                                            uint32_t stage, Meta *meta, int lane)
{
    using Geom = I4Geom<D>;
    const int pos = c.blk * kBlock;
    const int n_valid = min(kBlock, c.ctx - pos);
    int pi = pos >> a.log2_page;
    if (pi >= c.pbase + 32) {   // 32 pages hold whole blocks: a block's pages share a window
        c.pbase += 32;
        c.page = c.page_next;
        const int pages = (c.ctx + (1 << a.log2_page) - 1) >> a.log2_page;
        const int32_t *row = a.block_table + static_cast<size_t>(c.s) * a.bt_stride;
        c.page_next = c.pbase + 32 + lane < pages ? row[c.pbase + 32 + lane] : 0;
    }
    pi -= c.pbase;
    uint32_t page[2], off[2];
    page[0] = __shfl_sync(0xffffffffu, c.page, pi);
    page[1] = __shfl_sync(0xffffffffu, c.page, (pi + (16 >> a.log2_page)) & 31);
    off[0] = pos & ((1 << a.log2_page) - 1);
    off[1] = (pos + 16) & ((1 << a.log2_page) - 1);
    int live[2] = {n_valid, n_valid - 16};   // valid rows of each half
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (page[h] >= static_cast<uint32_t>(a.num_pages)) {
            if (lane == 0 && live[h] > 0)
                atomicOr(err_word(a), kErrPageRange);
            page[h] = 0;
            live[h] = 0;
        }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint8_t *k = l.k_row + static_cast<unsigned long long>(page[h]) * l.page_bytes +
                           off[h] * l.row_bytes;
        const int b0 = l.row < live[h] ? 16 : 0;
        const uint32_t d0 = stage + l.dst0 + h * Geom::kHalfCodes;
        copy_async16(d0, k, b0);
        copy_async16(d0 + Geom::kOffV, k + l.v_delta, b0);
        if (D == 128) {   // four lanes a row: the next row too
            const int b1 = l.row + 1 < live[h] ? 16 : 0;
            const uint32_t d1 = stage + l.dst1 + h * Geom::kHalfCodes;
            k += l.row_bytes;
            copy_async16(d1, k, b1);
            copy_async16(d1 + Geom::kOffV, k + l.v_delta, b1);
        }
    }
    // parameters: 16 bytes a lane
    if (D == 128 || lane < 16) {
        const uint32_t pg = l.par_half ? page[1] : page[0], of = l.par_half ? off[1] : off[0];
        const int lv = l.par_half ? live[1] : live[0];
        constexpr int kPer = 4 * Geom::kGroups;   // bytes of a position
        const int bytes = max(0, min(16, (lv - l.par_pos) * kPer));
        copy_async16(stage + l.dst_par,
                     l.par + static_cast<unsigned long long>(pg) * l.par_page_bytes + of * kPer,
                     bytes);
    }
    ++c.blk;
    --c.left;
    const bool last = c.blk == c.nb || c.left == 0;
    if (lane == 0) {
        const int flags = (c.fresh ? kFirst : 0) | (last ? kLast : 0) |
                          (c.from_start && c.blk == c.nb ? kWhole : 0);
        *reinterpret_cast<int4 *>(meta) = make_int4(c.s, n_valid, flags, 0);
    }
    c.fresh = false;
    if (last && c.left > 0) {
        ++c.s;
        c.blk = 0;
        if (!open_sequence(c, a, lane))
            c.left = 0;
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) paged_decode_int4_kernel(const Args a)
{
    pdl_wait();
    pdl_trigger();
    using Geom = I4Geom<D>;
    constexpr int NG = Geom::kGroups;     // groups of a vector
    constexpr int NC = Geom::kChunks;     // 16-byte chunks of a row: 32 dims each
    constexpr int NS = Geom::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int G = a.group;
    const int Hkv = a.kv_heads;
    uint8_t *ring = smem + warp * Geom::kWarpBytes;
    Meta *metas = reinterpret_cast<Meta *>(smem + kWarps * Geom::kWarpBytes) + warp * NS;
    long long *scratch =
        reinterpret_cast<long long *>(smem + kWarps * Geom::kWarpBytes + Geom::kMetaBytes);

    // ---- this warp's run: kv head kvh, blocks [g0, g1) of its order, beginning in sequence s0 ----
    const int gw = blockIdx.x * kWarps + warp;
    const int kvh = gw % Hkv;
    const int run = gw / Hkv;
    Cursor c;
    int run_len = 0;   // (a run's blocks: far below 2^31 for tables that fit the memory)
    const long long *bound_end = nullptr;   // the index of the first block past the run
    if (a.per_unit) {
        if (run >= a.num_seqs)
            return;
        bool over;
        c.ctx = clamped_ctx(a, run, &over);
        if (over && lane == 0 && kvh == 0)
            atomicOr(err_word(a), kErrContextRange);
        if (c.ctx == 0) {   // no positions: the rows are 0
            const size_t row0 = static_cast<size_t>(run) * a.q_heads + static_cast<size_t>(kvh) * G;
            for (int i = lane; i < G * D; i += 32)
                store_out(a.out, a.out_f32, row0 * D + i, 0.0f);
            return;
        }
        c.s = run;
        c.blk = 0;
        run_len = blocks_of(c.ctx);
    } else {
        // Prefix sums of the sequences' blocks over the CTA; then the bounds of the few runs this
        // CTA's warps have, each found by the thread whose sequences hold it.
        const int S = a.num_seqs;
        const int per = (S + kThreads - 1) / kThreads;
        const int lo = min(S, static_cast<int>(threadIdx.x) * per);
        const int hi = min(S, lo + per);
        long long mine = 0;
        for (int s = lo; s < hi; ++s) {
            bool over;
            mine += blocks_of(clamped_ctx(a, s, &over));
            if (over && blockIdx.x == 0)
                atomicOr(err_word(a), kErrContextRange);
        }
        long long incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off)
                incl += v;
        }
        if (lane == 31)
            scratch[warp] = incl;
        __syncthreads();
        long long acc = incl - mine, total = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            const long long t = scratch[i];
            if (i < warp)
                acc += t;
            total += t;
        }
        const long long n_runs = min(static_cast<long long>(a.runs), total);
        const long long cost = kBlockCost * total + kPieceCost * S;
        const int run_lo = blockIdx.x * kWarps / Hkv;
        const int n_bounds = (blockIdx.x * kWarps + kWarps - 1) / Hkv - run_lo + 2;   // 2 .. 9
        long long *bound_cost = scratch + kWarps;            // [9]
        long long *bound_g = bound_cost + kWarps + 1;        // [9] first block at or past it
        long long *bound_s = bound_g + kWarps + 1;           // [9] its sequence
        long long *bound_blk = bound_s + kWarps + 1;         // [9] and its block in the sequence
        // (cost and n_runs are taken up again after the loop: scratch[kScratchCost], + 1)
        if (total == 0)
            return;   // every row is written by the merge
        if (threadIdx.x == kThreads - 1) {
            scratch[kScratchCost] = cost;
            scratch[kScratchCost + 1] = n_runs;
        }
        if (threadIdx.x < n_bounds) {
            const long long b = run_lo + static_cast<long long>(threadIdx.x);
            bound_cost[threadIdx.x] = b < n_runs ? run_start(b, cost, n_runs) : cost;
            bound_g[threadIdx.x] = total;   // what the end of the last run stays at
            bound_s[threadIdx.x] = S;
            bound_blk[threadIdx.x] = 0;
        }
        __syncthreads();
        for (int s = lo; s < hi; ++s) {
            // sequence s covers the costs [kPieceCost s + kBlockCost B, kPieceCost (s + 1) +
            // kBlockCost (B + nb)), B blocks before it: they tile [0, cost)
            const long long nb = blocks_of(clamped_ctx(a, s));
            const long long first = block_cost(acc, s);
            for (int i = 0; i < n_bounds; ++i) {
                const long long x = bound_cost[i];
                if (x >= first - kPieceCost && x < first + kBlockCost * nb) {
                    const long long off =
                        min(nb, max(0LL, (x - first + kBlockCost - 1) / kBlockCost));
                    bound_g[i] = acc + off;
                    bound_s[i] = off < nb ? s : s + 1;
                    bound_blk[i] = off < nb ? off : 0;
                }
            }
            acc += nb;
        }
        __syncthreads();
        const int i = run - run_lo;
        run_len = static_cast<int>(bound_g[i + 1] - bound_g[i]);
        if (run >= n_runs || run_len <= 0)
            return;
        c.s = static_cast<int>(bound_s[i]);
        c.blk = static_cast<int>(bound_blk[i]);
        bound_end = &bound_g[i + 1];
    }
    c.left = run_len;
    if (!open_sequence(c, a, lane))
        return;

    LaneCopies l;
    {
        constexpr int kRow = Geom::kRow;
        const int P = 1 << a.log2_page;
        const int chunk = lane & (NC - 1);
        l.row = NC == 4 ? 2 * (lane >> 2) : 2 * ((lane >> 1) & 7) + (lane >> 4);
        l.row_bytes = a.hnd ? kRow : Hkv * kRow;
        l.page_bytes = static_cast<uint32_t>(P) * Hkv * kRow;
        l.k_row = a.k_codes + static_cast<size_t>(kvh) * (a.hnd ? P * kRow : kRow) +
                  static_cast<size_t>(l.row) * l.row_bytes + chunk * 16;
        l.v_delta = a.v_codes - a.k_codes;
        l.dst0 = half_offset<D>(l.row, chunk);
        l.dst1 = half_offset<D>(l.row + 1, chunk);
        // 4 NG lanes hold the 16 positions of one half of one tensor, 4 / NG positions each
        const bool is_v = lane >= 8 * NG;
        l.par_half = (lane / (4 * NG)) & 1;
        const int c16 = lane % (4 * NG);
        l.par_pos = c16 * (4 / NG);
        l.par_page_bytes = static_cast<uint32_t>(Hkv) * P * NG * 4;
        l.par = (is_v ? a.v_params : a.k_params) + static_cast<size_t>(kvh) * P * NG * 4 + c16 * 16;
        l.dst_par = (is_v ? Geom::kOffVp : Geom::kOffKp) + (l.par_half * 4 * NG + c16) * 16;
    }

    // ---- the first blocks on their way ----
    const uint32_t ring32 = smem_addr(ring);
    int fetched = 0;   // stage of the next fetch
    int pending = 0;   // blocks fetched and not yet computed
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) {
        if (c.left > 0) {
            fetch_block<D>(c, a, l, ring32 + fetched * Geom::kStageBytes, &metas[fetched], lane);
            ++pending;
        }
        copy_commit();
        fetched = fetched + 1 == NS ? 0 : fetched + 1;
    }
    __syncwarp();

    const int r = lane >> 2;
    const int t = lane & 3;
    // K: the 8 bytes of group 0 that this thread reads of position 2 r (group 1: 32 bytes on, a
    // turn of the chunk) and of position 2 r + 1; V: this lane's row of the transposing loads
    const int k_off[2] = {half_offset<D>(2 * r, t >> 1) + (t & 1) * 8,
                          half_offset<D>(2 * r + 1, t >> 1) + (t & 1) * 8};
    const int v_off = half_offset<D>(lane & 15, lane >> 4);

    uint32_t qb[NG][2][2][2];   // B fragments: [group][word][nibble][register]
    float o[NC][2][4];          // O^T: [32 dims][whole byte, high half][fragment]
    float zacc[NG][2];          // sum of p lo, heads 2 t and 2 t + 1
    float m_run[2], l_run[2], m_thr[2], mf[2], f[2], hq[NG][2];
    float vnorm = 1.0f, v_thr = 0.0f;
    int stage = 0;

    for (; pending > 0; --pending) {
        const int4 mt = *reinterpret_cast<const int4 *>(&metas[stage]);
        const int s = mt.x, n_valid = mt.y, flags = mt.z;
        const size_t row0 = static_cast<size_t>(s) * a.q_heads + static_cast<size_t>(kvh) * G;
        uint4 qw[NG][2];
        if (flags & kFirst) {   // the query rows travel with the block's last bytes
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    a.q + (row0 + (r < G ? r : 0)) * D + 64 * g + 16 * t);
                qw[g][0] = src[0];
                qw[g][1] = src[1];
            }
        }
        copy_wait<NS - 2>();
        __syncwarp();
        if (c.left > 0) {
            fetch_block<D>(c, a, l, ring32 + fetched * Geom::kStageBytes, &metas[fetched], lane);
            ++pending;
        }
        copy_commit();
        fetched = fetched + 1 == NS ? 0 : fetched + 1;

        if (flags & kFirst) {
            float qv[NG][16], qmax = 0.0f, qsum[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                qsum[g] = 0.0f;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t w4[4] = {qw[g][j].x, qw[g][j].y, qw[g][j].z, qw[g][j].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x0 = r < G ? __uint_as_float(w4[e] << 16) : 0.0f;
                        const float x1 = r < G ? __uint_as_float(w4[e] & 0xFFFF0000u) : 0.0f;
                        qv[g][8 * j + 2 * e] = x0;
                        qv[g][8 * j + 2 * e + 1] = x1;
                        qsum[g] += x0 + x1;
                        qmax = fmaxf(qmax, fmaxf(fabsf(x0), fabsf(x1)));
                    }
                }
            }
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) {
                qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, off));
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    qsum[g] += __shfl_xor_sync(0xffffffffu, qsum[g], off);
            }
            // q 2^(9 - e), e the exponent of the row's largest |q| (held to [-100, 100])
            const int e = min(100, max(-100, static_cast<int>(__float_as_uint(qmax) >> 23) - 127));
            const float up = __uint_as_float(static_cast<uint32_t>(127 + 9 - e) << 23);
            const float down = __uint_as_float(static_cast<uint32_t>(127 - 9 + e) << 23);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float *v = &qv[g][8 * j];
                    const float up16 = up * 16.0f;
                    qb[g][j][0][0] = pack_f16x2(v[0] * up16, v[4] * up16);
                    qb[g][j][0][1] = pack_f16x2(v[2] * up16, v[6] * up16);
                    qb[g][j][1][0] = pack_f16x2(v[1] * up, v[5] * up);
                    qb[g][j][1][1] = pack_f16x2(v[3] * up, v[7] * up);
                }
            }
            // Scores are kept as y = sum_g s_g acc_g + lo_g h_g with log2 score = f y: acc is
            // q u 2^(9 - e - 20), so f = scale log2(e) 2^(11 + e) and h = sum(q_g) 2^-(11 + e)
            const float h_scale = up * 9.5367431640625e-07f;   // 2^(9 - e) 2^-20
#pragma unroll
            for (int j = 0; j < 2; ++j) {   // heads 2 t and 2 t + 1
                const int src = (2 * t + j) * 4;
                f[j] = __shfl_sync(0xffffffffu, down, src) * 1048576.0f * a.scale_log2;
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    hq[g][j] = __shfl_sync(0xffffffffu, qsum[g] * h_scale, src);
                m_run[j] = m_thr[j] = -INFINITY;
                mf[j] = 0.0f;
                l_run[j] = 0.0f;
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    zacc[g][j] = 0.0f;
            }
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    o[n][b][0] = o[n][b][1] = o[n][b][2] = o[n][b][3] = 0.0f;
            vnorm = 1.0f;
            v_thr = 0.0f;   // any positive value scale sets vnorm
        }

        const uint8_t *st = ring + stage * Geom::kStageBytes;
        // parameters of this thread's positions: 16 T + 2 r and 16 T + 2 r + 1
        uint32_t kp[2][2][NG], vp[2][2][NG];
#pragma unroll
        for (int T = 0; T < 2; ++T) {
            const uint8_t *kpp = st + Geom::kOffKp + (16 * T + 2 * r) * NG * 4;
            const uint8_t *vpp = st + Geom::kOffVp + (16 * T + 2 * r) * NG * 4;
            if constexpr (NG == 2) {
                const uint4 x = *reinterpret_cast<const uint4 *>(kpp);
                const uint4 y = *reinterpret_cast<const uint4 *>(vpp);
                kp[T][0][0] = x.x;
                kp[T][0][1] = x.y;
                kp[T][1][0] = x.z;
                kp[T][1][1] = x.w;
                vp[T][0][0] = y.x;
                vp[T][0][1] = y.y;
                vp[T][1][0] = y.z;
                vp[T][1][1] = y.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2 *>(kpp);
                const uint2 y = *reinterpret_cast<const uint2 *>(vpp);
                kp[T][0][0] = x.x;
                kp[T][1][0] = x.y;
                vp[T][0][0] = y.x;
                vp[T][1][0] = y.y;
            }
        }

        // ---- scores: y[T][position][head] ----
        float y[2][2][2];
#pragma unroll
        for (int T = 0; T < 2; ++T) {
            float acc[NG][4];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                acc[g][0] = acc[g][1] = acc[g][2] = acc[g][3] = 0.0f;
                const uint2 w0 = *reinterpret_cast<const uint2 *>(
                    st + T * Geom::kHalfCodes + (k_off[0] ^ (32 * g)));
                const uint2 w1 = *reinterpret_cast<const uint2 *>(
                    st + T * Geom::kHalfCodes + (k_off[1] ^ (32 * g)));
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t x0 = j ? w0.y : w0.x, x1 = j ? w1.y : w1.x;
                    const uint32_t z0 = x0 >> 8, z1 = x1 >> 8;
                    mma_f16_16816(acc[g], x0 & 0x000F000Fu, x1 & 0x000F000Fu, z0 & 0x000F000Fu,
                                  z1 & 0x000F000Fu, qb[g][j][0][0], qb[g][j][0][1]);
                    mma_f16_16816(acc[g], x0 & 0x00F000F0u, x1 & 0x00F000F0u, z0 & 0x00F000F0u,
                                  z1 & 0x00F000F0u, qb[g][j][1][0], qb[g][j][1][1]);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)   // position 2 r + i
#pragma unroll
                for (int j = 0; j < 2; ++j) {   // head 2 t + j
                    float v = 0.0f;
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        const float sc = __uint_as_float(kp[T][i][g] << 16);
                        const float lo = __uint_as_float(kp[T][i][g] & 0xFFFF0000u);
                        v = g == 0 ? sc * acc[g][2 * i + j] : fmaf(sc, acc[g][2 * i + j], v);
                        v = fmaf(lo, hq[g][j], v);
                    }
                    y[T][i][j] = v;
                }
        }
        if (n_valid < kBlock) {
#pragma unroll
            for (int T = 0; T < 2; ++T)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (16 * T + 2 * r + i >= n_valid)
                        y[T][i][0] = y[T][i][1] = -INFINITY;
        }

        // ---- running maxima, and the power of two on the value scales ----
        float mb[2], vmax = 0.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            mb[j] = fmaxf(fmax3(y[0][0][j], y[0][1][j], y[1][0][j]), y[1][1][j]);
#pragma unroll
        for (int T = 0; T < 2; ++T)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    vmax = fmaxf(vmax, __uint_as_float(vp[T][i][g] << 16));
        if (__any_sync(0xffffffffu, mb[0] > m_thr[0] || mb[1] > m_thr[1] || vmax > v_thr)) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                mb[0] = fmaxf(mb[0], __shfl_xor_sync(0xffffffffu, mb[0], off));
                mb[1] = fmaxf(mb[1], __shfl_xor_sync(0xffffffffu, mb[1], off));
                vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, off));
            }
            float fix[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float m_new = fmaxf(m_run[j], mb[j]);
                fix[j] = m_run[j] == -INFINITY ? 0.0f : fast_exp2((m_run[j] - m_new) * f[j]);
                l_run[j] *= fix[j];
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    zacc[g][j] *= fix[j];
                m_run[j] = m_new;
                m_thr[j] = m_new + kLagLog2 / f[j];
                mf[j] = m_new == -INFINITY ? 0.0f : m_new * f[j];
            }
            float turn = 1.0f;
            if (vmax > v_thr) {   // the same in every lane that shares the maximum: all of them
                // vnorm = 2^(10 - e) for the largest scale's exponent e: vmax vnorm in [2^10, 2^11)
                const int e = max(-100, static_cast<int>(__float_as_uint(vmax) >> 23) - 127);
                const float vn = __uint_as_float(static_cast<uint32_t>(127 + 10 - e) << 23);
                turn = v_thr > 0.0f ? vn / vnorm : 1.0f;   // unset: every code product was 0
                vnorm = vn;
                v_thr = kMaxScaled / vn;
            }
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    o[n][b][0] *= fix[0] * turn;
                    o[n][b][1] *= fix[1] * turn;
                    o[n][b][2] *= fix[0] * turn;
                    o[n][b][3] *= fix[1] * turn;
                }
        }

        // ---- probabilities, and out ----
#pragma unroll
        for (int T = 0; T < 2; ++T) {
            float p[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    p[i][j] = fast_exp2(fmaf(y[T][i][j], f[j], -mf[j]));
                    l_run[j] += p[i][j];
                }
            uint32_t pb[NG][2];   // B fragments of the PV product
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float sc = __uint_as_float(vp[T][i][g] << 16) * vnorm;
                    const float lo = __uint_as_float(vp[T][i][g] & 0xFFFF0000u);
                    zacc[g][0] = fmaf(p[i][0], lo, zacc[g][0]);
                    zacc[g][1] = fmaf(p[i][1], lo, zacc[g][1]);
                    pb[g][i] = movmatrix_trans(pack_f16x2(p[i][0] * sc, p[i][1] * sc));
                }
            const uint32_t vb = ring32 + stage * Geom::kStageBytes + Geom::kOffV +
                                T * Geom::kHalfCodes;
#pragma unroll
            for (int g = 0; g < NG; ++g) {   // chunks 2 g and 2 g + 1
                uint32_t e[4];
                ldsm_x2_trans_b8(vb + (v_off ^ (32 * g)), e[0], e[1], e[2], e[3]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    // whole bytes (low + 16 high) and their high halves: one operation a pair
                    // each, where the low halves would also need the shift
                    const uint32_t x0 = e[2 * k], x1 = e[2 * k + 1];
                    const uint32_t z0 = __byte_perm(x0, 0u, 0x4341u);   // bytes 1 and 3
                    const uint32_t z1 = __byte_perm(x1, 0u, 0x4341u);
                    mma_f16_16816(o[2 * g + k][0], x0 & 0x00FF00FFu, x1 & 0x00FF00FFu, z0, z1,
                                  pb[g][0], pb[g][1]);
                    mma_f16_16816(o[2 * g + k][1], x0 & 0x00F000F0u, x1 & 0x00F000F0u,
                                  z0 & 0x00F000F0u, z1 & 0x00F000F0u, pb[g][0], pb[g][1]);
                }
            }
        }

        // ---- the end of a piece: normalised rows to the output or to the piece's slot ----
        if (flags & kLast) {
            float inv[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    l_run[j] += __shfl_xor_sync(0xffffffffu, l_run[j], off);
#pragma unroll
                    for (int g = 0; g < NG; ++g)
                        zacc[g][j] += __shfl_xor_sync(0xffffffffu, zacc[g][j], off);
                }
                inv[j] = 1.0f / l_run[j];   // the piece holds a position: the sum is at least 1
            }
            const bool whole = flags & kWhole;
            if (whole && !a.per_unit && lane == 0)   // the merge has nothing to do for it
                a.unit_info[static_cast<size_t>(s) * Hkv + kvh] = make_int2(0, 1);
            // pieces of kv head h own slots [h (S + R), (h + 1) (S + R)), piece (s, run) s + run
            // there: distinct for every piece, consecutive for one unit's
            const int slot = kvh * (a.num_seqs + a.runs) + s + run;
            const float v_inv = 1.0f / vnorm;   // a power of two: exact
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int head = 2 * t + j;
                if (head < G) {
#pragma unroll
                    for (int n = 0; n < NC; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {   // dims 32 n + 16 i + 2 r, + 1
                            const float z = zacc[n / 2][j];
                            float2 v;
                            const float whole_byte = o[n][0][2 * i + j], high = o[n][1][2 * i + j];
                            v.x = fmaf((whole_byte - high) * 16777216.0f, v_inv, z) * inv[j];
                            v.y = fmaf(high * 1048576.0f, v_inv, z) * inv[j];
                            const int dim = 32 * n + 16 * i + 2 * r;
                            if (whole)
                                store_out2(a.out, a.out_f32, (row0 + head) * D + dim, v);
                            else
                                *reinterpret_cast<float2 *>(
                                    a.part_o + (static_cast<size_t>(slot) * G + head) * D + dim) = v;
                        }
                    if (!whole && r == 0)
                        a.part_lse[static_cast<size_t>(slot) * G + head] =
                            (mf[j] + log2f(l_run[j])) * kLn2;
                }
            }
        }
        stage = stage + 1 == NS ? 0 : stage + 1;
    }
    copy_wait<0>();
    // A unit that begins in this run and goes on past it (only the run's last piece can): where its
    // pieces' slots begin, and the run that holds its last block.
    if (bound_end != nullptr && lane == 0 && c.from_start && c.blk < c.nb) {
        const long long g_last = *bound_end - 1 + (c.nb - c.blk);
        const long long last = run_of(block_cost(g_last, c.s), scratch[kScratchCost],
                                      scratch[kScratchCost + 1]);
        a.unit_info[static_cast<size_t>(c.s) * Hkv + kvh] = make_int2(
            kvh * (a.num_seqs + a.runs) + c.s + run, static_cast<int>(last - run + 1));
    }
}

// out[row] = sum_j exp(lse_j - M) o_j / sum_j exp(lse_j - M) over the pieces of the row's unit,
// W warps a row (8 where a unit has many pieces: few sequences, long contexts).  Rows whose unit is
// one whole piece were written by it; rows of a sequence with no positions are 0.
template <int D, int W>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W) merge_int4_kernel(const Args a)
{
    pdl_wait();
    pdl_trigger();
    constexpr int V = D / 32;
    constexpr int kRows = W == 1 ? 4 : 1;
    __shared__ float part[W == 1 ? 1 : W][D + 1];
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * kRows + (W == 1 ? warp : 0);
    if (row >= a.num_seqs * a.q_heads)
        return;
    const int s = row / a.q_heads;
    const int h = row - s * a.q_heads;
    const int G = a.group;
    const int kvh = h / G;
    const int ctx = clamped_ctx(a, s);
    float acc[V], sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
        acc[v] = 0.0f;
    if (ctx > 0) {
        const int2 info = __ldcg(a.unit_info + static_cast<size_t>(s) * a.kv_heads + kvh);
        const int count = info.y;
        if (count <= 1)
            return;
        const size_t first = static_cast<size_t>(info.x) * G + (h - kvh * G);
        const float *lse = a.part_lse + first;
        const float *po = a.part_o + first * D + lane * V;
        const size_t po_step = static_cast<size_t>(G) * D;
        float M = -INFINITY;
        for (int j = lane; j < count; j += 32)
            M = fmaxf(M, __ldcg(lse + static_cast<size_t>(j) * G));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        const float mu = M == -INFINITY ? 0.0f : M;
#pragma unroll 4
        for (int j = W == 1 ? 0 : warp; j < count; j += W) {
            const float w = fast_exp2((__ldcg(lse + static_cast<size_t>(j) * G) - mu) * kLog2e);
            sum += w;
            const float *src = po + static_cast<size_t>(j) * po_step;
#pragma unroll
            for (int v = 0; v < V; ++v)
                acc[v] = fmaf(w, __ldcg(src + v), acc[v]);
        }
    }
    if constexpr (W > 1) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            part[warp][lane * V + v] = acc[v];
        if (lane == 0)
            part[warp][D] = sum;
        __syncthreads();
        if (warp != 0)
            return;
        for (int w = 1; w < W; ++w) {
            sum += part[w][D];
#pragma unroll
            for (int v = 0; v < V; ++v)
                acc[v] += part[w][lane * V + v];
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const size_t base = static_cast<size_t>(row) * D + lane * V;
    if constexpr (V == 4)
        store_out4(a.out, a.out_f32, base,
                   make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv));
    else
        store_out2(a.out, a.out_f32, base, make_float2(acc[0] * inv, acc[1] * inv));
}

template <int D>
cudaError_t launch_t(const DecodeInt4Launch &l, cudaStream_t stream)
{
    Args a;
    a.q = static_cast<const __nv_bfloat16 *>(l.q);
    a.k_codes = static_cast<const uint8_t *>(l.pools.k_codes);
    a.v_codes = static_cast<const uint8_t *>(l.pools.v_codes);
    a.k_params = static_cast<const uint8_t *>(l.pools.k_params);
    a.v_params = static_cast<const uint8_t *>(l.pools.v_params);
    a.out = l.out;
    a.out_f32 = l.out_f32;
    a.part_o = l.part_o;
    a.part_lse = l.part_lse;
    a.unit_info = static_cast<int2 *>(l.unit_info);
    a.runs = l.per_unit ? l.num_seqs : l.runs;
    a.block_table = l.block_table;
    a.bt_stride = l.bt_stride;
    a.context_lens = l.context_lens;
    a.num_seqs = l.num_seqs;
    a.q_heads = l.q_heads;
    a.kv_heads = l.pools.kv_heads;
    a.group = l.q_heads / l.pools.kv_heads;
    a.log2_page = l.pools.page_size == 16 ? 4 : l.pools.page_size == 32 ? 5 : 6;
    a.num_pages = l.pools.num_pages;
    a.per_unit = l.per_unit ? 1 : 0;
    a.hnd = l.pools.hnd ? 1 : 0;
    a.scale_log2 = l.scale * kLog2e;
    a.err = current_error_word();
    constexpr size_t smem = I4Geom<D>::kSmemBytes;
    auto kernel = paged_decode_int4_kernel<D>;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(smem));
    if (err != cudaSuccess)
        return err;
    const long long warps = static_cast<long long>(a.runs) * a.kv_heads;
    const unsigned grid = static_cast<unsigned>((warps + kWarps - 1) / kWarps);
    err = launch_pdl(kernel, dim3(grid), dim3(kThreads), smem, stream, a);
    if (err != cudaSuccess || l.per_unit)
        return err;
    const int rows = l.num_seqs * l.q_heads;
    if (l.runs > 8LL * l.num_seqs)
        return launch_pdl(merge_int4_kernel<D, 8>, dim3(rows), dim3(256), 0, stream, a);
    return launch_pdl(merge_int4_kernel<D, 1>, dim3((rows + 3) / 4), dim3(128), 0, stream, a);
}

}  // namespace

cudaError_t launch_decode_int4(const DecodeInt4Launch &l, cudaStream_t stream)
{
    if (l.num_seqs == 0)
        return cudaSuccess;
    return l.pools.head_dim == 64 ? launch_t<64>(l, stream) : launch_t<128>(l, stream);
}

cudaError_t read_and_clear_decode_int4_errors(uint32_t *flags)
{
    uint32_t zero = 0;
    cudaError_t err = cudaMemcpyFromSymbol(flags, g_decode_int4_errors, sizeof(uint32_t));
    if (err != cudaSuccess)
        return err;
    return cudaMemcpyToSymbol(g_decode_int4_errors, &zero, sizeof(uint32_t));
}

}  // namespace kvc
