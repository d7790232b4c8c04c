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
// K the two weights are evened out in the query (the dims in low nibbles carry 16 q), for V at the
// end.  Putting the nibble under an exponent and subtracting the bias would double the conversion.
// Query rows enter as fp16 scaled by a power of two of their own (largest |q| in [2^9, 2^10), so bf16's
// eight bits are exact wherever they matter); probabilities times value scales as fp16 scaled by a
// power of two of each group of 64 dims that follows the group's largest value scale seen (vnorm),
// because a scale may have any exponent of bf16.  A product is rounded by at most 2^-11 of itself or,
// where it is an fp16 subnormal, by 2^-35 of that largest scale: a position whose scale is 2^24 below
// another one's of the same group loses bits, and so does one that weighs 2^-24 of the heaviest.  Sums,
// maxima, the minimum's part of both products and the accumulators are fp32.
//
// Work.  For each kv head the positions of all sequences, in 64-position blocks (sequence-major), are
// cut into runs of equal cost.  A group of warps, one per kv head (up to 8 heads, else the largest
// divisor of their number up to 8), works through a run in step: a block of all its heads is one
// stage of the group's ring in shared memory, and as many groups as fit 8 warps make a CTA (one per
// SM).  One producer warp fills the rings: four lanes keep a group's cursor, each issues the TMA
// boxes of one page (its codes and parameters for all heads of the group); page ids, and the next
// sequence's length and first ids, are requested blocks ahead.  A TMA operation costs the SM about 85 cycles
// whatever its size (1 and 2 KB boxes, one warp's heads apiece, took 84 us on the batched decode,
// and 16-byte cp.async by every warp 56: their addresses were a quarter of its instructions).
// Eight warps with 216 registers each, not 16 with 104: the products' operands and sums spill below
// about 200, and a warp has 64 positions' independent products to overlap (16 warps with 32-position
// stages: 61 us on the batched decode, 251 on the long one; 8 warps that the compiler held to 168
// registers 43.3 and 162; as it is 41.6 and 153).
// Consumer warps never wait for one another except through a stage's release.  A piece (the blocks
// of one sequence in a run) that is all of its sequence writes the output rows, the others a
// partial, merged by a second launch.
//
// Products.  S^T = K Q^T and O^T += V^T P'^T on mma.sync m16n8k16 (16 positions, or dims, by the
// query heads of the group padded to 8: too thin for tcgen05's 128-row tiles).  The contraction
// order is free in both: thread (r, t) = (lane / 4, lane % 4) takes 8 t .. 8 t + 7 of each half of
// K's row bytes, and V's transposing 8-bit ldmatrix hands thread (r, t) the bytes of positions
// 4 t .. 4 t + 3, so contraction index k is position 4 ((k % 8) / 2) + 2 (k % 2) + k / 8 and score
// rows r and r + 8 are positions 2 r and 2 r + 1.
//
// Bound: HBM, 2 (D / 2 + D / 16) bytes a position and kv head.  8 sequences of up to 131,072 positions
// (920 MB): 153 us, 6.0 TB/s, 89% of the measured copy.  64 sequences of up to 4,096 (172 MB): 41.6 us,
// of which 26 are streaming; the rest is the start (the cut of the runs, page ids and the first copies
// one after the other, 5 us), runs that end apart, and the merge's launch.
#include <math.h>

#include "kvc_device.cuh"
#include "kvc_launch.h"

namespace kvc {

namespace {

__device__ uint32_t g_decode_int4_errors;

constexpr int kWarps = kInt4Warps;   // consumer warps
// ... and the producer's, in a warpgroup of its own: three of four have nothing to do, but registers move
// between whole warpgroups.  A block is launched with 168 a thread (an SM quarter's 16,384 hold three
// warps of up to 170); the producer's four warps keep 72 of them and the consumers get 216:
// 128 * 72 + 256 * 216 = 384 * 168.
constexpr int kThreads = (kWarps + 4) * 32;
constexpr int kProducerRegs = 72, kConsumerRegs = 216;
static_assert(128 * kProducerRegs + kWarps * 32 * kConsumerRegs <= kThreads * 168, "registers");
constexpr int kBlock = kInt4Block;   // positions of one ring stage
constexpr int kTiles = kBlock / 16;  // of 16 positions, the rows of a product
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
// The running maximum may lag the true one by this much (log2): probabilities reach 2^4, and
// most blocks skip the reduction over the warp and the rescale.
constexpr float kLagLog2 = 4.0f;
constexpr float kMaxScaled = 2048.0f;   // largest value scale times vnorm: 2^4 * 2^11 < 65504

// Cost of a block and of a piece's start in the cut of the runs (a start as 12 or 16: 41.6 us on the
// batched decode, as 8 or 24 42.4, as 4 or 32 42.7 and 43.2).
constexpr long long kBlockCost = 16;
constexpr long long kPieceCost = 16;

// Scratch of the cut (64-bit words): the warps' block sums, four arrays of up to kWarps + 1 bounds.
constexpr int kBlockWarps = kThreads / 32;
constexpr int kScratchWords = kBlockWarps + 4 * (kWarps + 1);

template <int D>
struct I4Geom {
    static constexpr int kRow = D / 2;            // code bytes of a vector
    static constexpr int kChunks = kRow / 16;     // 16-byte chunks of a row
    static constexpr int kGroups = D / 64;
    static constexpr int kStages = D == 128 ? 3 : 5;
    static constexpr int kTileCodes = 16 * kRow;  // codes of 16 positions
    static constexpr int kTilePar = 16 * kGroups * 4;
    static constexpr int kOffV = kTiles * kTileCodes;
    static constexpr int kOffKp = 2 * kOffV;      // parameters
    // per head and tensor, 4 bytes a position and group; up to twice that is used at D = 64, where
    // an odd number of heads' 64 bytes is padded to the 128 that a TMA destination is aligned to
    static constexpr int kParBytes = 512;
    static constexpr int kOffVp = kOffKp + kParBytes;
    static constexpr int kStageBytes = kOffVp + kParBytes;   // of one head; a group's stage holds
                                                             // K codes of all heads, V codes, ...
    static constexpr int kOffMeta = kWarps * kStages * kStageBytes;
    static constexpr int kOffBar = kOffMeta + kWarps * kStages * 16;   // full, empty
    static constexpr int kOffScratch = kOffBar + 2 * kWarps * kStages * 8;
    static constexpr size_t kSmemBytes = 1024 + kOffScratch + kScratchWords * 8;
    static_assert(kStageBytes % (8 * kRow) == 0, "stages keep the phase of the swizzle");
    // bytes from one page's parameters of `heads` heads to the next one's, `box` positions a page
    static __host__ __device__ constexpr int page_par(int heads, int box)
    {
        return (heads * box * kGroups * 4 + 127) & ~127;
    }
    static_assert(4 * page_par(1, 16) <= kParBytes && 4 * page_par(3, 16) <= 3 * kParBytes &&
                      4 * page_par(5, 16) <= 5 * kParBytes && 4 * page_par(7, 16) <= 7 * kParBytes &&
                      4 * page_par(8, 16) <= 8 * kParBytes,
                  "four pages' parameters");
    static_assert(kSmemBytes <= 232448, "shared memory");
};

struct Args {
    const __nv_bfloat16 *q;
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
    int heads;          // kv heads (warps) of a group of warps
    int groups;         // groups of a CTA
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

// Where 16-byte chunk c of stage row `row` lies: rows of 64 bytes under the TMA's 64-byte swizzle
// (chunk c of row r at c ^ (r / 2) % 4), or of 32 bytes under the 32-byte one (c ^ (r / 4) % 2).
// The transposing loads touch every bank once; the K reads (8 bytes of rows 2 r) take two turns.
template <int D>
__device__ __forceinline__ int code_offset(int row, int c)
{
    return D == 128 ? row * 64 + ((c ^ ((row >> 1) & 3)) << 4)
                    : row * 32 + ((c ^ ((row >> 2) & 1)) << 4);
}

// c = a[16x16] * b[16x8]: the first product of a sum.
__device__ __forceinline__ void mma_f16_16816_zero(float (&c)[4], uint32_t a0, uint32_t a1,
                                                   uint32_t a2, uint32_t a3, uint32_t b0,
                                                   uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// What the producer leaves for the consumer, per stage.
constexpr int kFirst = 1, kLast = 2, kWhole = 4, kEnd = 8;
struct __align__(16) Meta {
    int s, n_valid, flags, unused;
};

constexpr int kAhead = 3;   // blocks whose page ids are requested ahead

// A producer lane: where its group's run is, and what has been requested ahead.
struct Cursor {
    int s, blk, nb, ctx;
    int left;            // blocks of the run not yet fetched
    int now[kAhead];     // the lane's page ids of blocks blk, blk + 1, ...
    int next_ctx;        // of sequence s + 1 (clamped), and the page ids of its first blocks
    int next[kAhead];
    bool fresh;          // the next block starts a piece
    bool from_start;     // the piece began at the sequence's first block
};

// The id of page `sub` of a block (0 past the block-table row, and where the block has fewer pages).
__device__ __forceinline__ int page_id(const Args &a, int s, int blk, int sub)
{
    const int pi = ((blk * kBlock) >> a.log2_page) + sub;
    return pi < a.bt_stride ? a.block_table[static_cast<size_t>(s) * a.bt_stride + pi] : 0;
}

// Requests what a switch to sequence c.s + 1 needs; nothing here waits for it.
__device__ __forceinline__ void request_next(Cursor &c, const Args &a, int sub)
{
    c.next_ctx = 0;
    if (c.s + 1 < a.num_seqs) {
        c.next_ctx = clamped_ctx(a, c.s + 1);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            c.next[i] = page_id(a, c.s + 1, i, sub);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_decode_int4_kernel(const __grid_constant__ CUtensorMap tmap_k,
                             const __grid_constant__ CUtensorMap tmap_v,
                             const __grid_constant__ CUtensorMap tmap_kp,
                             const __grid_constant__ CUtensorMap tmap_vp, const Args a)
{
    if (threadIdx.x == kWarps * 32) {   // before the wait: nothing writes these
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
        prefetch_tensormap(&tmap_kp);
        prefetch_tensormap(&tmap_vp);
    }
    pdl_wait();
    pdl_trigger();
    using Geom = I4Geom<D>;
    constexpr int NG = Geom::kGroups;     // groups of a vector
    constexpr int NC = Geom::kChunks;     // 16-byte chunks of a row: 32 dims each
    constexpr int NS = Geom::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int G = a.group;
    const int Hkv = a.kv_heads;
    const int HW = a.heads;
    const int head_groups = Hkv / HW;
    Meta *metas = reinterpret_cast<Meta *>(smem + Geom::kOffMeta);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Geom::kOffBar);   // [groups][NS]
    uint64_t *empty = full + kWarps * NS;
    long long *scratch = reinterpret_cast<long long *>(smem + Geom::kOffScratch);
    long long *bound_cost = scratch + kBlockWarps;       // [kWarps + 1]
    long long *bound_g = bound_cost + kWarps + 1;        // first block at or past it
    long long *bound_s = bound_g + kWarps + 1;           // its sequence
    long long *bound_blk = bound_s + kWarps + 1;         // and its block in the sequence

    for (int i = threadIdx.x; i < kWarps * NS; i += kThreads) {
        mbar_init(&full[i], 1);     // the producer's arrival and the bytes
        mbar_init(&empty[i], HW);   // one arrival per warp of the group
    }
    fence_mbar_init();

    // ---- the runs of this CTA's groups: blocks [g0, g1) of a kv head's order, first sequence ----
    const int gg0 = blockIdx.x * a.groups;
    const int run_lo = gg0 / head_groups;
    long long n_runs = a.runs, cost = 0;
    if (!a.per_unit) {
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
        for (int i = 0; i < kBlockWarps; ++i) {
            const long long t = scratch[i];
            if (i < warp)
                acc += t;
            total += t;
        }
        if (total == 0)
            return;   // every row is written by the merge
        n_runs = min(static_cast<long long>(a.runs), total);
        cost = kBlockCost * total + kPieceCost * S;
        const int n_bounds = (gg0 + a.groups - 1) / head_groups - run_lo + 2;   // 2 .. kWarps + 1
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
    }
    __syncthreads();   // the bounds and the barriers

    // the group of this warp, or of this producer lane, and its run
    const int grp = warp >= kWarps ? lane >> 2 : warp / HW;
    const int head0 = (gg0 + grp) % head_groups * HW;
    const int run = (gg0 + grp) / head_groups;
    int run_len = 0;   // (a run's blocks: far below 2^31 for tables that fit the memory)
    if (grp < a.groups) {
        if (a.per_unit)
            run_len = run < a.num_seqs ? blocks_of(clamped_ctx(a, run)) : 0;
        else if (run < n_runs)
            run_len = static_cast<int>(bound_g[run - run_lo + 1] - bound_g[run - run_lo]);
    }
    const uint32_t group_stage = HW * Geom::kStageBytes;
    uint8_t *ring = smem + grp * NS * group_stage;

    if (warp >= kWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" : : "n"(kProducerRegs));
        if (warp > kWarps)
            return;
        // ------------- producer: lanes 4 g .. 4 g + 3 fill group g's ring, a page each -------------
        const int P = 1 << a.log2_page;
        const int box = min(P, kBlock);               // positions of a TMA box
        const int sub = lane & 3;
        const uint32_t page_tx = HW * box * (2 * Geom::kRow + 2 * NG * 4);
        const uint64_t policy = l2_policy_evict_first();
        Cursor c;
        c.left = run_len;
        c.s = a.per_unit ? run : 0;
        c.blk = 0;
        c.nb = 0;
        c.from_start = true;
        c.fresh = true;
        if (run_len > 0) {
            if (!a.per_unit) {
                c.s = static_cast<int>(bound_s[run - run_lo]);
                c.blk = static_cast<int>(bound_blk[run - run_lo]);
                for (; c.s < a.num_seqs; ++c.s, c.blk = 0) {   // past empty sequences
                    c.ctx = clamped_ctx(a, c.s);
                    c.nb = blocks_of(c.ctx);
                    if (c.blk < c.nb)
                        break;
                }
            } else {
                bool over;
                c.ctx = clamped_ctx(a, c.s, &over);
                c.nb = blocks_of(c.ctx);
                if (over && head0 == 0 && sub == 0)
                    atomicOr(err_word(a), kErrContextRange);
            }
            if (c.s < a.num_seqs) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    c.now[i] = page_id(a, c.s, c.blk + i, sub);
                request_next(c, a, sub);
            }
            c.from_start = c.blk == 0;
        }
        int issued = 0, st = 0;
        uint32_t phase = 1;   // of the empty barrier that the next fetch waits for, after NS fetches
        bool ended = run_len <= 0;
        bool ok = true;
        long long since = clock64();
        while (__any_sync(0xffffffffu, !ended)) {
            bool ready = !ended && (issued < NS || mbar_test(&empty[grp * NS + st], phase));
            ready = __shfl_sync(0xffffffffu, ready, lane & ~3);   // the group's lanes go together
            if (!__any_sync(0xffffffffu, ready)) {
                if (warp_wait_over(since)) {
                    ok = false;
                    break;
                }
                __nanosleep(20);
                continue;
            }
            since = clock64();
            uint64_t *bar = &full[grp * NS + st];
            const bool more = c.s < a.num_seqs;   // false: the contexts changed under the launch
            const int pos = c.blk * kBlock;
            const int n_valid = more ? min(kBlock, c.ctx - pos) : 0;
            const int np = (n_valid + box - 1) >> (box == 16 ? 4 : box == 32 ? 5 : 6);
            const bool last = c.blk + 1 == c.nb || c.left == 1;
            const bool whole = c.from_start && c.blk + 1 == c.nb;
            if (ready && sub == 0) {
                const int flags = !more ? kEnd
                                        : (c.fresh ? kFirst : 0) | (last ? kLast : 0) |
                                              (whole ? kWhole : 0) | (c.left == 1 ? kEnd : 0);
                *reinterpret_cast<int4 *>(&metas[grp * NS + st]) = make_int4(c.s, n_valid, flags, 0);
                mbar_arrive_expect_tx(bar, np * page_tx);
            }
            __syncwarp();
            if (ready) {
                if (sub < np) {
                    uint8_t *stage = ring + st * group_stage;
                    const int off = pos & (P - 1);
                    int page = c.now[0];
                    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.num_pages)) {
                        atomicOr(err_word(a), kErrPageRange);
                        page = 0;
                    }
                    // boxes land as [head][position]; one page after all of the one before
                    const int c1 = a.hnd ? off : (page << a.log2_page) + off;
                    const int c2 = a.hnd ? page * Hkv + head0 : head0;
                    uint8_t *codes = stage + sub * HW * box * Geom::kRow;
                    uint8_t *par = stage + HW * Geom::kOffKp + sub * Geom::page_par(HW, box);
                    tma_load_3d(codes, &tmap_k, 0, c1, c2, bar, policy);
                    tma_load_3d(codes + HW * Geom::kOffV, &tmap_v, 0, c1, c2, bar, policy);
                    tma_load_3d(par, &tmap_kp, off * (NG * 2), head0, page, bar, policy);
                    tma_load_3d(par + HW * Geom::kParBytes, &tmap_vp, off * (NG * 2), head0, page, bar,
                                policy);
                }
                ++c.blk;
                --c.left;
                c.fresh = false;
                // where the merge finds the unit's pieces: nowhere, or from this run's slot to that
                // of the run that holds the unit's last block
                if (more && last && !a.per_unit && c.from_start && sub == 0) {
                    int first = 0, count = 1;
                    if (!whole) {
                        const long long g_last = bound_g[run - run_lo + 1] - 1 + (c.nb - c.blk);
                        first = c.s + run;
                        count = static_cast<int>(run_of(block_cost(g_last, c.s), cost, n_runs) -
                                                 run + 1);
                    }
                    for (int h = head0; h < head0 + HW; ++h)
                        a.unit_info[static_cast<size_t>(c.s) * Hkv + h] =
                            make_int2(h * (a.num_seqs + a.runs) + first, count);
                }
                if (!more || c.left == 0) {
                    ended = true;
                } else if (last) {   // on to the next sequence, requested long ago
                    ++c.s;
                    c.blk = 0;
                    c.ctx = c.next_ctx;
                    c.nb = blocks_of(c.ctx);
#pragma unroll
                    for (int i = 0; i < kAhead; ++i)
                        c.now[i] = c.next[i];
                    while (c.nb == 0 && ++c.s < a.num_seqs) {   // past empty sequences
                        c.ctx = clamped_ctx(a, c.s);
                        c.nb = blocks_of(c.ctx);
#pragma unroll
                        for (int i = 0; i < kAhead; ++i)
                            c.now[i] = page_id(a, c.s, i, sub);
                    }
                    c.fresh = true;
                    c.from_start = true;
                    if (c.s < a.num_seqs)
                        request_next(c, a, sub);
                } else {
#pragma unroll
                    for (int i = 0; i + 1 < kAhead; ++i)
                        c.now[i] = c.now[i + 1];
                    c.now[kAhead - 1] = page_id(a, c.s, c.blk + kAhead - 1, sub);
                }
                ++issued;
                if (++st == NS) {
                    st = 0;
                    phase ^= 1u;
                }
            }
            __syncwarp();
        }
        if (!ok) {
            if (lane == 0)
                atomicOr(err_word(a), kErrDecodeEmptyWait);
            // every copy in flight lands before the CTA can exit
            if (grp < a.groups && sub == 0)
                for (int b = max(0, issued - NS); b < issued; ++b)
                    if (!mbar_wait(&full[grp * NS + b % NS], (b / NS) & 1))
                        atomicOr(err_word(a), kErrDrainWait);
        }
        return;
    }

    // ------------------------------------ consumers ------------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" : : "n"(kConsumerRegs));
    const int in_group = warp - grp * HW;
    const int kvh = head0 + in_group;
    if (run_len <= 0) {
        if (a.per_unit && grp < a.groups && run < a.num_seqs) {   // no positions: the rows are 0
            const size_t row0 = static_cast<size_t>(run) * a.q_heads + static_cast<size_t>(kvh) * G;
            for (int i = lane; i < G * D; i += 32)
                store_out(a.out, a.out_f32, row0 * D + i, 0.0f);
        }
        return;
    }
    const uint32_t ring32 = smem_addr(ring);
    metas += grp * NS;
    full += grp * NS;
    empty += grp * NS;
    // This head's tiles in a stage: the boxes of one page lie as [head][position], so tile 1 is the
    // next 16 positions of the head or the next page (page size 16), tile 2 the next but one or the
    // next page (32), and tile 3 as far from tile 2 as 1 from 0.
    const int box = min(1 << a.log2_page, kBlock);
    const int head_codes = in_group * box * Geom::kRow;
    const int head_par = HW * Geom::kOffKp + in_group * box * NG * 4;
    const int codes1 = box == 16 ? HW * Geom::kTileCodes : Geom::kTileCodes;
    const int codes2 = box == 64 ? 2 * Geom::kTileCodes : 2 * HW * Geom::kTileCodes;
    const int par1 = box == 16 ? Geom::page_par(HW, 16) : Geom::kTilePar;
    const int par2 = box == 64   ? 2 * Geom::kTilePar
                     : box == 32 ? Geom::page_par(HW, 32)
                                 : 2 * Geom::page_par(HW, 16);
    const int v_codes = HW * Geom::kOffV, v_par = HW * Geom::kParBytes;   // V's from K's
    const int r = lane >> 2;
    const int t = lane & 3;
    // K: the 8 bytes of group 0 that this thread reads of position 2 r (group 1: 32 bytes on, a
    // turn of the chunk) and of position 2 r + 1; V: this lane's row of the transposing loads
    const int k_off[2] = {code_offset<D>(2 * r, t >> 1) + (t & 1) * 8,
                          code_offset<D>(2 * r + 1, t >> 1) + (t & 1) * 8};
    const int v_off = code_offset<D>(lane & 15, lane >> 4);

    uint32_t qb[NG][2][2][2];   // B fragments: [group][word][nibble][register]
    float o[NC][2][4];          // O^T: [32 dims][low nibble, high nibble][fragment]
    float zacc[NG][2];          // sum of p lo, heads 2 t and 2 t + 1
    // heads 2 t and 2 t + 1: the sum; the maximum in use times f, and the y from which it moves
    float l_run[2], mf[2], m_thr[2], f[2], hq[NG][2];
    float vnorm[NG], v_thr[NG];   // and the value scale from which vnorm moves
    int stage = 0;
    uint32_t phase = 0;

    while (true) {
        if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], phase))) {
            if (lane == 0)
                atomicOr(err_word(a), kErrDecodeFullWait);
            return;
        }
        const int4 mt = *reinterpret_cast<const int4 *>(&metas[stage]);
        const int s = mt.x, n_valid = mt.y, flags = mt.z;
        if (n_valid == 0)
            return;   // the contexts changed under the launch
        const size_t row0 = static_cast<size_t>(s) * a.q_heads + static_cast<size_t>(kvh) * G;

        if (flags & kFirst) {
            uint4 qw[NG][2];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    a.q + (row0 + (r < G ? r : 0)) * D + 64 * g + 16 * t);
                qw[g][0] = src[0];
                qw[g][1] = src[1];
            }
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
                m_thr[j] = -INFINITY;
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
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                vnorm[g] = 1.0f;
                v_thr[g] = 0.0f;   // any positive value scale sets vnorm
            }
        }

        const uint8_t *st = ring + stage * group_stage;
        // this thread's positions are 16 T + 2 r and 16 T + 2 r + 1
        auto load_params = [&](uint32_t (&w)[2][NG], const uint8_t *p) {
            if constexpr (NG == 2) {
                const uint4 x = *reinterpret_cast<const uint4 *>(p);
                w[0][0] = x.x;
                w[0][NG - 1] = x.y;
                w[1][0] = x.z;
                w[1][NG - 1] = x.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2 *>(p);
                w[0][0] = x.x;
                w[1][0] = x.y;
            }
        };
        const uint8_t *par = st + head_par + 2 * r * NG * 4;

        // ---- scores: y[T][position][head] ----
        float y[kTiles][2][2];
#pragma unroll
        for (int T = 0; T < kTiles; ++T) {
            const int at = (T & 1) * codes1 + (T >> 1) * codes2;
            uint32_t kp[2][NG];
            load_params(kp, par + (T & 1) * par1 + (T >> 1) * par2);
            float acc[NG][4];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const uint2 w0 = *reinterpret_cast<const uint2 *>(
                    st + head_codes + at + (k_off[0] ^ (32 * g)));
                const uint2 w1 = *reinterpret_cast<const uint2 *>(
                    st + head_codes + at + (k_off[1] ^ (32 * g)));
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t x0 = j ? w0.y : w0.x, x1 = j ? w1.y : w1.x;
                    const uint32_t z0 = x0 >> 8, z1 = x1 >> 8;
                    if (j == 0)
                        mma_f16_16816_zero(acc[g], x0 & 0x000F000Fu, x1 & 0x000F000Fu,
                                           z0 & 0x000F000Fu, z1 & 0x000F000Fu, qb[g][j][0][0],
                                           qb[g][j][0][1]);
                    else
                        mma_f16_16816(acc[g], x0 & 0x000F000Fu, x1 & 0x000F000Fu,
                                      z0 & 0x000F000Fu, z1 & 0x000F000Fu, qb[g][j][0][0],
                                      qb[g][j][0][1]);
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
                        const float sc = __uint_as_float(kp[i][g] << 16);
                        const float lo = __uint_as_float(kp[i][g] & 0xFFFF0000u);
                        v = g == 0 ? sc * acc[g][2 * i + j] : fmaf(sc, acc[g][2 * i + j], v);
                        v = fmaf(lo, hq[g][j], v);
                    }
                    y[T][i][j] = v;
                }
        }
        uint32_t vp[kTiles][2][NG];
#pragma unroll
        for (int T = 0; T < kTiles; ++T)
            load_params(vp[T], par + v_par + (T & 1) * par1 + (T >> 1) * par2);
        if (n_valid < kBlock) {
#pragma unroll
            for (int T = 0; T < kTiles; ++T)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (16 * T + 2 * r + i >= n_valid) {
                        // what lies in unused slots is any code and any parameter, NaN too
                        y[T][i][0] = y[T][i][1] = -INFINITY;
#pragma unroll
                        for (int g = 0; g < NG; ++g)
                            vp[T][i][g] = 0u;
                    }
        }

        // ---- running maxima, and the powers of two on the value scales ----
        float mb[2], vmax[NG];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            mb[j] = fmaxf(y[0][0][j], y[0][1][j]);
#pragma unroll
            for (int T = 1; T < kTiles; ++T)
                mb[j] = fmax3(mb[j], y[T][0][j], y[T][1][j]);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            vmax[g] = 0.0f;
#pragma unroll
            for (int T = 0; T < kTiles; ++T)
                vmax[g] = fmax3(vmax[g], __uint_as_float(vp[T][0][g] << 16),
                                __uint_as_float(vp[T][1][g] << 16));
        }
        if (__any_sync(0xffffffffu, mb[0] > m_thr[0] || mb[1] > m_thr[1] || vmax[0] > v_thr[0] ||
                                        vmax[NG - 1] > v_thr[NG - 1])) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                mb[0] = fmaxf(mb[0], __shfl_xor_sync(0xffffffffu, mb[0], off));
                mb[1] = fmaxf(mb[1], __shfl_xor_sync(0xffffffffu, mb[1], off));
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    vmax[g] = fmaxf(vmax[g], __shfl_xor_sync(0xffffffffu, vmax[g], off));
            }
            float fix[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                fix[j] = 1.0f;
                if (mb[j] > m_thr[j]) {   // the same in every lane of the head
                    const float mf_new = mb[j] * f[j];
                    fix[j] = m_thr[j] == -INFINITY ? 0.0f : fast_exp2(mf[j] - mf_new);
                    l_run[j] *= fix[j];
#pragma unroll
                    for (int g = 0; g < NG; ++g)
                        zacc[g][j] *= fix[j];
                    m_thr[j] = mb[j] + kLagLog2 / f[j];
                    mf[j] = mf_new;
                }
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float turn = 1.0f;
                if (vmax[g] > v_thr[g]) {   // the same in every lane that shares the maximum: all of them
                    // vnorm = 2^(10 - e) for the largest scale's exponent e: vmax vnorm in [2^10, 2^11)
                    const int e = max(-100, static_cast<int>(__float_as_uint(vmax[g]) >> 23) - 127);
                    const float vn = __uint_as_float(static_cast<uint32_t>(127 + 10 - e) << 23);
                    turn = v_thr[g] > 0.0f ? vn / vnorm[g] : 1.0f;   // unset: every code product was 0
                    vnorm[g] = vn;
                    v_thr[g] = kMaxScaled / vn;
                }
#pragma unroll
                for (int n = 2 * g; n < 2 * g + 2; ++n)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        o[n][b][0] *= fix[0] * turn;
                        o[n][b][1] *= fix[1] * turn;
                        o[n][b][2] *= fix[0] * turn;
                        o[n][b][3] *= fix[1] * turn;
                    }
            }
        }

        // ---- probabilities, and out ----
        // The tensor cores cut their sums off instead of rounding them, all terms here are positive,
        // and the sum of minima takes most of the result away again: over thousands of products
        // the cuts would add up to a part of what is left (a fifth of the output's norm at 131,072
        // positions).  So their sums are a block's, and the blocks are added up with rounding.
        const uint32_t vb = ring32 + stage * group_stage + v_codes + head_codes;
        float part[NC][2][4];
#pragma unroll
        for (int T = 0; T < kTiles; ++T) {
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
                    const float sc = __uint_as_float(vp[T][i][g] << 16) * vnorm[g];
                    const float lo = __uint_as_float(vp[T][i][g] & 0xFFFF0000u);
                    zacc[g][0] = fmaf(p[i][0], lo, zacc[g][0]);
                    zacc[g][1] = fmaf(p[i][1], lo, zacc[g][1]);
                    pb[g][i] = movmatrix_trans(pack_f16x2(p[i][0] * sc, p[i][1] * sc));
                }
            const uint32_t va = vb + (T & 1) * codes1 + (T >> 1) * codes2;
#pragma unroll
            for (int g = 0; g < NG; ++g) {   // chunks 2 g and 2 g + 1
                uint32_t e[4];
                ldsm_x2_trans_b8(va + (v_off ^ (32 * g)), e[0], e[1], e[2], e[3]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t x0 = e[2 * k], x1 = e[2 * k + 1];
                    const uint32_t z0 = x0 >> 8, z1 = x1 >> 8;
                    if (T == 0) {
                        mma_f16_16816_zero(part[2 * g + k][0], x0 & 0x000F000Fu, x1 & 0x000F000Fu,
                                           z0 & 0x000F000Fu, z1 & 0x000F000Fu, pb[g][0], pb[g][1]);
                        mma_f16_16816_zero(part[2 * g + k][1], x0 & 0x00F000F0u, x1 & 0x00F000F0u,
                                           z0 & 0x00F000F0u, z1 & 0x00F000F0u, pb[g][0], pb[g][1]);
                    } else {
                        mma_f16_16816(part[2 * g + k][0], x0 & 0x000F000Fu, x1 & 0x000F000Fu,
                                      z0 & 0x000F000Fu, z1 & 0x000F000Fu, pb[g][0], pb[g][1]);
                        mma_f16_16816(part[2 * g + k][1], x0 & 0x00F000F0u, x1 & 0x00F000F0u,
                                      z0 & 0x00F000F0u, z1 & 0x00F000F0u, pb[g][0], pb[g][1]);
                    }
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[n][b][i] += part[n][b][i];

        __syncwarp();
        if (lane == 0)
            mbar_arrive(&empty[stage]);

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
            // pieces of kv head h own slots [h (S + R), (h + 1) (S + R)), piece (s, run) s + run
            // there: distinct for every piece, consecutive for one unit's
            const int slot = kvh * (a.num_seqs + a.runs) + s + run;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int head = 2 * t + j;
                if (head < G) {
#pragma unroll
                    for (int n = 0; n < NC; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {   // dims 32 n + 16 i + 2 r, + 1
                            const float z = zacc[n / 2][j];
                            const float v_inv = 1.0f / vnorm[n / 2];   // a power of two: exact
                            float2 v;
                            v.x = fmaf(o[n][0][2 * i + j] * 16777216.0f, v_inv, z) * inv[j];
                            v.y = fmaf(o[n][1][2 * i + j] * 1048576.0f, v_inv, z) * inv[j];
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
        if (flags & kEnd)
            return;
        if (++stage == NS) {
            stage = 0;
            phase ^= 1u;
        }
    }
}

// The row's unit: where its pieces' partials are.  Before the wait only its context is read: a merge
// starts once every CTA of the decode has triggered, which they do after their own wait, so what ran
// before the decode is done.
struct Pieces {
    int count;           // 0 or 1: nothing to merge, the decode wrote the row
    const float *lse;    // piece j's at lse[j G]
    const float *o;      // and its row at o + j G D
};

template <int D>
__device__ __forceinline__ Pieces pieces_of(const Args &a, int s, int h)
{
    const int kvh = h / a.group;
    const int2 info = __ldcg(a.unit_info + static_cast<size_t>(s) * a.kv_heads + kvh);
    Pieces p;
    // (a sequence whose context changes while the decode runs may have left no such slots)
    p.count = info.x >= 0 && info.y <= a.kv_heads * (a.num_seqs + a.runs) - info.x ? info.y : 0;
    const size_t first = static_cast<size_t>(info.x) * a.group + (h - kvh * a.group);
    p.lse = a.part_lse + first;
    p.o = a.part_o + first * D;
    return p;
}

// V values of the output, from element `at` on.
template <int V>
__device__ __forceinline__ void store_values(const Args &a, size_t at, const float *v)
{
    if constexpr (V == 4)
        store_out4(a.out, a.out_f32, at, make_float4(v[0], v[1], v[2], v[3]));
    else
        store_out2(a.out, a.out_f32, at, make_float2(v[0], v[1]));
}

// out[row] = sum_j exp(lse_j - M) o_j / sum_j exp(lse_j - M) over the pieces of the row's unit,
// W warps a row.  Rows whose unit is one whole piece were written by it; rows of a sequence with no
// positions are 0.
template <int D, int W>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W) merge_int4_kernel(const Args a)
{
    constexpr int V = D / 32;
    constexpr int kRows = W == 1 ? 4 : 1;
    constexpr int kPre = 4;
    __shared__ float part[W == 1 ? 1 : W][D + 1];
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int w0 = W == 1 ? 0 : warp;   // this warp's first piece
    const int row = blockIdx.x * kRows + (W == 1 ? warp : 0);
    if (row >= a.num_seqs * a.q_heads)
        return;
    const int s = row / a.q_heads;
    const int G = a.group;
    const int raw = __ldcg(a.context_lens + s);
    pdl_wait();
    pdl_trigger();
    const Pieces p = pieces_of<D>(a, s, row - s * a.q_heads);
    float acc[V], sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
        acc[v] = 0.0f;
    if (raw > 0) {
        const int count = p.count;
        if (count <= 1)
            return;
        const float *lse = p.lse;
        const float *po = p.o + lane * V;
        const size_t po_step = static_cast<size_t>(G) * D;
        // one round trip: every piece's lse (lane j holds pieces j, j + 32, ...) and the rows of
        // this warp's first pieces
        float pre[kPre][V];
#pragma unroll
        for (int u = 0; u < kPre; ++u) {
            const int j = w0 + u * W;
            if (j < count) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    pre[u][v] = __ldcg(po + static_cast<size_t>(j) * po_step + v);
            }
        }
        const float mine = lane < count ? __ldcg(lse + static_cast<size_t>(lane) * G) : -INFINITY;
        float M = mine;
        for (int j = lane + 32; j < count; j += 32)
            M = fmaxf(M, __ldcg(lse + static_cast<size_t>(j) * G));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        const float mu = M == -INFINITY ? 0.0f : M;
        auto weight = [&](int j) {
            const float l = j < 32 ? __shfl_sync(0xffffffffu, mine, j)
                                   : __ldcg(lse + static_cast<size_t>(j) * G);
            return fast_exp2((l - mu) * kLog2e);
        };
#pragma unroll
        for (int u = 0; u < kPre; ++u) {
            const int j = w0 + u * W;
            if (j < count) {
                const float w = weight(j);
                sum += w;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    acc[v] = fmaf(w, pre[u][v], acc[v]);
            }
        }
#pragma unroll 4
        for (int j = w0 + kPre * W; j < count; j += W) {
            const float w = weight(j);
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
#pragma unroll
    for (int v = 0; v < V; ++v)
        acc[v] *= inv;
    store_values<V>(a, static_cast<size_t>(row) * D + lane * V, acc);
}

// The same for units of many pieces (very few sequences, long contexts), a CTA for 32 dims of a row: a
// thread per piece's weight, and eight warps that each take every eighth piece, kFly of them in
// flight, so that 128 pieces are one round trip.
constexpr int kWideThreads = 256;

template <int D>
__global__ void __launch_bounds__(kWideThreads) merge_wide_int4_kernel(const Args a)
{
    constexpr int W = kWideThreads / 32;
    constexpr int kFly = 16;
    constexpr int kParts = D / 32;
    static_assert(kWideThreads % (kFly * W) == 0, "a batch of rows has its weights in one tile");
    __shared__ float weight[kWideThreads], high[W], part[W][33];
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x / kParts;
    const int dim = blockIdx.x % kParts * 32 + lane;
    const int s = row / a.q_heads;
    const int raw = __ldcg(a.context_lens + s);
    pdl_wait();
    pdl_trigger();
    const Pieces p = pieces_of<D>(a, s, row - s * a.q_heads);
    float acc = 0.0f, sum = 0.0f;
    if (raw > 0) {
        if (p.count <= 1)
            return;
        const float *po = p.o + dim;
        const size_t po_step = static_cast<size_t>(a.group) * D;
        float x[kFly];   // of this warp's next pieces: those from j on
        auto load = [&](int j) {
#pragma unroll
            for (int u = 0; u < kFly; ++u)
                if (j + u * W < p.count)
                    x[u] = __ldcg(po + (j + u * W) * po_step);
        };
        load(warp);
        float M = -INFINITY;
        for (int j = threadIdx.x; j < p.count; j += kWideThreads)
            M = fmaxf(M, __ldcg(p.lse + static_cast<size_t>(j) * a.group));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        if (lane == 0)
            high[warp] = M;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w)
            M = fmaxf(M, high[w]);
        const float mu = M == -INFINITY ? 0.0f : M;
        for (int base = 0; base < p.count; base += kWideThreads) {
            const int mine = base + threadIdx.x;
            weight[threadIdx.x] =
                mine < p.count
                    ? fast_exp2((__ldcg(p.lse + static_cast<size_t>(mine) * a.group) - mu) * kLog2e)
                    : 0.0f;
            __syncthreads();
#pragma unroll 1
            for (int j = base + warp; j < min(p.count, base + kWideThreads); j += kFly * W) {
                if (j > warp)
                    load(j);
#pragma unroll
                for (int u = 0; u < kFly; ++u)
                    if (j + u * W < p.count) {
                        const float w = weight[j + u * W - base];
                        sum += w;
                        acc = fmaf(w, x[u], acc);
                    }
            }
            __syncthreads();
        }
    }
    part[warp][lane] = acc;
    if (lane == 0)
        part[warp][32] = sum;
    __syncthreads();
    if (warp != 0)
        return;
    for (int w = 1; w < W; ++w) {
        sum += part[w][32];
        acc += part[w][lane];
    }
    store_out(a.out, a.out_f32, static_cast<size_t>(row) * D + dim, sum == 0.0f ? 0.0f : acc / sum);
}

template <int D>
cudaError_t launch_t(const DecodeInt4Launch &l, const CUtensorMap (&maps)[4], cudaStream_t stream)
{
    Args a;
    a.q = static_cast<const __nv_bfloat16 *>(l.q);
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
    a.heads = int4_group_heads(l.pools.kv_heads);
    a.groups = kWarps / a.heads;
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
    const long long groups = static_cast<long long>(a.runs) * (a.kv_heads / a.heads);
    const unsigned grid = static_cast<unsigned>((groups + a.groups - 1) / a.groups);
    err = launch_pdl(kernel, dim3(grid), dim3(kThreads), smem, stream, maps[0], maps[1], maps[2],
                     maps[3], a);
    if (err != cudaSuccess || l.per_unit)
        return err;
    const int rows = l.num_seqs * l.q_heads;
    // Few sequences have many pieces a row.  1 sequence of 65,536 positions: 24.4 us with the wide
    // merge, 38.2 with 8 warps a row; 4 of 32,768: 35.9 and 38.6; 8 of 8,192: 25.0 and 23.8.  16 of 4,096
    // take 21.4 with 8 warps a row and 27.4 with one, 32 31.0 and 33.3, 48 41.2 and 41.1, 64 52.8 and 51.3.
    if (l.runs > 32LL * l.num_seqs)
        return launch_pdl(merge_wide_int4_kernel<D>, dim3(rows * (D / 32)), dim3(kWideThreads), 0,
                          stream, a);
    if (l.runs > 4LL * l.num_seqs)
        return launch_pdl(merge_int4_kernel<D, 8>, dim3(rows), dim3(256), 0, stream, a);
    return launch_pdl(merge_int4_kernel<D, 1>, dim3((rows + 3) / 4), dim3(128), 0, stream, a);
}

}  // namespace

// A divisor, because a box holds the heads of a whole group: the eight warps of a CTA are all busy for 1,
// 2, 4, 8 and 16 heads, seven for 7, six for 3, 6, 9 and 12, five for 5 and 10, and 11 and 13 take groups
// of one head, whose boxes cost the most TMA operations.  64 sequences of up to 4,096 positions
// (G = 4, D = 128), share of the HBM floor: 4 heads 30.0 us (42%), 5 40.7 (39%), 7 41.8 (53%), 8 42.3
// (60%), 9 66.1 (43%), 12 67.7 (56%), 16 69.9 (72%), but 11 118 (29%) and 13 137 (30%); 8 of up to
// 131,072: 3 heads 83 (61%), 4 85 (80%), 5 151 (56%), 8 153 (89%), 9 222 (69%), 11 265 (70%).
int int4_group_heads(int kv_heads)
{
    int n = kv_heads < 8 ? kv_heads : 8;
    while (kv_heads % n != 0)
        --n;
    return n;
}

cudaError_t launch_decode_int4(const DecodeInt4Launch &l, const CUtensorMap (&maps)[4],
                               cudaStream_t stream)
{
    if (l.num_seqs == 0)
        return cudaSuccess;
    return l.pools.head_dim == 64 ? launch_t<64>(l, maps, stream) : launch_t<128>(l, maps, stream);
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
