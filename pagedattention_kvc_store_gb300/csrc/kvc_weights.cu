// kvc_weights.cu -- paged decode attention that also adds up the attention weights.
//
// What it computes: kvc_decode's output, bit for bit (the same kernel code, and a single split writes its
// rows itself here too, NaN and all), and for every position p and kv head h
//   weights[row(s)][h][p] += sum over the G query heads g of h's group of softmax_p(q_g . K[p] scale),
// the measure by which kvc_evict keeps positions.
//
// A weight needs its row's final log-sum-exp, which no CTA knows while it holds the position's
// score.  Reading K again for the weights would cost half of the pass once more; the scores are
// 4 G bytes a position against the 4 D bytes of its K and V (G = 4, D = 128: 3%), so the decode CTAs
// write them, and the launch that merges the partials also turns them into weights: its first
// blocks merge (one warp a row; none where there is one split), the others take 1,024 positions of one
// (sequence, kv head) each.
// Nothing is added with atomics: every position has one writer, and the sum over the group has
// one order.  The weights' denominator is the sum of the unrounded probabilities (the output
// divides by the sum of the bf16-rounded ones that its numerator uses, up to 2^-9 off for a single
// position).
//
// Bound: HBM.  64 sequences of up to 4,096 positions (32 / 8 heads, D = 128, 617 MB): 108 us, 97 of them
// the decode with its scores and 11 the second launch; 8 of up to 131,072 (64 / 8 heads, 3.3 GB): 569 to
// 582 us call after call, 5.7 to 5.8 TB/s (510 and 43 each by itself), the scores (205 MB, written and
// read) going through HBM.
#include <math.h>

#include "kvc_decode_cta.cuh"

namespace kvc {

namespace {

__device__ uint32_t g_weights_errors;

using namespace dec;

// 4 or 8 positions a thread are within 0.5%, 2 or 16 and 512 threads 2 to 6% slower.
constexpr int kFinishThreads = 256;
static_assert(kFinishThreads / 32 >= kMaxGroup, "one warp per query head of a group");
constexpr int kPerThread = 4;
constexpr int kTile = kFinishThreads * kPerThread;   // positions of one weights block

template <int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 2)
    paged_decode_weights_kernel(const __grid_constant__ CUtensorMap tmap_k,
                                const __grid_constant__ CUtensorMap tmap_v, const Args a)
{
    pdl_wait();
    pdl_trigger();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    decode_cta<D, SPLIT, true>(&tmap_k, &tmap_v, a, blockIdx.x, blockIdx.y, blockIdx.z, smem,
                              a.err ? a.err : &g_weights_errors);
}

struct FinishArgs {
    Args d;
    float *weights;
    const int32_t *rows;   // row of each sequence, or null (row s)
    int num_rows, weight_stride;
    int num_seqs, max_ctx, merge_blocks, tiles;
};

// WIDE: the rows of many splits, merged by D / 32 warps each (more registers than the weights need).
template <int D, bool WIDE>
__global__ void __launch_bounds__(kFinishThreads) finish_kernel(const FinishArgs f)
{
    pdl_wait();
    pdl_trigger();
    const Args &a = f.d;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (blockIdx.x < f.merge_blocks) {
        constexpr int kRowWarps = WIDE ? D / 32 : 1;
        const int unit = blockIdx.x * (kFinishThreads / 32) + warp;
        const int row = unit / kRowWarps;
        if (row >= f.num_seqs * a.q_heads)
            return;
        if constexpr (WIDE)
            merge_row_part<D>(a.out, a.out_f32, a.part_o, a.part_lse, row, unit % kRowWarps,
                              a.n_split, nullptr);
        else
            merge_row<D>(a.out, a.out_f32, a.part_o, a.part_lse, row, a.n_split, nullptr);
        return;
    }
    // block -> (tile of positions, kv head, sequence), tile fastest, from the last: what the decode
    // wrote last is still in L2
    const int b = gridDim.x - 1 - blockIdx.x;
    const int tile = b % f.tiles;
    const int unit = b / f.tiles;
    const int kvh = unit % a.kv_heads;
    const int s = unit / a.kv_heads;
    const int raw = a.context_lens[s];
    const int ctx = min(raw, f.max_ctx);   // which the rows, the scores and the table row hold
    const int row = f.rows ? f.rows[s] : s;
    if (threadIdx.x == 0 && tile == 0 && kvh == 0) {
        if (raw > f.max_ctx && row >= 0)
            atomicOr(a.err ? a.err : &g_weights_errors, kErrContextRange);
        if (row >= f.num_rows)
            atomicOr(a.err ? a.err : &g_weights_errors, kErrSlotRange);
    }
    const int p0 = tile * kTile + threadIdx.x;
    if (tile * kTile >= ctx || row < 0 || row >= f.num_rows)
        return;
    __shared__ float lse[kMaxGroup];
    const size_t q0 = static_cast<size_t>(s) * a.q_heads + static_cast<size_t>(kvh) * a.group;
    if (warp < a.group) {   // one warp per query head of the group
        const float *part = a.part_lse2 + (q0 + warp) * a.split_stride;
        float M = -INFINITY;
        for (int j = lane; j < a.n_split; j += 32)
            M = fmaxf(M, part[j]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        const float mu = M == -INFINITY ? 0.0f : M;
        float sum = 0.0f;
        for (int j = lane; j < a.n_split; j += 32)
            sum += fast_exp2(part[j] - mu);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (lane == 0)
            lse[warp] = mu + log2f(sum);
    }
    __syncthreads();
    float *dst = f.weights + (static_cast<size_t>(row) * a.kv_heads + kvh) * f.weight_stride;
    const float *src = a.scores + q0 * a.score_stride;
    float w[kPerThread], old[kPerThread];
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
        const int p = p0 + k * kFinishThreads;
        w[k] = 0.0f;
        old[k] = p < ctx ? dst[p] : 0.0f;
    }
    for (int g = 0; g < a.group; ++g) {
        const float m = lse[g];
#pragma unroll
        for (int k = 0; k < kPerThread; ++k) {
            const int p = p0 + k * kFinishThreads;
            if (p < ctx)
                w[k] += fast_exp2(src[p] - m);
        }
        src += a.score_stride;
    }
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
        const int p = p0 + k * kFinishThreads;
        if (p < ctx)
            dst[p] = old[k] + w[k];
    }
}

template <int D>
cudaError_t launch_t(const DecodeLaunch &l, const WeightsLaunch &w, const CUtensorMap &tk,
                     const CUtensorMap &tv, cudaStream_t stream)
{
    Args a = make_args(l);
    a.scores = w.scores;
    a.score_stride = w.score_stride;
    a.part_lse2 = w.part_lse2;
    const size_t smem = DecodeGeom<D>::kSmemBytes;
    const bool split = l.n_split > 1;   // else the decode writes the rows
    auto kernel = split ? paged_decode_weights_kernel<D, true> : paged_decode_weights_kernel<D, false>;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(smem));
    if (err != cudaSuccess)
        return err;
    err = launch_pdl(kernel, dim3(l.n_split, l.kv_heads, l.num_seqs), dim3(kThreads), smem, stream,
                     tk, tv, a);
    if (err != cudaSuccess)
        return err;
    FinishArgs f;
    f.d = a;
    f.weights = w.weights;
    f.rows = w.rows;
    f.num_rows = w.num_rows;
    f.weight_stride = w.weight_stride;
    f.num_seqs = l.num_seqs;
    f.max_ctx = w.max_ctx;
    const int rows_per_block = kFinishThreads / 32;   // (warps)
    const bool wide = l.n_split > kWideMergeSplits;
    f.merge_blocks =
        split ? (l.num_seqs * l.q_heads * (wide ? D / 32 : 1) + rows_per_block - 1) / rows_per_block
              : 0;
    f.tiles = (w.max_ctx + kTile - 1) / kTile;
    const long long grid =
        f.merge_blocks + static_cast<long long>(f.tiles) * l.kv_heads * l.num_seqs;
    if (grid > 0x7FFFFFFFLL)
        return cudaErrorInvalidValue;
    return launch_pdl(wide ? finish_kernel<D, true> : finish_kernel<D, false>, dim3(static_cast<unsigned>(grid)), dim3(kFinishThreads), 0,
                      stream, f);
}

}  // namespace

cudaError_t launch_decode_weights(const DecodeLaunch &l, const WeightsLaunch &w,
                                  const CUtensorMap &tk, const CUtensorMap &tv,
                                  cudaStream_t stream)
{
    if (l.num_seqs == 0)
        return cudaSuccess;
    return l.head_dim == 128 ? launch_t<128>(l, w, tk, tv, stream)
                             : launch_t<64>(l, w, tk, tv, stream);
}

cudaError_t read_and_clear_weights_errors(uint32_t *flags)
{
    uint32_t zero = 0;
    cudaError_t err = cudaMemcpyFromSymbol(flags, g_weights_errors, sizeof(uint32_t));
    if (err != cudaSuccess)
        return err;
    return cudaMemcpyToSymbol(g_weights_errors, &zero, sizeof(uint32_t));
}

}  // namespace kvc
