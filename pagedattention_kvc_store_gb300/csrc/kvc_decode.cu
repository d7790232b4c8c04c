// kvc_decode.cu -- paged decode attention (one new token per sequence, GQA) with a split-K
// partition and the log-sum-exp merge of its partials.
//
// What it computes: "KV Cache Management and PagedAttention", "Compute attention over
// scattered KV" -- attention of the newest token's query over every valid position of its
// sequence, reading K/V in place from the pages its block table lists (no gather buffer),
// excluding unused slots of the last page and every other sequence's pages.  GQA: the G
// query heads of a group share one kv head.
//
// Kernel design (GB300):
//   * one CTA per (split, kv head, sequence); 4 consumer warps + 1 TMA producer warp;
//   * the producer streams 64-position stages of K and V into a 3-deep shared-memory ring
//     with cp.async.bulk.tensor (one box per page, both 64-column halves, 128-byte swizzle so
//     that ldmatrix reads are bank-conflict free), completion counted on mbarriers;
//   * each consumer warp takes 16 of the 64 positions of every stage: S = Q K^T and O += P V
//     on the tensor cores (mma.sync m16n8k16, the G query heads padded to 16 rows -- too thin
//     for tcgen05's 64/128-row tiles), online softmax in base 2 with warp shuffles;
//   * the 4 warps' (max, sum, O) are combined through shared memory at the end; with one
//     split the CTA writes the final output, otherwise an fp32 partial and its lse.
// Masked positions (past the context) are excluded before the exponential and their V
// entries are zeroed in registers, so NaN/Inf left in unused slots never reaches a sum.
#include <math.h>

#include "kvc_decode_cta.cuh"

namespace kvc {

namespace {

__device__ uint32_t g_decode_errors;

using namespace dec;

template <int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 2)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tmap_k,
                        const __grid_constant__ CUtensorMap tmap_v, const Args a)
{
    pdl_wait();
    pdl_trigger();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    decode_cta<D, SPLIT>(&tmap_k, &tmap_v, a, blockIdx.x, blockIdx.y, blockIdx.z, smem,
                         a.err ? a.err : &g_decode_errors);
}

// A warp per row, or (WIDE) per 32 dims of one.
template <int D, bool WIDE>
__global__ void __launch_bounds__(128) merge_kernel(void *out, int out_f32,
                                                    const float *__restrict__ part_o,
                                                    const float *__restrict__ part_lse,
                                                    int rows, int n_split, float *lse_out)
{
    pdl_wait();
    pdl_trigger();
    const long long warp = blockIdx.x * 4LL + (threadIdx.x >> 5);
    if constexpr (WIDE) {
        const int row = static_cast<int>(warp / (D / 32));
        if (row < rows)
            merge_row_part<D>(out, out_f32, part_o, part_lse, row, static_cast<int>(warp % (D / 32)),
                              n_split, lse_out);
    } else if (warp < rows) {
        merge_row<D>(out, out_f32, part_o, part_lse, static_cast<int>(warp), n_split, lse_out);
    }
}

template <int D, bool SPLIT>
cudaError_t launch_decode_t(const DecodeLaunch &l, const CUtensorMap &tk, const CUtensorMap &tv,
                            cudaStream_t stream)
{
    const Args a = make_args(l);
    const size_t smem = DecodeGeom<D>::kSmemBytes;
    auto kernel = paged_decode_kernel<D, SPLIT>;
    cudaError_t err =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem));
    if (err != cudaSuccess)
        return err;
    dim3 grid(l.n_split, l.kv_heads, l.num_seqs);
    return launch_pdl(kernel, grid, dim3(kThreads), smem, stream, tk, tv, a);
}

// The bounded wait every kernel uses, on an mbarrier phase that nothing completes: it gives
// up after kWaitLimitCycles and the CTA records kErrSelftestWait and returns, leaving the
// context usable.  Then the wait of a warp that polls for itself (warp_wait_over), its lanes' clocks as
// far apart as half the limit: all of them have to give up in the same turn.  And a wait for work, first with its
// one turn run out, then with many that the first one's end cuts short.  A diagnostic of the failure path, with
// no fault and no hang.
__global__ void __launch_bounds__(32) selftest_wait_kernel(uint32_t *word)
{
    __shared__ uint64_t bar;
    __shared__ uint32_t gave_up;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
        gave_up = 0;
    }
    __syncwarp();
    const bool waited = __all_sync(0xffffffffu, mbar_wait(&bar, 0));
    const long long since = clock64() - threadIdx.x * (kWaitLimitCycles / 64);
    unsigned turns = 0;
    while (!mbar_test(&bar, 0) && !warp_wait_over(since))
        ++turns;
    int together;
    __match_all_sync(0xffffffffu, turns, &together);
    bool ended = false;
    if (threadIdx.x == 0) {
        ended = !mbar_wait_work(&bar, 0, 1, &gave_up) && gave_up == 1;
        ended = !mbar_wait_work(&bar, 0, 64, &gave_up) && ended;
    }
    if (!waited && together && ended)
        atomicOr(word ? word : &g_decode_errors, kErrSelftestWait);
}

}  // namespace

cudaError_t launch_decode(const DecodeLaunch &l, const CUtensorMap &tk, const CUtensorMap &tv,
                          cudaStream_t stream)
{
    if (l.num_seqs == 0)
        return cudaSuccess;
    const bool split = l.n_split > 1 || l.split_stride > 1 || l.key_start != nullptr;
    if (l.head_dim == 128)
        return split ? launch_decode_t<128, true>(l, tk, tv, stream)
                     : launch_decode_t<128, false>(l, tk, tv, stream);
    return split ? launch_decode_t<64, true>(l, tk, tv, stream)
                 : launch_decode_t<64, false>(l, tk, tv, stream);
}

cudaError_t launch_merge(void *out, int out_f32, const float *part_o, const float *part_lse,
                         int rows, int n_split, int head_dim, float *lse_out, cudaStream_t stream)
{
    if (rows == 0)
        return cudaSuccess;
    const bool wide = n_split > kWideMergeSplits;
    const long long warps = static_cast<long long>(rows) * (wide ? head_dim / 32 : 1);
    const long long blocks = (warps + 3) / 4;
    if (blocks > 0x7FFFFFFFLL)
        return cudaErrorInvalidValue;
    auto kernel = head_dim == 128 ? (wide ? merge_kernel<128, true> : merge_kernel<128, false>)
                                  : (wide ? merge_kernel<64, true> : merge_kernel<64, false>);
    return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(128), 0, stream, out, out_f32,
                      part_o, part_lse, rows, n_split, lse_out);
}

cudaError_t launch_selftest_wait(cudaStream_t stream)
{
    selftest_wait_kernel<<<1, 32, 0, stream>>>(current_error_word());
    return cudaGetLastError();
}

cudaError_t read_and_clear_decode_errors(uint32_t *flags)
{
    uint32_t zero = 0;
    cudaError_t err = cudaMemcpyFromSymbol(flags, g_decode_errors, sizeof(uint32_t));
    if (err != cudaSuccess)
        return err;
    return cudaMemcpyToSymbol(g_decode_errors, &zero, sizeof(uint32_t));
}

}  // namespace kvc
