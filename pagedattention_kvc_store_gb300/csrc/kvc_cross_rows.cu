// kvc_cross_rows.cu -- cross attention for few query rows: the single tokens of a source's beams.
//
// The same result as kvc_cross.cu's kernel, for at most 32 rows (token, query head of the group) of a (source,
// kv head).  It is bound by reading K and V once, and the tensor cores' 128-row tiles would stand
// nearly empty: a CTA takes one chunk of one (source, kv head), a TMA warp streams its pages (one box per page,
// both column halves) through a ring of 64-position stages, and four warps hold the rows in tiles of 16 for
// mma.sync, the warps of a tile splitting a stage's positions and joining at the end.  Two CTAs an SM, so that
// one's start and end lie under the other's stream.
// Against that kernel, us (calls back to back, with the join): 64 sources of 512-4,096 positions, 8 kv heads, groups
// of 4, 16-position pages: 1 token 98 / 101, 4 tokens 101 / 100, 8 tokens (32 rows) 114 / 99; 64 sources of 150 x 4
// tokens 11.5 / 24.7, 4 of 2,000 11.7 / 14.0, 16 of 500-3,000 x 4 with 20 kv heads of one query head and 64 dims 40 /
// 48; 8 of 32k-131k, groups of 8, 1 token 412 / 420, 32 rows 424 / 416 (6.0 TB/s): ahead by most where sources are
// short or rows few, behind at 32 rows of many positions.  64 rows in tiles of this kind (the shared-prefix
// decode's) took 241 when the other kernel took 142.
// P is rounded to bf16 for the product; sums are of the unrounded values, as there.
#include <math.h>

#include "kvc_device.cuh"
#include "kvc_launch.h"

namespace kvc {

namespace {

__device__ uint32_t g_cross_rows_errors;

constexpr int kConsumerWarps = 4;
constexpr int kThreads = (kConsumerWarps + 1) * 32;
constexpr int kStages = 3;
constexpr int kMaxRows = kCrossFewRows;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Geom {
    static constexpr int kTileBytes = kStageKeys * D * 2;
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kRingBytes = kStages * kStageBytes;
    static constexpr int kCombineBytes =
        kConsumerWarps * 16 * (D + 8) * 4 + 2 * kConsumerWarps * 16 * 4 +
        kMaxRows * kConsumerWarps * 4 + kMaxRows * 8;
    static_assert(kCombineBytes <= kRingBytes, "the combine area lies over the ring");
    static constexpr size_t kSmemBytes = 1024 + kRingBytes + 2 * kStages * 8;
};

struct Args {
    const __nv_bfloat16 *q;
    void *out;                  // rows [T][q_heads], or the partials [T][q_heads][n_split] when split
    int out_f32;
    float *lse;                 // of the same rows, or null (one split)
    const int32_t *block_table;
    int bt_stride;
    const int32_t *q_indptr, *source_lens;
    int q_heads, kv_heads, group, page_size;
    int num_tokens, max_q_len, max_src, chunk, n_split;
    float scale_log2;
    int hnd;
    uint32_t *err;
};

template <int D, int NMT>
__global__ void __launch_bounds__(kThreads, 2)
    cross_rows_kernel(const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v, const Args a)
{
    pdl_wait();
    pdl_trigger();
    using G_ = Geom<D>;
    constexpr int kWarpsPerTile = kConsumerWarps / NMT;   // warps sharing one 16-row tile
    constexpr int kKeysPerWarp = kStageKeys / kWarpsPerTile;
    constexpr int kNT = kKeysPerWarp / 8;                  // n-tiles of S per warp and stage

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + G_::kRingBytes);
    uint64_t *empty = full + kStages;
    uint32_t *const err_word = a.err ? a.err : &g_cross_rows_errors;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int split = blockIdx.x, kvh = blockIdx.y, src = blockIdx.z;
    const int G = a.group;
    const int P = a.page_size;
    const int tok0 = a.q_indptr[src];
    bool in_range;
    const int n_tok = source_tokens(tok0, a.q_indptr[src + 1], a.num_tokens, in_range);
    const int len = a.source_lens[src];
    const int most = min(a.max_src, a.bt_stride * P);
    if ((len > most || n_tok > a.max_q_len || !in_range) && threadIdx.x == 0)
        atomicOr(err_word, kErrContextRange);
    const int rows = min(n_tok, a.max_q_len) * G;
    if (rows <= 0)
        return;
    const int k_begin = split * a.chunk;
    const int k_end = min(min(len, most), k_begin + a.chunk);
    // where row r goes, counted in rows
    auto out_row = [&](int r) {
        const int m = r / G;
        return (static_cast<long long>(tok0 + m) * a.q_heads + static_cast<long long>(kvh) * G + r - m * G) *
                   a.n_split + split;
    };
    if (k_begin >= k_end) {
        // no position: zeros and -inf; an empty split's row is not read
        for (int idx = threadIdx.x; idx < rows * (D / 4); idx += kThreads) {
            const int r = idx / (D / 4), c = idx - r * (D / 4);
            if (a.n_split == 1)
                store_out4(a.out, a.out_f32, static_cast<size_t>(out_row(r)) * D + 4 * c,
                           make_float4(0.0f, 0.0f, 0.0f, 0.0f));
            if (c == 0 && a.lse != nullptr)
                a.lse[out_row(r)] = -INFINITY;
        }
        return;
    }
    const int n_blocks = (k_end - k_begin + kStageKeys - 1) / kStageKeys;
    const int n_pages = (k_end - k_begin + P - 1) / P;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kConsumerWarps);
        }
        fence_mbar_init();
    }
    __syncthreads();

    if (warp == kConsumerWarps) {
        // ------------------------ TMA producer (whole warp) -------------------------------
        const int32_t *bt_row = a.block_table + static_cast<size_t>(src) * a.bt_stride + k_begin / P;
        if (lane == 0) {
            prefetch_tensormap(&tmap_k);
            prefetch_tensormap(&tmap_v);
        }
        const uint64_t policy = l2_policy_evict_first();
        int cached_base = 0;
        int cached_page = lane < n_pages ? bt_row[lane] : 0;
        int issued = 0;
        bool ok = true;
        for (int b = 0; b < n_blocks; ++b) {
            const int st = b % kStages;
            if (b >= kStages &&
                !__all_sync(0xffffffffu, mbar_wait(&empty[st], ((b / kStages) - 1) & 1))) {
                ok = false;
                break;
            }
            const int keys = min(kStageKeys, k_end - k_begin - b * kStageKeys);
            const int np = (keys + P - 1) / P;
            if (lane == 0)
                mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(np * P * D * 2 * 2));
            __syncwarp();
            uint8_t *kdst = smem + st * G_::kStageBytes;
            uint8_t *vdst = kdst + G_::kTileBytes;
            const int lp0 = b * kStageKeys / P;   // first page of the stage inside this chunk
            if (lp0 + np > cached_base + 32) {
                cached_base = lp0;
                cached_page = (lp0 + lane < n_pages) ? bt_row[lp0 + lane] : 0;
            }
            // lane 2 i loads page i of K, lane 2 i + 1 page i of V
            const int i = lane >> 1;
            const int page = __shfl_sync(0xffffffffu, cached_page, (lp0 - cached_base + i) & 31);
            if (i < np) {
                const int off = i * P * D * 2;
                // NHD maps {64, slot, half, kv head}; HND maps {64, offset, half, block}
                const int c1 = a.hnd ? 0 : page * P;
                const int c3 = a.hnd ? page * a.kv_heads + kvh : kvh;
                tma_load_4d_hint((lane & 1 ? vdst : kdst) + off, lane & 1 ? &tmap_v : &tmap_k, 0, c1, 0, c3,
                                 &full[st], policy);
            }
            issued = b + 1;
        }
        if (!ok && lane == 0) {
            atomicOr(err_word, kErrCrossWait);
            for (int b = max(0, issued - kStages); b < issued; ++b)
                if (!mbar_wait(&full[b % kStages], (b / kStages) & 1))
                    atomicOr(err_word, kErrDrainWait);
        }
        return;
    }

    // --------------------------------- consumers -----------------------------------------
    const int mt = warp / kWarpsPerTile;   // this warp's 16-row tile
    const int ksl = warp % kWarpsPerTile;  // its slice of every stage's positions
    const int cq = (lane & 3) * 2;
    const int ra = mt * 16 + (lane >> 2);  // fragment rows ra and ra + 8
    const int rb = ra + 8;
    const bool va = ra < rows, vb = rb < rows;
    auto q_row_ptr = [&](int r) {
        const int m = r / G;
        const int gh = r - m * G;
        return a.q + (static_cast<size_t>(tok0 + m) * a.q_heads + static_cast<size_t>(kvh) * G + gh) * D;
    };
    uint32_t qa[D / 16][4];
    {
        const __nv_bfloat16 *qa_row = va ? q_row_ptr(ra) : nullptr;
        const __nv_bfloat16 *qb_row = vb ? q_row_ptr(rb) : nullptr;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const int c = kk * 16 + cq;
            qa[kk][0] = va ? *reinterpret_cast<const uint32_t *>(qa_row + c) : 0u;
            qa[kk][1] = vb ? *reinterpret_cast<const uint32_t *>(qb_row + c) : 0u;
            qa[kk][2] = va ? *reinterpret_cast<const uint32_t *>(qa_row + c + 8) : 0u;
            qa[kk][3] = vb ? *reinterpret_cast<const uint32_t *>(qb_row + c + 8) : 0u;
        }
    }
    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
        o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
    float m_a = -INFINITY, m_b = -INFINITY;

    // ldmatrix addresses.  Inside a stage tile, row `row` of half `h` starts at
    // ((row / P) * (D / 64) + h) * P * 128 + (row % P) * 128, and 16-byte chunk c of it sits
    // at chunk c ^ (row & 7).  Every row a lane addresses has row & 7 equal to lane & 7, so the
    // swizzled chunk of column tile j is (2 (j % 4) + c0) ^ (lane & 7), i.e. (32 (j % 4)) ^ x
    // bytes for a per-lane x: one add per ldmatrix once the row's offset is known.
    const int log2p = __ffs(P) - 1;
    const int half_bytes = P * 128;
    constexpr int kHalves = D / 64;
    constexpr int kPairs = kNT / 2;             // 16-key groups of a warp's slice
    const int k_row = ksl * kKeysPerWarp + (lane & 7) + ((lane >> 4) << 3);
    const int v_row = ksl * kKeysPerWarp + (lane & 7) + (((lane >> 3) & 1) << 3);
    auto row_offset = [&](int row) {
        return static_cast<uint32_t>(((row >> log2p) * kHalves) * half_bytes +
                                     (row & (P - 1)) * 128);
    };
    uint32_t k_x[4], v_x[4];
    {
        const uint32_t xk = static_cast<uint32_t>((((lane >> 3) & 1) ^ (lane & 7)) << 4);
        const uint32_t xv = static_cast<uint32_t>(((lane >> 4) ^ (lane & 7)) << 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            k_x[j] = (32u * j) ^ xk;
            v_x[j] = (32u * j) ^ xv;
        }
    }
    float l_a = 0.0f, l_b = 0.0f;   // this thread's columns' share of the rows' sums
    const float sl2 = a.scale_log2;
    bool ok = true;

    for (int b = 0; b < n_blocks; ++b) {
        const int st = b % kStages;
        if (!__all_sync(0xffffffffu, mbar_wait(&full[st], (b / kStages) & 1))) {
            ok = false;
            break;
        }
        const uint32_t kbase = smem_addr(smem + st * G_::kStageBytes);
        const uint32_t vbase = kbase + G_::kTileBytes;
        const int n_valid = k_end - (k_begin + b * kStageKeys + ksl * kKeysPerWarp);
        if (n_valid > 0) {
            float sc[kNT][4];
#pragma unroll
            for (int n = 0; n < kNT; ++n)
                sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
#pragma unroll
            for (int pr = 0; pr < kPairs; ++pr) {
                const uint32_t krow = kbase + row_offset(pr * 16 + k_row);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t b0, b1, b2, b3;
                    ldsm_x4(krow + (kk / 4) * half_bytes + k_x[kk % 4], b0, b1, b2, b3);
                    mma_bf16_16816(sc[2 * pr], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], b0,
                                   b1);
                    mma_bf16_16816(sc[2 * pr + 1], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3],
                                   b2, b3);
                }
            }
            if (n_valid < kKeysPerWarp) {   // warp-uniform: only the last slice of a chunk
#pragma unroll
                for (int n = 0; n < kNT; ++n) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (n * 8 + cq + e >= n_valid) {
                            sc[n][e] = -INFINITY;
                            sc[n][2 + e] = -INFINITY;
                        }
                    }
                }
            }
            float mx_a = fmax3(sc[0][0], sc[0][1], sc[1][0]);
            float mx_b = fmax3(sc[0][2], sc[0][3], sc[1][2]);
            mx_a = fmaxf(mx_a, sc[1][1]);
            mx_b = fmaxf(mx_b, sc[1][3]);
#pragma unroll
            for (int n = 2; n < kNT; ++n) {
                mx_a = fmax3(mx_a, sc[n][0], sc[n][1]);
                mx_b = fmax3(mx_b, sc[n][2], sc[n][3]);
            }
            mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, 1));
            mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, 2));
            mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, 1));
            mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, 2));
            const float mn_a = fmaxf(m_a, mx_a * sl2), mn_b = fmaxf(m_b, mx_b * sl2);
            if (__any_sync(0xffffffffu, (mn_a > m_a) || (mn_b > m_b))) {
                const float al_a = (m_a == -INFINITY) ? 0.0f : fast_exp2(m_a - mn_a);
                const float al_b = (m_b == -INFINITY) ? 0.0f : fast_exp2(m_b - mn_b);
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    o[n][0] *= al_a;
                    o[n][1] *= al_a;
                    o[n][2] *= al_b;
                    o[n][3] *= al_b;
                }
                l_a *= al_a;
                l_b *= al_b;
                m_a = mn_a;
                m_b = mn_b;
            }
            const float nu_a = (m_a == -INFINITY) ? 0.0f : -m_a;
            const float nu_b = (m_b == -INFINITY) ? 0.0f : -m_b;
            uint32_t pa[kNT][2];
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
                const float a0 = fast_exp2(fmaf(sc[n][0], sl2, nu_a));
                const float a1 = fast_exp2(fmaf(sc[n][1], sl2, nu_a));
                const float b0 = fast_exp2(fmaf(sc[n][2], sl2, nu_b));
                const float b1 = fast_exp2(fmaf(sc[n][3], sl2, nu_b));
                l_a += a0 + a1;
                l_b += b0 + b1;
                pa[n][0] = pack_bf16x2(a0, a1);
                pa[n][1] = pack_bf16x2(b0, b1);
            }
#pragma unroll
            for (int ks = 0; ks < kPairs; ++ks) {
                if (ks * 16 >= n_valid)
                    break;
                const bool partial = n_valid < (ks + 1) * 16;
                const uint32_t vrow = vbase + row_offset(ks * 16 + v_row);
#pragma unroll
                for (int dt = 0; dt < D / 16; ++dt) {
                    uint32_t v0, v1, v2, v3;
                    ldsm_x4_trans(vrow + (dt / 4) * half_bytes + v_x[dt % 4], v0, v1, v2, v3);
                    if (partial) {
                        v0 = keep_keys(v0, ks * 16 + cq, n_valid);
                        v1 = keep_keys(v1, ks * 16 + 8 + cq, n_valid);
                        v2 = keep_keys(v2, ks * 16 + cq, n_valid);
                        v3 = keep_keys(v3, ks * 16 + 8 + cq, n_valid);
                    }
                    mma_bf16_16816(o[2 * dt], pa[2 * ks][0], pa[2 * ks][1], pa[2 * ks + 1][0],
                                   pa[2 * ks + 1][1], v0, v1);
                    mma_bf16_16816(o[2 * dt + 1], pa[2 * ks][0], pa[2 * ks][1],
                                   pa[2 * ks + 1][0], pa[2 * ks + 1][1], v2, v3);
                }
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&empty[st]);
    }
    if (!ok)
        atomicOr(err_word, kErrCrossWait);
    l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
    l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
    l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
    l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);

    // ------------------- combine the warps of each tile, write partials --------------------
    // Warp w of tile t leaves its unnormalised o (rows of D + 8 floats: the pad spreads the
    // 8 rows a store instruction touches over distinct banks), its running max and row sum.
    // One thread per output row then folds the tile's warps into weights 2^(m_w - M) / L
    // and finds where the row goes; the write-out is float4 loads and stores.
    constexpr int kRowStride = D + 8;
    named_barrier(1, kConsumerWarps * 32);   // every warp is done with the ring
    float *red_o = reinterpret_cast<float *>(smem);                        // [W][16][D + 8]
    float *red_m = red_o + kConsumerWarps * 16 * kRowStride;                // [W][16]
    float *red_l = red_m + kConsumerWarps * 16;                             // [W][16]
    float *row_w = red_l + kConsumerWarps * 16;                             // [rows][W / tile]
    long long *row_slot = reinterpret_cast<long long *>(row_w + kMaxRows * kWarpsPerTile);
    {
        const int la = lane >> 2, lb = la + 8;
        float *dst_a = red_o + (warp * 16 + la) * kRowStride + cq;
        float *dst_b = red_o + (warp * 16 + lb) * kRowStride + cq;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            *reinterpret_cast<float2 *>(dst_a + n * 8) = make_float2(o[n][0], o[n][1]);
            *reinterpret_cast<float2 *>(dst_b + n * 8) = make_float2(o[n][2], o[n][3]);
        }
        if ((lane & 3) == 0) {
            red_m[warp * 16 + la] = m_a;
            red_l[warp * 16 + la] = l_a;
            red_m[warp * 16 + lb] = m_b;
            red_l[warp * 16 + lb] = l_b;
        }
    }
    named_barrier(1, kConsumerWarps * 32);
    for (int r = threadIdx.x; r < rows; r += kConsumerWarps * 32) {
        const int slot0 = (r >> 4) * kWarpsPerTile * 16 + (r & 15);
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarpsPerTile; ++w)
            M = fmaxf(M, red_m[slot0 + w * 16]);
        float f[kWarpsPerTile];
        float L = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarpsPerTile; ++w) {
            const float mw = red_m[slot0 + w * 16];
            f[w] = (mw == -INFINITY) ? 0.0f : fast_exp2(mw - M);
            L += f[w] * red_l[slot0 + w * 16];
        }
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;   // NaN stays NaN
#pragma unroll
        for (int w = 0; w < kWarpsPerTile; ++w)
            row_w[r * kWarpsPerTile + w] = f[w] * inv;
        row_slot[r] = out_row(r);
        if (a.lse != nullptr)
            a.lse[row_slot[r]] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
    }
    named_barrier(1, kConsumerWarps * 32);
    constexpr int kVec = D / 4;
    for (int idx = threadIdx.x; idx < rows * kVec; idx += kConsumerWarps * 32) {
        const int r = idx / kVec;
        const int c = (idx - r * kVec) * 4;
        const float *src = red_o + ((r >> 4) * kWarpsPerTile * 16 + (r & 15)) * kRowStride + c;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarpsPerTile; ++w) {
            const float wt = row_w[r * kWarpsPerTile + w];
            const float4 v = *reinterpret_cast<const float4 *>(src + w * 16 * kRowStride);
            acc.x = fmaf(wt, v.x, acc.x);
            acc.y = fmaf(wt, v.y, acc.y);
            acc.z = fmaf(wt, v.z, acc.z);
            acc.w = fmaf(wt, v.w, acc.w);
        }
        store_out4(a.out, a.out_f32, static_cast<size_t>(row_slot[r]) * D + c, acc);
    }
}


template <int D, int NMT>
cudaError_t launch_t(const CrossLaunch &l, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t stream)
{
    Args a;
    const bool split = l.n_split > 1;
    a.q = static_cast<const __nv_bfloat16 *>(l.q);
    a.out = split ? l.part_o : l.out;
    a.out_f32 = split || l.out_f32 ? 1 : 0;
    a.lse = split ? l.part_lse : l.lse;
    a.block_table = l.block_table;
    a.bt_stride = l.bt_stride;
    a.q_indptr = l.q_indptr;
    a.source_lens = l.source_lens;
    a.q_heads = l.q_heads;
    a.kv_heads = l.kv_heads;
    a.group = l.q_heads / l.kv_heads;
    a.page_size = l.page_size;
    a.num_tokens = l.num_tokens;
    a.max_q_len = l.max_q_len;
    a.max_src = l.max_src;
    a.chunk = l.chunk;
    a.n_split = l.n_split;
    a.scale_log2 = l.scale * kLog2e;
    a.hnd = l.hnd ? 1 : 0;
    a.err = current_error_word();
    auto kernel = cross_rows_kernel<D, NMT>;
    const size_t smem = Geom<D>::kSmemBytes;
    const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(smem));
    if (err != cudaSuccess)
        return err;
    return launch_pdl(kernel, dim3(l.n_split, l.kv_heads, l.num_sources), dim3(kThreads), smem, stream, tk,
                      tv, a);
}

}  // namespace

cudaError_t launch_cross_rows(const CrossLaunch &l, const CUtensorMap &tmap_k, const CUtensorMap &tmap_v,
                              cudaStream_t stream)
{
    const int rows = l.max_q_len * (l.q_heads / l.kv_heads);
    if (rows > kCrossFewRows || l.kv_heads > 65535)
        return cudaErrorInvalidValue;
    if (l.head_dim == 128)
        return rows <= 16 ? launch_t<128, 1>(l, tmap_k, tmap_v, stream)
                          : launch_t<128, 2>(l, tmap_k, tmap_v, stream);
    return rows <= 16 ? launch_t<64, 1>(l, tmap_k, tmap_v, stream)
                      : launch_t<64, 2>(l, tmap_k, tmap_v, stream);
}

cudaError_t read_and_clear_cross_rows_errors(uint32_t *flags)
{
    uint32_t zero = 0;
    cudaError_t err = cudaMemcpyFromSymbol(flags, g_cross_rows_errors, sizeof(uint32_t));
    if (err != cudaSuccess)
        return err;
    return cudaMemcpyToSymbol(g_cross_rows_errors, &zero, sizeof(uint32_t));
}

}  // namespace kvc
