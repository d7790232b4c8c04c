// kvc_launch.h -- host-side launchers of the kvc kernels (internal; the C ABI is kvc.h).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kvc {

// The device word that the calling host thread named with kvc_set_error_word, or nullptr (the
// kernels then set bits in their translation unit's own word, read by kvc_device_errors).
uint32_t *current_error_word();

// Streaming multiprocessors of the current device (152 where there is none).
int current_sm_count();

// Launch with programmatic stream serialisation (see pdl_wait / pdl_trigger in kvc_device.cuh):
// the kernel may start before the previous launch on the stream has finished and waits for it
// in its first instruction.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args &&>(args)...);
}

struct DecodeLaunch {
    const void *q;
    void *out;
    int out_f32;
    float *part_o;            // [S][Hq][n_split][D] when n_split > 1
    float *part_lse;          // [S][Hq][n_split]
    const int32_t *block_table;
    int bt_stride;
    const int32_t *context_lens;
    int num_seqs, q_heads, kv_heads, head_dim, page_size;
    int chunk, n_split;
    float scale;
    // Optional, for decode over a suffix: keys start at key_start[s] (a multiple of page
    // size), and the partials of this launch are splits split_base .. of split_stride.
    const int32_t *key_start = nullptr;
    int split_base = 0;
    int split_stride = 0;   // 0: n_split
    bool hnd = false;       // pools in the HND layout (the tensor maps follow it too)
    // Fused store (kvc_decode_store): new K / V [S][Hkv][D] and the writable pools.
    const void *k_new = nullptr, *v_new = nullptr;
    void *k_pool_w = nullptr, *v_pool_w = nullptr;
    int num_slots = 0;
};

// Decode over INT8 pages (head_dim 64 or 128): codes like a bf16 pool, scales [pages][Hkv][P].
// The positions of all (sequence, kv head) units are cut into n_ctas equal runs of 64-position
// blocks (one CTA each), whose pieces are merged by a second launch; per_unit runs one CTA per
// unit instead and writes the output directly (no workspace, no merge).
struct DecodeInt8Launch {
    const void *q;
    const float *k_scales, *v_scales;
    void *out;
    int out_f32;
    float *part_o = nullptr;      // [units + n_ctas][G][D]
    float *part_lse = nullptr;    // [units + n_ctas][G]
    void *unit_info = nullptr;    // [units] int2: first partial slot, piece count
    const int32_t *block_table;
    int bt_stride;
    const int32_t *context_lens;
    int num_seqs, q_heads, kv_heads, page_size;
    int n_ctas = 1;
    bool per_unit = false;
    float scale;
    // fused store (kvc_decode_int8_store): new K/V [S][Hkv][D] bf16 and the pools to write
    const void *k_new = nullptr, *v_new = nullptr;
    void *k_codes_w = nullptr, *v_codes_w = nullptr;
    float *k_scales_w = nullptr, *v_scales_w = nullptr;
    int num_slots = 0;
    int head_dim = 128;
    bool hnd = false;   // codes [pages][Hkv][P][D] (the tensor maps follow it too)
};
cudaError_t launch_decode_int8(const DecodeInt8Launch &l, const CUtensorMap &tmap_k,
                               const CUtensorMap &tmap_v, cudaStream_t stream);
cudaError_t read_and_clear_decode_int8_errors(uint32_t *flags);

// Pools of 4-bit pages: codes [pages][P][Hkv][D / 2] (HND: [pages][Hkv][P][D / 2]), two to a byte;
// parameters [pages][Hkv][P][D / 64] pairs of bf16 (scale, minimum).
struct Int4Pools {
    void *k_codes, *v_codes, *k_params, *v_params;
    int num_pages, page_size, kv_heads, head_dim;
    bool hnd;
};
cudaError_t launch_store_int4(const Int4Pools &p, const void *k_new, const void *v_new,
                              const int32_t *slots, int num_tokens, cudaStream_t stream);
cudaError_t launch_load_int4(const Int4Pools &p, void *k_out, void *v_out, bool out_f32,
                             const int32_t *slots, int num_tokens, cudaStream_t stream);
cudaError_t read_and_clear_store_int4_errors(uint32_t *flags);

// Decode over 4-bit pages: the positions of all sequences, in kInt4Block-position blocks, are cut
// into `runs` runs of equal cost per kv head (one warp each); per_unit: one run per sequence, no
// workspace and no merge.
constexpr int kInt4Block = 64;
constexpr int kInt4Warps = 8;   // consumer warps of a CTA, one CTA per SM
// kv heads that a group of warps takes together: the largest divisor of their number up to 8.
int int4_group_heads(int kv_heads);
struct DecodeInt4Launch {
    Int4Pools pools;
    const void *q;
    void *out;
    bool out_f32;
    float *part_o = nullptr;      // [Hkv (S + runs)][G][D]
    float *part_lse = nullptr;    // [Hkv (S + runs)][G]
    void *unit_info = nullptr;    // [S][Hkv] int2: first partial slot, piece count
    const int32_t *block_table;
    int bt_stride;
    const int32_t *context_lens;
    int num_seqs, q_heads;
    int runs = 1;
    bool per_unit = false;
    float scale;
};
// maps: K and V codes, K and V parameters, with boxes of min(page_size, kInt4Block) positions of
// int4_group_heads(kv_heads) kv heads, which land as [head][position][bytes].
cudaError_t launch_decode_int4(const DecodeInt4Launch &l, const CUtensorMap (&maps)[4],
                               cudaStream_t stream);
cudaError_t read_and_clear_decode_int4_errors(uint32_t *flags);

// kvc_decode_weights: the decode of `l` (its partials for every split, also when there is one), its
// scores [S][Hq][score_stride] and exact log2-sum-exp2s [S][Hq][n_split], added up into weights
// [num_rows][Hkv][weight_stride].
struct WeightsLaunch {
    float *weights;
    const int32_t *rows;   // [S] or null
    int num_rows, weight_stride, max_ctx;
    float *scores;
    size_t score_stride;
    float *part_lse2;
};
cudaError_t launch_decode_weights(const DecodeLaunch &l, const WeightsLaunch &w,
                                  const CUtensorMap &tmap_k, const CUtensorMap &tmap_v,
                                  cudaStream_t stream);
cudaError_t read_and_clear_weights_errors(uint32_t *flags);

// kvc_evict: the moves of each (sequence, kv head), lists [S][Hkv][2][list_cap] and counts
// [S][Hkv][2].
constexpr int kEvictCtaSlots = 1 << 19;   // slots of one CTA (masks of 2 bits each)
constexpr int kEvictMaxCtx = 1 << 22;     // slots of a row: 8 CTAs
struct EvictLaunch {
    void *k_pool, *v_pool;
    const int32_t *block_table;
    int bt_stride;
    const int32_t *context_lens;
    int num_seqs, max_ctx;
    const float *weights;
    const int32_t *positions;
    float *weights_out;
    int32_t *positions_out;
    const int32_t *rows;   // [S] or null
    int num_rows, stride;
    int budget, recent;
    int32_t *new_lens;
    int32_t *lists = nullptr, *counts = nullptr;   // null without a possible move (list_cap 0)
    int list_cap = 0;
    int kv_heads, head_dim, page_size, num_pages;
    bool hnd;
};
cudaError_t launch_evict(const EvictLaunch &l, cudaStream_t stream);
cudaError_t read_and_clear_evict_errors(uint32_t *flags);

// Rotary positions: of each pair its angle per unit of position, as a 64-bit fraction of a turn, and the
// axis (row of positions) that it goes by.
constexpr int kRopePairs = 64;
constexpr int kRopeAxes = 8;
struct RopeAngles {
    uint64_t turns[kRopePairs];
    uint8_t axis[kRopePairs];
};
struct RopeLaunch {
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;         // elements between tokens
    void *q_out, *k_out, *v_out;                    // with slots: k_out and v_out are the pools
    long long q_out_stride, k_out_stride = 0;
    const int32_t *positions;                       // [axes][num_tokens]
    const int32_t *slots = nullptr;                 // null: k_out takes the rows, no values
    int num_tokens, q_heads, kv_heads, head_dim, rotary_dim;
    int page_size = 1, num_slots = 0;
    bool hnd = false, adjacent = false;
    RopeAngles angles;
};
cudaError_t launch_rope(const RopeLaunch &l, cudaStream_t stream);
cudaError_t read_and_clear_rope_errors(uint32_t *flags);

// Pages handed out, shared, given back and closed up: a table of rows, the references of every page, and the
// arrays whose pages are copied along.
struct PageArray {
    void *data;
    long long page_bytes;
};
struct PagesLaunch {
    int32_t *block_table;
    int bt_stride;
    int32_t *context_lens;
    int num_seqs;
    int32_t *page_refs;
    int num_pages, page_size;
    const PageArray *arrays = nullptr;   // host
    int num_arrays = 0;
};
size_t reserve_workspace_bytes(int num_seqs, int num_pages);
size_t compact_workspace_bytes(int num_pages);
cudaError_t launch_truncate(const PagesLaunch &l, const int32_t *new_lens, cudaStream_t stream);
cudaError_t launch_fork(const PagesLaunch &l, int32_t *out_rows, int out_stride, int32_t *out_lens,
                        const int32_t *parents, const int32_t *share_lens, int num_out, cudaStream_t stream);
cudaError_t launch_reserve(const PagesLaunch &l, const int32_t *new_tokens, int32_t *missing,
                           void *workspace, cudaStream_t stream);
cudaError_t launch_compact(const PagesLaunch &l, int32_t *page_map, int32_t *num_live, void *workspace,
                           cudaStream_t stream);
cudaError_t read_and_clear_pages_errors(uint32_t *flags);

// Grouped decode over a shared prefix: for each group, the first prefix_len[g] positions are
// the same pages for every member (the leader's block-table row lists them).
struct GroupedPrefixLaunch {
    const void *q;
    float *part_o;            // [S][Hq][split_stride][D]
    float *part_lse;          // [S][Hq][split_stride]
    const int32_t *block_table;
    int bt_stride;
    const int32_t *group_indptr;   // [num_groups + 1] into group_seqs
    const int32_t *group_seqs;
    const int32_t *prefix_len;     // [num_groups]
    int num_groups, max_rows;      // max_rows = largest group size * G (<= 64)
    int num_seqs, q_heads, kv_heads, head_dim, page_size;
    int chunk, n_split, split_stride;
    float scale;
    bool hnd = false;
    // at most this many prefix CTAs, each taking every max_prefix_ctas-th work item after its
    // first (0: one CTA per item)
    int max_prefix_ctas = 0;
};

struct AppendLaunch {
    const void *q;
    void *out;
    int out_f32;
    const int32_t *block_table;
    int bt_stride;
    const int32_t *q_indptr;
    const int32_t *context_lens;
    int num_seqs, num_tokens, max_q_len, q_heads, kv_heads, head_dim, page_size;
    float scale;
    bool hnd = false;
    // kvc_append_store: the chunk's K/V come from k_new / v_new (tmap_kn / tmap_vn) and the
    // kernel writes them to the pools (k_pool_w / v_pool_w), except the boundary tokens
    // launch_store_boundary wrote before.
    bool fused = false;
    void *k_pool_w = nullptr, *v_pool_w = nullptr;
    int num_pages = 0;   // pages of the pools (fused: a page id outside them is skipped)
};

// kvc_append_int8: AppendLaunch over INT8 pages (head_dim 64 or 128) plus the scale arrays.
struct AppendInt8Launch {
    void *out;
    int out_f32;
    const float *k_scales, *v_scales;   // [num_pages][kv_heads][page_size]
    const int32_t *block_table;
    int bt_stride;
    const int32_t *q_indptr;
    const int32_t *context_lens;
    int num_seqs, num_tokens, max_q_len, q_heads, kv_heads, page_size;
    float scale;
    int head_dim = 128;
    bool hnd = false;   // codes [pages][Hkv][P][D] (the tensor maps follow it too)
};

// kvc_cross: queries against a source's pages, every position seen by every query; positions in n_split
// chunks of `chunk` (a multiple of kCrossBlock), joined by a second launch when there are several.
constexpr int kCrossBlock = 128;
constexpr int kCrossFewRows = 32;   // rows of a (source, kv head) up to which launch_cross_rows may take them
struct CrossLaunch {
    const void *q;
    void *out;
    bool out_f32;
    float *lse;                                      // [T][Hq] or null
    float *part_o = nullptr, *part_lse = nullptr;    // [T][Hq][n_split][D], [T][Hq][n_split]
    const int32_t *block_table;
    int bt_stride;
    const int32_t *q_indptr, *source_lens;
    int num_sources, num_tokens, max_q_len, max_src, q_heads, kv_heads, head_dim, page_size;
    int chunk, n_split;
    float scale;
    bool hnd;
};
// A (source, kv head) has few rows: chunks of a multiple of kStageKeys, maps as for launch_decode.
cudaError_t launch_cross_rows(const CrossLaunch &l, const CUtensorMap &tmap_k, const CUtensorMap &tmap_v,
                              cudaStream_t stream);
// The join of either kernel's splits.
cudaError_t launch_cross_merge(const CrossLaunch &l, cudaStream_t stream);
cudaError_t read_and_clear_cross_rows_errors(uint32_t *flags);
// tmap_q as for launch_append_tc; tmap_k / tmap_v with a box per page, [group of 8 positions][column half][8][64]
cudaError_t launch_cross(const CrossLaunch &l, const CUtensorMap &tmap_q, const CUtensorMap &tmap_k,
                         const CUtensorMap &tmap_v, cudaStream_t stream);
cudaError_t read_and_clear_cross_errors(uint32_t *flags);

// kvc_validate: the smallest offending index of each check (INT32_MAX when it passed), then two
// bitmaps over the pool's slots.
constexpr int kValidateChecks = 4;
struct ValidateRecord {
    int first_bad[kValidateChecks];
};
size_t validate_workspace_bytes(long long num_slots);
cudaError_t launch_validate(const int32_t *block_table, int bt_stride, const int32_t *context_lens,
                            int num_seqs, const int32_t *slots, int num_tokens, int page_size,
                            int num_pages, void *workspace, cudaStream_t stream);

// Each returns cudaSuccess or the launch error.
cudaError_t launch_slot_mapping(int32_t *slots, const int32_t *block_table, int bt_stride,
                                const int32_t *context_lens, const int32_t *q_indptr,
                                int num_seqs, int num_tokens, int max_q_len, int page_size,
                                cudaStream_t stream);
cudaError_t launch_store(void *k_pool, void *v_pool, int kv_heads, int head_dim,
                         int num_slots, const void *k_new, const void *v_new,
                         const int32_t *slots, int num_tokens, cudaStream_t stream,
                         bool hnd = false, int page_size = 1);
cudaError_t launch_store_int8(void *k_codes, void *v_codes, float *k_scales, float *v_scales,
                              int kv_heads, int head_dim, int page_size, int num_slots,
                              const void *k_new, const void *v_new, const int32_t *slots,
                              int num_tokens, cudaStream_t stream, bool hnd = false);
cudaError_t launch_copy_pages(void *k_pool, void *v_pool, int num_pages, int page_size,
                              int kv_heads, int head_dim, const int32_t *src_pages,
                              const int32_t *dst_pages, int num_copies, cudaStream_t stream);
cudaError_t launch_decode(const DecodeLaunch &a, const CUtensorMap &tmap_k,
                          const CUtensorMap &tmap_v, cudaStream_t stream);
cudaError_t launch_merge(void *out, int out_f32, const float *part_o, const float *part_lse,
                         int rows, int n_split, int head_dim, float *lse_out,
                         cudaStream_t stream);
// Grouped decode: sets key_start to 0, then each group's members' key_start to the group's
// prefix length (one block; the grouped grid marks the empty prefix partials itself).
cudaError_t launch_grouped_setup(int32_t *key_start, const int32_t *group_indptr,
                                 const int32_t *group_seqs, const int32_t *prefix_len,
                                 int num_groups, int num_seqs, int page_size, int bt_stride,
                                 cudaStream_t stream);
// Groups from block tables (adjacent sequences agreeing on leading shareable pages), one CTA:
// group_indptr[num_seqs / 2 + 1], group_seqs[num_seqs], prefix_len[num_seqs / 2], num_groups[1].
cudaError_t launch_group_detect(const int32_t *block_table, int bt_stride,
                                const int32_t *context_lens, int num_seqs, int page_size,
                                int max_members, int32_t *group_indptr, int32_t *group_seqs,
                                int32_t *prefix_len, int32_t *num_groups, cudaStream_t stream);
// The prefix CTAs of `p` and the suffix decode of `l` (key_start set, partials after the
// prefix splits) in one grid.
cudaError_t launch_grouped_decode(const GroupedPrefixLaunch &p, const DecodeLaunch &l,
                                  const CUtensorMap &tmap_k, const CUtensorMap &tmap_v,
                                  cudaStream_t stream);
// tmap_q views q as [T][kv_heads][G][head_dim] with 128-row boxes; tmap_kn / tmap_vn (fused
// only) view k_new / v_new as {head_dim, kv head, token} with {64, 1, page_size} boxes.
cudaError_t launch_append_tc(const AppendLaunch &a, const CUtensorMap &tmap_q,
                             const CUtensorMap &tmap_k, const CUtensorMap &tmap_v,
                             cudaStream_t stream, const CUtensorMap *tmap_kn = nullptr,
                             const CUtensorMap *tmap_vn = nullptr);
// The new tokens that share a page with cached positions (the chunk's first page when
// (ctx - q_len) % page_size != 0), stored at their slots from the block table.
cudaError_t launch_store_boundary(void *k_pool, void *v_pool, int kv_heads, int head_dim,
                                  int page_size, int num_slots, bool hnd, const void *k_new,
                                  const void *v_new, const int32_t *block_table, int bt_stride,
                                  const int32_t *q_indptr, const int32_t *context_lens,
                                  int num_seqs, bool whole, cudaStream_t stream);
// tmap_q as for launch_append_tc; tmap_k / tmap_v are the INT8 page maps (one box per page).
cudaError_t launch_append_int8(const AppendInt8Launch &a, const CUtensorMap &tmap_q,
                               const CUtensorMap &tmap_k, const CUtensorMap &tmap_v,
                               cudaStream_t stream);

// Device error words, one per translation unit that owns bounded waits.
cudaError_t read_and_clear_decode_errors(uint32_t *flags);
// One CTA whose bounded wait runs out (about a second): sets kErrSelftestWait.
cudaError_t launch_selftest_wait(cudaStream_t stream);
cudaError_t read_and_clear_store_errors(uint32_t *flags);
cudaError_t read_and_clear_append_tc_errors(uint32_t *flags);
cudaError_t read_and_clear_grouped_errors(uint32_t *flags);
cudaError_t read_and_clear_append_int8_errors(uint32_t *flags);

// Record a failure reason for kvc_last_error() from another translation unit.
int set_last_error(int status, const char *message);

// Stage geometry shared by the decode and append pipelines: a stage holds kStageKeys
// positions of one kv head as whole pages, each page stored [half][page_size rows][64 columns]
// with 128-byte swizzle (one TMA box per page).
constexpr int kStageKeys = 64;   // positions per pipeline stage

}  // namespace kvc
