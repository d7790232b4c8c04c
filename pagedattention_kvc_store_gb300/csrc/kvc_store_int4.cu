// kvc_store_int4.cu -- 4-bit pages: quantising store of new keys/values, and the way back.
//
// A vector (one kv head at one position, D values) is held as D / 64 groups of 64 values.  With
// lo and hi a group's smallest and largest value,
//   scale = bf16((hi / 2 - lo / 2) / 7.5),  code = clamp(rint((x / 2 - lo / 2) / (scale / 2)), 0, 15),
// all in fp32 with round-to-nearest (the halves keep hi - lo inside fp32 for every bf16 input and
// change nothing else), and x stands for scale * code + lo.  lo is one of the bf16 inputs, so it
// is exact in bf16; the rounding of scale to bf16 moves the largest value by at most
// 15 * 2^-9 = 0.03 of a step, against the half step that the codes lose anyway, and keeps the
// parameters at 4 bytes a group (72 bytes a vector at D = 128, 3.6 times below bf16).  A group
// with equal values stores scale 0 and is exact; one with a NaN or an infinity cannot be
// represented and stores NaN for both, so that attention over it is NaN rather than wrong.
//
// Codes: byte j of a vector holds dim 2 j in its low and 2 j + 1 in its high four bits; vectors lie
// as in a bf16 pool ([slot][kv head], or [page][kv head][offset] for HND).  Parameters: bf16
// (scale, lo) at [page][kv head][offset][group], so the page's run for one kv head is contiguous.
//
// Both kernels are bound by HBM (328 bytes a vector at D = 128).  Eight lanes take a group, one
// 16-byte load of 8 values each; the K and V vectors of one (token, kv head) go to neighbouring
// lanes.  The codes need a correctly rounded quotient, but a division per value would make the
// store bound by instructions (about 12 a value): the product with the approximate reciprocal
// is off by less than 1e-5 of a step, so only quotients that close to a tie take the division.
#include <math.h>

#include "kvc_device.cuh"
#include "kvc_launch.h"

namespace kvc {

namespace {

__device__ uint32_t g_store_int4_errors;

constexpr int kThreads = 256;

// The vector (K or V of one token and kv head) that a lane works on, and its place in the pools.
struct Place {
    bool live;        // the token has a slot inside the pool
    size_t code_row;  // vector index in the code pool
    size_t par_row;   // vector index in the parameter pool
};

__device__ __forceinline__ Place place_of(int slot, int g, int kv_heads, int log2_page,
                                          int num_slots, bool hnd, uint32_t *err, bool report)
{
    Place p;
    p.live = slot >= 0 && slot < num_slots;
    if (slot >= num_slots && report)
        atomicOr(err, kErrSlotRange);
    const int page = slot >> log2_page;
    const int off = slot & ((1 << log2_page) - 1);
    p.par_row = ((static_cast<size_t>(page) * kv_heads + g) << log2_page) + off;
    p.code_row = hnd ? p.par_row : static_cast<size_t>(slot) * kv_heads + g;
    return p;
}

// L lanes per vector (D = 8 L).  Work item w = (token, kv head, K or V), V fastest: 2 L lanes read
// the K and V vectors of one (token, kv head).
template <int L>
__global__ void __launch_bounds__(kThreads)
    store_int4_kernel(uint32_t *__restrict__ k_codes, uint32_t *__restrict__ v_codes,
                      uint32_t *__restrict__ k_params, uint32_t *__restrict__ v_params,
                      const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new,
                      const int32_t *__restrict__ slots, int num_tokens, int kv_heads,
                      int log2_page, int num_slots, bool hnd, uint32_t *word)
{
    pdl_wait();
    pdl_trigger();
    uint32_t *err = word ? word : &g_store_int4_errors;
    const long long items = static_cast<long long>(num_tokens) * kv_heads * 2;
    const long long step = static_cast<long long>(gridDim.x) * (kThreads / L);
    const int c = threadIdx.x % L;   // 16-byte chunk of the vector
    // every lane of a warp goes round together (the shuffles below), so the bound is the warp's
    const long long w_first = static_cast<long long>(blockIdx.x) * (kThreads / L) + threadIdx.x / L;
    const long long warp_first = w_first - (threadIdx.x & 31) / L;
    for (long long w0 = warp_first; w0 < items; w0 += step) {
        const long long w = w0 + (threadIdx.x & 31) / L;
        const bool in = w < items;
        const bool is_v = w & 1;
        const long long vec = in ? w >> 1 : 0;
        const int t = static_cast<int>(vec / kv_heads);
        const int g = static_cast<int>(vec - static_cast<long long>(t) * kv_heads);
        const int slot = in ? __ldcg(slots + t) : -1;
        const Place p = place_of(slot, g, kv_heads, log2_page, num_slots, hnd, err,
                                 c == 0 && g == 0);
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (p.live)
            x = load_streaming((is_v ? v_new : k_new) + vec * L + c);
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(xw[i] << 16);
            f[2 * i + 1] = __uint_as_float(xw[i] & 0xFFFF0000u);
        }
        // smallest and largest value, and whether all are finite (|x| of the bits below the
        // exponent of infinity)
        float lo = f[0], hi = f[0];
        bool finite = true;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo = fminf(lo, f[i]);
            hi = fmaxf(hi, f[i]);
            finite = finite && (__float_as_uint(f[i]) & 0x7F800000u) != 0x7F800000u;
        }
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
        }
        const uint32_t bad = __ballot_sync(0xffffffffu, !finite);
        const bool group_ok = ((bad >> (threadIdx.x & 24)) & 0xFFu) == 0;
        if (!p.live)
            continue;
        const float lo_half = lo * 0.5f;
        const __nv_bfloat16 scale16 =
            __float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi * 0.5f, lo_half), 7.5f));
        const float scale_half = __bfloat162float(scale16) * 0.5f;
        uint32_t packed = 0;
        uint32_t param = 0x7FC07FC0u;   // NaN, NaN
        if (group_ok) {
            param = static_cast<uint32_t>(__bfloat16_as_ushort(scale16)) |
                    (__float_as_uint(lo) & 0xFFFF0000u);
            if (scale_half > 0.0f) {
                const float inv = __frcp_rn(scale_half);   // infinite for the smallest scales:
                                                           // the quotient is then divided out
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float a = __fsub_rn(f[i] * 0.5f, lo_half);
                    float q = a * inv;
                    float r = rintf(q);
                    if (!(fabsf(q - r) < 0.4999f))
                        r = rintf(__fdiv_rn(a, scale_half));
                    packed |= static_cast<uint32_t>(fminf(r, 15.0f)) << (4 * i);
                }
            }
        }
        (is_v ? v_codes : k_codes)[p.code_row * L + c] = packed;
        if ((c & 7) == 0)
            (is_v ? v_params : k_params)[p.par_row * (L / 8) + c / 8] = param;
    }
}

// The values that 4-bit pages hold at the given slots, as bf16 (rounded to nearest even) or fp32:
// scale * code is exact in fp32 (4 by 8 bits) and the sum with lo rounds once.
template <int L, bool F32>
__global__ void __launch_bounds__(kThreads)
    load_int4_kernel(uint4 *__restrict__ k_out, uint4 *__restrict__ v_out,
                     const uint32_t *__restrict__ k_codes, const uint32_t *__restrict__ v_codes,
                     const uint32_t *__restrict__ k_params, const uint32_t *__restrict__ v_params,
                     const int32_t *__restrict__ slots, int num_tokens, int kv_heads,
                     int log2_page, int num_slots, bool hnd, uint32_t *word)
{
    pdl_wait();
    pdl_trigger();
    uint32_t *err = word ? word : &g_store_int4_errors;
    const long long items = static_cast<long long>(num_tokens) * kv_heads * 2;
    const long long step = static_cast<long long>(gridDim.x) * (kThreads / L);
    const int c = threadIdx.x % L;
    for (long long w = static_cast<long long>(blockIdx.x) * (kThreads / L) + threadIdx.x / L;
         w < items; w += step) {
        const bool is_v = w & 1;
        const long long vec = w >> 1;
        const int t = static_cast<int>(vec / kv_heads);
        const int g = static_cast<int>(vec - static_cast<long long>(t) * kv_heads);
        const Place p = place_of(__ldcg(slots + t), g, kv_heads, log2_page, num_slots, hnd, err,
                                 c == 0 && g == 0);
        float v[8];
        if (p.live) {
            const uint32_t codes = __ldcg((is_v ? v_codes : k_codes) + p.code_row * L + c);
            const uint32_t par = __ldcg((is_v ? v_params : k_params) + p.par_row * (L / 8) + c / 8);
            const float scale = __uint_as_float(par << 16);
            const float lo = __uint_as_float(par & 0xFFFF0000u);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = fmaf(scale, static_cast<float>((codes >> (4 * i)) & 15u), lo);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = 0.0f;
        }
        uint4 *out = is_v ? v_out : k_out;
        if (F32) {
            out += (vec * L + c) * 2;
            out[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]),
                                __float_as_uint(v[2]), __float_as_uint(v[3]));
            out[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]),
                                __float_as_uint(v[6]), __float_as_uint(v[7]));
        } else {
            out[vec * L + c] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                          pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        }
    }
}

int log2_of(int x)
{
    int n = 0;
    while ((1 << n) < x)
        ++n;
    return n;
}

// Blocks of kThreads for `items` work items of L lanes, at most 8 blocks per SM.
int blocks_for(long long items, int lanes)
{
    const long long wanted = (items * lanes + kThreads - 1) / kThreads;
    const long long cap = static_cast<long long>(current_sm_count()) * 8;
    return static_cast<int>(wanted < cap ? wanted : cap);
}

}  // namespace

cudaError_t launch_store_int4(const Int4Pools &p, const void *k_new, const void *v_new,
                              const int32_t *slots, int num_tokens, cudaStream_t stream)
{
    if (num_tokens == 0)
        return cudaSuccess;
    const int lanes = p.head_dim / 8;
    const int blocks = blocks_for(2LL * num_tokens * p.kv_heads, lanes);
    auto kernel = lanes == 16 ? store_int4_kernel<16> : store_int4_kernel<8>;
    return launch_pdl(kernel, dim3(blocks), dim3(kThreads), 0, stream,
                      static_cast<uint32_t *>(p.k_codes), static_cast<uint32_t *>(p.v_codes),
                      static_cast<uint32_t *>(p.k_params), static_cast<uint32_t *>(p.v_params),
                      static_cast<const uint4 *>(k_new), static_cast<const uint4 *>(v_new), slots,
                      num_tokens, p.kv_heads, log2_of(p.page_size), p.num_pages * p.page_size,
                      p.hnd, current_error_word());
}

cudaError_t launch_load_int4(const Int4Pools &p, void *k_out, void *v_out, bool out_f32,
                             const int32_t *slots, int num_tokens, cudaStream_t stream)
{
    if (num_tokens == 0)
        return cudaSuccess;
    const int lanes = p.head_dim / 8;
    const int blocks = blocks_for(2LL * num_tokens * p.kv_heads, lanes);
    auto kernel = lanes == 16 ? (out_f32 ? load_int4_kernel<16, true> : load_int4_kernel<16, false>)
                              : (out_f32 ? load_int4_kernel<8, true> : load_int4_kernel<8, false>);
    return launch_pdl(kernel, dim3(blocks), dim3(kThreads), 0, stream,
                      static_cast<uint4 *>(k_out), static_cast<uint4 *>(v_out),
                      static_cast<const uint32_t *>(p.k_codes),
                      static_cast<const uint32_t *>(p.v_codes),
                      static_cast<const uint32_t *>(p.k_params),
                      static_cast<const uint32_t *>(p.v_params), slots, num_tokens, p.kv_heads,
                      log2_of(p.page_size), p.num_pages * p.page_size, p.hnd,
                      current_error_word());
}

cudaError_t read_and_clear_store_int4_errors(uint32_t *flags)
{
    uint32_t zero = 0;
    cudaError_t err = cudaMemcpyFromSymbol(flags, g_store_int4_errors, sizeof(uint32_t));
    if (err != cudaSuccess)
        return err;
    return cudaMemcpyToSymbol(g_store_int4_errors, &zero, sizeof(uint32_t));
}

}  // namespace kvc
