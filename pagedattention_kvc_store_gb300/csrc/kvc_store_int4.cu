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
// Both kernels are bound by HBM (328 bytes a vector at D = 128), but only if they spend few instructions:
// a lane takes 16 values of K and the same of V at a time (four lanes a group), minima and maxima
// go two to a word, the arithmetic two to an instruction (f32x2), and token and head come from a
// multiplication by a reciprocal that the host makes.  The codes need a correctly rounded quotient;
// a division per value would be about 12 instructions, and a cheaper check that falls back to it
// falls back all the time, because bf16 values lie on exact ties often (78 us for the 50,000 tokens
// that take 45 us with the corrected product below).
#include <math.h>

#include <algorithm>

#include "kvc_device.cuh"
#include "kvc_launch.h"

namespace kvc {

namespace {

__device__ uint32_t g_store_int4_errors;

constexpr int kThreads = 256;

// Work item = vector (token, kv head), K and V together.
struct Shape {
    int kv_heads, log2_page, num_slots, hnd;
    unsigned long long recip;   // ceil(2^64 / kv_heads), 0 for one head
};

// Token and head of a vector, and its places in the pools.
struct Place {
    bool live;        // the token has a slot inside the pool
    size_t code_row;  // vector index in the code pools
    size_t par_row;   // vector index in the parameter pools
};

__device__ __forceinline__ Place place_of(const Shape &s, const int32_t *slots, uint32_t vec,
                                          bool report, uint32_t *err)
{
    const uint32_t t = s.recip ? static_cast<uint32_t>(__umul64hi(s.recip, vec)) : vec;
    const uint32_t g = vec - t * s.kv_heads;
    const int slot = __ldcg(slots + t);
    Place p;
    p.live = slot >= 0 && slot < s.num_slots;
    if (slot >= s.num_slots && report && g == 0)
        atomicOr(err, kErrSlotRange);
    const int page = slot >> s.log2_page;
    const int off = slot & ((1 << s.log2_page) - 1);
    p.par_row = ((static_cast<size_t>(page) * s.kv_heads + g) << s.log2_page) + off;
    p.code_row = s.hnd ? p.par_row : static_cast<size_t>(slot) * s.kv_heads + g;
    return p;
}

// The smaller of two bf16 pairs, element by element; a NaN on either side wins.
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The larger ones, alike.
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ float approx_rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Codes (16 values: 8 bytes) and parameter of a quarter of a group; four neighbouring lanes hold one.
__device__ __forceinline__ uint2 quantise16(const uint32_t (&x)[8], uint32_t &param)
{
    // lo and hi of the lane's values, two to a word; then lo and -hi of the group
    uint32_t lo2 = x[0], hi2 = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo2 = min2_nan(lo2, x[i]);
        hi2 = max2_nan(hi2, x[i]);
    }
    const uint32_t nhi2 = hi2 ^ 0x80008000u;
    uint32_t m = min2_nan(__byte_perm(lo2, nhi2, 0x5410), __byte_perm(lo2, nhi2, 0x7632));
    m = min2_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = min2_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const float lo_half = __uint_as_float(m << 16) * 0.5f;
    const float hi_half = -__uint_as_float(m & 0xFFFF0000u) * 0.5f;
    const __nv_bfloat16 scale16 = __float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi_half, lo_half), 7.5f));
    const float scale_half = __bfloat162float(scale16) * 0.5f;
    // NaN anywhere, or an infinite end: the exponent bits of either end are all ones
    if (((m & 0x7F80u) == 0x7F80u) || ((m & 0x7F800000u) == 0x7F800000u)) {
        param = 0x7FC07FC0u;
        return make_uint2(0u, 0u);
    }
    param = static_cast<uint32_t>(__bfloat16_as_ushort(scale16)) | (m << 16);
    if (!(scale_half > 0.0f))
        return make_uint2(0u, 0u);
    // a = x / 2 - lo / 2 (one rounding), b = scale / 2, and q the quotient a / b as a division rounds
    // it: the product with the reciprocal, corrected by its remainder a - q b (a fused operation
    // gives it to 2^-24 of itself), is off by 2^-44 before its last rounding.  That rounds as the
    // exact quotient does wherever it matters, next to a half k + 1/2: (k + 1/2) b has 13 bits, so
    // an a that is not equal to it is at least 2^-24 away, and a quotient of either kind stays
    // 2^-37 off the point where the rounding would turn.  Equality gives k + 1/2 itself.  r is then
    // the nearest integer: 1.5 2^23 added and taken away, ties to even.  scale is at most 2^-8 of
    // itself off, so r needs no clamp.
    // The codes come out as floats 1.5 2^23 + r: r in the low bits.
    uint64_t r2[8];
    if (scale_half >= 1e-30f) {
        const float inv = approx_rcp(scale_half);
        const uint64_t half2 = f2_pack(0.5f, 0.5f), nlo2 = f2_pack(-lo_half, -lo_half);
        const uint64_t inv2 = f2_pack(inv, inv), nb2 = f2_pack(-scale_half, -scale_half);
        const uint64_t magic2 = f2_pack(12582912.0f, 12582912.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint64_t v =
                f2_pack(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xFFFF0000u));
            const uint64_t a = f2_fma(v, half2, nlo2);
            const uint64_t q = f2_mul(a, inv2);
            const uint64_t q1 = f2_fma(f2_fma(q, nb2, a), inv2, q);
            r2[i] = f2_add(q1, magic2);
        }
    } else {   // near and among the subnormals the products above would lose bits, and scale is coarse
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a0 = fmaf(__uint_as_float(x[i] << 16), 0.5f, -lo_half);
            const float a1 = fmaf(__uint_as_float(x[i] & 0xFFFF0000u), 0.5f, -lo_half);
            r2[i] = f2_pack(fminf(rintf(__fdiv_rn(a0, scale_half)), 15.0f) + 12582912.0f,
                            fminf(rintf(__fdiv_rn(a1, scale_half)), 15.0f) + 12582912.0f);
        }
    }
    // a byte is even + 16 odd: the floats' upper bits, 16 times too, stay above it
    uint32_t byte[8], code[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float even, odd;
        f2_unpack(r2[i], even, odd);
        byte[i] = __float_as_uint(even) + 16u * __float_as_uint(odd);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        code[h] = __byte_perm(__byte_perm(byte[4 * h], byte[4 * h + 1], 0x0040),
                              __byte_perm(byte[4 * h + 2], byte[4 * h + 3], 0x0040), 0x5410);
    return make_uint2(code[0], code[1]);
}

// L lanes per vector, 16 values each (D = 16 L).
// (five CTAs an SM: with 54 registers and four of them 1% slower, with six 40 registers spill)
template <int L>
__global__ void __launch_bounds__(kThreads, 5)
    store_int4_kernel(uint2 *__restrict__ k_codes, uint2 *__restrict__ v_codes,
                      uint32_t *__restrict__ k_params, uint32_t *__restrict__ v_params,
                      const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new,
                      const int32_t *__restrict__ slots, uint32_t vectors, const Shape shape,
                      uint32_t *word)
{
    pdl_wait();
    pdl_trigger();
    uint32_t *err = word ? word : &g_store_int4_errors;
    const int c = threadIdx.x % L;
    const uint32_t step = gridDim.x * (kThreads / L);
    // a warp's lanes go round together (the group's shuffles)
    const uint32_t in_warp = (threadIdx.x & 31) / L;
    for (uint32_t w0 = (blockIdx.x * kThreads + (threadIdx.x & ~31u)) / L; w0 < vectors; w0 += step) {
        const uint32_t vec = min(w0 + in_warp, vectors - 1);   // the last one again: stored alike
        // padding tokens' values are read too: one round trip to memory instead of two
        const size_t at = (static_cast<size_t>(vec) * L + c) * 2;
        const uint4 k0 = __ldcs(k_new + at), k1 = __ldcs(k_new + at + 1);
        const uint4 v0 = __ldcs(v_new + at), v1 = __ldcs(v_new + at + 1);
        const Place p = place_of(shape, slots, vec, c == 0, err);
        const uint32_t xk[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
        const uint32_t xv[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        uint32_t kp, vp;
        const uint2 kc = quantise16(xk, kp), vc = quantise16(xv, vp);
        if (p.live) {
            k_codes[p.code_row * L + c] = kc;
            v_codes[p.code_row * L + c] = vc;
            if ((c & 3) == 0) {
                k_params[p.par_row * (L / 4) + c / 4] = kp;
                v_params[p.par_row * (L / 4) + c / 4] = vp;
            }
        }
    }
}

// The values that 4-bit pages hold at the given slots, as bf16 (rounded to nearest even) or fp32:
// scale * code is exact in fp32 (4 by 8 bits) and the sum with lo rounds once.  A lane takes the
// 8 values of chunk c and, at D = 128, of chunk c + 8, of K and V, so that stores are whole
// 16-byte chunks side by side.  A nibble under the exponent of 2^23 is 2^23 + code.
template <int D, bool F32>
__global__ void __launch_bounds__(kThreads)
    load_int4_kernel(uint4 *__restrict__ k_out, uint4 *__restrict__ v_out,
                     const uint32_t *__restrict__ k_codes, const uint32_t *__restrict__ v_codes,
                     const uint32_t *__restrict__ k_params, const uint32_t *__restrict__ v_params,
                     const int32_t *__restrict__ slots, uint32_t vectors, const Shape shape,
                     uint32_t *word)
{
    pdl_wait();
    pdl_trigger();
    uint32_t *err = word ? word : &g_store_int4_errors;
    constexpr int L = 8;            // lanes of a vector
    constexpr int NG = D / 64;
    const int c = threadIdx.x % L;
    const uint32_t step = gridDim.x * (kThreads / L);
    for (uint32_t vec = blockIdx.x * (kThreads / L) + threadIdx.x / L; vec < vectors; vec += step) {
        const Place p = place_of(shape, slots, vec, c == 0, err);
        uint32_t codes[2][NG] = {}, par[2][NG] = {};
        if (p.live) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                codes[0][g] = __ldcg(k_codes + p.code_row * (NG * L) + g * L + c);
                codes[1][g] = __ldcg(v_codes + p.code_row * (NG * L) + g * L + c);
                par[0][g] = __ldcg(k_params + p.par_row * NG + g);
                par[1][g] = __ldcg(v_params + p.par_row * NG + g);
            }
        }
#pragma unroll
        for (int which = 0; which < 2; ++which) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const float scale = __uint_as_float(par[which][g] << 16);
                const float lo = __uint_as_float(par[which][g] & 0xFFFF0000u);
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t u = (codes[which][g] >> (4 * i)) & 15u;
                    v[i] = fmaf(scale, __uint_as_float(0x4B000000u | u) - 8388608.0f, lo);
                }
                const size_t at = static_cast<size_t>(vec) * (NG * L) + g * L + c;
                uint4 *out = which ? v_out : k_out;
                if (F32) {
                    __stcs(out + 2 * at, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]),
                                                    __float_as_uint(v[2]), __float_as_uint(v[3])));
                    __stcs(out + 2 * at + 1,
                           make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]),
                                      __float_as_uint(v[6]), __float_as_uint(v[7])));
                } else {
                    __stcs(out + at,
                           make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                      pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
                }
            }
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

// Blocks of kThreads for `vectors` work items of L lanes, at most `per_sm` per SM.  Many short blocks
// spread the stores and even out the SMs' ends: 50,000 tokens are stored and loaded in 86.9 us with 20
// blocks an SM for the store and 8 for the load, 86.2 with 40 and 8, 82.1 with 20 and 32, 81.4 with 20
// and 64.
constexpr int kStoreBlocks = 40, kLoadBlocks = 64;

int blocks_for(long long vectors, int lanes, int per_sm)
{
    const long long wanted = (vectors * lanes + kThreads - 1) / kThreads;
    const long long cap = static_cast<long long>(current_sm_count()) * per_sm;
    return static_cast<int>(wanted < cap ? wanted : cap);
}

Shape shape_of(const Int4Pools &p)
{
    Shape s;
    s.kv_heads = p.kv_heads;
    s.log2_page = log2_of(p.page_size);
    s.num_slots = p.num_pages * p.page_size;
    s.hnd = p.hnd;
    s.recip = p.kv_heads == 1 ? 0 : ~0ull / p.kv_heads + 1;
    return s;
}

// Tokens of one launch: vector indices stay below 2^31.
long long tokens_per_launch(const Int4Pools &p)
{
    return std::max(1LL, (1LL << 30) / p.kv_heads);
}

}  // namespace

cudaError_t launch_store_int4(const Int4Pools &p, const void *k_new, const void *v_new,
                              const int32_t *slots, int num_tokens, cudaStream_t stream)
{
    const int lanes = p.head_dim / 16;
    auto kernel = lanes == 8 ? store_int4_kernel<8> : store_int4_kernel<4>;
    const long long most = tokens_per_launch(p);
    for (long long t = 0; t < num_tokens; t += most) {
        const long long vectors = std::min(most, num_tokens - t) * p.kv_heads;
        const size_t at = static_cast<size_t>(t) * p.kv_heads * lanes * 2;
        const cudaError_t err = launch_pdl(
            kernel, dim3(blocks_for(vectors, lanes, kStoreBlocks)), dim3(kThreads), 0, stream,
            static_cast<uint2 *>(p.k_codes), static_cast<uint2 *>(p.v_codes),
            static_cast<uint32_t *>(p.k_params), static_cast<uint32_t *>(p.v_params),
            static_cast<const uint4 *>(k_new) + at, static_cast<const uint4 *>(v_new) + at,
            slots + t, static_cast<uint32_t>(vectors), shape_of(p), current_error_word());
        if (err != cudaSuccess)
            return err;
    }
    return cudaSuccess;
}

cudaError_t launch_load_int4(const Int4Pools &p, void *k_out, void *v_out, bool out_f32,
                             const int32_t *slots, int num_tokens, cudaStream_t stream)
{
    auto kernel = p.head_dim == 128
                      ? (out_f32 ? load_int4_kernel<128, true> : load_int4_kernel<128, false>)
                      : (out_f32 ? load_int4_kernel<64, true> : load_int4_kernel<64, false>);
    const long long most = tokens_per_launch(p);
    for (long long t = 0; t < num_tokens; t += most) {
        const long long vectors = std::min(most, num_tokens - t) * p.kv_heads;
        const size_t at = static_cast<size_t>(t) * p.kv_heads * (p.head_dim / 8) * (out_f32 ? 2 : 1);
        const cudaError_t err = launch_pdl(
            kernel, dim3(blocks_for(vectors, 8, kLoadBlocks)), dim3(kThreads), 0, stream,
            static_cast<uint4 *>(k_out) + at, static_cast<uint4 *>(v_out) + at,
            static_cast<const uint32_t *>(p.k_codes), static_cast<const uint32_t *>(p.v_codes),
            static_cast<const uint32_t *>(p.k_params), static_cast<const uint32_t *>(p.v_params),
            slots + t, static_cast<uint32_t>(vectors), shape_of(p), current_error_word());
        if (err != cudaSuccess)
            return err;
    }
    return cudaSuccess;
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
