// kvc_rope.cu -- rotary positions with several axes, and the store of rotated keys into pages.
//
// Pair f of a head (of rotary / 2 pairs) turns by a = position[axis(f)] * inv_freq(f):
//   y0 = x0 cos a - x1 sin a,   y1 = x1 cos a + x0 sin a.
// Angles are held as turns in 64-bit fixed point: inv_freq / (2 pi) modulo 1 as a 64-bit fraction, so
// position * fraction modulo 2^64 is the angle's fraction of a turn, exact to position * 2^-64 on top of
// the fraction's own roundings (2^-52 of inv_freq / (2 pi)) however far the position is; in fp32 the angle
// of position 131,072 would be off by up to 2^-8.  Its upper 32 bits become an fp32 number of half turns
// in [-1, 1] for sincospif.  The rotation itself is fp32, rounded once to bf16.
//
// HBM-bound: a token's heads are read once and written once.  A thread holds the 8 cosines and sines of
// one pair of 16-byte chunks (dims 8 c .. and 8 c + rotary / 2 .., or two chunks in a row where pairs
// are adjacent dims) and goes over heads of its token with them, kRows heads at a time so that all their
// loads are in flight together; values, and dims past rotary, go through unchanged.  50,000 tokens of 32 + 8 + 8
// heads of 128 dims into pages (1.15 GB from and to memory: one token in eleven is padding and stores nothing): 183 us,
// 6.3 TB/s, 93% of a copy; blocks of 256 threads 187 us, 3 heads at a time 181 us but 70.3 us against 66.7 for 9,973
// tokens of 64 + 8 + 8 heads.  Rows of the same queries and keys (1.02 GB), in place or not: 182 us, 5.6 TB/s.
#include "kvc_device.cuh"
#include "kvc_launch.h"

namespace kvc {

namespace {

__device__ uint32_t g_rope_errors;

constexpr int kThreads = 128;
constexpr int kRows = 2;   // heads whose loads a thread has in flight

struct Args {
    const uint8_t *q, *k, *v;               // rows of heads, strides in bytes between tokens
    long long q_stride, k_stride, v_stride;
    uint8_t *q_out, *k_out, *v_out;         // k_out: rows of heads, or the pool
    long long q_out_stride, k_out_stride;
    const int32_t *positions, *slots;
    int num_tokens, q_heads, kv_heads, v_heads;   // v_heads 0: keys alone, not into pages
    int pairs;                              // 16-dim pieces of a head that turn
    int lanes_log2;                         // threads (of one pair of chunks) to a token
    int page_log2, num_slots, hnd;
    uint32_t *err;
    RopeAngles angles;
};

template <int D, bool ADJACENT, bool STORE>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ Args a)
{
    pdl_wait();
    pdl_trigger();
    constexpr int kPieces = D / 16;         // pairs of chunks of a head
    const int piece = threadIdx.x % kPieces;
    const int unit = threadIdx.x / kPieces;
    const int lanes = 1 << a.lanes_log2;
    const int lane = unit & (lanes - 1);
    const int t = blockIdx.x * ((kThreads / kPieces) >> a.lanes_log2) + (unit >> a.lanes_log2);
    if (t >= a.num_tokens)
        return;
    const bool turns = piece < a.pairs;
    // this thread's chunks, in 16-byte units
    const int c0 = (ADJACENT || !turns) ? 2 * piece : piece;
    const int c1 = (ADJACENT || !turns) ? 2 * piece + 1 : piece + a.pairs;

    const int heads = a.q_heads + a.kv_heads + a.v_heads;
    uint4 x[kRows][2];
    auto load = [&](int h0) {
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int h = h0 + u * lanes;
            const uint8_t *src;
            if (h < a.q_heads)
                src = a.q + t * a.q_stride + h * (D * 2);
            else if (h < a.q_heads + a.kv_heads)
                src = a.k + t * a.k_stride + (h - a.q_heads) * (D * 2);
            else
                src = a.v + t * a.v_stride + (h - a.q_heads - a.kv_heads) * (D * 2);
            if (h < heads) {
                x[u][0] = __ldcs(reinterpret_cast<const uint4 *>(src) + c0);
                x[u][1] = __ldcs(reinterpret_cast<const uint4 *>(src) + c1);
            }
        }
    };
    load(lane);   // on its way while the angles are made

    long long k_row = 0, k_head = D * 2;    // bytes: this token's first key row, and between heads
    bool store = true;
    if (STORE) {
        const int slot = __ldg(a.slots + t);
        store = slot >= 0 && slot < a.num_slots;
        if (slot >= a.num_slots && lane == 0 && piece == 0)
            atomicOr(a.err ? a.err : &g_rope_errors, kErrSlotRange);
        const long long page = slot >> a.page_log2, off = slot & ((1 << a.page_log2) - 1);
        k_row = a.hnd ? (((page * a.kv_heads) << a.page_log2) + off) * (D * 2)
                      : static_cast<long long>(slot) * a.kv_heads * (D * 2);
        k_head = a.hnd ? (static_cast<long long>(D * 2) << a.page_log2) : D * 2;
    } else {
        k_row = t * a.k_out_stride;
    }

    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        cs[i] = 1.0f;
        sn[i] = 0.0f;
        if (turns) {
            const int f = 8 * piece + i;
            const int p = __ldg(a.positions + static_cast<size_t>(a.angles.axis[f]) * a.num_tokens + t);
            const uint64_t turn = static_cast<uint64_t>(static_cast<long long>(p)) * a.angles.turns[f];
            // the upper half as a signed fraction of a turn, in half turns
            sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &sn[i], &cs[i]);
        }
    }

    for (int h0 = lane;;) {
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int h = h0 + u * lanes;
            uint8_t *dst;
            if (h < a.q_heads)
                dst = a.q_out + t * a.q_out_stride + h * (D * 2);
            else if (h < a.q_heads + a.kv_heads)
                dst = a.k_out + k_row + (h - a.q_heads) * k_head;
            else
                dst = a.v_out + k_row + (h - a.q_heads - a.kv_heads) * k_head;
            if (h >= heads || (h >= a.q_heads && !store))
                continue;
            if (turns && h < a.q_heads + a.kv_heads) {
                uint32_t w[8] = {x[u][0].x, x[u][0].y, x[u][0].z, x[u][0].w,
                                 x[u][1].x, x[u][1].y, x[u][1].z, x[u][1].w};
                if (ADJACENT) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float lo = __uint_as_float(w[i] << 16);
                        const float hi = __uint_as_float(w[i] & 0xFFFF0000u);
                        w[i] = pack_bf16x2(fmaf(lo, cs[i], -(hi * sn[i])),
                                           fmaf(hi, cs[i], lo * sn[i]));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float a0 = __uint_as_float(w[i] << 16);
                        const float a1 = __uint_as_float(w[i] & 0xFFFF0000u);
                        const float b0 = __uint_as_float(w[i + 4] << 16);
                        const float b1 = __uint_as_float(w[i + 4] & 0xFFFF0000u);
                        const int j = 2 * i;
                        w[i] = pack_bf16x2(fmaf(a0, cs[j], -(b0 * sn[j])),
                                           fmaf(a1, cs[j + 1], -(b1 * sn[j + 1])));
                        w[i + 4] = pack_bf16x2(fmaf(b0, cs[j], a0 * sn[j]),
                                               fmaf(b1, cs[j + 1], a1 * sn[j + 1]));
                    }
                }
                x[u][0] = make_uint4(w[0], w[1], w[2], w[3]);
                x[u][1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
            reinterpret_cast<uint4 *>(dst)[c0] = x[u][0];
            reinterpret_cast<uint4 *>(dst)[c1] = x[u][1];
        }
        h0 += kRows * lanes;
        if (h0 >= heads)
            break;
        load(h0);
    }
}

template <int D, bool ADJACENT, bool STORE>
cudaError_t launch_t(const RopeLaunch &l, cudaStream_t stream)
{
    Args a;
    a.q = static_cast<const uint8_t *>(l.q);
    a.k = static_cast<const uint8_t *>(l.k);
    a.v = static_cast<const uint8_t *>(l.v);
    a.q_stride = l.q_stride * 2;
    a.k_stride = l.k_stride * 2;
    a.v_stride = l.v_stride * 2;
    a.q_out = static_cast<uint8_t *>(l.q_out);
    a.k_out = static_cast<uint8_t *>(l.k_out);
    a.v_out = static_cast<uint8_t *>(l.v_out);
    a.q_out_stride = l.q_out_stride * 2;
    a.k_out_stride = l.k_out_stride * 2;
    a.positions = l.positions;
    a.slots = l.slots;
    a.num_tokens = l.num_tokens;
    a.q_heads = l.q_heads;
    a.kv_heads = l.kv_heads;
    a.v_heads = STORE ? l.kv_heads : 0;
    a.pairs = l.rotary_dim / 16;
    a.page_log2 = 0;
    while ((1 << a.page_log2) < l.page_size)
        ++a.page_log2;
    a.num_slots = l.num_slots;
    a.hnd = l.hnd ? 1 : 0;
    a.err = current_error_word();
    a.angles = l.angles;
    constexpr int kUnits = kThreads / (D / 16);
    // Threads to a token: each computes the angles again, so few where tokens are many (4 of them; 50,000
    // tokens of 48 heads: 183 us, with 8 threads 187, with 32 452), and more, down to kRows heads each, until
    // the blocks are many to an SM, for their last ones to end together (9,973 tokens of 80 heads: 8 threads
    // 66.7 us, 4 72.2).
    const int heads = a.q_heads + a.kv_heads + a.v_heads;
    const long long many = 32LL * current_sm_count();
    a.lanes_log2 = 0;
    while ((2 << a.lanes_log2) <= kUnits && (kRows << a.lanes_log2) < heads &&
           (a.lanes_log2 < 2 || (static_cast<long long>(l.num_tokens) << a.lanes_log2) / kUnits < many))
        ++a.lanes_log2;
    const int per_block = kUnits >> a.lanes_log2;
    const int blocks = (l.num_tokens + per_block - 1) / per_block;
    return launch_pdl(rope_kernel<D, ADJACENT, STORE>, dim3(blocks), dim3(kThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_rope(const RopeLaunch &l, cudaStream_t stream)
{
    if (l.num_tokens == 0)
        return cudaSuccess;
    const bool store = l.slots != nullptr;
    if (l.head_dim == 128) {
        if (l.adjacent)
            return store ? launch_t<128, true, true>(l, stream) : launch_t<128, true, false>(l, stream);
        return store ? launch_t<128, false, true>(l, stream) : launch_t<128, false, false>(l, stream);
    }
    if (l.adjacent)
        return store ? launch_t<64, true, true>(l, stream) : launch_t<64, true, false>(l, stream);
    return store ? launch_t<64, false, true>(l, stream) : launch_t<64, false, false>(l, stream);
}

cudaError_t read_and_clear_rope_errors(uint32_t *flags)
{
    uint32_t zero = 0;
    cudaError_t err = cudaMemcpyFromSymbol(flags, g_rope_errors, sizeof(uint32_t));
    if (err != cudaSuccess)
        return err;
    return cudaMemcpyToSymbol(g_rope_errors, &zero, sizeof(uint32_t));
}

}  // namespace kvc
