// kv_rotary.cu -- the paged cache's write with rotary positions on the way: K rotated (and quantised) into
// its pages, V as it is, Q rotated beside it, in one pass over the three.
//
// The rotation is rotary.cu's; what it gives goes to the quantisation in fp32 (of the 8-bit formats: scale =
// max(bf16(amax / 127), 2^-126), code = x / scale to the nearest), so that a key is rounded once. What bounds it:
// HBM, and with an 8-bit cache nearly as much the instructions (40 % of the issue slots at 16 warps an SM, which 128
// registers a thread allow): the quantisation's 16 values a lane wait for the row's maximum. Measured on the GPU, 32 query
// heads and 8 kv heads of 128 values: 8 prompts of 2048 tokens 8-bit 62 us (370 MB, 6.0 TB/s; the rotation and
// the write one after the other read and write 1.3 times as much), bf16 66 us (403 MB, 6.1 TB/s; 4 bytes a thread
// spill); 64 requests of one token 3.9 and 4.0 us (start, length, page and row are loads that depend on one another).
#include <climits>
#include <type_traits>

#include "kv_device.cuh"
#include "launch_stream.h"
#include "rotary_device.cuh"

namespace lora {
namespace {

// Scale and codes of the 16 fp32 values of this lane; the row's kLanes lanes take part. y = x (1 / s) is corrected by what
// it leaves of x, (x - y s) (1 / s) (Markstein 1990): x / s to half a step of fp32, and exactly where it is a number of
// fp32, as ties are. So a code is within 1/2 + 2^-18 of a step of x, and a bf16 row's codes are those of exact arithmetic.
// (The write of bf16 rows, kv_cache.cu, does with a rounding of y to a multiple of 2^-11 ahead of the one to a whole
// number, which moves codes of fp32 values that lie 2^-12 beside a tie.)
template <int kLanes>
__device__ __forceinline__ uint4 quantise16f(const float (&x)[16], uint16_t *scale_bits)
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool finite = top < 0x7F800000u;
    const uint32_t sb = pack_bf16x2(__fdiv_rn(__uint_as_float(top), 127.0f), 0.0f) & 0xFFFFu;
    const float s = fmaxf(__uint_as_float(sb << 16), 1.17549435e-38f);  // 2^-126
    *scale_bits = finite ? (uint16_t)(__float_as_uint(s) >> 16) : (uint16_t)0x7FC0;
    const float inv = __frcp_rn(s);
    const uint64_t inv2 = pack2(inv, inv);
    const uint64_t neg = pack2(-s, -s);
    const uint64_t whole = pack2(12582912.0f, 12582912.0f);  // 1.5 2^23: the code in the low byte
    uint32_t c[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t v[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint64_t xs = pack2(x[4 * q + 2 * e], x[4 * q + 2 * e + 1]), y = mul2(xs, inv2);
            float lo, hi;
            unpack2(add2(fma2(fma2(y, neg, xs), inv2, y), whole), &lo, &hi);
            v[e] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x0040);
        }
        c[q] = finite ? __byte_perm(v[0], v[1], 0x5410) : 0u;
    }
    return make_uint4(c[0], c[1], c[2], c[3]);
}

constexpr int kBatch = 4;  // blocks loaded before any is stored

// A row is one head of one token: Hq of Q, H of K, H of V. D / 16 lanes hold one, a block is the 512 / D rows of one
// of them that a warp holds at a time. A warp takes a chunk of consecutive tokens, or a part of one token's
// blocks; the tokens are looked up 32 at a time, a lane a token, and a lane's eight angles serve all its
// rows of a token.
template <int D, bool kInt8, bool kHalf>
__global__ void __launch_bounds__(RotaryGrid::kWarps * 32, RotaryGrid::kCtas)
    kv_write_rotary_kernel(KvDev kv, KvBatchDev b, const __grid_constant__ RotaryDev rot, KvRotaryArgs a, int parts)
{
    constexpr int kLanes = D / 16, kRows = 32 / kLanes;
    const int lane = threadIdx.x & 31;
    const int sub = lane / kLanes, c = lane % kLanes;
    const int q_blocks = (a.Hq + kRows - 1) / kRows, h_blocks = (kv.H + kRows - 1) / kRows, all = q_blocks + 2 * h_blocks;
    const RotaryShare me(b.T, all, parts);
    const int b0 = me.b0, b1 = me.b1;
    int d0, d1;
    rotary_runs(rot, D, c, &d0, &d1);
    const bool turns = 16 * c < rot.dim;

    // Of the warp's token number 32 y + lane: its position, and its cache row for head 0 (-1: none); kNowhere: padding
    // behind the last sequence, or a bad sequence.
    constexpr int kNowhere = INT_MIN;
    int my_pos = kNowhere;
    int64_t my_row = -1;
    auto look_up = [&](int first) {
        int seq = max(0, kv_find_seq(b, first, lane));
        my_pos = kNowhere;
        my_row = -1;
        const int t = first + lane * me.step;
        if (t >= me.t1) return;
        KvSeq s;
        for (;; ++seq) {  // (a chunk may end in a later sequence; among bad starts the search may stop early)
            if (seq >= b.n_seqs) return;
            s = kv_seq(b, kv.page_shift, seq, kv.err);
            if (t < s.row0) return;
            if (t - s.row0 < s.n) break;
        }
        my_pos = s.L - s.n + (t - s.row0);
        if (my_pos >= 0 && b1 > q_blocks) my_row = kv_row(kv, b, seq, my_pos);
    };

#pragma unroll 1
    for (int t = me.t0, i = 0; t < me.t1; t += me.step, ++i) {
        if ((i & 31) == 0) look_up(t);
        const int pos = __shfl_sync(0xffffffffu, my_pos, i & 31);
        const int64_t cache_row = __shfl_sync(0xffffffffu, my_row, i & 31);
        if (pos == kNowhere) continue;
        Turn8 turn;
        if (turns) turn = rotary_turn<kHalf>(rot, c, pos, false);

        // Q's blocks of this warp
        {
            const uint16_t *const src = a.Q + (int64_t)t * a.q_stride + sub * D;
            uint16_t *const dst = a.Q_out + (int64_t)t * a.qo_stride + sub * D;
            const int end = min(b1 * kRows, a.Hq) - sub;
#pragma unroll 1
            for (int r0 = b0 * kRows; r0 < end; r0 += kBatch * kRows) {
                uint4 v[kBatch][2];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (r0 + i * kRows < end) {
                        v[i][0] = *reinterpret_cast<const uint4 *>(src + (r0 + i * kRows) * D + d0);
                        v[i][1] = *reinterpret_cast<const uint4 *>(src + (r0 + i * kRows) * D + d1);
                    }
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (r0 + i * kRows < end) {
                        if (turns) {
                            float f[16];
                            unpack16(v[i], f);
                            rotary_pairs<kHalf>(turn, f);
                            v[i][0] = pack8(f);
                            v[i][1] = pack8(f + 8);
                        }
                        if (pos < 0) v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(dst + (r0 + i * kRows) * D + d0) = v[i][0];
                        *reinterpret_cast<uint4 *>(dst + (r0 + i * kRows) * D + d1) = v[i][1];
                    }
            }
        }
        // K's and V's
        if (cache_row < 0) continue;
#pragma unroll 1
        for (int blk = max(b0, q_blocks); blk < b1; blk += kBatch) {
            uint4 v[kBatch][2];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
                const bool is_v = blk + i - q_blocks >= h_blocks;
                const int h = (blk + i - q_blocks - (is_v ? h_blocks : 0)) * kRows + sub;
                if (blk + i >= b1 || h >= kv.H) continue;
                const uint16_t *const src = (is_v ? a.V + (int64_t)t * a.v_stride : a.K + (int64_t)t * a.k_stride) + h * D;
                v[i][0] = *reinterpret_cast<const uint4 *>(src + d0);
                v[i][1] = *reinterpret_cast<const uint4 *>(src + d1);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (blk + i >= b1) break;
                const bool is_v = blk + i - q_blocks >= h_blocks;
                const int h = (blk + i - q_blocks - (is_v ? h_blocks : 0)) * kRows + sub;
                const int64_t row = cache_row + ((int64_t)h << kv.page_shift);
                float f[16];
                unpack16(v[i], f);
                if (turns && !is_v) rotary_pairs<kHalf>(turn, f);
                if constexpr (kInt8) {
                    uint16_t scale;
                    const uint4 q = quantise16f<kLanes>(f, &scale);
                    if (h < kv.H) {
                        uint8_t *const to = static_cast<uint8_t *>(is_v ? kv.v : kv.k) + row * D;
                        *reinterpret_cast<uint2 *>(to + d0) = make_uint2(q.x, q.y);
                        *reinterpret_cast<uint2 *>(to + d1) = make_uint2(q.z, q.w);
                        if (c == 0) (is_v ? kv.vs : kv.ks)[row] = scale;
                    }
                } else if (h < kv.H) {
                    uint16_t *const to = static_cast<uint16_t *>(is_v ? kv.v : kv.k) + row * D;
                    *reinterpret_cast<uint4 *>(to + d0) = pack8(f);
                    *reinterpret_cast<uint4 *>(to + d1) = pack8(f + 8);
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_kv_write_rotary(const KvDev &kv, bool int8, const KvBatchDev &b, const lora_rotary *rotary,
                                   const KvRotaryArgs &a, int num_sms, cudaStream_t stream)
{
    auto pick = [&](auto half) {
        constexpr bool kHalf = decltype(half)::value;
        return kv.D == 128 ? (int8 ? kv_write_rotary_kernel<128, true, kHalf> : kv_write_rotary_kernel<128, false, kHalf>)
                           : (int8 ? kv_write_rotary_kernel<64, true, kHalf> : kv_write_rotary_kernel<64, false, kHalf>);
    };
    auto fn = rotary->layout == LORA_ROTARY_HALF ? pick(std::true_type()) : pick(std::false_type());
    const int per = 512 / kv.D;
    const RotaryGrid g(b.T, (a.Hq + per - 1) / per + 2 * ((kv.H + per - 1) / per), num_sms);
    return launch_stream(g.streams, false, fn, g.ctas, RotaryGrid::kWarps * 32, stream, kv, b, rotary_view(rotary), a, g.parts);
}

}  // namespace lora
