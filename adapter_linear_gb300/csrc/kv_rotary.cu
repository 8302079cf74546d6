// kv_rotary.cu -- the paged cache's write with rotary positions on the way: K rotated (and quantised) into
// its pages, V as it is, Q rotated beside it, in one pass over the three.
#include <algorithm>

#include "kv_device.cuh"
#include "rotary_device.cuh"

namespace lora {
namespace {

constexpr int kBatch = 4;  // blocks of rows loaded before any is stored

// Scale and codes of the 16 fp32 values of this lane; the row's kLanes lanes take part. As the write of bf16
// rows quantises (kv_cache.cu), of which a bf16 x is a case: y = x (1 / s) is rounded to a multiple of 2^-11
// and then to a whole number, so a code is off by at most 1/2 + 2^-12 + 2^-16 of a step, and a bf16 row's
// codes are those of exact arithmetic.
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
    const uint64_t grid = pack2(6144.0f, 6144.0f), back = pack2(-6144.0f, -6144.0f);  // 1.5 2^12: multiples of 2^-11
    const uint64_t whole = pack2(12582912.0f, 12582912.0f);  // 1.5 2^23: the code in the low byte
    uint32_t c[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t v[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float lo, hi;
            unpack2(add2(add2(fma2(pack2(x[4 * q + 2 * e], x[4 * q + 2 * e + 1]), inv2, grid), back), whole), &lo, &hi);
            v[e] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x0040);
        }
        c[q] = finite ? __byte_perm(v[0], v[1], 0x5410) : 0u;
    }
    return make_uint4(c[0], c[1], c[2], c[3]);
}

// A row is one head of one token: Hq of Q, H of K, H of V. D / 16 lanes hold one. A warp takes `blocks` blocks
// of 512 / D rows of one token, which is looked up once and whose angles (8 a lane) serve all of them.
template <int D, bool kInt8>
__global__ void __launch_bounds__(256) kv_write_rotary_kernel(KvDev kv, KvBatchDev b, const __grid_constant__ RotaryDev rot,
                                                              KvRotaryArgs a, int parts, int blocks)
{
    constexpr int kLanes = D / 16, kRows = 32 / kLanes;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int64_t t64 = w / parts;
    if (t64 >= b.T) return;
    const int t = (int)t64;
    const int sub = lane / kLanes, c = lane % kLanes;
    const int rows = a.Hq + 2 * kv.H;
    const int first = (int)(w - t64 * parts) * blocks * kRows, last = min(rows, first + blocks * kRows);
    int d0, d1;
    rotary_runs(rot, c, &d0, &d1);

    // rows of the tensors, from this lane's in the block that starts at r0
    uint4 x[kBatch][2];
    auto load = [&](int r0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + i * kRows + sub;
            x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
            if (r >= last) continue;
            const uint16_t *src = r < a.Hq          ? a.Q + (int64_t)t * a.q_stride + r * D
                                  : r < a.Hq + kv.H ? a.K + (int64_t)t * a.k_stride + (r - a.Hq) * D
                                                    : a.V + (int64_t)t * a.v_stride + (r - a.Hq - kv.H) * D;
            x[i][0] = *reinterpret_cast<const uint4 *>(src + d0);
            x[i][1] = *reinterpret_cast<const uint4 *>(src + d1);
        }
    };
    load(first);  // on their way while the token is looked up

    // the token's sequence, position and cache row (-1: none)
    int seq = kv_find_seq(b, t, lane);
    KvSeq s{0, 0, 0};
    bool there = seq >= 0;
    if (there) {
        for (;; ++seq) {  // (among bad starts the search may stop before t's sequence)
            if (seq >= b.n_seqs) {
                there = false;
                break;
            }
            s = kv_seq(b, kv.page_shift, seq, kv.err);
            if (t < s.row0) there = false;
            if (!there || t - s.row0 < s.n) break;
        }
    }
    if (!there) return;  // padding, or a bad sequence
    const int pos = s.L - s.n + (t - s.row0);
    const int64_t cache_row = pos >= 0 && last > a.Hq ? kv_row(kv, b, seq, pos) : -1;
    const bool turns = 16 * c < rot.dim;
    Turn8 turn;
    if (turns) turn = rotary_turn(rot, c, pos, false);

    for (int r0 = first; r0 < last; r0 += kBatch * kRows) {
        if (r0 > first) load(r0);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + i * kRows + sub;
            if (r0 + i * kRows >= last) break;
            float f[16];
            unpack8(x[i][0], f);
            unpack8(x[i][1], f + 8);
            if (turns && r < a.Hq + kv.H) rotary_pairs(rot.half, turn, f);
            const bool is_v = r >= a.Hq + kv.H;
            const int64_t row = cache_row + ((int64_t)(r - a.Hq - (is_v ? kv.H : 0)) << kv.page_shift);
            if constexpr (kInt8) {
                if (r0 + (i + 1) * kRows > a.Hq) {  // some of the block's rows go to the cache
                    uint16_t scale;
                    const uint4 q = quantise16f<kLanes>(f, &scale);
                    if (r >= a.Hq && r < last && cache_row >= 0) {
                        uint8_t *const to = static_cast<uint8_t *>(is_v ? kv.v : kv.k) + row * D;
                        *reinterpret_cast<uint2 *>(to + d0) = make_uint2(q.x, q.y);
                        *reinterpret_cast<uint2 *>(to + d1) = make_uint2(q.z, q.w);
                        if (c == 0) (is_v ? kv.vs : kv.ks)[row] = scale;
                    }
                }
            } else if (r >= a.Hq && r < last && cache_row >= 0) {
                uint16_t *const to = static_cast<uint16_t *>(is_v ? kv.v : kv.k) + row * D;
                *reinterpret_cast<uint4 *>(to + d0) = pack8(f);
                *reinterpret_cast<uint4 *>(to + d1) = pack8(f + 8);
            }
            if (r < a.Hq && r < last) {
                uint16_t *const to = a.Q_out + (int64_t)t * a.qo_stride + r * D;
                const bool zero = pos < 0;
                const uint4 none = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4 *>(to + d0) = zero ? none : pack8(f);
                *reinterpret_cast<uint4 *>(to + d1) = zero ? none : pack8(f + 8);
            }
        }
    }
}

}  // namespace

cudaError_t launch_kv_write_rotary(const KvDev &kv, bool int8, const KvBatchDev &b, const lora_rotary *rotary,
                                   const KvRotaryArgs &a, int num_sms, cudaStream_t stream)
{
    auto fn = kv.D == 128 ? (int8 ? kv_write_rotary_kernel<128, true> : kv_write_rotary_kernel<128, false>)
                          : (int8 ? kv_write_rotary_kernel<64, true> : kv_write_rotary_kernel<64, false>);
    const cudaError_t e = ensure_smem_attr((const void *)fn, 0);
    if (e != cudaSuccess) return e;
    const int per = 512 / kv.D;
    const int64_t all = (a.Hq + 2 * kv.H + per - 1) / per;  // blocks of a token
    const int64_t blocks = std::min(all, std::max<int64_t>(1, b.T * all / (16 * (int64_t)num_sms)));
    const int64_t parts = (all + blocks - 1) / blocks;
    fn<<<(unsigned)((b.T * parts + 7) / 8), 256, 0, stream>>>(kv, b, rotary_view(rotary), a, (int)parts, (int)blocks);
    return cudaGetLastError();
}

}  // namespace lora
