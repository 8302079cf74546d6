// rotary_device.cuh -- rotary positions: a pair's angle, and the rotation of the 16 values a lane holds.
#pragma once

#include "../../include/lora_rotary.h"
#include "device_common.cuh"

namespace lora {

// The rotation as the kernels see it (a kernel parameter: lanes read their own entries of `step`). Its layout, pairs
// (i, i + dim / 2) or else (2 i, 2 i + 1), is the kernels' kHalf.
struct RotaryDev {
    uint64_t step[LORA_ROTARY_MAX_DIM / 2];  // of a pair: turns from one position to the next, times 2^64
    float factor;
    int dim;    // values of a head that are rotated, a multiple of 16
};

// A lane holds 16 values of a head as two runs of 8, one of each half of the rotated values (or of the others), so that
// neighbouring lanes' 16-byte accesses fill sectors, and that no lane needs another's values: half layout, the
// runs are pairs 8 c .. 8 c + 7 (c: the lane of the head); interleaved, 4 pairs each. (Runs side by side, two
// half sectors a lane: 30011 tokens interleaved 111 us with loads past L1, 91 with L1 making up for it.)
__device__ __forceinline__ void rotary_runs(const RotaryDev &rot, int head_dim, int c, int *d0, int *d1)
{
    const bool turns = 16 * c < rot.dim;
    const int first = turns ? 0 : rot.dim, n = turns ? rot.dim : head_dim - rot.dim;
    *d0 = first + 8 * c - first / 2;
    *d1 = *d0 + n / 2;
}

// cos and sin, times the factor, of the lane's pairs at position p. p times the pair's turns modulo one
// is exact in 64-bit integers; its upper 32 bits, signed, are the angle in units of pi / 2^31.
struct Turn8 {
    float c[8], s[8];
};
template <bool kHalf>
__device__ __forceinline__ Turn8 rotary_turn(const RotaryDev &rot, int c, int p, bool inverse)
{
    Turn8 t;
    const float f = inverse ? -rot.factor : rot.factor;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int pair = kHalf ? 8 * c + e : 4 * c + (e & 3) + (e < 4 ? 0 : rot.dim / 4);
        const uint64_t turns = (uint64_t)(int64_t)p * rot.step[pair];
        float s, co;
        sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &co);
        t.c[e] = co * rot.factor;
        t.s[e] = s * f;
    }
    return t;
}

__device__ __forceinline__ void unpack8(const uint4 &v, float *x)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float *x)
{
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// Two runs of 8 bf16 values, as floats: x[0..7], x[8..15].
__device__ __forceinline__ void unpack16(const uint4 (&v)[2], float (&x)[16])
{
    unpack8(v[0], x);
    unpack8(v[1], x + 8);
}

// The two runs, turned.
template <bool kHalf>
__device__ __forceinline__ void rotary_pairs(const Turn8 &t, float (&x)[16])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float &a = kHalf ? x[e] : x[2 * e], &b = kHalf ? x[8 + e] : x[2 * e + 1];
        const float u = a * t.c[e] - b * t.s[e], v = fmaf(a, t.s[e], b * t.c[e]);
        a = u;
        b = v;
    }
}

// How T tokens of `all` blocks of rows each are shared out. Many tokens: a chunk of consecutive ones a CTA, its warps
// taking turns, so that what a CTA reads at a time lies together. Few: a part of one token's blocks a warp.
struct RotaryGrid {
    static constexpr int kWarps = 8, kCtas = 2;  // of a CTA, of an SM
    int parts;  // 1: chunks
    unsigned ctas;
    bool streams;  // a call that reads and writes far more than L1 and the SMs hold at a time
    RotaryGrid(int64_t T, int64_t all, int num_sms)
    {
        const int64_t warps = (int64_t)kWarps * kCtas * num_sms;
        parts = (int)(T >= warps ? 1 : (warps + T - 1) / T < all ? (warps + T - 1) / T : all);
        ctas = (unsigned)(T >= warps ? kCtas * num_sms : (T * parts + kWarps - 1) / kWarps);
        streams = T * all >= 8 * warps;
    }
};
// This warp's tokens t0, t0 + step, .. below t1, and its blocks [b0, b1) of them.
struct RotaryShare {
    int t0, t1, step, b0, b1;
    __device__ __forceinline__ RotaryShare(int T, int all, int parts)
    {
        const int warp = threadIdx.x >> 5;
        if (parts == 1) {
            t0 = (int)((int64_t)blockIdx.x * T / gridDim.x) + warp;
            t1 = (int)((int64_t)(blockIdx.x + 1) * T / gridDim.x);
            step = RotaryGrid::kWarps;
            b0 = 0;
            b1 = all;
        } else {
            const int64_t w = (int64_t)blockIdx.x * RotaryGrid::kWarps + warp;
            const int part = (int)(w % parts);
            t0 = (int)(w / parts);
            t1 = min(T, t0 + 1);
            step = 1;
            b0 = (int)((int64_t)part * all / parts);
            b1 = (int)((int64_t)(part + 1) * all / parts);
        }
    }
};

inline RotaryDev rotary_view(const lora_rotary *r)
{
    RotaryDev v;
    for (int i = 0; i < LORA_ROTARY_MAX_DIM / 2; ++i) v.step[i] = r->step[i];
    v.factor = r->factor;
    v.dim = r->rotary_dim;
    return v;
}

// A rotation that lora_rotary_init may have filled.
inline bool rotary_ok(const lora_rotary *r)
{
    return r && r->rotary_dim >= 16 && r->rotary_dim <= LORA_ROTARY_MAX_DIM && r->rotary_dim % 16 == 0 &&
           (r->layout == LORA_ROTARY_HALF || r->layout == LORA_ROTARY_INTERLEAVED);
}

}  // namespace lora
