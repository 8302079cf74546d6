// rotary_device.cuh -- rotary positions: a pair's angle, and the rotation of the 16 values a lane holds.
#pragma once

#include "../../include/lora_rotary.h"
#include "device_common.cuh"

namespace lora {

// The rotation as the kernels see it (a kernel parameter: lanes read their own entries of `step`).
struct RotaryDev {
    uint64_t step[LORA_ROTARY_MAX_DIM / 2];  // of a pair: turns from one position to the next, times 2^64
    float factor;
    int dim;    // values of a head that are rotated, a multiple of 16
    int half;   // pairs (i, i + dim / 2), else (2 i, 2 i + 1)
};

// A lane holds 16 values of a head as two runs of 8: in the rotated part those of pairs 8 c .. 8 c + 7
// (c: the lane of the head), so that no lane needs another's. Their offsets:
__device__ __forceinline__ void rotary_runs(const RotaryDev &rot, int c, int *d0, int *d1)
{
    const bool split = rot.half && 16 * c < rot.dim;
    *d0 = split ? 8 * c : 16 * c;
    *d1 = split ? rot.dim / 2 + 8 * c : 16 * c + 8;
}

// cos and sin, times the factor, of pairs 8 c .. 8 c + 7 at position p. p times the pair's turns modulo one
// is exact in 64-bit integers; its upper 32 bits, signed, are the angle in units of pi / 2^31.
struct Turn8 {
    float c[8], s[8];
};
__device__ __forceinline__ Turn8 rotary_turn(const RotaryDev &rot, int c, int p, bool inverse)
{
    Turn8 t;
    const float f = inverse ? -rot.factor : rot.factor;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint64_t turns = (uint64_t)(int64_t)p * rot.step[8 * c + e];
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

// The two runs, turned.
__device__ __forceinline__ void rotary_pairs(bool half, const Turn8 &t, float (&x)[16])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float a = half ? x[e] : x[2 * e], b = half ? x[8 + e] : x[2 * e + 1];
        const float u = a * t.c[e] - b * t.s[e], v = fmaf(a, t.s[e], b * t.c[e]);
        if (half) {
            x[e] = u;
            x[8 + e] = v;
        } else {
            x[2 * e] = u;
            x[2 * e + 1] = v;
        }
    }
}

inline RotaryDev rotary_view(const lora_rotary *r)
{
    RotaryDev v;
    for (int i = 0; i < LORA_ROTARY_MAX_DIM / 2; ++i) v.step[i] = r->step[i];
    v.factor = r->factor;
    v.dim = r->rotary_dim;
    v.half = r->layout == LORA_ROTARY_HALF;
    return v;
}

// A rotation that lora_rotary_init may have filled.
inline bool rotary_ok(const lora_rotary *r)
{
    return r && r->rotary_dim >= 16 && r->rotary_dim <= LORA_ROTARY_MAX_DIM && r->rotary_dim % 16 == 0 &&
           (r->layout == LORA_ROTARY_HALF || r->layout == LORA_ROTARY_INTERLEAVED);
}

}  // namespace lora
