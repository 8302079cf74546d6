// kv_device.cuh -- device helpers of the paged key/value cache: finding a row's sequence and
// a token's cache row, and the conversions between 8-bit codes and values.
#pragma once

#include <cuda_fp16.h>

#include "device_common.cuh"
#include "kv_internal.h"

namespace lora {

__device__ __forceinline__ void kv_flag_range(int *err) { atomicOr(err, kErrRangeBit); }

// Sequence b's rows [row0, row0 + n) and length L, checked: a start outside 0..T or a length
// beyond the table flags the error word and reads as an empty sequence.
struct KvSeq {
    int row0, n, L;
};

__device__ __forceinline__ KvSeq kv_seq(const KvBatchDev &b, int page_shift, int seq, int *err)
{
    KvSeq s;
    s.row0 = b.start[seq];
    const int end = b.start[seq + 1];
    s.n = end - s.row0;
    s.L = b.kv_len[seq];
    if (s.row0 < 0 || end > b.T || s.n < 0 || s.L < 0 ||
        (int64_t)s.L > ((int64_t)b.table_stride << page_shift)) {
        kv_flag_range(err);
        s.n = 0;
        s.L = 0;
    }
    return s;
}

// The sequence whose rows hold row t (called by a whole warp, the same t in every lane): the
// last b with start[b] <= t, by a 32-way search: a round narrows the range to a 32nd, so 1024
// sequences take two dependent loads. -1: before the first row.
__device__ __forceinline__ int kv_find_seq(const KvBatchDev &b, int t, int lane)
{
    int lo = 0, len = b.n_seqs;  // the answer is lo - 1 + (number of starts <= t in [lo, lo + len))
    while (len > 0) {
        const int step = (len + 31) >> 5;
        const int at = lo + (lane + 1) * step - 1;  // the last entry of this lane's part
        const bool le = at < lo + len && b.start[at] <= t;
        const int full = __popc(__ballot_sync(0xffffffffu, le));  // parts that lie wholly below
        const int end = lo + len;
        lo += full * step;
        len = min(step - 1, end - lo);
    }
    return lo - 1;
}

// Cache row of the token at `pos` of sequence `seq` for head 0, or -1 (a bad table entry).
__device__ __forceinline__ int64_t kv_row(const KvDev &kv, const KvBatchDev &b, int seq, int pos)
{
    const int page = b.table[(int64_t)seq * b.table_stride + (pos >> kv.page_shift)];
    if (page < 0 || page >= kv.num_pages) {
        kv_flag_range(kv.err);
        return -1;
    }
    return (((int64_t)page * kv.H) << kv.page_shift) + (pos & ((1 << kv.page_shift) - 1));
}

constexpr float kLn2 = 0.6931471805599453f;

// 2^x, to about 2^-22 of it; 0 for -inf
__device__ __forceinline__ float fast_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (x & mask) | bits in one instruction: with both constants known the compiler makes two of it,
// so `bits` comes from a register it cannot see through (kv_opaque).
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(mask), "r"(bits));
    return r;
}
__device__ __forceinline__ uint32_t kv_opaque(uint32_t v)
{
    uint32_t r;
    asm volatile("mov.b32 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// Two 8-bit codes to two bf16, exactly. x holds code a in bits 0..7 and code b in bits 16..23
// (the other bits are ignored). A code is (low 7 bits) - (its sign bit's 128), and in bf16
// 0x4300 | v is 128 + v for v < 128 and 0x4380 is 256: code = (128 + low) - (128 or 256).
// base: 0x43004300 from kv_opaque.
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t x, uint32_t base)
{
    const uint32_t low = and_or(x, 0x007F007Fu, base);
    const uint32_t sign = and_or(x, 0x00800080u, base);
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&low),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&sign));
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The four codes of a word, in order, as two f16 pairs, exactly: 0x6400 | v is 1024 + v in f16,
// v = code + 128.
__device__ __forceinline__ void codes4_to_f16(uint32_t w, uint32_t *lo, uint32_t *hi)
{
    w ^= 0x80808080u;
    const uint32_t bias = 0x64806480u;  // 1024 + 128, twice
    const uint32_t x[2] = {__byte_perm(w, 0x64646464u, 0x4140), __byte_perm(w, 0x64646464u, 0x4342)};
    const __half2 l = __hsub2(*reinterpret_cast<const __half2 *>(&x[0]), *reinterpret_cast<const __half2 *>(&bias));
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&x[1]), *reinterpret_cast<const __half2 *>(&bias));
    *lo = *reinterpret_cast<const uint32_t *>(&l);
    *hi = *reinterpret_cast<const uint32_t *>(&h);
}

// Code i (0..3) of word a and code i of word b as a bf16 pair.
__device__ __forceinline__ uint32_t codes_pair_to_bf16(uint32_t a, uint32_t b, int i, uint32_t base)
{
    return codes_to_bf16(__byte_perm(a, b, 0x0400u + 0x0101u * (uint32_t)i), base);
}

}  // namespace lora
