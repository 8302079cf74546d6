// kv_device.cuh -- device helpers of the paged key/value cache: finding a row's sequence and
// a token's cache row, and the conversions between 8-bit codes and values.
#pragma once

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

// Two 8-bit codes to two bf16, exactly. x holds code a in bits 0..7 and code b in bits 16..23
// (the other bits are ignored). A code is (low 7 bits) - (its sign bit's 128), and in bf16
// 0x4300 | v is 128 + v for v < 128 and 0x4380 is 256: code = (128 + low) - (128 or 256).
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t x)
{
    const uint32_t low = (x & 0x007F007Fu) | 0x43004300u;
    const uint32_t sign = (x & 0x00800080u) | 0x43004300u;
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&low),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&sign));
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The four codes of a word, in order, as two bf16 pairs.
__device__ __forceinline__ void codes4_to_bf16(uint32_t w, uint32_t *lo, uint32_t *hi)
{
    *lo = codes_to_bf16(__byte_perm(w, 0, 0x4140));
    *hi = codes_to_bf16(__byte_perm(w, 0, 0x4342));
}

// Code i (0..3) of word a and code i of word b as a bf16 pair.
__device__ __forceinline__ uint32_t codes_pair_to_bf16(uint32_t a, uint32_t b, int i)
{
    return codes_to_bf16(__byte_perm(a, b, 0x0400u + 0x0101u * (uint32_t)i));
}

}  // namespace lora
