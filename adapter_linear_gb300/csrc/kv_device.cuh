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

}  // namespace lora
