// kv_internal.h -- what the translation units of the paged key/value cache share: the
// handle, the views the kernels take and the launchers (not part of the public ABI).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/lora_kv.h"
#include "internal.h"

namespace lora {

// The cache as the kernels see it. Row (page, head, r) starts at ((page * H + head) * p + r)
// * D values of k / v (bytes or bf16) and holds its scale at the same row index.
struct KvDev {
    void *k, *v;
    uint16_t *ks, *vs;  // bf16 bits (int8 caches)
    int num_pages;
    int page_shift;     // log2 of the tokens per page
    int H, D;
    int *err;
};

// The batch as the kernels see it (device pointers).
struct KvBatchDev {
    const int32_t *table, *start, *kv_len;
    int table_stride, n_seqs, T;
};

cudaError_t launch_kv_write(const KvDev &kv, bool int8, const KvBatchDev &b, const uint16_t *K, int64_t k_stride,
                            const uint16_t *V, int64_t v_stride, int num_sms, cudaStream_t stream);
cudaError_t launch_kv_read(const KvDev &kv, bool int8, const KvBatchDev &b, uint16_t *K, int64_t k_stride,
                           uint16_t *V, int64_t v_stride, int num_sms, cudaStream_t stream);

// The write with rotary positions: K, V as for the write; Q (Hq heads, 0: none) rotated into Q_out.
struct KvRotaryArgs {
    const uint16_t *K, *V, *Q;
    uint16_t *Q_out;
    int64_t k_stride, v_stride, q_stride, qo_stride;
    int Hq;
};
cudaError_t launch_kv_write_rotary(const KvDev &kv, bool int8, const KvBatchDev &b, const lora_rotary *rotary,
                                   const KvRotaryArgs &a, int num_sms, cudaStream_t stream);

// One attention call.
struct KvAttn {
    const uint16_t *Q;
    uint16_t *O;
    float *lse;          // or nullptr
    int64_t q_stride, o_stride;
    int Hq, G;           // query heads; query heads per kv head
    uint32_t g_mul;      // x / G = x g_mul >> (32 + g_shift) for 0 <= x < 2^31, G > 1
    int g_shift;
    int window;          // 0: none
    float scale;
};

// Attention over a prefix that the sequences of a group share (kv_shared.cu) runs the attention kernels in two
// more modes.
//   kPrefix: the "sequences" are groups: all rows of one see all tokens of its prefix, in the pages of its first
//     sequence with rows. O and lse (in units of log2) go to the arrays below, fp32; the group of an empty
//     prefix is left out.
//   kOwn: sequence b starts at token lo[b] (a multiple of the page's tokens); where that is above 0 its rows
//     are joined with what the first mode left there.
enum KvMode { kPlain = 0, kPrefix = 1, kOwn = 2 };
//     The tcgen05 kernel leaves the pieces of an item that several CTAs share in `part` (row major). What they
//     are pieces of is in items[first CTA], for a kernel that joins them, and in where[row], for one that
//     reads the pieces themselves (pieces).
constexpr int kShareRows = 256;  // rows of a slot of `part`
constexpr uint32_t kJoined = 0xFFFFFFFFu;
struct KvShareItem {
    int last, row0, head, rows;  // last CTA with a piece (-1: nothing to join), the first token's row, kv head, rows
    int first_row, pad[3];       // the first row's number among the group's rows
};
// Where a CTA's share of the prefixes' work begins, from the plan: the item's group (as in groups), its number and
// tile of rows, and in the tcgen05 kernel's units the share [u, u_end), the tile's first one, and all of them.
struct KvShareBegin {
    int4 group;
    int64_t u, u_end, tile0, total;
    int seq, tile, shares, pad;
};
static_assert(sizeof(KvShareBegin) == 64, "read as four pieces");
// What where[row] says of the pieces [c0, c0 + n) of a row's prefix. After a wait of the prefix's kernel has run
// out a row has none, and the word there is what the memory held before: then kJoined, whose O and lse2 are the row's own
// places, so that nothing outside the scratch is read (grid: of the prefix's kernel).
__host__ __device__ inline uint2 kv_where(uint2 w, int grid)
{
    const uint32_t c0 = w.x & 0xFFFFu, c1 = w.x >> 16;
    if (w.x != kJoined && !(c0 <= c1 && c1 < (uint32_t)grid && w.y < (uint32_t)kShareRows)) w.x = kJoined;
    return w;
}
struct KvShareDev {
    KvShareBegin *begins;  // [grid of the tcgen05 kernel]
    int64_t *group_at;     // [n_groups] the plan's own
    float *part;         // [2 grid][256][D], then (m, l) [2 grid][256][2]
    KvShareItem *items;  // [grid]
    uint2 *where;        // [T][Hq] last and first CTA with a piece of the row, 16 bits each, and its row in their blocks;
                         // x == kJoined: none, O and lse2 are there
    bool pieces;         // read the pieces; else all are joined
    int pieces_grid;     // the grid of the kernel that left them
    bool two_parts;      // the tcgen05 kernel gives every weight of a prefix two bf16 parts
    int64_t ml_at;       // where in part (m, l) begin
    int4 *groups;  // a group's sequence whose pages are read, tokens of its prefix, first row, rows
    int32_t *lo;   // [n_seqs]
    // Work of the short-chunk kernel on the sequences' own tokens: the first item of each sequence [n_seqs + 1],
    // and of all {items (-1: too many to be numbered), the most units of one, units (64 bits, the lower half first)}.
    int32_t *own_first;
    int4 *own_sums;
    float *O;      // [T][Hq][D]
    float *lse2;   // [T][Hq]
};

// The kernel for short chunks. It takes the sequences of at most max_rows rows (new tokens times
// G); max_new is the caller's bound on the new tokens of one. part, count: scratch of
// kv_decode_part_floats floats and kv_decode_grid ints (zero between calls), used by one call at a
// time.
int kv_decode_grid(int num_sms);
size_t kv_decode_part_floats(int D, int num_sms);
cudaError_t launch_kv_decode(const KvDev &kv, bool int8, const KvBatchDev &b, const KvAttn &a, int max_new,
                             int max_rows, float *part, int *count, int num_sms, cudaStream_t stream);

// The kernel for longer chunks (tcgen05): the sequences of at least min_rows rows. part, count:
// as above, kv_prefill_part_floats floats and 8 kv_prefill_grid ints.
int kv_prefill_grid(int num_sms);
size_t kv_prefill_part_floats(int D, int num_sms);
cudaError_t launch_kv_prefill(const KvDev &kv, bool int8, const KvBatchDev &b, const KvAttn &a, int min_rows,
                              float *part, int *count, int num_sms, cudaStream_t stream);

// The pieces that launch_kv_prefill_shared(kPrefix) left, joined into share.O and share.lse2.
size_t kv_share_part_floats(int D, int num_sms);
cudaError_t launch_kv_share_join(const KvDev &kv, bool int8, const KvAttn &a, const KvShareDev &share, int num_sms,
                                 cudaStream_t stream);

// Both for groups that share prefixes. early: the kernel may start before the one ahead of it has ended; it waits for
// that one itself, kPrefix before it reads the plan, kOwn before it reads the prefixes' results. The plan fills
// share.groups and share.lo.
// own_rows: rows of an item of launch_kv_decode_shared(kOwn), kv_decode_rows(max_new * G); it takes sequences of up to
// max_rows. shares: kv_prefill_grid where launch_kv_prefill_shared(kPrefix) is next, else 0.
constexpr int kDecodeUnit = 64, kDecodeHeadUnits = 4;
inline int kv_decode_rows(int64_t rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 24; }
cudaError_t launch_kv_share_plan(const KvDev &kv, const KvBatchDev &b, const int32_t *seq_start,
                                 const int32_t *prefix_len, int n_groups, int G, int own_rows, int max_rows, int shares,
                                 const KvShareDev &share, cudaStream_t stream);
cudaError_t launch_kv_decode_shared(KvMode mode, const KvDev &kv, bool int8, const KvBatchDev &b, const KvAttn &a,
                                    const KvShareDev &share, int max_new, int max_rows, float *part, int *count,
                                    int num_sms, bool early, cudaStream_t stream);
cudaError_t launch_kv_prefill_shared(KvMode mode, const KvDev &kv, bool int8, const KvBatchDev &b, const KvAttn &a,
                                     const KvShareDev &share, int min_rows, float *part, int *count, int num_sms,
                                     cudaStream_t stream);

}  // namespace lora
