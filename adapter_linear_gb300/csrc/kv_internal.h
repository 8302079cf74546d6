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

}  // namespace lora
