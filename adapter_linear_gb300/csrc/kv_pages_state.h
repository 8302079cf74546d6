// kv_pages_state.h -- the host-side state of a lora_kv_pages (private to the library).
#pragma once

#include <algorithm>

#include <cuda_runtime.h>

#include "../../include/lora_kv.h"
#include "kv_internal.h"
#include "pool_state.h"

struct lora_kv_pages {
    int device = 0;
    int num_pages = 0, page_shift = 0, max_seqs = 0, stride = 0;
    int32_t *table = nullptr, *kv_len = nullptr, *refs = nullptr;  // the caller's
    int32_t *scratch = nullptr;
    int *d_err = nullptr;               // [0] the error word, [1] its value at the last read, [2] pages used
    int *h_err = nullptr;               // pinned
    cudaEvent_t ev = nullptr;           // the calls so far
    cudaStream_t ctl_stream = nullptr;  // error-word reads
    // pairs of a move list: a compaction moves at most half of the pages, an update copies one page a slot
    int cap() const { return std::max(num_pages / 2 + 1, max_seqs); }
};

namespace lora {

constexpr int kErrPagesBit = 8;  // not enough free pages

cudaError_t launch_kv_copy(const KvDev &kv, bool int8, const int32_t *src, const int32_t *dst, const int32_t *rows,
                           const int32_t *n_dev, int n, int num_sms, cudaStream_t stream);
cudaError_t launch_kv_copy_moves(const KvDev &kv, bool int8, const lora_kv_pages *p, int num_sms, cudaStream_t stream);
// Around the kernels of one call that uses p's tables: it follows the calls so far.
lora_status kv_pages_begin(lora_kv_pages *p, cudaStream_t stream, bool *tracked);
lora_status kv_pages_end(lora_kv_pages *p, cudaStream_t stream, bool tracked, cudaError_t e);

}  // namespace lora
