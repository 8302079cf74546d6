// kv_state.h -- the host-side state of a lora_kv (private to the library).
#pragma once

#include <vector>

#include <cuda_runtime.h>

#include "../../include/lora_kv.h"
#include "kv_internal.h"
#include "pool_state.h"

struct lora_kv {
    int device = 0, num_sms = 0;
    int num_pages = 0, page_shift = 0, H = 0, D = 0;
    bool int8 = false;
    void *k = nullptr, *v = nullptr;           // the caller's arenas
    uint16_t *ks = nullptr, *vs = nullptr;
    int *d_err = nullptr;                      // [0] the error word, [1] its value at the last read
    int *h_err = nullptr;                      // pinned copy of d_err[1]
    // the writes and reads so far on each stream that has been used, the most recent stream's at the end
    struct Call {
        cudaStream_t stream;
        cudaEvent_t ev;
    };
    std::vector<Call> calls;
    // the attention's scratch, used by one call at a time; attn_ev: the attention calls so far
    cudaEvent_t attn_ev = nullptr;
    float *dec_part = nullptr, *pre_part = nullptr;  // pre_part: from the first call or reserve
    int *count = nullptr;                            // the short-chunk kernel's, then the other's
    cudaStream_t ctl_stream = nullptr;         // error-word reads
};
