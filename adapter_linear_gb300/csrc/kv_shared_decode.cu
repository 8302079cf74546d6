// kv_shared_decode.cu -- the short-chunk attention kernel over shared prefixes and over what is behind them.
#include "kv_decode_kernel.cuh"

namespace lora {

cudaError_t launch_kv_decode_shared(KvMode mode, const KvDev &kv, bool int8, const KvBatchDev &b, const KvAttn &a,
                                    const KvShareDev &share, int max_new, int max_rows, float *part, int *count,
                                    int num_sms, bool early, cudaStream_t stream)
{
    return mode == kPrefix ? launch_kv_decode_mode<kPrefix>(kv, int8, b, a, share, max_new, max_rows, part, count,
                                                            num_sms, early, stream)
                           : launch_kv_decode_mode<kOwn>(kv, int8, b, a, share, max_new, max_rows, part, count,
                                                         num_sms, early, stream);
}

}  // namespace lora
