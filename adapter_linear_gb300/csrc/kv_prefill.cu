// kv_prefill.cu -- attention of longer chunks over the paged cache (kv_prefill_kernel.cuh), every sequence by itself.
#include "kv_prefill_kernel.cuh"

namespace lora {

int kv_prefill_grid(int num_sms) { return num_sms; }

size_t kv_prefill_part_floats(int D, int num_sms)
{
    return (size_t)2 * kv_prefill_grid(num_sms) * kBlockRows * (D + 2);
}

cudaError_t launch_kv_prefill(const KvDev &kv, bool int8, const KvBatchDev &b, const KvAttn &a, int min_rows,
                              float *part, int *count, int num_sms, cudaStream_t stream)
{
    return launch_kv_prefill_mode<kPlain>(kv, int8, b, a, KvShareDev{}, min_rows, part, count, num_sms, stream);
}

}  // namespace lora
