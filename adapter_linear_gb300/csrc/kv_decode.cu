// kv_decode.cu -- attention of short chunks over the paged cache (kv_decode_kernel.cuh), every sequence by itself.
#include "kv_decode_kernel.cuh"

namespace lora {

int kv_decode_grid(int num_sms) { return kMaxCtas * num_sms; }

// two pieces a CTA
size_t kv_decode_part_floats(int D, int num_sms) { return (size_t)2 * kPartRows * num_sms * (D + 2); }

cudaError_t launch_kv_decode(const KvDev &kv, bool int8, const KvBatchDev &b, const KvAttn &a, int max_new,
                             int max_rows, float *part, int *count, int num_sms, cudaStream_t stream)
{
    return launch_kv_decode_mode<kPlain>(kv, int8, b, a, KvShareDev{}, max_new, max_rows, part, count, num_sms, false,
                                         stream);
}

}  // namespace lora
