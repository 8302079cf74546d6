// kv_attention.cu -- attention of a chunk of new tokens over the paged cache.
//
// For row t at position pos of its sequence, query head h and its kv head:
//   z_j = scale * <Q[t,h], K_j> over the visible j,  O = sum_j softmax(z)_j V_j,
// in one pass over the keys with the running maximum m and sum l of the softmax: a key with
// z_j > m scales l and O down by exp(m - z_j).
#include "kv_device.cuh"

namespace lora {
namespace {

// One warp per (row, query head): lane i holds D / 32 dimensions of Q, O and of each key and
// value it reads, one key at a time.
template <int D, bool kInt8>
__global__ void __launch_bounds__(256) kv_attention_kernel(KvDev kv, KvBatchDev b, KvAttn a)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (w >= (int64_t)b.T * a.Hq) return;
    const int t = (int)(w / a.Hq), h = (int)(w % a.Hq);
    const int seq = kv_find_seq(b, t, lane);
    if (seq < 0) return;
    const KvSeq s = kv_seq(b, kv.page_shift, seq, kv.err);
    if (t - s.row0 >= s.n) return;
    const int pos = s.L - s.n + t - s.row0;
    const int j0 = a.window > 0 ? max(0, pos - a.window + 1) : 0;
    const int hk = h / a.G;

    float q[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const uint16_t v = a.Q[t * a.q_stride + h * D + lane * E + e];
        q[e] = __uint_as_float((uint32_t)v << 16) * a.scale;
        o[e] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    for (int j = j0; j <= pos; ++j) {
        int64_t row = kv_row(kv, b, seq, j);
        if (row < 0) break;
        row += (int64_t)hk << kv.page_shift;
        float k[E], v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int64_t at = row * D + lane * E + e;
            if (kInt8) {
                k[e] = (float)static_cast<const int8_t *>(kv.k)[at];
                v[e] = (float)static_cast<const int8_t *>(kv.v)[at];
            } else {
                k[e] = __uint_as_float((uint32_t)static_cast<const uint16_t *>(kv.k)[at] << 16);
                v[e] = __uint_as_float((uint32_t)static_cast<const uint16_t *>(kv.v)[at] << 16);
            }
        }
        float z = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) z = fmaf(q[e], k[e], z);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
        float vscale = 1.0f;
        if (kInt8) {
            z *= __uint_as_float((uint32_t)kv.ks[row] << 16);
            vscale = __uint_as_float((uint32_t)kv.vs[row] << 16);
        }
        const float m2 = fmaxf(m, z);
        const float down = m == -INFINITY ? 0.0f : expf(m - m2), p = expf(z - m2);
        l = l * down + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(p * vscale, v[e], o[e] * down);
        m = m2;
    }
    const float inv = pos < 0 ? 0.0f : 1.0f / l;
#pragma unroll
    for (int e = 0; e < E; ++e)
        a.O[t * a.o_stride + h * D + lane * E + e] = (uint16_t)(pack_bf16x2(o[e] * inv, 0.0f) & 0xFFFFu);
    if (a.lse && lane == 0) a.lse[(int64_t)t * a.Hq + h] = pos < 0 ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_kv_attention(const KvDev &kv, bool int8, const KvBatchDev &b, const KvAttn &a,
                                cudaStream_t stream)
{
    auto fn = kv.D == 128 ? (int8 ? kv_attention_kernel<128, true> : kv_attention_kernel<128, false>)
                          : (int8 ? kv_attention_kernel<64, true> : kv_attention_kernel<64, false>);
    const cudaError_t e = ensure_smem_attr((const void *)fn, 0);
    if (e != cudaSuccess) return e;
    const int64_t warps = (int64_t)b.T * a.Hq;
    fn<<<(unsigned)((warps + 7) / 8), 256, 0, stream>>>(kv, b, a);
    return cudaGetLastError();
}

}  // namespace lora
