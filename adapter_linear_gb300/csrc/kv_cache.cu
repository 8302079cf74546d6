// kv_cache.cu -- the paged key/value cache: the kernels that write tokens into their pages
// (quantised to 8 bits on the way) and read them back, and the C ABI of lora_kv.h.
#include <algorithm>
#include <climits>
#include <new>

#include "kv_device.cuh"
#include "kv_state.h"

using namespace lora;

namespace {

// ------------------------------------------------------------------- kernels
//
// A row (one token, one head, K or V) is D values; D / 8 lanes hold it, 8 values (16 bytes) a
// lane, so a warp holds 32 / (D / 8) rows. A token has 2 H rows (K's heads, then V's); warp w
// takes token w / C, rows (w % C) * (rows per warp) and on, C = chunks of a token.

template <int D>
struct RowMap {
    static constexpr int kLanes = D / 8;           // lanes per row
    static constexpr int kRows = 32 / kLanes;      // rows per warp
};

__device__ __forceinline__ float bf16_bits_f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// scale and 8 codes of this lane's 8 values; the row's kLanes lanes take part.
//   s = max(bf16(amax / 127), 2^-126), code = clamp(rint(x / s), -127, 127)
// x and s have 8 significant bits, so x / s is a tie or at least 2^-11 away from one:
// the fp32 division decides every code as exact arithmetic would.
template <int kLanes>
__device__ __forceinline__ uint2 quantise8(const uint4 &x, uint16_t *scale_bits)
{
    const float f[8] = {bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y),
                        bf16_lo(x.z), bf16_hi(x.z), bf16_lo(x.w), bf16_hi(x.w)};
    // the largest magnitude as an integer: the bits of |x| order like their values, and an
    // infinity or a NaN (exponent all ones) is larger than every finite value
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(f[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool finite = top < 0x7F800000u;
    const uint32_t sb = pack_bf16x2(__fdiv_rn(__uint_as_float(top), 127.0f), 0.0f) & 0xFFFFu;
    const float s = fmaxf(__uint_as_float(sb << 16), 1.17549435e-38f);  // 2^-126
    *scale_bits = finite ? (uint16_t)(__float_as_uint(s) >> 16) : (uint16_t)0x7FC0;
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = fminf(fmaxf(rintf(__fdiv_rn(f[i], s)), -127.0f), 127.0f);
        const int c = finite ? (int)q : 0;
        w[i >> 2] |= (uint32_t)(c & 0xFF) << (8 * (i & 3));
    }
    return make_uint2(w[0], w[1]);
}

// bf16(scale * code) of 8 codes: the product of a 7-bit code and an 8-bit scale is exact in
// fp32, so it is rounded once.
__device__ __forceinline__ uint4 dequantise8(uint2 c, uint16_t scale_bits)
{
    const float s = bf16_bits_f(scale_bits);
    uint32_t o[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const uint32_t w = p < 2 ? c.x : c.y;
        const int lo = (int)(int8_t)(w >> (16 * (p & 1))), hi = (int)(int8_t)(w >> (16 * (p & 1) + 8));
        o[p] = pack_bf16x2(s * (float)lo, s * (float)hi);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Where the token of row t of the call lies: its cache row for head 0; -1: a position below
// zero; -2: nowhere (padding after the last sequence, a bad table entry or length).
__device__ __forceinline__ int64_t token_row(const KvDev &kv, const KvBatchDev &b, int t, int lane)
{
    const int seq = kv_find_seq(b, t, lane);
    if (seq < 0) return -2;
    const KvSeq s = kv_seq(b, kv.page_shift, seq, kv.err);
    const int i = t - s.row0;
    if (i >= s.n) return -2;
    const int pos = s.L - s.n + i;
    if (pos < 0) return -1;
    const int64_t row = kv_row(kv, b, seq, pos);
    return row < 0 ? -2 : row;
}

template <int D, bool kInt8>
__global__ void __launch_bounds__(256) kv_write_kernel(KvDev kv, KvBatchDev b, const uint16_t *__restrict__ K,
                                                       int64_t k_stride, const uint16_t *__restrict__ V,
                                                       int64_t v_stride)
{
    using M = RowMap<D>;
    const int lane = threadIdx.x & 31;
    const int C = (2 * kv.H + M::kRows - 1) / M::kRows;
    const int64_t items = (int64_t)b.T * C;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); w < items; w += warps) {
        const int t = (int)(w / C);
        const int r = (int)(w % C) * M::kRows + lane / M::kLanes;
        const int d = (lane % M::kLanes) * 8;
        const bool on = r < 2 * kv.H;
        const bool is_v = r >= kv.H;
        const int h = is_v ? r - kv.H : r;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (on) x = ldg_nc_v4((is_v ? V + t * v_stride : K + t * k_stride) + h * D + d);
        const int64_t row0 = token_row(kv, b, t, lane);
        if (row0 < 0) continue;
        const int64_t row = row0 + ((int64_t)h << kv.page_shift);
        if (kInt8) {
            uint16_t s;
            const uint2 c = quantise8<M::kLanes>(x, &s);
            if (on) {
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(is_v ? kv.v : kv.k) + row * D + d) = c;
                if (d == 0) (is_v ? kv.vs : kv.ks)[row] = s;
            }
        } else if (on) {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(is_v ? kv.v : kv.k) + row * D + d) = x;
        }
    }
}

template <int D, bool kInt8>
__global__ void __launch_bounds__(256) kv_read_kernel(KvDev kv, KvBatchDev b, uint16_t *__restrict__ K,
                                                      int64_t k_stride, uint16_t *__restrict__ V,
                                                      int64_t v_stride)
{
    using M = RowMap<D>;
    const int lane = threadIdx.x & 31;
    const int C = (2 * kv.H + M::kRows - 1) / M::kRows;
    const int64_t items = (int64_t)b.T * C;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); w < items; w += warps) {
        const int t = (int)(w / C);
        const int r = (int)(w % C) * M::kRows + lane / M::kLanes;
        const int d = (lane % M::kLanes) * 8;
        const bool is_v = r >= kv.H;
        const int h = is_v ? r - kv.H : r;
        const int64_t row0 = token_row(kv, b, t, lane);
        if (row0 == -2 || r >= 2 * kv.H) continue;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (row0 >= 0) {
            const int64_t row = row0 + ((int64_t)h << kv.page_shift);
            if (kInt8)
                x = dequantise8(*reinterpret_cast<const uint2 *>(
                                    static_cast<const uint8_t *>(is_v ? kv.v : kv.k) + row * D + d),
                                (is_v ? kv.vs : kv.ks)[row]);
            else
                x = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(is_v ? kv.v : kv.k) +
                                                     row * D + d);
        }
        *reinterpret_cast<uint4 *>((is_v ? V + t * v_stride : K + t * k_stride) + h * D + d) = x;
    }
}

int row_grid(const KvDev &kv, int T, int num_sms)
{
    const int rows = 32 / (kv.D / 8);
    const int64_t items = (int64_t)T * ((2 * kv.H + rows - 1) / rows);
    return (int)std::min<int64_t>((items + 7) / 8, (int64_t)num_sms * 8);
}

// The error word read and cleared in one atomic step: [1] receives its value.
__global__ void kv_read_clear_kernel(int *err) { err[1] = atomicExch(err, 0); }

}  // namespace

namespace lora {

cudaError_t launch_kv_write(const KvDev &kv, bool int8, const KvBatchDev &b, const uint16_t *K, int64_t k_stride,
                            const uint16_t *V, int64_t v_stride, int num_sms, cudaStream_t stream)
{
    auto fn = kv.D == 128 ? (int8 ? kv_write_kernel<128, true> : kv_write_kernel<128, false>)
                          : (int8 ? kv_write_kernel<64, true> : kv_write_kernel<64, false>);
    const cudaError_t e = ensure_smem_attr((const void *)fn, 0);
    if (e != cudaSuccess) return e;
    fn<<<row_grid(kv, b.T, num_sms), 256, 0, stream>>>(kv, b, K, k_stride, V, v_stride);
    return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvDev &kv, bool int8, const KvBatchDev &b, uint16_t *K, int64_t k_stride,
                           uint16_t *V, int64_t v_stride, int num_sms, cudaStream_t stream)
{
    auto fn = kv.D == 128 ? (int8 ? kv_read_kernel<128, true> : kv_read_kernel<128, false>)
                          : (int8 ? kv_read_kernel<64, true> : kv_read_kernel<64, false>);
    const cudaError_t e = ensure_smem_attr((const void *)fn, 0);
    if (e != cudaSuccess) return e;
    fn<<<row_grid(kv, b.T, num_sms), 256, 0, stream>>>(kv, b, K, k_stride, V, v_stride);
    return cudaGetLastError();
}

}  // namespace lora

// ================================================================= the C ABI

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

bool tensor_ok(const void *p, int64_t stride, int64_t row)
{
    return p && aligned16(p) && stride >= row && stride % 8 == 0;
}

constexpr int kMaxTokens = 1 << 30;  // of a call or a sequence: positions stay clear of 32 bits

// A batch the kernels can take; *empty: there is nothing to do.
lora_status check_batch(const lora_kv_batch *b, int page_shift, bool *empty)
{
    *empty = false;
    if (!b || b->n_seqs < 0 || b->T < 0 || b->max_new < 0) return LORA_ERR_ARG;
    if (b->n_seqs == 0 || b->T == 0) {
        *empty = true;
        return LORA_OK;
    }
    if (!b->page_table || !b->start || !b->kv_len || b->table_stride < 1) return LORA_ERR_ARG;
    if (b->T > kMaxTokens || ((int64_t)b->table_stride << page_shift) > kMaxTokens) return LORA_ERR_ARG;
    return LORA_OK;
}

KvBatchDev batch_view(const lora_kv_batch *b)
{
    KvBatchDev v;
    v.table = b->page_table;
    v.start = b->start;
    v.kv_len = b->kv_len;
    v.table_stride = b->table_stride;
    v.n_seqs = b->n_seqs;
    v.T = b->T;
    return v;
}

KvDev kv_view(const lora_kv *p)
{
    KvDev v;
    v.k = p->k;
    v.v = p->v;
    v.ks = p->ks;
    v.vs = p->vs;
    v.num_pages = p->num_pages;
    v.page_shift = p->page_shift;
    v.H = p->H;
    v.D = p->D;
    v.err = p->d_err;
    return v;
}

constexpr int kDecodeRows = 16;

// The tcgen05 kernel's scratch (40 MB for D = 128), from the first call that needs it.
lora_status ensure_pre_part(lora_kv *p)
{
    if (p->pre_part) return LORA_OK;
    const size_t bytes = sizeof(float) * kv_prefill_part_floats(p->D, p->num_sms);
    if (cudaMalloc((void **)&p->pre_part, bytes) != cudaSuccess) {
        cudaGetLastError();
        p->pre_part = nullptr;
        return LORA_ERR_OOM;
    }
    return LORA_OK;
}

// Calls inside a graph capture are not tracked: the order of replays is the caller's.
lora_status is_tracked(cudaStream_t stream, bool *tracked)
{
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    CUDA_TRY(cudaStreamIsCapturing(stream, &cs));
    *tracked = cs == cudaStreamCaptureStatusNone;
    return LORA_OK;
}

// After a call on `stream`: the error-word read waits for it.
lora_status note_kv_call(lora_kv *p, cudaStream_t stream)
{
    bool tracked;
    const lora_status st = is_tracked(stream, &tracked);
    if (st != LORA_OK || !tracked) return st;
    CUDA_TRY(cudaEventRecord(p->ev_call, stream));
    CUDA_TRY(cudaStreamWaitEvent(p->ctl_stream, p->ev_call, 0));
    return LORA_OK;
}

}  // namespace

extern "C" {

lora_status lora_kv_create(int num_pages, int page_tokens, int n_kv_heads, int head_dim, int format,
                           void *k_pages, void *v_pages, void *k_scales, void *v_scales, lora_kv_t *out)
{
    if (!out) return LORA_ERR_ARG;
    *out = nullptr;
    if (format != LORA_KV_BF16 && format != LORA_KV_INT8) return LORA_ERR_ARG;
    if (page_tokens < 16 || page_tokens > 256 || (page_tokens & (page_tokens - 1)) != 0) return LORA_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 128) return LORA_ERR_SHAPE;
    if (n_kv_heads < 1 || n_kv_heads > 256 || num_pages < 1) return LORA_ERR_SHAPE;
    if ((int64_t)num_pages * page_tokens * n_kv_heads > INT_MAX) return LORA_ERR_SHAPE;
    const bool int8 = format == LORA_KV_INT8;
    if (!k_pages || !v_pages || !aligned16(k_pages) || !aligned16(v_pages)) return LORA_ERR_ARG;
    if (int8 != (k_scales != nullptr) || int8 != (v_scales != nullptr)) return LORA_ERR_ARG;
    if (!aligned16(k_scales) || !aligned16(v_scales)) return LORA_ERR_ARG;

    int dev = 0, major = 0, minor = 0, sms = 0;
    CUDA_TRY(cudaGetDevice(&dev));
    CUDA_TRY(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev));
    CUDA_TRY(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev));
    CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    if (major != 10 || minor != 3) return LORA_ERR_UNSUPPORTED;

    lora_kv *p = new (std::nothrow) lora_kv();
    if (!p) return LORA_ERR_OOM;
    p->device = dev;
    p->num_sms = sms;
    p->num_pages = num_pages;
    for (p->page_shift = 4; (1 << p->page_shift) < page_tokens;) ++p->page_shift;
    p->H = n_kv_heads;
    p->D = head_dim;
    p->int8 = int8;
    p->k = k_pages;
    p->v = v_pages;
    p->ks = static_cast<uint16_t *>(k_scales);
    p->vs = static_cast<uint16_t *>(v_scales);
    const size_t counts = sizeof(int) * (size_t)(kv_decode_grid(sms) + 8 * kv_prefill_grid(sms));
    if (cudaMalloc((void **)&p->d_err, 2 * sizeof(int)) != cudaSuccess ||
        cudaMalloc((void **)&p->dec_part, sizeof(float) * kv_decode_part_floats(head_dim, sms)) != cudaSuccess ||
        cudaMalloc((void **)&p->count, counts) != cudaSuccess ||
        cudaHostAlloc((void **)&p->h_err, sizeof(int), cudaHostAllocDefault) != cudaSuccess) {
        cudaGetLastError();
        lora_kv_destroy(p);
        return LORA_ERR_OOM;
    }
    if (cudaMemset(p->d_err, 0, 2 * sizeof(int)) != cudaSuccess ||
        cudaMemset(p->count, 0, counts) != cudaSuccess ||
        cudaEventCreateWithFlags(&p->ev_call, cudaEventDisableTiming) != cudaSuccess ||
        cudaEventCreateWithFlags(&p->ev_attn, cudaEventDisableTiming) != cudaSuccess ||
        cudaStreamCreateWithFlags(&p->ctl_stream, cudaStreamNonBlocking) != cudaSuccess ||
        ensure_smem_attr((const void *)kv_read_clear_kernel, 0) != cudaSuccess ||
        cudaDeviceSynchronize() != cudaSuccess) {
        lora_kv_destroy(p);
        return LORA_ERR_CUDA;
    }
    *out = p;
    return LORA_OK;
}

lora_status lora_kv_destroy(lora_kv_t p)
{
    if (!p) return LORA_ERR_ARG;
    cudaDeviceSynchronize();
    if (p->ctl_stream) cudaStreamDestroy(p->ctl_stream);
    if (p->ev_call) cudaEventDestroy(p->ev_call);
    if (p->ev_attn) cudaEventDestroy(p->ev_attn);
    if (p->dec_part) cudaFree(p->dec_part);
    if (p->pre_part) cudaFree(p->pre_part);
    if (p->count) cudaFree(p->count);
    if (p->d_err) cudaFree(p->d_err);
    if (p->h_err) cudaFreeHost(p->h_err);
    delete p;
    return LORA_OK;
}

lora_status lora_kv_reserve(lora_kv_t p, int max_tokens, int n_heads, int max_seqs)
{
    if (!p || max_tokens < 0 || max_seqs < 0) return LORA_ERR_ARG;
    if (n_heads < 1 || n_heads > 1024 || n_heads % p->H != 0) return LORA_ERR_SHAPE;
    return max_tokens > max_seqs ? ensure_pre_part(p) : LORA_OK;  // single tokens never need it
}

lora_status lora_kv_write(lora_kv_t p, const void *K, int64_t k_stride, const void *V, int64_t v_stride,
                          const lora_kv_batch *batch, lora_stream_t stream)
{
    if (!p) return LORA_ERR_ARG;
    bool empty;
    lora_status st = check_batch(batch, p->page_shift, &empty);
    if (st != LORA_OK || empty) return st;
    const int64_t row = (int64_t)p->H * p->D;
    if (!tensor_ok(K, k_stride, row) || !tensor_ok(V, v_stride, row)) return LORA_ERR_ARG;
    CUDA_TRY(launch_kv_write(kv_view(p), p->int8, batch_view(batch), static_cast<const uint16_t *>(K), k_stride,
                             static_cast<const uint16_t *>(V), v_stride, p->num_sms, stream));
    return note_kv_call(p, stream);
}

lora_status lora_kv_read(lora_kv_t p, void *K, int64_t k_stride, void *V, int64_t v_stride,
                         const lora_kv_batch *batch, lora_stream_t stream)
{
    if (!p) return LORA_ERR_ARG;
    bool empty;
    lora_status st = check_batch(batch, p->page_shift, &empty);
    if (st != LORA_OK || empty) return st;
    const int64_t row = (int64_t)p->H * p->D;
    if (!tensor_ok(K, k_stride, row) || !tensor_ok(V, v_stride, row)) return LORA_ERR_ARG;
    CUDA_TRY(launch_kv_read(kv_view(p), p->int8, batch_view(batch), static_cast<uint16_t *>(K), k_stride,
                            static_cast<uint16_t *>(V), v_stride, p->num_sms, stream));
    return note_kv_call(p, stream);
}

lora_status lora_kv_attention(lora_kv_t p, const void *Q, int64_t q_stride, int n_heads,
                              const lora_kv_batch *batch, float scale, int window, void *O, int64_t o_stride,
                              float *lse, lora_stream_t stream)
{
    if (!p || window < 0) return LORA_ERR_ARG;
    if (n_heads < 1 || n_heads > 1024 || n_heads % p->H != 0) return LORA_ERR_SHAPE;
    bool empty;
    lora_status st = check_batch(batch, p->page_shift, &empty);
    if (st != LORA_OK || empty) return st;
    if ((int64_t)batch->T * n_heads > INT_MAX) return LORA_ERR_ARG;
    const int64_t row = (int64_t)n_heads * p->D;
    if (!tensor_ok(Q, q_stride, row) || !tensor_ok(O, o_stride, row)) return LORA_ERR_ARG;
    KvAttn a;
    a.Q = static_cast<const uint16_t *>(Q);
    a.O = static_cast<uint16_t *>(O);
    a.lse = lse;
    a.q_stride = q_stride;
    a.o_stride = o_stride;
    a.Hq = n_heads;
    a.G = n_heads / p->H;
    a.window = std::min(window, kMaxTokens);
    a.scale = scale;
    // Sequences of up to kDecodeRows rows of a kv head go to the short-chunk kernel, others to
    // the tcgen05 kernel; where max_new says that there is only one kind, one launch takes all.
    const bool prefill = (int64_t)batch->max_new * a.G > kDecodeRows;
    const bool decode = !prefill || batch->T < (int64_t)batch->n_seqs * batch->max_new;
    if (prefill && (st = ensure_pre_part(p)) != LORA_OK) return st;
    bool tracked;
    if ((st = is_tracked(stream, &tracked)) != LORA_OK) return st;
    // the scratch belongs to one call at a time: after the last one, if that ran elsewhere
    if (tracked && p->attn_any && stream != p->attn_stream) CUDA_TRY(cudaStreamWaitEvent(stream, p->ev_attn, 0));
    const KvDev kv = kv_view(p);
    const KvBatchDev bd = batch_view(batch);
    if (decode)
        CUDA_TRY(launch_kv_decode(kv, p->int8, bd, a, batch->max_new, prefill ? kDecodeRows : INT_MAX, p->dec_part,
                                  p->count, p->num_sms, stream));
    if (prefill)
        CUDA_TRY(launch_kv_prefill(kv, p->int8, bd, a, decode ? kDecodeRows + 1 : 0, p->pre_part,
                                   p->count + kv_decode_grid(p->num_sms), p->num_sms, stream));
    if (!tracked) return LORA_OK;
    CUDA_TRY(cudaEventRecord(p->ev_attn, stream));
    CUDA_TRY(cudaStreamWaitEvent(p->ctl_stream, p->ev_attn, 0));
    p->attn_stream = stream;
    p->attn_any = true;
    return LORA_OK;
}

lora_status lora_kv_check_errors(lora_kv_t p)
{
    if (!p) return LORA_ERR_ARG;
    // on the control stream, which follows every call enqueued on the cache
    kv_read_clear_kernel<<<1, 1, 0, p->ctl_stream>>>(p->d_err);
    if (cudaGetLastError() != cudaSuccess ||
        cudaMemcpyAsync(p->h_err, p->d_err + 1, sizeof(int), cudaMemcpyDeviceToHost, p->ctl_stream) !=
            cudaSuccess ||
        cudaStreamSynchronize(p->ctl_stream) != cudaSuccess)
        return LORA_ERR_CUDA;
    if (*p->h_err & kErrTimeoutBit) return LORA_ERR_TIMEOUT;
    if (*p->h_err & kErrRangeBit) return LORA_ERR_RANGE;
    return LORA_OK;
}

}  // extern "C"
