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
// A row is one token, one head, K or V: D values. A token has 2 H rows, K's heads, then V's. A
// warp takes a run of consecutive tokens (1 to kRun) and kRows neighbouring rows of each; a lane
// holds 16 values of a row of an 8-bit cache (32 bytes of bf16, 16 of codes) or 8 of a bf16 one.
//
// HBM bounds both at thousands of tokens (write: 2 D bytes read and D + 2 written a row of an 8-bit
// cache, read the reverse), the chain of dependent loads (sequence, length, page) at a few.
// So a run is looked up once, a lane a token, and then copied four tokens at a time, loads
// ahead of stores; few tokens get runs of one, so that as many warps as possible share them.
// Measured, 8 kv heads of 128 values, 8-bit: 141741 tokens read 153 us (5.7 TB/s; runs of 16 157, of
// 4 160), 16384 written and read 47 us (two kernels of 100 MB). More resident warps do not help: with
// 48 registers a thread the copies in flight spill (177 and 63 us).
constexpr int kRun = 8;
constexpr int kBatch = 4;  // tokens loaded before any is stored

template <int D, bool kInt8>
struct RowMap {
    static constexpr int kValues = kInt8 ? 16 : 8;   // of a lane
    static constexpr int kLanes = D / kValues;       // of a row
    static constexpr int kRows = 32 / kLanes;        // of a warp
    static constexpr int kVec = kValues / 8;         // 16-byte vectors of bf16 a lane
};

// scale and 16 codes of this lane's 16 values; the row's kLanes lanes take part.
//   s = max(bf16(amax / 127), 2^-126), code = rint(x / s), ties to even
// (at most 127: s is at least amax / 127.499). x and s have 8 significant bits, so x / s is either a
// tie or more than 2^-10 away from one. y = x * (1 / s) is off by less than 2^-15, so rounding it
// to a multiple of 2^-11 first gives the ties exactly and moves nothing else across one: the codes
// are those of exact arithmetic without a division each (a division each: 16384 tokens written
// and read back 76 us, so 56).
template <int kLanes>
__device__ __forceinline__ uint4 quantise16(const uint4 (&x)[2], uint16_t *scale_bits)
{
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    // the largest magnitude as an integer: the bits of |x| order like their values, and an
    // infinity or a NaN (exponent all ones) is larger than every finite value
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool finite = top < 0x7F80u;
    const uint32_t sb = pack_bf16x2(__fdiv_rn(__uint_as_float(top << 16), 127.0f), 0.0f) & 0xFFFFu;
    const float s = fmaxf(__uint_as_float(sb << 16), 1.17549435e-38f);  // 2^-126
    *scale_bits = finite ? (uint16_t)(__float_as_uint(s) >> 16) : (uint16_t)0x7FC0;
    const float inv = __frcp_rn(s);
    const uint64_t inv2 = pack2(inv, inv);
    const uint64_t grid = pack2(6144.0f, 6144.0f), back = pack2(-6144.0f, -6144.0f);  // 1.5 2^12: multiples of 2^-11
    const uint64_t whole = pack2(12582912.0f, 12582912.0f);  // 1.5 2^23: the code in the low byte
    uint32_t c[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t v[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t b = w[2 * q + e];
            float lo, hi;
            unpack2(add2(add2(fma2(pack2(bf16_lo(b), bf16_hi(b)), inv2, grid), back), whole), &lo, &hi);
            v[e] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x0040);
        }
        c[q] = finite ? __byte_perm(v[0], v[1], 0x5410) : 0u;
    }
    return make_uint4(c[0], c[1], c[2], c[3]);
}

// bf16(scale * code) of 8 codes: codes are exact in bf16, and a bf16 product rounds the exact one
// once. s: the scale, twice.
__device__ __forceinline__ uint4 dequantise8(uint32_t c0, uint32_t c1, __nv_bfloat162 s, uint32_t base)
{
    uint32_t o[4];
    codes4_to_bf16(c0, base, &o[0], &o[1]);
    codes4_to_bf16(c1, base, &o[2], &o[3]);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&o[p]), s);
        o[p] = *reinterpret_cast<const uint32_t *>(&v);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ uint4 shfl_xor_v4(uint4 v, int d)
{
    return make_uint4(__shfl_xor_sync(0xffffffffu, v.x, d), __shfl_xor_sync(0xffffffffu, v.y, d),
                      __shfl_xor_sync(0xffffffffu, v.z, d), __shfl_xor_sync(0xffffffffu, v.w, d));
}

// Where the tokens of rows t0 + lane, lane < run, lie: the cache row for head 0; -1: a position
// below zero; -2: nowhere (padding after the last sequence, a bad table entry or length).
__device__ __forceinline__ int64_t run_rows(const KvDev &kv, const KvBatchDev &b, int t0, int run, int lane)
{
    int seq = max(0, kv_find_seq(b, t0, lane));
    const int t = t0 + lane;
    if (lane >= run) return -2;
    KvSeq s;
    for (;; ++seq) {  // a run may end in a later sequence
        if (seq >= b.n_seqs) return -2;
        s = kv_seq(b, kv.page_shift, seq, kv.err);
        if (t < s.row0) return -2;
        if (t - s.row0 < s.n) break;
    }
    const int pos = s.L - s.n + (t - s.row0);
    if (pos < 0) return -1;
    const int64_t row = kv_row(kv, b, seq, pos);
    return row < 0 ? -2 : row;
}

template <int D, bool kInt8>
__global__ void __launch_bounds__(256) kv_write_kernel(KvDev kv, KvBatchDev b, const uint16_t *__restrict__ K,
                                                       int64_t k_stride, const uint16_t *__restrict__ V,
                                                       int64_t v_stride, int run_len)
{
    using M = RowMap<D, kInt8>;
    const int lane = threadIdx.x & 31;
    const int C = (2 * kv.H + M::kRows - 1) / M::kRows;
    const int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int64_t t0_ = w / C * run_len;
    if (t0_ >= b.T) return;
    const int t0 = (int)t0_, run = min(run_len, b.T - t0);
    const int r = (int)(w % C) * M::kRows + lane / M::kLanes;
    const int d = (lane % M::kLanes) * M::kValues;
    const bool on = r < 2 * kv.H, is_v = r >= kv.H;
    const int h = on ? (is_v ? r - kv.H : r) : 0;
    const int64_t stride = is_v ? v_stride : k_stride;
    const uint16_t *src = (is_v ? V : K) + (int64_t)t0 * stride + h * D + d;
    const int64_t head = (int64_t)h << kv.page_shift;
    uint4 x[kBatch][M::kVec];
    auto load = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int v = 0; v < M::kVec; ++v) {
                x[i][v] = make_uint4(0, 0, 0, 0);
                if (i0 + i < run && on) x[i][v] = ldg_nc_v4(src + (i0 + i) * stride + v * 8);
            }
    };
    load(0);  // on their way while the run is looked up
    const int64_t rows = run_rows(kv, b, t0, run, lane);
    for (int i0 = 0; i0 < run; i0 += kBatch) {
        if (i0 > 0) load(i0);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int64_t row = __shfl_sync(0xffffffffu, rows, min(i0 + i, 31)) + head;
            const bool there = i0 + i < run && row >= head && on;
            if constexpr (kInt8) {
                uint16_t s;
                const uint4 c = quantise16<M::kLanes>(x[i], &s);
                if (there) {
                    *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(is_v ? kv.v : kv.k) + row * D + d) = c;
                    if (d == 0) (is_v ? kv.vs : kv.ks)[row] = s;
                }
            } else if (there) {
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(is_v ? kv.v : kv.k) + row * D + d) = x[i][0];
            }
        }
    }
}

template <int D, bool kInt8>
__global__ void __launch_bounds__(256) kv_read_kernel(KvDev kv, KvBatchDev b, uint16_t *__restrict__ K,
                                                      int64_t k_stride, uint16_t *__restrict__ V,
                                                      int64_t v_stride, int run_len)
{
    using M = RowMap<D, kInt8>;
    const int lane = threadIdx.x & 31;
    const int C = (2 * kv.H + M::kRows - 1) / M::kRows;
    const int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int64_t t0_ = w / C * run_len;
    if (t0_ >= b.T) return;
    const int t0 = (int)t0_, run = min(run_len, b.T - t0);
    const int r = (int)(w % C) * M::kRows + lane / M::kLanes;
    const int d = (lane % M::kLanes) * M::kValues;
    const bool on = r < 2 * kv.H, is_v = r >= kv.H;
    const int h = on ? (is_v ? r - kv.H : r) : 0;
    const int64_t stride = is_v ? v_stride : k_stride;
    uint16_t *dst = (is_v ? V : K) + (int64_t)t0 * stride + h * D + d;
    const uint32_t base = kv_opaque(0x43004300u);
    const bool odd = lane & 1;
    const int64_t head = (int64_t)h << kv.page_shift;
    const int64_t rows = run_rows(kv, b, t0, run, lane);
    for (int i0 = 0; i0 < run; i0 += kBatch) {
        uint4 x[kBatch];
        uint16_t s[kBatch];
        int64_t row[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            row[i] = __shfl_sync(0xffffffffu, rows, min(i0 + i, 31));
            if (i0 + i >= run || !on) row[i] = -2;
            x[i] = make_uint4(0, 0, 0, 0);
            s[i] = 0;
            if (row[i] >= 0) {
                const int64_t at = row[i] + head;
                x[i] = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(is_v ? kv.v : kv.k) +
                                                        (at * D + d) * (kInt8 ? 1 : 2));
                if (kInt8) s[i] = (is_v ? kv.vs : kv.ks)[at];
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            uint16_t *const to = dst + (i0 + i) * stride;
            if constexpr (kInt8) {
                // two neighbouring lanes swap halves, so that each store fills 32-byte sectors
                // (141741 tokens read: 175 us without, so 165), and what is written makes room
                // in L2 first (157)
                const __nv_bfloat162 f = q4_scale_pair(s[i]);
                const uint4 lo = dequantise8(x[i].x, x[i].y, f, base), hi = dequantise8(x[i].z, x[i].w, f, base);
                const uint4 got = shfl_xor_v4(odd ? lo : hi, 1);
                if (row[i] == -2) continue;
                __stcs(reinterpret_cast<uint4 *>(odd ? to - 8 : to), odd ? got : lo);
                __stcs(reinterpret_cast<uint4 *>(odd ? to + 8 : to + 16), odd ? hi : got);
            } else if (row[i] != -2) {
                *reinterpret_cast<uint4 *>(to) = x[i];
            }
        }
    }
}

// Run length and blocks (8 warps): runs of 1 until four warps a scheduler have one each, then
// longer ones.
struct RowGrid {
    int run;
    unsigned blocks;
};
RowGrid row_grid(const KvDev &kv, bool int8, int T, int num_sms)
{
    const int rows = 32 / (kv.D / (int8 ? 16 : 8));
    const int64_t C = (2 * kv.H + rows - 1) / rows;
    RowGrid g;
    g.run = (int)std::min<int64_t>(kRun, std::max<int64_t>(1, T * C / (16 * (int64_t)num_sms)));
    g.blocks = (unsigned)(((T + g.run - 1) / g.run * C + 7) / 8);
    return g;
}

// The error word read and cleared in one atomic step: [1] receives its value.
__global__ void kv_read_clear_kernel(int *err) { err[1] = atomicExch(err, 0); }

// What calls leave behind whose waits ran out (lora_kv_selftest_timeout).
__global__ void kv_abandon_kernel(int *err, int *count, int n)
{
    for (int i = threadIdx.x; i < n; i += blockDim.x) count[i] = 1 + i % 3;
    if (threadIdx.x == 0) atomicOr(err, kErrTimeoutBit);
}

}  // namespace

namespace lora {

cudaError_t launch_kv_write(const KvDev &kv, bool int8, const KvBatchDev &b, const uint16_t *K, int64_t k_stride,
                            const uint16_t *V, int64_t v_stride, int num_sms, cudaStream_t stream)
{
    auto fn = kv.D == 128 ? (int8 ? kv_write_kernel<128, true> : kv_write_kernel<128, false>)
                          : (int8 ? kv_write_kernel<64, true> : kv_write_kernel<64, false>);
    const cudaError_t e = ensure_smem_attr((const void *)fn, 0);
    if (e != cudaSuccess) return e;
    const RowGrid g = row_grid(kv, int8, b.T, num_sms);
    fn<<<g.blocks, 256, 0, stream>>>(kv, b, K, k_stride, V, v_stride, g.run);
    return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvDev &kv, bool int8, const KvBatchDev &b, uint16_t *K, int64_t k_stride,
                           uint16_t *V, int64_t v_stride, int num_sms, cudaStream_t stream)
{
    auto fn = kv.D == 128 ? (int8 ? kv_read_kernel<128, true> : kv_read_kernel<128, false>)
                          : (int8 ? kv_read_kernel<64, true> : kv_read_kernel<64, false>);
    const cudaError_t e = ensure_smem_attr((const void *)fn, 0);
    if (e != cudaSuccess) return e;
    const RowGrid g = row_grid(kv, int8, b.T, num_sms);
    fn<<<g.blocks, 256, 0, stream>>>(kv, b, K, k_stride, V, v_stride, g.run);
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

// A batch the kernels can take, with the cache's device current; *empty: there is nothing to do.
lora_status check_batch(const lora_kv *p, const lora_kv_batch *b, bool *empty)
{
    *empty = false;
    int dev = -1;
    CUDA_TRY(cudaGetDevice(&dev));
    if (dev != p->device) return LORA_ERR_ARG;
    if (!b || b->n_seqs < 0 || b->T < 0 || b->max_new < 0) return LORA_ERR_ARG;
    if (b->n_seqs == 0 || b->T == 0) {
        *empty = true;
        return LORA_OK;
    }
    if (!b->page_table || !b->start || !b->kv_len || b->table_stride < 1) return LORA_ERR_ARG;
    if (b->T > kMaxTokens || ((int64_t)b->table_stride << p->page_shift) > kMaxTokens) return LORA_ERR_ARG;
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

// Arrival counters of both attention kernels.
int count_ints(const lora_kv *p) { return kv_decode_grid(p->num_sms) + 8 * kv_prefill_grid(p->num_sms); }

// Rows (query heads of new tokens) of a kv head up to which the short-chunk kernel takes a sequence: 32
// requests of 6 tokens on 4 query heads (24 rows) take 82 us there, 161 on the tcgen05 kernel, of
// whose 256 rows they use 24; with 28 and 32 rows the short-chunk kernel's accumulators spill (192
// against 160).
constexpr int kDecodeRows = 24;

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

bool capturing(cudaStream_t stream, lora_status *st)
{
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    *st = cudaStreamIsCapturing(stream, &cs) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
    if (*st != LORA_OK) cudaGetLastError();
    return cs != cudaStreamCaptureStatusNone;
}

// `ev` now stands for what it stood for and for the work of `stream` so far. Two streams may have
// one handle (the per-thread stream of two threads, a stream made after another was destroyed), so the
// old record is waited for before it is replaced; on one stream that is nothing.
lora_status extend_event(cudaEvent_t ev, cudaStream_t stream)
{
    CUDA_TRY(cudaStreamWaitEvent(stream, ev, 0));
    CUDA_TRY(cudaEventRecord(ev, stream));
    return LORA_OK;
}

// After a write or a read on `stream`: an event of that stream, for the error-word read. Calls inside a
// graph capture are not tracked: the order of replays is the caller's.
lora_status note_kv_call(lora_kv *p, cudaStream_t stream)
{
    lora_status st;
    if (capturing(stream, &st) || st != LORA_OK) return st;
    // the entry of this stream, or a new one, becomes the last
    for (size_t i = p->calls.size(); i-- > 0;)
        if (p->calls[i].stream == stream) {
            std::swap(p->calls[i], p->calls.back());
            return extend_event(p->calls.back().ev, stream);
        }
    lora_kv::Call c{stream, nullptr};
    CUDA_TRY(cudaEventCreateWithFlags(&c.ev, cudaEventDisableTiming));
    if (cudaEventRecord(c.ev, stream) != cudaSuccess) {
        cudaGetLastError();
        cudaEventDestroy(c.ev);
        return LORA_ERR_CUDA;
    }
    try {
        p->calls.push_back(c);
    } catch (...) {
        cudaEventDestroy(c.ev);
        return LORA_ERR_OOM;
    }
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
    const size_t counts = sizeof(int) * (size_t)count_ints(p);
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
        cudaStreamCreateWithFlags(&p->ctl_stream, cudaStreamNonBlocking) != cudaSuccess ||
        cudaEventCreateWithFlags(&p->attn_ev, cudaEventDisableTiming) != cudaSuccess ||
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
    for (const lora_kv::Call &c : p->calls) cudaEventDestroy(c.ev);
    if (p->attn_ev) cudaEventDestroy(p->attn_ev);
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
    // all of them may be one sequence's
    return (int64_t)max_tokens * (n_heads / p->H) > kDecodeRows ? ensure_pre_part(p) : LORA_OK;
}

lora_status lora_kv_write(lora_kv_t p, const void *K, int64_t k_stride, const void *V, int64_t v_stride,
                          const lora_kv_batch *batch, lora_stream_t stream)
{
    if (!p) return LORA_ERR_ARG;
    bool empty;
    lora_status st = check_batch(p, batch, &empty);
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
    lora_status st = check_batch(p, batch, &empty);
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
    lora_status st = check_batch(p, batch, &empty);
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
    // 2^(s + 1) >= G > 2^s: the multiplier, 2^(32 + s) / G rounded up, times G is off from 2^(32 + s) by less than
    // G, which shows from x = 2^31 on
    a.g_shift = 0;
    while ((2 << a.g_shift) < a.G) ++a.g_shift;
    a.g_mul = a.G > 1 ? (uint32_t)(((1ull << (32 + a.g_shift)) + a.G - 1) / a.G) : 0;
    a.window = std::min(window, kMaxTokens);
    a.scale = scale;
    // Sequences of up to kDecodeRows rows of a kv head go to the short-chunk kernel, others to
    // the tcgen05 kernel; where max_new says that there is only one kind, one launch takes all. (No
    // sequence has more than T rows, so that a loose bound needs no scratch that lora_kv_reserve leaves out.)
    const int max_new = std::min(batch->max_new, batch->T);
    const bool prefill = (int64_t)max_new * a.G > kDecodeRows;
    const bool decode = !prefill || batch->T < (int64_t)batch->n_seqs * max_new;
    if (prefill && (st = ensure_pre_part(p)) != LORA_OK) return st;
    // The scratch belongs to one call at a time: after the last attention call, whatever stream that
    // ran on (captured calls: the order of replays is the caller's).
    const bool tracked = !capturing(stream, &st);
    if (st != LORA_OK) return st;
    if (tracked) CUDA_TRY(cudaStreamWaitEvent(stream, p->attn_ev, 0));
    const KvDev kv = kv_view(p);
    const KvBatchDev bd = batch_view(batch);
    cudaError_t e = cudaSuccess;
    if (decode)
        e = launch_kv_decode(kv, p->int8, bd, a, max_new, prefill ? kDecodeRows : INT_MAX, p->dec_part, p->count,
                             p->num_sms, stream);
    if (prefill && e == cudaSuccess)
        e = launch_kv_prefill(kv, p->int8, bd, a, decode ? kDecodeRows + 1 : 0, p->pre_part,
                              p->count + kv_decode_grid(p->num_sms), p->num_sms, stream);
    // (the first launch may have run when the second failed; the event stands for all calls so far,
    // each having waited for the one before)
    if (tracked && cudaEventRecord(p->attn_ev, stream) != cudaSuccess && e == cudaSuccess) e = cudaErrorUnknown;
    if (e != cudaSuccess) {
        cudaGetLastError();
        return LORA_ERR_CUDA;
    }
    return LORA_OK;
}

lora_status lora_kv_check_errors(lora_kv_t p)
{
    if (!p) return LORA_ERR_ARG;
    // on the control stream, after every call
    CUDA_TRY(cudaStreamWaitEvent(p->ctl_stream, p->attn_ev, 0));
    for (const lora_kv::Call &c : p->calls) CUDA_TRY(cudaStreamWaitEvent(p->ctl_stream, c.ev, 0));
    kv_read_clear_kernel<<<1, 1, 0, p->ctl_stream>>>(p->d_err);
    if (cudaGetLastError() != cudaSuccess ||
        cudaMemcpyAsync(p->h_err, p->d_err + 1, sizeof(int), cudaMemcpyDeviceToHost, p->ctl_stream) !=
            cudaSuccess ||
        cudaStreamSynchronize(p->ctl_stream) != cudaSuccess)
        return LORA_ERR_CUDA;
    if (*p->h_err & kErrTimeoutBit) {
        // pieces of that call never arrived: the counters start from zero again
        CUDA_TRY(cudaMemsetAsync(p->count, 0, sizeof(int) * (size_t)count_ints(p), p->ctl_stream));
        CUDA_TRY(cudaStreamSynchronize(p->ctl_stream));
        return LORA_ERR_TIMEOUT;
    }
    if (*p->h_err & kErrRangeBit) return LORA_ERR_RANGE;
    return LORA_OK;
}

lora_status lora_kv_selftest_timeout(lora_kv_t p, lora_stream_t stream)
{
    if (!p) return LORA_ERR_ARG;
    kv_abandon_kernel<<<1, 256, 0, stream>>>(p->d_err, p->count, count_ints(p));
    CUDA_TRY(cudaGetLastError());
    return note_kv_call(p, stream);
}

}  // extern "C"
