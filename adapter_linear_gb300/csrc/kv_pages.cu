// kv_pages.cu -- page tables of sequences that fork, grow, shrink and go: the update and the compaction of
// the tables, and the copies of pages that they ask for.
#include <algorithm>
#include <climits>
#include <new>

#include <cooperative_groups.h>

#include "kv_pages_state.h"
#include "kv_state.h"

namespace cg = cooperative_groups;
using namespace lora;

namespace {

// The tables are some hundred kilobytes, in L2, and the work on them a handful of steps that each need all of
// the one before (who names a page, which pages are free, who gets them), so latency bounds it: one cluster
// of kCtas CTAs does all steps, a cluster barrier between them.
constexpr int kCtas = 8, kThreads = 1024;
constexpr int kUnit = 128;  // table entries a warp takes at a time, four a lane

struct PagesDev {
    int32_t *table, *kv_len, *refs;
    int P, S, W, shift;        // pages, slots, entries a slot, log2 of a page's tokens
    int32_t *old_table;        // [S][W] the table before the call, where it is used
    int32_t *kept, *src;       // [S] tokens kept, and of which slot (-1: none)
    int32_t *base;             // [S] the first new page of a slot among all, 2 x + (keeps the page it ends in)
    int32_t *held;             // [S] entries used before
    int32_t *count, *claim;    // [P] slots that have all of a page; the first that ends inside (kNone: none)
    int32_t *fresh;            // [P] new pages, in order
    int32_t *moves;            // [3][cap]: page, page, rows
    int32_t *moves_n;          // [1]
    int cap;
    int *err;
};

constexpr int kNone = INT_MAX;

// What the CTAs of the cluster tell each other, in the first one's shared memory.
struct Common {
    int bad[2];            // error bits of the first two steps, each looked at behind its step's barrier
    int found[kCtas];      // free (update) or used (compaction) pages of each CTA's part
    int need, copies;      // new pages and copies in all
    int below;             // compaction: used pages below n
};

__device__ __forceinline__ int entries(int tokens, int shift) { return (tokens + (1 << shift) - 1) >> shift; }

// Sum over a block of v, in every thread. sm: 33 values.
template <class T>
__device__ __forceinline__ T block_sum(T v, T *sm)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    __syncthreads();
    if (lane == 0) sm[warp] = v;
    __syncthreads();
    if (warp == 0) {
        T s = sm[lane];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        if (lane == 0) sm[32] = s;
    }
    __syncthreads();
    return sm[32];
}

// Exclusive prefix of v over a block; *all: the sum.
template <class T>
__device__ __forceinline__ T block_scan(T v, T *sm, T *all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T s = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T o = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += o;
    }
    __syncthreads();
    if (lane == 31) sm[warp] = s;
    __syncthreads();
    if (warp == 0) {
        T x = sm[lane], y = x;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const T o = __shfl_up_sync(0xffffffffu, y, d);
            if (lane >= d) y += o;
        }
        sm[lane] = y - x;
        if (lane == 31) sm[32] = y;
    }
    __syncthreads();
    *all = sm[32];
    return sm[warp] + s - v;
}

// Calls fn(slot, entry) for the entries below used(slot) of all slots, spread over the cluster's warps.
template <class Used, class Fn>
__device__ __forceinline__ void each_entry(const PagesDev &p, int cta, Used used, Fn fn)
{
    const int lane = threadIdx.x & 31;
    const int per = (p.W + kUnit - 1) / kUnit;
    for (int64_t u = cta * (kThreads / 32) + (threadIdx.x >> 5); u < (int64_t)p.S * per; u += kCtas * (kThreads / 32)) {
        const int s = (int)(u / per), j0 = (int)(u % per) * kUnit;
        const int n = used(s);
#pragma unroll
        for (int k = 0; k < kUnit / 32; ++k)
            if (j0 + k * 32 + lane < n) fn(s, j0 + k * 32 + lane);
    }
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1)
    kv_pages_update_kernel(PagesDev p, const int32_t *parent, const int32_t *keep, const int32_t *room)
{
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ Common mine;
    __shared__ int64_t sm[33];
    int *const sm32 = reinterpret_cast<int *>(sm);
    const int cta = blockIdx.x, tid = cta * kThreads + threadIdx.x;
    Common *const all = cluster.map_shared_rank(&mine, 0);
    if (threadIdx.x < 2) mine.bad[threadIdx.x] = 0;
    cluster.sync();

    // ---- 1: what is asked for; the counts start from zero; the table as it is
    const int capacity = (int)min((int64_t)p.W << p.shift, (int64_t)INT_MAX);
    for (int i = tid; i < p.S; i += kCtas * kThreads) {
        const int from = parent ? parent[i] : i, here = p.kv_len[i];
        const int extra = room ? room[i] : 0;
        bool wrong = from < -1 || from >= p.S || extra < 0 || here < 0 || here > capacity;
        int n = 0;
        if (!wrong && from >= 0) {
            n = p.kv_len[from];
            wrong = n < 0 || n > capacity;
            if (keep) n = min(n, max(0, keep[i]));
        }
        wrong = wrong || (int64_t)n + extra > capacity;
        if (wrong) atomicOr(&all->bad[0], kErrRangeBit);
        p.kept[i] = wrong ? 0 : n;
        p.src[i] = wrong ? -1 : from;
        p.held[i] = wrong ? 0 : entries(here, p.shift);
    }
    for (int x = tid; x < p.P; x += kCtas * kThreads) {
        p.count[x] = 0;
        p.claim[x] = kNone;
    }
    each_entry(p, cta, [&](int s) { return min(p.W, max(0, entries(min(p.kv_len[s], capacity), p.shift))); },
               [&](int s, int j) { p.old_table[(int64_t)s * p.W + j] = p.table[(int64_t)s * p.W + j]; });
    cluster.sync();
    int bad = all->bad[0];
    if (bad) goto refuse;

    // ---- 2: who has a page, who ends inside one
    each_entry(p, cta, [&](int s) { return entries(__ldcg(p.kept + s), p.shift); },
               [&](int s, int j) {
                   const int x = __ldcg(p.old_table + (int64_t)__ldcg(p.src + s) * p.W + j);
                   if (x < 0 || x >= p.P) {
                       atomicOr(&all->bad[1], kErrRangeBit);
                   } else if (j < __ldcg(p.kept + s) >> p.shift) {
                       atomicAdd(p.count + x, 1);
                   } else {
                       atomicMin(p.claim + x, s + (__ldcg(p.src + s) == s ? 0 : p.S));
                   }
               });
    cluster.sync();
    bad = all->bad[1];
    if (bad) goto refuse;

    {
        // ---- 3: free pages of this CTA's part (a page that someone ends inside and nobody has stays with the
        // first who asked); the first CTA: the new pages and copies of every slot
        const int part = (p.P + kCtas - 1) / kCtas, x0 = min(p.P, cta * part), x1 = min(p.P, x0 + part);
        int free = 0;
        for (int x = x0 + threadIdx.x; x < x1; x += kThreads)
            free += __ldcg(p.count + x) == 0 && __ldcg(p.claim + x) == kNone;
        free = block_sum(free, sm32);
        if (threadIdx.x == 0) all->found[cta] = free;
        if (cta == 0) {
            int64_t before = 0;  // new pages, and in the upper half copies
            for (int s0 = 0; s0 < p.S; s0 += kThreads) {
                const int s = s0 + threadIdx.x;
                int64_t v = 0;
                int stays = 0, n = 0, old = -1, to = -1;
                if (s < p.S) {
                    n = __ldcg(p.kept + s);
                    const int total = n + (room ? room[s] : 0), full = n >> p.shift;
                    if (n & ((1 << p.shift) - 1)) {
                        to = __ldcg(p.src + s);
                        old = __ldcg(p.old_table + (int64_t)to * p.W + full);
                        stays = __ldcg(p.claim + old) == s + (to == s ? 0 : p.S) && __ldcg(p.count + old) == 0;
                        if (!stays) v = 1ll << 32;
                    }
                    v += entries(total, p.shift) - full - stays;
                }
                int64_t sum;
                const int64_t at = before + block_scan(v, sm, &sum);
                if (s < p.S) {
                    p.base[s] = 2 * (int)(uint32_t)at + stays;
                    if (v >> 32) {
                        const int k = (int)(at >> 32);
                        p.moves[k] = old;
                        p.moves[p.cap + k] = (int)(uint32_t)at;  // (which new page: its number below)
                        p.moves[2 * p.cap + k] = n & ((1 << p.shift) - 1);
                    }
                }
                before += sum;
            }
            if (threadIdx.x == 0) {
                mine.need = (int)(uint32_t)before;
                mine.copies = (int)(before >> 32);
            }
        }
        cluster.sync();

        // ---- 4: the lowest free pages, as many as are needed
        const int need = all->need;
        int before = 0, there = 0;
        for (int c = 0; c < kCtas; ++c) {
            if (c < cta) before += all->found[c];
            there += all->found[c];
        }
        if (need > there) {
            bad = kErrPagesBit;
            goto refuse;
        }
        for (int y0 = x0; y0 < x1 && before < need; y0 += kThreads) {
            const int x = y0 + threadIdx.x;
            const int v = x < x1 && __ldcg(p.count + x) == 0 && __ldcg(p.claim + x) == kNone;
            int sum;
            const int at = before + block_scan(v, sm32, &sum);
            if (v && at < need) {
                p.fresh[at] = x;
                p.count[x] = 1;
            }
            before += sum;
        }
        cluster.sync();

        // ---- 5: the new state
        for (int x = tid; x < p.P; x += kCtas * kThreads) {
            const int c = __ldcg(p.count + x);
            p.refs[x] = c == 0 && __ldcg(p.claim + x) != kNone ? 1 : c;
        }
        each_entry(p, cta,
                   [&](int s) {
                       return max(__ldcg(p.held + s), entries(__ldcg(p.kept + s) + (room ? room[s] : 0), p.shift));
                   },
                   [&](int s, int j) {
                       const int n = __ldcg(p.kept + s), b = __ldcg(p.base + s);
                       const int old = (n >> p.shift) + (b & 1);  // entries that stay
                       int x = -1;
                       if (j < old)
                           x = __ldcg(p.old_table + (int64_t)__ldcg(p.src + s) * p.W + j);
                       else if (j < entries(n + (room ? room[s] : 0), p.shift))
                           x = __ldcg(p.fresh + (b >> 1) + j - old);
                       p.table[(int64_t)s * p.W + j] = x;
                   });
        for (int s = tid; s < p.S; s += kCtas * kThreads) p.kv_len[s] = __ldcg(p.kept + s) + (room ? room[s] : 0);
        const int copies = all->copies;
        for (int k = tid; k < copies; k += kCtas * kThreads)
            p.moves[p.cap + k] = __ldcg(p.fresh + __ldcg(p.moves + p.cap + k));
        if (tid == 0) *p.moves_n = copies;
        cluster.sync();  // the first CTA's shared memory is still read
        return;
    }

refuse:
    if (tid == 0) {
        atomicOr(p.err, bad);
        *p.moves_n = 0;
    }
    cluster.sync();
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1)
    kv_pages_compact_kernel(PagesDev p, int32_t *table_out, int32_t *refs_out)
{
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ Common mine;
    __shared__ int sm[33];
    const int cta = blockIdx.x, tid = cta * kThreads + threadIdx.x;
    Common *const all = cluster.map_shared_rank(&mine, 0);
    const int part = (p.P + kCtas - 1) / kCtas, x0 = min(p.P, cta * part), x1 = min(p.P, x0 + part);
    cluster.sync();  // all have started

    int used = 0;
    for (int x = x0 + threadIdx.x; x < x1; x += kThreads) used += p.refs[x] > 0;
    used = block_sum(used, sm);
    if (threadIdx.x == 0) all->found[cta] = used;
    cluster.sync();
    int n = 0, before = 0;
    for (int c = 0; c < kCtas; ++c) {
        if (c < cta) before += all->found[c];
        n += all->found[c];
    }
    // used pages below n: counted by the CTA whose part n is in
    if (n >= x0 && (n < x1 || (x1 == p.P && n == p.P && x0 < x1))) {
        int v = 0;
        for (int x = x0 + threadIdx.x; x < min(n, x1); x += kThreads) v += p.refs[x] > 0;
        v = block_sum(v, sm);
        if (threadIdx.x == 0) all->below = before + v;
    }
    cluster.sync();
    const int below = all->below, moved = n - below;
    // the k-th used page from n on, the k-th free one below n
    for (int y0 = x0; y0 < x1; y0 += kThreads) {
        const int x = y0 + threadIdx.x;
        const int r = x < x1 ? p.refs[x] : 0;
        int sum;
        const int at = before + block_scan((int)(r > 0), sm, &sum);
        if (x < x1 && x >= n && r > 0) {
            p.moves[at - below] = x;
            p.moves[2 * p.cap + at - below] = 1 << p.shift;
            p.count[x] = at - below;  // its move
            p.claim[at - below] = r;
        }
        if (x < x1 && x < n && r == 0) p.moves[p.cap + x - at] = x;
        before += sum;
    }
    cluster.sync();

    for (int x = tid; x < p.P; x += kCtas * kThreads) {
        const int r = p.refs[x];
        if (x >= n)
            refs_out[x] = 0;
        else if (r > 0 && refs_out != p.refs)
            refs_out[x] = r;
    }
    for (int k = tid; k < moved; k += kCtas * kThreads) refs_out[__ldcg(p.moves + p.cap + k)] = __ldcg(p.claim + k);
    const int capacity = (int)min((int64_t)p.W << p.shift, (int64_t)INT_MAX);
    each_entry(p, cta,
               [&](int s) {
                   if (table_out != p.table) return p.W;
                   return max(0, entries(min(p.kv_len[s], capacity), p.shift));
               },
               [&](int s, int j) {
                   const int64_t e = (int64_t)s * p.W + j;
                   const int x = p.table[e];
                   const bool inside = j < entries(max(0, min(p.kv_len[s], capacity)), p.shift);
                   const bool bad = inside && (x < 0 || x >= p.P);
                   if (bad) atomicOr(p.err, kErrRangeBit);
                   // (a page that refs does not count has no move)
                   int to = x;
                   if (inside && !bad && x >= n && x < p.P) {
                       const int k = __ldcg(p.count + x);
                       if (k >= 0 && k < moved && __ldcg(p.moves + k) == x)
                           to = __ldcg(p.moves + p.cap + k);
                       else
                           atomicOr(p.err, kErrRangeBit);
                   }
                   if (to != x || table_out != p.table) table_out[e] = to;
               });
    if (tid == 0) *p.moves_n = moved;
    cluster.sync();  // the first CTA's shared memory is still read
}

__global__ void __launch_bounds__(kThreads) kv_pages_used_kernel(const int32_t *refs, int P, int *out)
{
    __shared__ int sm[33];
    int used = 0;
    for (int x = threadIdx.x; x < P; x += kThreads) used += refs[x] > 0;
    used = block_sum(used, sm);
    if (threadIdx.x == 0) *out = used;
}

__global__ void kv_pages_read_clear_kernel(int *err) { err[1] = atomicExch(err, 0); }

// Copies of pages: HBM bounds them. The rows of a page, a head, K or V are contiguous; a warp copies up to
// kSlice bytes of them at a time, all loads ahead of the stores.
constexpr int kSlice = 4096;

struct CopyList {
    const int32_t *src, *dst, *rows;  // rows: or nullptr, all
    const int32_t *n_dev;             // or nullptr: n
    int n;
};

__global__ void __launch_bounds__(256) kv_copy_kernel(KvDev kv, int row_bytes, CopyList list)
{
    const int lane = threadIdx.x & 31;
    const int n = list.n_dev ? min(*list.n_dev, list.n) : list.n;
    const int tokens = 1 << kv.page_shift;
    const int slices = (tokens * row_bytes + kSlice - 1) / kSlice;
    const int per = 2 * kv.H * slices;  // units of a pair: slices of heads of K, then of V
    for (int64_t u = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); u < (int64_t)n * per;
         u += (int64_t)gridDim.x * (blockDim.x >> 5)) {
        const int i = (int)(u / per), y = (int)(u % per);
        const int slice = y % slices, h = y / slices % kv.H;
        const bool is_v = y >= kv.H * slices;
        const int a = list.src[i], b = list.dst[i], rows = list.rows ? list.rows[i] : tokens;
        if (a < 0 || b < 0 || a == b) continue;
        if (a >= kv.num_pages || b >= kv.num_pages || rows < 0 || rows > tokens) {
            if (lane == 0) atomicOr(kv.err, kErrRangeBit);
            continue;
        }
        const int64_t from = ((int64_t)a * kv.H + h) << kv.page_shift, to = ((int64_t)b * kv.H + h) << kv.page_shift;
        uint8_t *const values = static_cast<uint8_t *>(is_v ? kv.v : kv.k);
        const uint8_t *const src = values + from * row_bytes;
        uint8_t *const dst = values + to * row_bytes;
        const int end = min(rows * row_bytes, (slice + 1) * kSlice);
        const int at = slice * kSlice + lane * 16;
        uint4 v[kSlice / 512];
#pragma unroll
        for (int k = 0; k < kSlice / 512; ++k)
            if (at + k * 512 < end) v[k] = __ldcs(reinterpret_cast<const uint4 *>(src + at + k * 512));
#pragma unroll
        for (int k = 0; k < kSlice / 512; ++k)
            if (at + k * 512 < end) *reinterpret_cast<uint4 *>(dst + at + k * 512) = v[k];
        if (kv.ks && slice == 0) {
            uint16_t *const scales = is_v ? kv.vs : kv.ks;
            for (int r = lane; r < rows; r += 32) scales[to + r] = scales[from + r];
        }
    }
}

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

lora_status on_device(int device)
{
    int dev = -1;
    CUDA_TRY(cudaGetDevice(&dev));
    return dev == device ? LORA_OK : LORA_ERR_ARG;
}

// Between the two the caller enqueues one call's kernels on `stream`: they follow the calls so far. Calls inside
// a capture are ordered by whoever replays the graph.
lora_status begin_call(lora_kv_pages *p, cudaStream_t stream, bool *tracked)
{
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(stream, &cs) != cudaSuccess) {
        cudaGetLastError();
        return LORA_ERR_CUDA;
    }
    *tracked = cs == cudaStreamCaptureStatusNone;
    if (*tracked) CUDA_TRY(cudaStreamWaitEvent(stream, p->ev, 0));
    return LORA_OK;
}
lora_status end_call(lora_kv_pages *p, cudaStream_t stream, bool tracked, cudaError_t e)
{
    if (tracked && cudaEventRecord(p->ev, stream) != cudaSuccess && e == cudaSuccess) e = cudaErrorUnknown;
    if (e == cudaSuccess) return LORA_OK;
    cudaGetLastError();
    return LORA_ERR_CUDA;
}

PagesDev pages_view(const lora_kv_pages *p)
{
    PagesDev v;
    v.table = p->table;
    v.kv_len = p->kv_len;
    v.refs = p->refs;
    v.P = p->num_pages;
    v.S = p->max_seqs;
    v.W = p->stride;
    v.shift = p->page_shift;
    const size_t P = (size_t)p->num_pages, S = (size_t)p->max_seqs;
    int32_t *at = p->scratch;
    auto take = [&](size_t n) {
        int32_t *const x = at;
        at += n;
        return x;
    };
    v.old_table = take(S * (size_t)p->stride);
    v.kept = take(S);
    v.src = take(S);
    v.base = take(S);
    v.held = take(S);
    v.count = take(P);
    v.claim = take(P);
    v.fresh = take(P);
    v.cap = p->cap();
    v.moves = take(3 * (size_t)p->cap());
    v.moves_n = take(1);
    v.err = p->d_err;
    return v;
}

}  // namespace

namespace lora {

cudaError_t launch_kv_copy(const KvDev &kv, bool int8, const int32_t *src, const int32_t *dst, const int32_t *rows,
                           const int32_t *n_dev, int n, int num_sms, cudaStream_t stream)
{
    const cudaError_t e = ensure_smem_attr((const void *)kv_copy_kernel, 0);
    if (e != cudaSuccess) return e;
    const int row_bytes = kv.D * (int8 ? 1 : 2);
    const int64_t slices = (((int64_t)row_bytes << kv.page_shift) + kSlice - 1) / kSlice;
    const int64_t units = (int64_t)n * 2 * kv.H * slices;
    const int64_t ctas = std::min<int64_t>((units + 7) / 8, 8 * (int64_t)num_sms);
    kv_copy_kernel<<<(unsigned)ctas, 256, 0, stream>>>(kv, row_bytes, CopyList{src, dst, rows, n_dev, n});
    return cudaGetLastError();
}

// The moves of the last update or compaction of `p`.
cudaError_t launch_kv_copy_moves(const KvDev &kv, bool int8, const lora_kv_pages *p, int num_sms, cudaStream_t stream)
{
    const PagesDev v = pages_view(p);
    return launch_kv_copy(kv, int8, v.moves, v.moves + v.cap, v.moves + 2 * (size_t)v.cap, v.moves_n, v.cap, num_sms,
                          stream);
}

lora_status kv_pages_begin(lora_kv_pages *p, cudaStream_t stream, bool *tracked)
{
    return begin_call(p, stream, tracked);
}
lora_status kv_pages_end(lora_kv_pages *p, cudaStream_t stream, bool tracked, cudaError_t e)
{
    return end_call(p, stream, tracked, e);
}

}  // namespace lora

extern "C" {

lora_status lora_kv_pages_create(int num_pages, int page_tokens, int max_seqs, int table_stride, int32_t *page_table,
                                 int32_t *kv_len, int32_t *refs, lora_kv_pages_t *out)
{
    if (!out) return LORA_ERR_ARG;
    *out = nullptr;
    if (num_pages < 1 || num_pages > (1 << 27)) return LORA_ERR_SHAPE;
    if (page_tokens < 16 || page_tokens > 256 || (page_tokens & (page_tokens - 1)) != 0) return LORA_ERR_SHAPE;
    if (max_seqs < 1 || max_seqs > 65536 || table_stride < 1) return LORA_ERR_SHAPE;
    if ((int64_t)max_seqs * table_stride > INT_MAX || (int64_t)table_stride * page_tokens > (1 << 30))
        return LORA_ERR_SHAPE;
    if (!page_table || !kv_len || !refs || !aligned4(page_table) || !aligned4(kv_len) || !aligned4(refs))
        return LORA_ERR_ARG;
    int dev = 0, major = 0, minor = 0;
    CUDA_TRY(cudaGetDevice(&dev));
    CUDA_TRY(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev));
    CUDA_TRY(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev));
    if (major != 10 || minor != 3) return LORA_ERR_UNSUPPORTED;
    lora_kv_pages *p = new (std::nothrow) lora_kv_pages();
    if (!p) return LORA_ERR_OOM;
    p->device = dev;
    p->num_pages = num_pages;
    for (p->page_shift = 4; (1 << p->page_shift) < page_tokens;) ++p->page_shift;
    p->max_seqs = max_seqs;
    p->stride = table_stride;
    p->table = page_table;
    p->kv_len = kv_len;
    p->refs = refs;
    const size_t ints = (size_t)max_seqs * table_stride + 4 * (size_t)max_seqs + 3 * (size_t)num_pages +
                        3 * (size_t)p->cap() + 1;
    if (cudaMalloc((void **)&p->d_err, 3 * sizeof(int)) != cudaSuccess ||
        cudaMalloc((void **)&p->scratch, sizeof(int32_t) * ints) != cudaSuccess ||
        cudaHostAlloc((void **)&p->h_err, sizeof(int), cudaHostAllocDefault) != cudaSuccess) {
        cudaGetLastError();
        lora_kv_pages_destroy(p);
        return LORA_ERR_OOM;
    }
    if (cudaMemset(p->d_err, 0, 3 * sizeof(int)) != cudaSuccess ||
        cudaMemset(pages_view(p).moves_n, 0, sizeof(int)) != cudaSuccess ||
        cudaStreamCreateWithFlags(&p->ctl_stream, cudaStreamNonBlocking) != cudaSuccess ||
        cudaEventCreateWithFlags(&p->ev, cudaEventDisableTiming) != cudaSuccess ||
        ensure_smem_attr((const void *)kv_pages_update_kernel, 0) != cudaSuccess ||
        ensure_smem_attr((const void *)kv_pages_compact_kernel, 0) != cudaSuccess ||
        ensure_smem_attr((const void *)kv_pages_used_kernel, 0) != cudaSuccess ||
        ensure_smem_attr((const void *)kv_pages_read_clear_kernel, 0) != cudaSuccess ||
        cudaDeviceSynchronize() != cudaSuccess) {
        cudaGetLastError();
        lora_kv_pages_destroy(p);
        return LORA_ERR_CUDA;
    }
    *out = p;
    return LORA_OK;
}

lora_status lora_kv_pages_destroy(lora_kv_pages_t p)
{
    if (!p) return LORA_ERR_ARG;
    cudaDeviceSynchronize();
    if (p->ctl_stream) cudaStreamDestroy(p->ctl_stream);
    if (p->ev) cudaEventDestroy(p->ev);
    if (p->scratch) cudaFree(p->scratch);
    if (p->d_err) cudaFree(p->d_err);
    if (p->h_err) cudaFreeHost(p->h_err);
    delete p;
    return LORA_OK;
}

lora_status lora_kv_pages_update(lora_kv_pages_t p, const int32_t *parent, const int32_t *keep, const int32_t *room,
                                 lora_stream_t stream)
{
    if (!p || !aligned4(parent) || !aligned4(keep) || !aligned4(room)) return LORA_ERR_ARG;
    lora_status st = on_device(p->device);
    bool tracked;
    if (st == LORA_OK) st = begin_call(p, stream, &tracked);
    if (st != LORA_OK) return st;
    kv_pages_update_kernel<<<kCtas, kThreads, 0, stream>>>(pages_view(p), parent, keep, room);
    return end_call(p, stream, tracked, cudaGetLastError());
}

lora_status lora_kv_pages_compact(lora_kv_pages_t p, int32_t *table_out, int32_t *refs_out, lora_stream_t stream)
{
    if (!p || (table_out != nullptr) != (refs_out != nullptr) || !aligned4(table_out) || !aligned4(refs_out))
        return LORA_ERR_ARG;
    lora_status st = on_device(p->device);
    bool tracked;
    if (st == LORA_OK) st = begin_call(p, stream, &tracked);
    if (st != LORA_OK) return st;
    kv_pages_compact_kernel<<<kCtas, kThreads, 0, stream>>>(pages_view(p), table_out ? table_out : p->table,
                                                            refs_out ? refs_out : p->refs);
    return end_call(p, stream, tracked, cudaGetLastError());
}

lora_status lora_kv_pages_used(lora_kv_pages_t p, int *used)
{
    if (!p || !used) return LORA_ERR_ARG;
    const lora_status st = on_device(p->device);
    if (st != LORA_OK) return st;
    CUDA_TRY(cudaStreamWaitEvent(p->ctl_stream, p->ev, 0));
    kv_pages_used_kernel<<<1, kThreads, 0, p->ctl_stream>>>(p->refs, p->num_pages, p->d_err + 2);
    if (cudaGetLastError() != cudaSuccess ||
        cudaMemcpyAsync(p->h_err, p->d_err + 2, sizeof(int), cudaMemcpyDeviceToHost, p->ctl_stream) != cudaSuccess ||
        cudaStreamSynchronize(p->ctl_stream) != cudaSuccess)
        return LORA_ERR_CUDA;
    *used = *p->h_err;
    return LORA_OK;
}

lora_status lora_kv_pages_check_errors(lora_kv_pages_t p)
{
    if (!p) return LORA_ERR_ARG;
    CUDA_TRY(cudaStreamWaitEvent(p->ctl_stream, p->ev, 0));
    kv_pages_read_clear_kernel<<<1, 1, 0, p->ctl_stream>>>(p->d_err);
    if (cudaGetLastError() != cudaSuccess ||
        cudaMemcpyAsync(p->h_err, p->d_err + 1, sizeof(int), cudaMemcpyDeviceToHost, p->ctl_stream) != cudaSuccess ||
        cudaStreamSynchronize(p->ctl_stream) != cudaSuccess)
        return LORA_ERR_CUDA;
    if (*p->h_err & kErrRangeBit) return LORA_ERR_RANGE;
    if (*p->h_err & kErrPagesBit) return LORA_ERR_OOM;
    return LORA_OK;
}

}  // extern "C"
