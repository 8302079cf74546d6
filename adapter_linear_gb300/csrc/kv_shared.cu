// kv_shared.cu -- attention of groups of sequences that share a prefix's pages.
//
// The softmax over a row's keys splits into any sets of them: with (O1, lse1) over the prefix and (O2, lse2) over
// the sequence's own tokens,
//   O = (w1 O1 + w2 O2) / (w1 + w2),  lse = log(w1 + w2) + max(lse1, lse2),  w = exp(lse - max(lse1, lse2)).
// So a group's rows attend to its prefix together, as one chunk that sees all of it: the prefix is read once for
// all of them, and many rows fill the tcgen05 kernel's tiles where each sequence alone would read it again for
// a handful of rows. Then every sequence attends to its own tokens, and the kernel that does this joins the two
// where it writes its result. O1 is kept in fp32.
//
// What bounds it: the prefix's kernel takes 4500 (bf16) or 7200 (8-bit) cycles a key tile of one or two tiles of 128
// rows, the softmax's as in kv_prefill_kernel.cuh with both parts of every weight, and 9 us of each call go by before its first
// scores: the plan 2, the share's first segment, tokens and Q 4, cold code of each role the rest. The own
// tokens' kernel starts while it ends and waits for it only before its epilogue, which reads the prefix's pieces (19
// of an item where one group's heads are all there is). Measured on the GPU, 32 query heads on 8 kv heads of 128
// values: 8 sequences over one prefix of 1000, 8-bit, 19 us; 64 over 8192 with up to 500 of their own, 8-bit,
// 58 us (prefix's kernel 34, own tokens' 30, overlapping); 16 groups of 16 over 500 to 4000 with up to 400 of their
// own, bf16, 115 us (365 MB: 3.2 TB/s); 3 groups of 16 over 9000 to 16000 with 3 to 6 new tokens, 8-bit, 165 us
// (0.29 PFLOP/s); 8 prompts of 300 behind 2000, 8-bit 194 us, bf16 167. Every sequence by itself
// (lora_kv_attention, whose reads of common pages come from L2), 30 tokens of its own, 8-bit, and shared: 8 sequences
// over 1000, 4000, 16000 tokens 14, 22, 49 us and 19, 24, 38; 64 sequences 33, 92, 316 and 30, 36, 55; the 8 prompts 155 and
// 194. So it takes many short chunks over a long prefix to pay; long chunks did not in any case measured.
#include <algorithm>
#include <climits>

#include "kv_prefill_kernel.cuh"

namespace lora {
namespace {

// x / y, not negative
__device__ __forceinline__ int64_t plan_div(int64_t x, int64_t y)
{
    return (x | y) >> 32 == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}

// A group's prefix: what is asked for, but no further than the new tokens of any of its sequences, in
// whole pages. A group of one sequence, or one with a sequence whose start or length is bad, has none.
//
// Then the kernels' work is counted here, once, not by every CTA of theirs, whose code and loads are cold (7 of the
// 20 us of 8 sequences over 1000 tokens, 9 us of 256 sequences' own tokens). Two CTAs at the same time: the first
// writes the groups and shares out the prefixes' units (begins), the second writes lo and numbers the items of
// the own tokens.
constexpr int kPlanGroups = 1024;  // whose sums shared memory holds
__global__ void __launch_bounds__(1024) kv_share_plan_kernel(KvDev kv, KvBatchDev b, const int32_t *seq_start,
                                                             const int32_t *prefix_len, int n_groups, int G, int own_rows,
                                                             int max_rows, int shares, KvShareDev share)
{
    __shared__ int64_t sm_at[kPlanGroups], sm_sums[32];
    __shared__ int sm_most[32];
    __shared__ unsigned long long sm_units;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const bool prefixes = blockIdx.x == 0;
    int64_t *const at = n_groups <= kPlanGroups ? sm_at : share.group_at;
    pdl_launch_dependents();
    if (!prefixes)
        for (int i = threadIdx.x; i < b.n_seqs; i += blockDim.x) share.lo[i] = 0;
    bool ordered = true;
    for (int g = threadIdx.x; g < n_groups; g += blockDim.x)
        ordered = ordered && seq_start[g] >= 0 && seq_start[g] <= seq_start[g + 1] && seq_start[g + 1] <= b.n_seqs;
    ordered = __syncthreads_and(ordered);
    if (!ordered && threadIdx.x == 0) kv_flag_range(kv.err);
    auto item_units = [&](int e) { return kHeadUnits + max(1, (e + kKeys - 1) / kKeys); };  // e tokens, a head, a tile
    for (int g = threadIdx.x >> 5; g < n_groups; g += blockDim.x >> 5) {
        const int s0 = ordered ? seq_start[g] : 0, s1 = ordered ? seq_start[g + 1] : 0;
        int before = INT32_MAX, first = INT32_MAX, rows = 0, with_rows = 0;
        bool ok = true;
        for (int i = s0 + lane; i < s1; i += 32) {
            const KvSeq s = kv_seq(b, kv.page_shift, i, kv.err);
            ok = ok && s.n == b.start[i + 1] - b.start[i];
            if (s.n > 0) {
                before = min(before, s.L - s.n);
                first = min(first, i);
                rows += s.n;
                ++with_rows;
            }
        }
        before = __reduce_min_sync(0xffffffffu, before);
        first = __reduce_min_sync(0xffffffffu, first);
        rows = __reduce_add_sync(0xffffffffu, rows);
        with_rows = __reduce_add_sync(0xffffffffu, with_rows);
        ok = __all_sync(0xffffffffu, ok) && with_rows > 1;
        int e = ok ? max(0, min(before, prefix_len[g])) : 0;
        e = e >> kv.page_shift << kv.page_shift;
        if (prefixes) {
            if (lane == 0) {
                share.groups[g] = e > 0 ? make_int4(first, e, b.start[first], rows) : make_int4(0, 0, 0, 0);
                const int64_t tiles = ((int64_t)rows * G + kBlockRows - 1) / kBlockRows;
                if (shares > 0) at[g] = e > 0 ? tiles * kv.H * item_units(e) : 0;
            }
        } else if (e > 0) {
            for (int i = s0 + lane; i < s1; i += 32) share.lo[i] = e;
        }
    }
    __syncthreads();

    // total plus `mine` of the threads before this one; then all of the block's are in total, too
    auto before_me = [&](int64_t mine, int64_t &total) {
        int64_t x = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += o;
        }
        __syncthreads();
        if (lane == 31) sm_sums[warp] = x;
        __syncthreads();
        x += total - mine;
        for (int y = 0; y < warps; ++y) {
            total += sm_sums[y];
            if (y < warp) x += sm_sums[y];
        }
        return x;
    };
    if (prefixes) {
        if (shares == 0) return;
        int64_t total = 0;  // at[g]: from its units to those of the groups before it
        for (int g0 = 0; g0 < n_groups; g0 += blockDim.x) {
            const int g = g0 + threadIdx.x;
            const int64_t x = before_me(g < n_groups ? at[g] : 0, total);
            if (g < n_groups) at[g] = x;
        }
        __syncthreads();
        const int64_t n = min((int64_t)shares, total), q = n > 0 ? plan_div(total, n) : 0, r = total - q * n;
        for (int c = threadIdx.x; c < shares; c += blockDim.x) {
            KvShareBegin begin{};
            if (c < n) {
                begin.u = c * q + c * (int)r / (int)n;  // c total / n
                begin.u_end = (c + 1) * q + (c + 1) * (int)r / (int)n;
                int g = 0;
                for (int hi = n_groups - 1; g < hi;) {  // the last whose units begin at u or before
                    const int mid = (g + hi + 1) >> 1;
                    if (at[mid] <= begin.u)
                        g = mid;
                    else
                        hi = mid - 1;
                }
                begin.group = share.groups[g];
                begin.seq = g;
                const int64_t tile = (int64_t)item_units(begin.group.y) * kv.H;
                begin.tile = (int)plan_div(begin.u - at[g], tile);
                begin.tile0 = at[g] + begin.tile * tile;
                begin.total = total;
                begin.shares = (int)n;
            }
            share.begins[c] = begin;
        }
        return;
    }

    // the items of what is behind, a sequence a thread (starts that decrease may make more than 2^31: then they have
    // no numbers)
    if (threadIdx.x == 0) sm_units = 0;
    int64_t before = 0;
    int most = 0;
    unsigned long long units = 0;
    for (int i0 = 0; i0 < b.n_seqs; i0 += blockDim.x) {
        const int i = i0 + threadIdx.x;
        int tiles = 0;
        if (i < b.n_seqs) {
            const KvSeq s = kv_seq(b, kv.page_shift, i, kv.err);
            const int64_t rows = (int64_t)s.n * G;
            if (rows <= max_rows) tiles = (int)((rows + own_rows - 1) / own_rows);
            const int lo = share.lo[i];
            for (int t = 0; t < tiles; ++t) {
                const int last = (int)min((int64_t)(t + 1) * own_rows, rows) - 1;
                const int hi = max(0, s.L - s.n + last / G + 1);
                const int n = max(1, (hi - min(lo, hi) + kDecodeUnit - 1) / kDecodeUnit);
                units += kDecodeHeadUnits + n;
                most = max(most, n);
            }
        }
        const int64_t x = before_me((int64_t)tiles * kv.H, before);  // (its barriers are sm_units', too)
        if (i < b.n_seqs) share.own_first[i] = (int)x;
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) sm_most[warp] = most;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) units += __shfl_xor_sync(0xffffffffu, units, d);
    if (lane == 0) atomicAdd(&sm_units, units);
    __syncthreads();
    if (warp == 0) {
        most = __reduce_max_sync(0xffffffffu, lane < warps ? sm_most[lane] : 0);
        if (lane == 0) {
            units = sm_units * kv.H;
            share.own_first[b.n_seqs] = (int)before;
            *share.own_sums = make_int4(before <= INT_MAX ? (int)before : -1, most, (int)(uint32_t)units, (int)(units >> 32));
        }
    }
}

// The pieces of the items that several CTAs of the prefix's kernel share: with few groups an item is cut into
// dozens. A unit of work is kJoinRows rows of one item; the blocks, all resident, take turns.
constexpr int kJoinRows = 8, kJoinThreads = 256, kMaxPieces = 256;
static_assert(kMaxPieces == kJoinThreads, "an item a thread");

template <int D, bool kInt8>
__global__ void __launch_bounds__(kJoinThreads) kv_share_join_kernel(KvAttn a, KvShareDev share, int grid)
{
    __shared__ float weight[kJoinRows][kMaxPieces];
    __shared__ int units_to[kMaxPieces], sums[kJoinThreads / 32];  // units of the items up to each
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    pdl_wait_prior();
    int n = 0;
    if (threadIdx.x < grid && share.items[threadIdx.x].last >= 0)
        n = (share.items[threadIdx.x].rows + kJoinRows - 1) / kJoinRows;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, n, d);
        if (lane >= d) n += o;
    }
    if (lane == 31) sums[warp] = n;
    __syncthreads();
    for (int x = 0; x < warp; ++x) n += sums[x];
    units_to[threadIdx.x] = n;
    __syncthreads();
    const float2 *const ml = reinterpret_cast<const float2 *>(share.part + share.ml_at);
    for (int u = blockIdx.x; u < units_to[kMaxPieces - 1]; u += gridDim.x) {
        int c0 = 0;  // the first item whose units go beyond u
#pragma unroll
        for (int step = kMaxPieces / 2; step > 0; step >>= 1)
            if (units_to[c0 + step - 1] <= u) c0 += step;
        const KvShareItem item = share.items[c0];
        const int r0 = (u - (c0 > 0 ? units_to[c0 - 1] : 0)) * kJoinRows, rows = min(kJoinRows, item.rows - r0);
        const int pieces = item.last - c0 + 1;
        auto slot = [&](int x) { return kv_slot(c0, x); };
        auto out_row = [&](int r) {
            const int row = item.first_row + r0 + r;
            return (int64_t)(item.row0 + row / a.G) * a.Hq + item.head * a.G + row % a.G;
        };
        // a row's maximum, sum and weights by one warp
        for (int r = warp; r < rows; r += kJoinThreads / 32) {
            float M = -INFINITY, sum = 0.0f;
            for (int x = lane; x < pieces; x += 32) {
                const float m = ml[slot(x) * kBlockRows + r0 + r].x;
                weight[r][x] = m;
                M = fmaxf(M, m);
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
            const float ref = M == -INFINITY ? 0.0f : M;
            for (int x = lane; x < pieces; x += 32) {
                const float w = fast_exp2(weight[r][x] - ref);
                sum += w * ml[slot(x) * kBlockRows + r0 + r].y;
                weight[r][x] = w;
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            for (int x = lane; x < pieces; x += 32) weight[r][x] *= inv;
            if (lane == 0) share.lse2[out_row(r)] = sum == 0.0f ? -INFINITY : M + log2f(sum);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < rows * (D / 4); i += kJoinThreads) {
            const int r = i / (D / 4), d = (i % (D / 4)) * 4;
            const float *const src = share.part + (int64_t)(r0 + r) * D + d;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int x = 0; x < pieces; ++x) {
                const float4 v = *reinterpret_cast<const float4 *>(src + (int64_t)slot(x) * kBlockRows * D);
                const float w = weight[r][x];
                acc.x = add_piece<kInt8>(w, v.x, acc.x);
                acc.y = add_piece<kInt8>(w, v.y, acc.y);
                acc.z = add_piece<kInt8>(w, v.z, acc.z);
                acc.w = add_piece<kInt8>(w, v.w, acc.w);
            }
            *reinterpret_cast<float4 *>(share.O + out_row(r) * D + d) = acc;
        }
        __syncthreads();  // the weights are free again
    }
}

}  // namespace

size_t kv_share_part_floats(int D, int num_sms)
{
    return (size_t)2 * kv_prefill_grid(num_sms) * kBlockRows * (D + 2);
}

cudaError_t launch_kv_share_join(const KvDev &kv, bool int8, const KvAttn &a, const KvShareDev &share, int num_sms,
                                 cudaStream_t stream)
{
    auto fn = kv.D == 128 ? (int8 ? kv_share_join_kernel<128, true> : kv_share_join_kernel<128, false>)
                          : (int8 ? kv_share_join_kernel<64, true> : kv_share_join_kernel<64, false>);
    const int grid = kv_prefill_grid(num_sms);
    if (grid > kMaxPieces) return cudaErrorInvalidConfiguration;
    const cudaError_t e = ensure_smem_attr((const void *)fn, 0);
    if (e != cudaSuccess) return e;
    return kv_launch(true, fn, dim3(2 * num_sms), kJoinThreads, 0, stream, a, share, grid);
}

cudaError_t launch_kv_share_plan(const KvDev &kv, const KvBatchDev &b, const int32_t *seq_start,
                                 const int32_t *prefix_len, int n_groups, int G, int own_rows, int max_rows, int shares,
                                 const KvShareDev &share, cudaStream_t stream)
{
    const cudaError_t e = ensure_smem_attr((const void *)kv_share_plan_kernel, 0);
    if (e != cudaSuccess) return e;
    // a sequence a thread, a group a warp, a share a thread
    const int64_t most = std::max<int64_t>({1, b.n_seqs, 32 * (int64_t)n_groups, shares});
    const int threads = (int)std::min<int64_t>(1024, (most + 31) / 32 * 32);
    kv_share_plan_kernel<<<2, threads, 0, stream>>>(kv, b, seq_start, prefix_len, n_groups, G, own_rows, max_rows, shares,
                                                    share);
    return cudaGetLastError();
}

cudaError_t launch_kv_prefill_shared(KvMode mode, const KvDev &kv, bool int8, const KvBatchDev &b, const KvAttn &a,
                                     const KvShareDev &share, int min_rows, float *part, int *count, int num_sms,
                                     cudaStream_t stream)
{
    return mode == kPrefix
               ? launch_kv_prefill_mode<kPrefix>(kv, int8, b, a, share, min_rows, part, count, num_sms, stream)
               : launch_kv_prefill_mode<kOwn>(kv, int8, b, a, share, min_rows, part, count, num_sms, stream);
}

}  // namespace lora
