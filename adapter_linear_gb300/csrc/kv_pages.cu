// kv_pages.cu -- page tables of sequences that fork, grow, shrink and go: the update and the compaction of
// the tables, and the copies of pages that they ask for.
//
// Slot i becomes the first n_i = min(keep_i, length of its parent) tokens of slot parent_i, with pages for room_i
// more. Whole pages are shared: refs[x] is the number of entries that name page x, and a page is free when that is 0.
// A page that n_i ends inside stays with one slot (the lowest that ends there, if no other has all of it),
// the others get a copy; new pages are the lowest free ones in order of slot and entry, so equal calls
// give equal tables. Measured on the GPU (tables of 16-token pages): 64 slots of up to 4000 tokens that keep a number of
// theirs and get 5 more 12.5 us; 4 prompts of up to 6000 tokens forked into 256 slots, and the copies, 18.5 us; room alone,
// one token more for each of 64 slots of 2000 tokens 7.6 us, 256 of 1000 10.2, 1024 of 400 34, and the copies' kernel,
// with nothing to do, 1.2 us more; the same trimmed to what they held before and extended 13, 18 and 74; 300 slots over
// 24000 pages, 55 % used, compacted, and 5900 pages of 64 KB copied, 135 us (5.8 TB/s).
#include <algorithm>
#include <climits>
#include <new>

#include <cooperative_groups.h>

#include "device_common.cuh"
#include "kv_pages_state.h"
#include "kv_state.h"
#include "launch_stream.h"

namespace cg = cooperative_groups;
using namespace lora;

namespace {

// The tables are some hundred kilobytes, in L2, and the work on them a handful of steps that each need all of
// the one before (who names a page, which pages are free, who gets them), so the latency of L2 and of the steps'
// ends bounds it (a hop to L2 0.5 us, a cluster barrier 0.6): one cluster of kCtas CTAs does all
// steps, a cluster barrier between them, and what all of them need of the slots is in every CTA's shared memory.
constexpr int kCtas = 8, kThreads = 1024;
constexpr int kUnit = 128;       // table entries a warp takes at a time, four a lane
constexpr int kTile = 4 * kThreads;  // pages a CTA scans at a time, four a thread
constexpr int kSlotsHere = 1024; // slots that fit the shared memory; of more the numbers lie in scratch

struct PagesDev {
    int32_t *table, *kv_len, *refs;
    int P, S, W, shift;        // pages, slots, entries a slot, log2 of a page's tokens
    int4 *slots;               // [S], where they do not fit the shared memory
    int32_t *stash;            // [S][W] entries that slots take over from others
    int32_t *last;             // [S] the page that a slot's kept tokens end inside
    int32_t *base;             // [S] the first new page of a slot among all, 2 x + (keeps the page it ends in)
    int32_t *count, *claim;    // [P] slots that have all of a page; the first that ends inside (kNone: none);
                               // 0 and kNone between calls
    int32_t *list;             // [P] free pages, in order, of each CTA's part of the pages
    int32_t *place, *named;    // compaction: [P] a page's place in the list, [P / 2 + 1] refs of those in the list
    int32_t *moves;            // [3][cap]: page, page, rows
    int32_t *moves_n;          // [1]
    int cap;
    int *err;
};

constexpr int kNone = 0x7F7F7F7F;  // (bytes that are all the same)

// A slot: tokens kept, of which slot (-1: none), tokens afterwards, entries used before.
__device__ __forceinline__ int kept_of(const int4 &s) { return s.x; }
__device__ __forceinline__ int from_of(const int4 &s) { return s.y; }
__device__ __forceinline__ int total_of(const int4 &s) { return s.z; }
__device__ __forceinline__ int held_of(const int4 &s) { return s.w; }

// What a CTA tells the others: they read it behind a cluster barrier.
struct Told {
    int bad[2];        // error bits of the first two steps
    int found;         // pages it found
    int need, copies;  // the last CTA: new pages and copies in all
};

__device__ __forceinline__ int entries(int tokens, int shift) { return (tokens + (1 << shift) - 1) >> shift; }

// Sum over a block of v, in every thread. sm: 33 values.
__device__ __forceinline__ int block_sum(int v, int *sm)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if (lane == 0) sm[warp] = v;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, sm[lane]);
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
    T x = sm[lane], y = x;  // every warp: the warps' sums
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T o = __shfl_up_sync(0xffffffffu, y, d);
        if (lane >= d) y += o;
    }
    *all = __shfl_sync(0xffffffffu, y, 31);
    return __shfl_sync(0xffffffffu, y - x, warp) + s - v;
}

// The cluster's warps share out pieces of kUnit entries of all slots: piece(slot, its first entry).
template <class Piece>
__device__ __forceinline__ void each_piece(const PagesDev &p, int cta, Piece piece)
{
    const uint32_t per = (p.W + kUnit - 1) / kUnit;  // S W is below 2^31
#pragma unroll 1
    for (uint32_t u = (threadIdx.x >> 5) * kCtas + cta; u < p.S * per; u += kCtas * (kThreads / 32))
        piece((int)(u / per), (int)(u % per) * kUnit);
}

// For the entries begin(slot) .. end(slot) - 1 of all slots: use(slot, entry, *at(slot, entry)). A lane's four
// loads are made whether they are needed or not (of some entry), behind no branch: all at once.
template <class Begin, class End, class At, class Use>
__device__ __forceinline__ void each_entry(const PagesDev &p, int cta, Begin begin, End end, At at, Use use)
{
    const int lane = threadIdx.x & 31;
    each_piece(p, cta, [&](int s, int first) {
        const int from = begin(s), n = end(s);
        if (first >= n || first + kUnit <= from) return;
        int x[kUnit / 32];
#pragma unroll
        for (int k = 0; k < kUnit / 32; ++k) x[k] = __ldcg(at(s, min(max(first + lane + k * 32, from), n - 1)));
#pragma unroll
        for (int k = 0; k < kUnit / 32; ++k) {
            const int j = first + lane + k * 32;
            if (j >= from && j < n) use(s, j, x[k]);
        }
    });
}

// A cluster barrier in two halves, which orders no memory beyond the CTA's own: the block's barrier ahead of it has
// every thread's reads of another CTA's shared memory done, and what the threads wrote into their own there for each other.
// The start of a kernel (all CTAs have started before the first reaches into another), and its end (arrive when
// this CTA has read, wait before it goes).
__device__ __forceinline__ void cluster_arrive()
{
    __syncthreads();
    asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait;" ::: "memory"); }

// value(told) of every CTA of the cluster into out[kCtas]; behind a cluster barrier, called by all threads.
template <class Value>
__device__ __forceinline__ void gather(cg::cluster_group &cluster, Told *mine, int *out, Value value)
{
    __syncthreads();
    if (threadIdx.x < kCtas) out[threadIdx.x] = value(*cluster.map_shared_rank(mine, threadIdx.x));
    __syncthreads();
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1)
    kv_pages_update_kernel(PagesDev p, const int32_t *parent, const int32_t *keep, const int32_t *room)
{
    pdl_launch_dependents();  // (the copies' kernel)
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ Told mine;
    __shared__ int4 slots_here[kSlotsHere];
    __shared__ int kids[kSlotsHere], least[kSlotsHere];  // slots that go on from a slot, the fewest whole pages of them
    __shared__ int last_here[kSlotsHere], base_here[kSlotsHere];  // the last CTA's: PagesDev::last, base
    __shared__ int64_t sm[33];
    __shared__ int others[kCtas];
    int *const sm32 = reinterpret_cast<int *>(sm);
    const int cta = blockIdx.x, tid = cta * kThreads + threadIdx.x, mask = (1 << p.shift) - 1;
    const bool here = p.S <= kSlotsHere;
    int4 *const slots = here ? slots_here : p.slots;
    const bool counted = !parent && !keep;  // every slot keeps what it has: refs are the counts
    if (threadIdx.x < 2) mine.bad[threadIdx.x] = 0;
    for (int i = threadIdx.x; i < kSlotsHere; i += kThreads) {
        kids[i] = 0;
        least[i] = INT_MAX;
    }
    cluster_arrive();  // all have started, before the first reaches into another's shared memory
    cluster_wait();

    // ---- 1: what is asked for. Each slot is read once, by one thread, which tells all CTAs where the slots fit
    // (so that they agree, whatever else may write what they read).
    const int capacity = (int)min((int64_t)p.W << p.shift, (int64_t)INT_MAX);
    for (int i = threadIdx.x * kCtas + cta; i < p.S; i += kCtas * kThreads) {
        const int from = parent ? parent[i] : i, now = p.kv_len[i];
        const int extra = room ? room[i] : 0, most = keep ? max(0, keep[i]) : INT_MAX;
        bool wrong = from < -1 || from >= p.S || extra < 0 || now < 0 || now > capacity;
        int n = 0;
        if (!wrong && from >= 0) {
            n = from == i ? now : p.kv_len[from];
            wrong = n < 0 || n > capacity;
            n = min(n, most);
        }
        wrong = wrong || (int64_t)n + extra > capacity;
        if (wrong) mine.bad[0] = kErrRangeBit;
        const int4 slot = wrong ? make_int4(0, -1, 0, 0) : make_int4(n, from, n + extra, entries(now, p.shift));
        if (here)
#pragma unroll
            for (int c = 0; c < kCtas; ++c) cluster.map_shared_rank(slots_here, c)[i] = slot;
        else
            slots[i] = slot;
    }
    cluster.sync();
    int bad = 0;
    gather(cluster, &mine, others, [](const Told &t) { return t.bad[0]; });
    for (int c = 0; c < kCtas; ++c) bad |= others[c];
    if (bad) {
        cluster_arrive();
        if (tid == 0) {
            atomicOr(p.err, bad);
            *p.moves_n = 0;
        }
        cluster_wait();
        return;
    }
    if (here && !counted) {
        for (int i = threadIdx.x; i < p.S; i += kThreads)
            if (from_of(slots_here[i]) >= 0) {
                atomicAdd(kids + from_of(slots_here[i]), 1);
                atomicMin(least + from_of(slots_here[i]), kept_of(slots_here[i]) >> p.shift);
            }
        __syncthreads();
    }
    int *const last = here ? cluster.map_shared_rank(last_here, kCtas - 1) : p.last;
    int *const base = here ? cluster.map_shared_rank(base_here, kCtas - 1) : p.base;

    // ---- 2: who has a page, who ends inside one. The pages that all slots that go on from one have are
    // counted once for all of them: an SM's atomics go 1.6 cycles a lane.
    if (counted) {  // known: the entries are only looked at (the result is asked for behind the next barrier)
        each_entry(p, cta, [&](int) { return 0; }, [&](int s) { return held_of(slots[s]); },
                   [&](int s, int j) { return p.table + (int64_t)s * p.W + j; },
                   [&](int s, int j, int x) {
                       // (a page that a slot ends inside is its own, unless the caller's tables have it otherwise)
                       if (x < 0 || x >= p.P || (j == kept_of(slots[s]) >> p.shift && p.refs[x] != 1))
                           mine.bad[1] = kErrRangeBit;
                   });
    } else {
        each_piece(p, cta, [&](int s, int first) {
            const int4 me = slots[s];
            const int from = from_of(me), n = entries(kept_of(me), p.shift), whole = kept_of(me) >> p.shift;
            const int to = here && kids[s] > 0 ? least[s] : 0;     // entries of this row that all its kids have
            const int since = here && from >= 0 ? least[from] : 0; // entries of the other row that are counted here
            if (first >= max(n, to)) return;
            const int32_t *const mine_row = p.table + (int64_t)s * p.W;
            const int32_t *const row = from >= 0 ? p.table + (int64_t)from * p.W : mine_row;
            int x[kUnit / 32], y[kUnit / 32];
#pragma unroll
            for (int k = 0; k < kUnit / 32; ++k) {
                const int j = first + (threadIdx.x & 31) + k * 32;
                x[k] = __ldcg(mine_row + min(j, p.W - 1));
                y[k] = __ldcg(row + min(j, p.W - 1));
            }
#pragma unroll
            for (int k = 0; k < kUnit / 32; ++k) {
                const int j = first + (threadIdx.x & 31) + k * 32;
                if (j < to) {
                    if (x[k] >= 0 && x[k] < p.P)
                        atomicAdd(p.count + x[k], kids[s]);
                    else
                        mine.bad[1] = kErrRangeBit;
                }
                if (j >= n) continue;
                const bool ok = y[k] >= 0 && y[k] < p.P;
                if (!ok) mine.bad[1] = kErrRangeBit;
                if (from != s) p.stash[(int64_t)s * p.W + j] = y[k];
                if (j == whole) {  // ends inside
                    if (ok) atomicMin(p.claim + y[k], s + (from == s ? 0 : p.S));
                    last[s] = ok ? y[k] : 0;
                } else if (j >= since && ok) {
                    atomicAdd(p.count + y[k], 1);
                }
            }
        });
        cluster.sync();
    }

    // ---- 3: the free pages of this CTA's part (a page that someone ends inside and nobody has stays with the
    // first who asked), in order; the last CTA, which has no part: the new pages and copies of every slot
    const int part = ((p.P + kCtas - 2) / (kCtas - 1) + 3) & ~3;
    const int x0 = min(p.P, cta * part), x1 = cta == kCtas - 1 ? x0 : min(p.P, x0 + part);
    auto pages4 = [&](int x, int (&c)[4], int (&cl)[4]) {  // counts and claims of pages x .. x + 3 below x1
        const int32_t *const from = counted ? p.refs : p.count;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int y = min(x + e, x1 - 1);
            c[e] = __ldcg(from + y);
            cl[e] = __ldcg((counted ? p.refs : p.claim) + y);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (x + e >= x1) c[e] = 1;
            if (counted) cl[e] = kNone;
        }
    };
    int found = 0;
    for (int y0 = x0; y0 < x1; y0 += kTile) {
        const int x = y0 + 4 * threadIdx.x;
        int c[4], cl[4], v = 0, sum;
        pages4(x, c, cl);
#pragma unroll
        for (int e = 0; e < 4; ++e) v += c[e] == 0 && cl[e] == kNone;
        int at = found + block_scan(v, sm32, &sum);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c[e] == 0 && cl[e] == kNone) {
                p.list[x0 + at] = x + e;
                if (!counted) p.count[x + e] = -1 - at;  // free: its place in the list
                ++at;
            }
        found += sum;
    }
    if (threadIdx.x == 0) mine.found = found;
    if (cta == kCtas - 1) {
        int64_t before = 0;  // new pages, and in the upper half copies
        for (int s0 = 0; s0 < p.S; s0 += kThreads) {
            const int s = s0 + threadIdx.x;
            int64_t v = 0, sum;
            int stays = 0, n = 0, old = -1;
            if (s < p.S) {
                n = kept_of(slots[s]);
                if (n & mask) {
                    if (counted) {
                        stays = 1;
                    } else {
                        old = last[s];
                        const int count = __ldcg(p.count + old);  // (a page that someone asked for is not in a list)
                        stays = __ldcg(p.claim + old) == s + (from_of(slots[s]) == s ? 0 : p.S) && count == 0;
                    }
                    if (!stays) v = 1ll << 32;
                }
                v += entries(total_of(slots[s]), p.shift) - (n >> p.shift) - stays;
            }
            const int64_t at = before + block_scan(v, sm, &sum);
            if (s < p.S) {
                base[s] = 2 * (int)(uint32_t)at + stays;
                if (v >> 32) {
                    const int k = (int)(at >> 32);
                    p.moves[k] = old;
                    p.moves[p.cap + k] = (int)(uint32_t)at;  // (which new page: its number below)
                    p.moves[2 * p.cap + k] = n & mask;
                }
            }
            before += sum;
        }
        if (threadIdx.x == 0) {
            mine.need = (int)min((int64_t)(uint32_t)before, (int64_t)INT_MAX);
            mine.copies = (int)(before >> 32);
        }
    }
    cluster.sync();

    // ---- 4: the new state
    gather(cluster, &mine, others, [](const Told &t) { return t.found | (t.bad[1] ? INT_MIN : 0); });
    const Told *const last_told = cluster.map_shared_rank(&mine, kCtas - 1);
    const int need = last_told->need, copies = last_told->copies;
    int there = 0, before = 0;
    for (int c = 0; c < kCtas; ++c) {
        const int f = others[c] & INT_MAX;
        bad |= others[c] < 0 ? kErrRangeBit : 0;
        if (c < cta) before += f;
        there += f;
    }
    if (!bad && need > there) bad = kErrPagesBit;
    if (!counted)
        for (int y0 = x0; y0 < x1; y0 += kTile) {
            const int x = y0 + 4 * threadIdx.x;
            int c[4], cl[4];
            pages4(x, c, cl);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (x + e < x1) {
                    if (!bad)
                        p.refs[x + e] = c[e] < 0 ? before - 1 - c[e] < need : c[e] == 0 && cl[e] != kNone ? 1 : c[e];
                    p.count[x + e] = 0;  // for the next call
                    p.claim[x + e] = kNone;
                }
        }
    if (bad) {
        cluster_arrive();
        if (tid == 0) {
            atomicOr(p.err, bad);
            *p.moves_n = 0;
        }
        cluster_wait();
        return;
    }
    auto new_page = [&](int i) {  // where the i-th of all free pages is listed
        int c = 0;
#pragma unroll
        for (int y = 0; y < kCtas - 2; ++y)
            if (c == y && i >= others[y]) {
                i -= others[y];
                ++c;
            }
        return p.list + c * part + i;
    };
    each_entry(p, cta,
               [&](int s) { return from_of(slots[s]) == s ? kept_of(slots[s]) >> p.shift : 0; },
               [&](int s) { return max(held_of(slots[s]), entries(total_of(slots[s]), p.shift)); },
               [&](int s, int j) -> const int32_t * {
                   const int4 me = slots[s];
                   const int b = base[s];
                   const int old = (kept_of(me) >> p.shift) + (b & 1);  // entries that stay
                   const int32_t *const there = (from_of(me) == s ? p.table : p.stash) + (int64_t)s * p.W + j;
                   return j < old || j >= entries(total_of(me), p.shift) ? there : new_page((b >> 1) + j - old);
               },
               [&](int s, int j, int x) {
                   const int4 me = slots[s];
                   const bool used = j < entries(total_of(me), p.shift);
                   p.table[(int64_t)s * p.W + j] = used ? x : -1;
                   if (counted && used && j >= entries(kept_of(me), p.shift)) p.refs[x] = 1;
               });
    cluster_arrive();  // nothing more of another CTA's shared memory
    for (int s = tid; s < p.S; s += kCtas * kThreads) p.kv_len[s] = total_of(slots[s]);
    for (int k = tid; k < copies; k += kCtas * kThreads) p.moves[p.cap + k] = __ldcg(new_page(__ldcg(p.moves + p.cap + k)));
    if (tid == 0) *p.moves_n = copies;
    cluster_wait();
}

// n pages are used. The used page x >= n with d used pages above it moves to the (moved - 1 - d)-th free page below n.
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1)
    kv_pages_compact_kernel(PagesDev p, int32_t *table_out, int32_t *refs_out)
{
    pdl_launch_dependents();  // (the copies' kernel)
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ Told mine;
    __shared__ int sm[33], others[kCtas];
    const int cta = blockIdx.x, tid = cta * kThreads + threadIdx.x;
    const int part = ((p.P + kCtas - 1) / kCtas + 3) & ~3;
    const int x0 = min(p.P, cta * part), x1 = min(p.P, x0 + part);
    auto refs4 = [&](int x, int (&r)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = __ldcg(p.refs + min(x + e, x1 - 1));
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (x + e >= x1) r[e] = 0;
    };

    int used = 0;
    for (int y0 = x0; y0 < x1; y0 += kTile) {
        int r[4];
        refs4(y0 + 4 * threadIdx.x, r);
#pragma unroll
        for (int e = 0; e < 4; ++e) used += r[e] > 0;
    }
    used = block_sum(used, sm);
    if (threadIdx.x == 0) mine.found = used;
    cluster.sync();
    gather(cluster, &mine, others, [](const Told &t) { return t.found; });
    int n = 0, before = 0;
    for (int c = 0; c < kCtas; ++c) {
        if (c < cta) before += others[c];
        n += others[c];
    }
    // the used pages from n on, from the last; the free ones below n, from the first
    int holes = 0;
    for (int y0 = x0; y0 < x1; y0 += kTile) {
        const int x = y0 + 4 * threadIdx.x;
        int r[4], v = 0, sum;
        refs4(x, r);
#pragma unroll
        for (int e = 0; e < 4; ++e) v += r[e] > 0;
        int at = before + block_scan(v, sm, &sum);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int y = x + e;
            if (y < x1 && r[e] > 0) {
                const int d = n - 1 - at;
                if (y >= n && d >= 0 && d < p.P / 2 + 1) {  // (as it is, unless refs change meanwhile)
                    p.list[d] = y;
                    p.place[y] = d;
                    p.named[d] = r[e];
                }
                ++at;
            } else if (y < x1 && y < n && y - at < p.cap) {
                p.moves[p.cap + y - at] = y;
                ++holes;
            }
        }
        before += sum;
    }
    holes = block_sum(holes, sm);
    if (threadIdx.x == 0) mine.need = holes;
    cluster.sync();
    gather(cluster, &mine, others, [](const Told &t) { return t.need; });
    cluster_arrive();  // nothing more of another CTA's shared memory
    int moved = 0;
    for (int c = 0; c < kCtas; ++c) moved += others[c];
    moved = min(moved, p.P / 2 + 1);

    for (int k = tid; k < moved; k += kCtas * kThreads) {
        const int d = moved - 1 - k;
        p.moves[k] = __ldcg(p.list + d);
        p.moves[2 * p.cap + k] = 1 << p.shift;
        refs_out[__ldcg(p.moves + p.cap + k)] = __ldcg(p.named + d);
    }
    for (int x = tid; x < p.P; x += kCtas * kThreads) {
        if (x >= n)
            refs_out[x] = 0;
        else if (refs_out != p.refs) {
            const int r = p.refs[x];
            if (r > 0) refs_out[x] = r;
        }
    }
    const int capacity = (int)min((int64_t)p.W << p.shift, (int64_t)INT_MAX);
    const bool copy = table_out != p.table;
    each_entry(p, cta, [&](int) { return 0; },
               [&](int s) { return copy ? p.W : max(0, entries(min(p.kv_len[s], capacity), p.shift)); },
               [&](int s, int j) { return p.table + (int64_t)s * p.W + j; },
               [&](int s, int j, int x) {
                   const int64_t e = (int64_t)s * p.W + j;
                   const bool inside = !copy || j < entries(max(0, min(p.kv_len[s], capacity)), p.shift);
                   int to = x;
                   if (inside && (x < 0 || x >= p.P)) {
                       atomicOr(p.err, kErrRangeBit);
                   } else if (inside && x >= n) {
                       const int d = __ldcg(p.place + x);
                       if (d >= 0 && d < moved && __ldcg(p.list + d) == x)
                           to = __ldcg(p.moves + p.cap + moved - 1 - d);
                       else  // a page that refs does not count has no move
                           atomicOr(p.err, kErrRangeBit);
                   }
                   if (to != x || copy) table_out[e] = to;
               });
    if (tid == 0) *p.moves_n = moved;
    cluster_wait();
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
// kSlice bytes of them at a time, all loads ahead of the stores. (The large compaction's: 125 us, 6.2 TB/s.)
constexpr int kSlice = 4096;

struct CopyList {
    const int32_t *src, *dst, *rows;  // rows: or nullptr, all
    const int32_t *n_dev;             // or nullptr: n
    int n;
};

__global__ void __launch_bounds__(256) kv_copy_kernel(KvDev kv, int row_bytes, CopyList list)
{
    // what is to be copied: the update's or compaction's kernel lets this one start (call after call a step of 64 slots
    // 17.4 us, so 14.7)
    pdl_wait_prior();
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
    v.slots = reinterpret_cast<int4 *>(take(4 * S));  // (cudaMalloc's alignment)
    v.stash = take(S * (size_t)p->stride);
    v.last = take(S);
    v.base = take(S);
    v.count = take(P);
    v.claim = take(P);
    v.list = take(P + 4 * kCtas);
    v.place = take(P);
    v.named = take(P / 2 + 1);
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
    const int row_bytes = kv.D * (int8 ? 1 : 2);
    const int64_t slices = (((int64_t)row_bytes << kv.page_shift) + kSlice - 1) / kSlice;
    const int64_t units = (int64_t)n * 2 * kv.H * slices;
    const int64_t ctas = std::min<int64_t>((units + 7) / 8, 8 * (int64_t)num_sms);
    return launch_stream(true, true, kv_copy_kernel, (unsigned)ctas, 256, stream, kv, row_bytes,
                         CopyList{src, dst, rows, n_dev, n});
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
    const size_t ints = (size_t)max_seqs * table_stride + 6 * (size_t)max_seqs + 4 * (size_t)num_pages +
                        (size_t)num_pages / 2 + 1 + 4 * kCtas + 3 * (size_t)p->cap() + 1;
    if (cudaMalloc((void **)&p->d_err, 3 * sizeof(int)) != cudaSuccess ||
        cudaMalloc((void **)&p->scratch, sizeof(int32_t) * ints) != cudaSuccess ||
        cudaHostAlloc((void **)&p->h_err, sizeof(int), cudaHostAllocDefault) != cudaSuccess) {
        cudaGetLastError();
        lora_kv_pages_destroy(p);
        return LORA_ERR_OOM;
    }
    if (cudaMemset(p->d_err, 0, 3 * sizeof(int)) != cudaSuccess ||
        cudaMemset(pages_view(p).moves_n, 0, sizeof(int)) != cudaSuccess ||
        cudaMemset(pages_view(p).count, 0, sizeof(int32_t) * (size_t)num_pages) != cudaSuccess ||
        cudaMemset(pages_view(p).claim, kNone & 0xff, sizeof(int32_t) * (size_t)num_pages) != cudaSuccess ||
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
    int dev = -1;
    if (cudaGetDevice(&dev) == cudaSuccess && dev != p->device) cudaSetDevice(p->device);
    cudaDeviceSynchronize();
    if (p->ctl_stream) cudaStreamDestroy(p->ctl_stream);
    if (p->ev) cudaEventDestroy(p->ev);
    if (p->scratch) cudaFree(p->scratch);
    if (p->d_err) cudaFree(p->d_err);
    if (p->h_err) cudaFreeHost(p->h_err);
    if (dev >= 0 && dev != p->device) cudaSetDevice(dev);
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
    const lora_status st = on_device(p->device);
    if (st != LORA_OK) return st;
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
