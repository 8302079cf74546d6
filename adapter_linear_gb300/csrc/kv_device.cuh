// kv_device.cuh -- device helpers of the paged key/value cache: finding a row's sequence and
// a token's cache row, and the conversions between 8-bit codes and values.
#pragma once

#include <cuda_fp16.h>

#include "device_common.cuh"
#include "kv_internal.h"

namespace lora {

__device__ __forceinline__ void kv_flag_range(int *err) { atomicOr(err, kErrRangeBit); }

// Sequence b's rows [row0, row0 + n) and length L, checked: a start outside 0..T, starts that
// decrease or a length beyond the table flag the error word and read as an empty sequence.
struct KvSeq {
    int row0, n, L;
};

__device__ __forceinline__ KvSeq kv_seq(const KvBatchDev &b, int page_shift, int seq, int *err)
{
    const int row0 = b.start[seq], end = b.start[seq + 1], L = b.kv_len[seq];
    // (compared before they are subtracted: the difference of two bad starts may wrap round)
    if (row0 < 0 || end < row0 || end > b.T || L < 0 || (int64_t)L > ((int64_t)b.table_stride << page_shift)) {
        kv_flag_range(err);
        return KvSeq{0, 0, 0};
    }
    return KvSeq{row0, end - row0, L};
}

// The sequence whose rows hold row t (called by a whole warp, the same t in every lane): the
// last b with start[b] <= t, by a 32-way search: a round narrows the range to a 32nd, so 1024
// sequences take two dependent loads. -1: before the first row. Among bad starts the search stops
// at the first that is above t, so it finds t's sequence or one before it.
__device__ __forceinline__ int kv_find_seq(const KvBatchDev &b, int t, int lane)
{
    int lo = 0, len = b.n_seqs;  // the answer is lo - 1 + (number of starts <= t in [lo, lo + len))
    while (len > 0) {
        const int step = (len + 31) >> 5;
        const int at = lo + (lane + 1) * step - 1;  // the last entry of this lane's part
        const bool le = at < lo + len && b.start[at] <= t;
        // parts that lie wholly below, up to the first that does not
        const int full = __clz(__brev(~__ballot_sync(0xffffffffu, le)));
        const int end = lo + len;
        lo += full * step;
        len = min(step - 1, end - lo);
    }
    return lo - 1;
}

// Cache row of the token at `pos` of sequence `seq` for head 0, or -1 (a bad table entry).
__device__ __forceinline__ int64_t kv_row(const KvDev &kv, const KvBatchDev &b, int seq, int pos)
{
    const int page = b.table[(int64_t)seq * b.table_stride + (pos >> kv.page_shift)];
    if (page < 0 || page >= kv.num_pages) {
        kv_flag_range(kv.err);
        return -1;
    }
    return (((int64_t)page * kv.H) << kv.page_shift) + (pos & ((1 << kv.page_shift) - 1));
}

// x / G for 0 <= x < 2^31 (KvAttn::g_mul, g_shift).
__device__ __forceinline__ int div_g(const KvAttn &a, int x)
{
    return a.G == 1 ? x : (int)(__umulhi((uint32_t)x, a.g_mul) >> a.g_shift);
}

// The work of an attention kernel and one CTA's share of it.
//
// An item is (sequence, tile of R rows, kv head); a row is one query head of one new token: row
// r of a sequence is token r / G, head r % G of the kv head's G. An item's visible tokens [lo,
// hi), lo rounded down to 16 (so that 16 tokens from there never cross a page), are cut into
// units of kUnit tokens, at least one (rows that see nothing still write their zeros), behind kHead
// empty units, which stand for what an item costs beside its tokens. Units are numbered
// sequence by sequence, tile by tile, head by head; CTA c of `grid` takes units [c total / grid,
// (c + 1) total / grid). Every member but next() is called by whole warps, which all
// compute the same. Sequences with n G outside min_rows..max_rows are left out.
template <int R, int kUnit, int kHead>
struct KvWork {
    const KvDev &kv;
    const KvBatchDev &b;
    const KvAttn &a;
    const int G, window, min_rows, max_rows, lane;
    int64_t total = 0;           // units of all items
    int64_t grid = 0, u_end = 0;
    int64_t u = 0, seg_end = 0;  // the current segment: units [u, seg_end) of one item
    int64_t item0 = 0;           // the item's first unit
    int64_t tile0 = 0;           // first unit of the tile's first head
    int seq = -1, tile = 0, tiles = 0, nu = 0, head = 0, lo = 0, hi = 0;
    int j0 = 0, j1 = 0;          // units of tokens: [j0, j1) of the item's nu - kHead
    KvSeq sh{0, 0, 0};

    __device__ __forceinline__ KvWork(const KvDev &kv_, const KvBatchDev &b_, const KvAttn &a_, int min_rows_,
                                      int max_rows_, int lane_)
        : kv(kv_), b(b_), a(a_), G(a_.G), window(a_.window), min_rows(min_rows_), max_rows(max_rows_), lane(lane_)
    {
        for (int s0 = 0; s0 < b.n_seqs; s0 += 32) {
            const int64_t v = units_of_32(s0);
            if (s0 == 0) first_ = v;
            total += v;
        }
        total = sum(total);
    }

    // Take share c of n; false: it is empty.
    __device__ __forceinline__ bool take_share(int64_t c, int64_t n)
    {
        grid = n;
        if (c >= n) return false;
        seg_end = c * total / n;
        u_end = (c + 1) * total / n;
        int64_t before = 0;
        for (int s0 = 0;; s0 += 32) {
            const int64_t mine = s0 == 0 ? first_ : units_of_32(s0);
            const int64_t incl = scan(mine);
            const uint32_t past = __ballot_sync(0xffffffffu, before + incl > seg_end);
            if (past) {
                const int k = __ffs(past) - 1;
                before += __shfl_sync(0xffffffffu, incl - mine, k);
                set_seq(s0 + k);
                break;
            }
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
        for (int t0 = 0;; t0 += 32) {  // the tile, 32 at a time
            const int64_t mine = t0 + lane < tiles ? (int64_t)units(sh, t0 + lane) * kv.H : 0;
            const int64_t incl = scan(mine);
            const uint32_t past = __ballot_sync(0xffffffffu, before + incl > seg_end);
            if (past) {
                const int k = __ffs(past) - 1;
                tile0 = before + __shfl_sync(0xffffffffu, incl - mine, k);
                set_tile(t0 + k);
                return true;
            }
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
    }

    // The share's next segment that has tokens' units; false at its end.
    __device__ __forceinline__ bool next()
    {
        do {
            if (!next_any()) return false;
            j0 = max(0, (int)(u - item0) - kHead);
            j1 = (int)(seg_end - item0) - kHead;
        } while (j1 <= 0);
        return true;
    }

    __device__ __forceinline__ bool first() const { return j0 == 0; }
    __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == nu - kHead; }
    // The CTAs that have the item's first and last tokens' units (total >= grid: no share is
    // empty).
    __device__ __forceinline__ int first_cta() const { return cta_of(item0 + kHead); }
    __device__ __forceinline__ int last_cta() const { return cta_of(item0 + nu - 1); }

private:
    int64_t first_ = 0;  // the units of sequence `lane`

    __device__ __forceinline__ int cta_of(int64_t x) const { return (int)(((x + 1) * grid - 1) / total); }
    __device__ __forceinline__ bool next_any()
    {
        u = seg_end;
        if (u >= u_end) return false;
        while (u >= tile0 + (int64_t)nu * kv.H) {
            tile0 += (int64_t)nu * kv.H;
            if (tile + 1 < tiles) {
                set_tile(tile + 1);
            } else {
                do set_seq(seq + 1);
                while (tiles == 0);
                set_tile(0);
            }
        }
        head = (int)((u - tile0) / nu);
        item0 = tile0 + (int64_t)head * nu;
        seg_end = min(item0 + nu, u_end);
        return true;
    }

    __device__ __forceinline__ int tiles_of(const KvSeq &s) const
    {
        const int64_t rows = (int64_t)s.n * G;
        return rows >= min_rows && rows <= max_rows ? (int)((rows + R - 1) / R) : 0;
    }
    __device__ __forceinline__ void range(const KvSeq &s, int t, int *lo_, int *hi_) const
    {
        // (n G < 2^31, and the last tile's last row may pass it)
        const int r1 = min(t * R + (R - 1u), s.n * (uint32_t)G - 1u);
        const int i0 = div_g(a, t * R), i1 = div_g(a, r1);
        const int p0 = s.L - s.n + i0, p1 = s.L - s.n + i1;
        *hi_ = max(0, p1 + 1);
        *lo_ = min((window > 0 ? max(0, p0 - window + 1) : 0) & ~15, *hi_);
    }
    __device__ __forceinline__ int units(const KvSeq &s, int t) const
    {
        int l, h;
        range(s, t, &l, &h);
        return kHead + max(1, (h - l + kUnit - 1) / kUnit);
    }
    // Units of sequence s0 + lane (0 past the last). Few tiles: a lane counts its own; a sequence
    // of many is counted by all lanes together.
    __device__ __forceinline__ int64_t units_of_32(int s0) const
    {
        KvSeq s{0, 0, 0};
        if (s0 + lane < b.n_seqs) s = kv_seq(b, kv.page_shift, s0 + lane, kv.err);
        const int n = tiles_of(s);
        int64_t v = 0;
        if (n <= 8)
            for (int t = 0; t < n; ++t) v += units(s, t);
        for (uint32_t todo = __ballot_sync(0xffffffffu, n > 8); todo; todo &= todo - 1) {
            const int k = __ffs(todo) - 1;
            const KvSeq q{0, __shfl_sync(0xffffffffu, s.n, k), __shfl_sync(0xffffffffu, s.L, k)};
            const int m = __shfl_sync(0xffffffffu, n, k);
            int64_t part = 0;
            for (int t = lane; t < m; t += 32) part += units(q, t);
            part = sum(part);
            if (lane == k) v = part;
        }
        return v * kv.H;
    }
    __device__ __forceinline__ void set_seq(int s)
    {
        seq = s;
        sh = kv_seq(b, kv.page_shift, s, kv.err);
        tiles = tiles_of(sh);
    }
    __device__ __forceinline__ void set_tile(int t)
    {
        tile = t;
        range(sh, t, &lo, &hi);
        nu = units(sh, t);
    }
    static __device__ __forceinline__ int64_t sum(int64_t v)
    {
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
        return v;
    }
    __device__ __forceinline__ int64_t scan(int64_t v) const
    {
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, v, x);
            if (lane >= x) v += o;
        }
        return v;
    }
};

// 16-byte asynchronous copy to shared memory; of the 16 bytes `bytes` are read, the rest are zeros
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float *a, float *b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// An infinity or a NaN of V in an unquantised cache belongs to every row that sees its token, whatever
// weight it has there: the row's value is NaN with a NaN or infinities of both signs, else that
// infinity. The products do not give that (0 or a negative second part of a weight times an
// infinity is NaN or the other infinity), so the kernels look for values of O that are not finite and
// work those out from V again; where some rows do not see all tokens, the bad values stay out of the
// product.
//
// Of a pair of bf16: the infinities and NaN become zeros (finite_part), or all but them do
// (the other half of the same xor).
__device__ __forceinline__ uint32_t finite_part(uint32_t v)
{
    const uint32_t lo = (v & 0x7F80u) == 0x7F80u ? 0u : v & 0xFFFFu;
    const uint32_t hi = (v & 0x7F800000u) == 0x7F800000u ? 0u : v & 0xFFFF0000u;
    return lo | hi;
}

// acc + wt v for a piece's weight, which may be 0 where its O is an infinity.
template <bool kInt8>
__device__ __forceinline__ float add_piece(float wt, float v, float acc)
{
    return fmaf(!kInt8 && wt == 0.0f && fabsf(v) == INFINITY ? 1.0f : wt, v, acc);
}

constexpr float kLn2 = 0.6931471805599453f;

// 2^x, to about 2^-22 of it; 0 for -inf
__device__ __forceinline__ float fast_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float fast_log2(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (x & mask) | bits in one instruction: with both constants known the compiler makes two of it,
// so `bits` comes from a register it cannot see through (kv_opaque).
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(mask), "r"(bits));
    return r;
}
__device__ __forceinline__ uint32_t kv_opaque(uint32_t v)
{
    uint32_t r;
    asm volatile("mov.b32 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// Two 8-bit codes to two bf16, exactly. x holds code a in bits 0..7 and code b in bits 16..23
// (the other bits are ignored). A code is (low 7 bits) - (its sign bit's 128), and in bf16
// 0x4300 | v is 128 + v for v < 128 and 0x4380 is 256: code = (128 + low) - (128 or 256).
// base: 0x43004300 from kv_opaque.
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t x, uint32_t base)
{
    const uint32_t low = and_or(x, 0x007F007Fu, base);
    const uint32_t sign = and_or(x, 0x00800080u, base);
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&low),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&sign));
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The four codes of a word, in order, as two f16 pairs, exactly: 0x6400 | v is 1024 + v in f16,
// v = code + 128.
__device__ __forceinline__ void codes4_to_f16(uint32_t w, uint32_t *lo, uint32_t *hi)
{
    w ^= 0x80808080u;
    const uint32_t bias = 0x64806480u;  // 1024 + 128, twice
    const uint32_t x[2] = {__byte_perm(w, 0x64646464u, 0x4140), __byte_perm(w, 0x64646464u, 0x4342)};
    const __half2 l = __hsub2(*reinterpret_cast<const __half2 *>(&x[0]), *reinterpret_cast<const __half2 *>(&bias));
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&x[1]), *reinterpret_cast<const __half2 *>(&bias));
    *lo = *reinterpret_cast<const uint32_t *>(&l);
    *hi = *reinterpret_cast<const uint32_t *>(&h);
}

// The four codes of a word, in order, as two bf16 pairs.
__device__ __forceinline__ void codes4_to_bf16(uint32_t w, uint32_t base, uint32_t *lo, uint32_t *hi)
{
    *lo = codes_to_bf16(__byte_perm(w, 0, 0x4140), base);
    *hi = codes_to_bf16(__byte_perm(w, 0, 0x4342), base);
}

// Code i (0..3) of word a and code i of word b as a bf16 pair.
__device__ __forceinline__ uint32_t codes_pair_to_bf16(uint32_t a, uint32_t b, int i, uint32_t base)
{
    return codes_to_bf16(__byte_perm(a, b, 0x0400u + 0x0101u * (uint32_t)i), base);
}

}  // namespace lora
