// kv_prefill_kernel.cuh -- attention of longer chunks over the paged cache: the products on the tcgen05
// tensor cores.
//
// For a row (one query head of one new token) at position pos and its visible keys j:
//   z_j = scale <Q, K_j>,  m near max z_j,  l = sum 2^(z_j - m),  O = sum 2^(z_j - m) V_j / l
// (z in units of log2), over tiles of 128 keys in one pass. m is any number near the maximum: it
// cancels in O / l, so it is moved, and O rescaled, only when a score passes it by much.
//
// A CTA works on 256 rows of one kv head: the G query heads that share it for 256 / G tokens, so
// K and V are read once for all of them, as two MMA tiles of 128 rows. Warps 0-3 and 4-7 do the
// softmax of one tile each (a thread holds a row), 8-11 bring K and V tiles into shared memory
// (8-bit codes become bf16 on the way), warps 12 and 13 issue the MMAs, warp 14
// hands out the work:
//   S_t = Q_t K^T  (both operands in shared memory, S in tensor memory, 128 columns a tile)
//   O_t += P_t V   (P, the bf16 weights, written by the softmax over S; O in tensor memory)
// in two halves of 64 keys: PV_t(j, h) follows as soon as that half's weights are there, and behind it
// S_t(j + 1, h) over the same columns, so that the next tile's scores of one half are made
// while the softmax works on the other half. MMAs of one thread execute in order, so S_t(j + 1, h)
// overwrites P_t(j, h) only after PV_t(j, h) has read it, and the commit behind S_t(j + 1, h) covers
// PV_t(j, h). (A product a tile, in turns of the two tiles: 8 prompts of 2048 bf16 379 us,
// halves 373; 512 tokens over 32000 int8 398, so 377. S with N = 64 reads Q twice, which costs
// 24 % of the products' time at D = 128.)
//
// The softmax of a row, a thread: 32 scores at a time from tensor memory into registers, the next
// 32 on their way while these become weights.
//
// What bounds it: the softmax. Of the 3500 cycles that a key tile of 2 x 128 rows takes at D = 128,
// bf16, it takes 2900 in each row's thread (44 % of the issue slots are used, the rest is
// latency between dependent instructions, two softmax warps a scheduler); with an 8-bit cache 6000 of
// 6200 (49 %), the multiplications by scales on top and, beside it, the codes' conversion: their stores,
// the loads of scales and the MMAs' operands use 86 % of shared memory's bandwidth. The tensor cores
// are active 47 and 45 % of the time. 32 query heads on 8 kv heads of 128 values: 8 prompts of
// 2048 tokens bf16 391 us (0.70 PFLOP/s), 512 tokens over 32000 8-bit 359 us (0.75), call included.
//
// An 8-bit cache's scales stay outside the products: the codes are exact in bf16, a key's scale
// multiplies its column of S and a value's its weight.
//
// A weight rounded to bf16 is off by up to 2^-8 of it, which averages out over many keys but shows
// where one key holds much of a row's weight. So where a key may hold more than a quarter of
// what its row has so far, the half's weights go to the product in two bf16 parts, the second with
// the rest (a second product for that half: a piece's first keys, then rarely). A prefix that short chunks share
// (KvShareDev::two_parts) has all its weights in two parts, as the short-chunk kernel has, which each of them alone would
// have gone to: 64 requests over 8192 tokens 8-bit 57 us, 56 with the rule; 16 prompts of 16 answers bf16 114.5 and 109;
// 48 drafts over 9000 to 16000 8-bit 163 and 150.
//
// Work is shared out like the short-chunk kernel's: the grid's CTAs (one an SM) take equal
// contiguous runs of 128-token units over all items, pieces of an item go to scratch as
// (m, l, O), and the warp that finishes a piece of 32 rows last joins them in CTA order.
#pragma once

#include <cmath>

#include "kv_device.cuh"

namespace lora {
namespace {

constexpr int kBlockRows = kShareRows, kTileRows = 128, kKeys = 128, kHalf = 64, kPart = 32;
constexpr int kSoftWarps = 8, kLoadWarps = 4;
constexpr int kThreads = (kSoftWarps + kLoadWarps + 4) * 32;  // two MMA warps, one that hands out the work, one idle
// Registers a thread of the softmax warps, the loading warps and the MMA warps' group: a block of
// 512 threads starts with 128 each, and 2 x 152 + 120 + 88 is 4 x 128. (Nothing may spill: shared
// memory leaves L1 28 KB, and a spilled register comes back from L2.)
constexpr int kSoftRegs = 152, kLoadRegs = 120, kMmaRegs = 88;
static_assert(2 * kSoftRegs + kLoadRegs + kMmaRegs <= 4 * 128, "register split");

// What an item costs beside its key tiles, in key tiles (its first tile's two parts, Q, the output):
// 8 prompts of 2048 bf16 442 us at 1, 388 at 2, 381 at 3; 40 mixed 8-bit requests 94, 94 and 95.
constexpr int kHeadUnits = 3;
constexpr int kSegments = 4;
constexpr int kOutPitch = 80;  // bytes of a row of 32 bf16 columns: rows start 5 x 16 bytes apart

template <int D>
struct Cfg {
    static constexpr int kTileBytes = 128 * D * 2;           // 128 rows of Q, K or V in bf16
    static constexpr int kStages = D == 128 ? 2 : 4;
    // Scales of a key tile: S of tile i - kStages is done (k_empty) before tile i's are written,
    // so the weights of the tile before that one are, too: kStages + 1 entries would do.
    static constexpr int kRing = kStages + 2;
    static constexpr int kQ = 0;
    static constexpr int kK = 2 * kTileBytes;
    static constexpr int kV = kK + kStages * kTileBytes;
    static constexpr int kScales = kV + kStages * kTileBytes;  // float [kRing][2][128]: the keys' (times the
                                                               // score's), the values'
    static constexpr int kSegs = kScales + kRing * 256 * 4;
    static constexpr int kBars = kSegs + kSegments * 64;
    static constexpr int kOut = kBars + 512;                   // a softmax warp's 32 rows x 32 columns of O
    static constexpr int kSmem = kOut + kSoftWarps * 32 * kOutPitch + 1024;           // and room to align to 1024
    static constexpr uint32_t kO = 256;                        // tensor memory column of O_0
};

// One segment of the CTA's share, as the warp that walks the share hands it to the others.
struct Segment {
    int seq, row0, n, L;    // the sequence whose pages are read (row0: its first row of the call's tensors)
    int tile, head;         // block of 256 rows, kv head
    int lo, hi;             // its visible tokens
    int j0, j1;             // key tiles [j0, j1) of them; j1 == 0: no more segments
    int whole, slot;        // all of the item? else the scratch slot of the piece
    int c0, c1;             // and the CTAs that have pieces of the item
    int bad;                // V had an infinity or a NaN in a tile that not all rows see (unquantised cache)
    int first;              // the sequence's first token of its own (kOwn)
};
static_assert(sizeof(Segment) == 64, "segment");

struct Bars {
    uint64_t seg_full[kSegments], seg_empty[kSegments], q_full[2], q_empty[2], k_full[4], k_empty[4], v_full[4],
        v_empty[4], sc_full[6], s_full[2][2], p_full[2][2], pv_half[2], o_full[2], drain[2];
};
static_assert(sizeof(Bars) <= 512, "barriers");

// The positions [x, y] that all rows of a segment's block see.
template <KvMode kMode>
__device__ __forceinline__ int2 seen_by_all(const Segment *w, int G, int window)
{
    if (kMode == kPrefix) return make_int2(0, w->L - 1);
    const int first = w->tile * kBlockRows, p0 = w->L - w->n;
    return make_int2(window > 0 ? p0 + (min(first + kBlockRows, w->n * G) - 1) / G - window + 1 : 0, p0 + first / G);
}
// Of 16 tokens from tok0, does some row not see one?
__device__ __forceinline__ bool edge_group(int tok0, int2 seen) { return tok0 + 15 > seen.y || tok0 < seen.x; }

struct Plan {
    int min_rows;
    float scale_log2;   // |scale| log2(e)
    uint32_t q_sign;    // 0x80008000 for a negative scale: flips the sign of a pair of Q's values
    float *part;   // [2 grid] slots of [256 / 32 warps][D / 4][32 rows][4], then [2 grid][256][2] (m, l)
    int *count;    // [grid][8] arrivals of a warp's rows at the item that starts in that CTA
};

// Where in a 128-row tile (halves of 64 values, rows of 128 bytes, 16-byte chunks swizzled as the
// tensor core's 128-byte pattern has them) chunk ch of row r lies.
__device__ __forceinline__ uint32_t tile_off(int r, int ch)
{
    return (uint32_t)((ch >> 3) * 16384 + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

// The same tile as an operand whose N runs along the row (V: N = the head's dims, K = the tokens):
// 64-value halves 16 KB apart, groups of 8 tokens 1 KB apart.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t smem_addr)
{
    uint64_t d = 0;
    d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(16384 >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// The MMA warp runs its loop with all lanes, so that operands stay in uniform registers (from a
// single lane's branch each MMA took 100 cycles to issue, moving them there); `lead` is
// non-zero in the lane that issues.
// D[tmem] (+)= A[smem] * B[smem]
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void commit_lead(uint32_t lead, uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(lead)
        : "memory");
}

// 32 columns into registers; they are there after tmem_wait32 on the same registers (which orders
// nothing else).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[kPart])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
                 "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                   "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
                   "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
                   "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[kPart])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]),
                   "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]),
                   "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}

__device__ __forceinline__ void tmem_ld8_wait(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_zero8(uint32_t taddr)
{
    const uint32_t z = 0;
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %1, %1, %1, %1, %1, %1, %1};" ::"r"(taddr), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int kRegs>
__device__ __forceinline__ void regs_up()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_down()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// mbar_wait with one place that tries: the roles' loops run through several waits a key tile, and
// their code must stay small.
__device__ __forceinline__ bool small_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *err)
{
    uint32_t n = 0;
    uint64_t start = 0;
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
        if ((++n & 255u) != 0) continue;
        const uint64_t now = global_timer_ns();
        if (n == 256) start = now;
        if (*abort_flag || now - start > kWaitTimeoutNs) {
            if (!*abort_flag) atomicOr(err, kErrTimeoutBit);
            *abort_flag = 1;
            return false;
        }
    }
    return true;
}

// A wait of a whole warp: every lane waits (and so sees what the barrier released), and all
// agree on whether it ran out.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *err)
{
    return __all_sync(0xffffffffu, small_wait(bar, parity, abort_flag, err));
}

// The row's scores of 32 keys in units of log2, in pairs: raw ones (as loaded) times mul or the
// keys' scales; returns the largest.
template <bool kInt8>
__device__ __forceinline__ float part_scores(const uint32_t (&s)[kPart], const float *sc, uint64_t mul,
                                             uint64_t (&z)[kPart / 2])
{
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < kPart / 2; ++i) {
        z[i] = pack2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
        if (kInt8) {
            const ulonglong2 c = *reinterpret_cast<const ulonglong2 *>(sc + 2 * (i & ~1));
            z[i] = mul2(z[i], i & 1 ? c.y : c.x);
        } else {
            z[i] = mul2(z[i], mul);
        }
        float a, b;
        unpack2(z[i], &a, &b);
        top[i & 1] = fmaxf(top[i & 1], fmaxf(a, b));
    }
    return fmaxf(top[0], top[1]);
}

// -inf for the keys that the row does not see: it sees columns above `low` up to `lim`; returns the
// largest score that is left.
__device__ __forceinline__ float mask_scores(uint64_t (&z)[kPart / 2], int lim, int low)
{
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPart / 2; ++i) {
        float a, b;
        unpack2(z[i], &a, &b);
        a = 2 * i <= lim && 2 * i > low ? a : -INFINITY;
        b = 2 * i + 1 <= lim && 2 * i + 1 > low ? b : -INFINITY;
        z[i] = pack2(a, b);
        top = fmaxf(top, fmaxf(a, b));
    }
    return top;
}

// The row's 32 weights 2^(z - m), times the values' scales (0 for a key the row does not see,
// whatever its scale is: kMask, 8-bit), as bf16 pairs: keys 16 i + 2 e, + 1 in column 16 i + e, and in column
// 16 i + 8 + e what rounding left of them (rest) or zeros. Returns the weights' sum.
template <bool kInt8, bool kMask>
__device__ __forceinline__ float part_weights(const uint64_t (&z)[kPart / 2], uint32_t tS, const float *sc, float m,
                                              bool rest)
{
    const uint64_t neg = pack2(-m, -m);
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int ch = 0; ch < kPart / 16; ++ch) {
        uint64_t w[8];
        uint32_t p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float e0, e1, z0, z1;
            unpack2(z[8 * ch + e], &z0, &z1);
            unpack2(add2(z[8 * ch + e], neg), &e0, &e1);
            e0 = fast_exp2(e0);
            e1 = fast_exp2(e1);
            w[e] = pack2(e0, e1);
            sum[e & 1] = add2(sum[e & 1], w[e]);
            if (kInt8) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(sc + 128 + 16 * ch + 2 * (e & ~1));
                w[e] = mul2(w[e], e & 1 ? v.y : v.x);
            }
            unpack2(w[e], &e0, &e1);
            if (kMask) {
                e0 = z0 == -INFINITY ? 0.0f : e0;
                e1 = z1 == -INFINITY ? 0.0f : e1;
                w[e] = pack2(e0, e1);
            }
            p[e] = pack_bf16x2(e0, e1);
        }
        tmem_st8(tS + ch * 16, p);
        if (rest) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float w0, w1;
                unpack2(w[e], &w0, &w1);
                p[e] = pack_bf16x2(w0 - bf16_lo(p[e]), w1 - bf16_hi(p[e]));
            }
            tmem_st8(tS + ch * 16 + 8, p);
        } else {
            tmem_zero8(tS + ch * 16 + 8);
        }
    }
    float a, b;
    unpack2(add2(sum[0], sum[1]), &a, &b);
    return a + b;
}

// A row's 8 columns of O, or of pairs of weights, times `down`.
__device__ __forceinline__ void scale_o(uint32_t tO, float down)
{
    uint32_t o[8];
    tmem_ld8_wait(tO, o);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * down);
    tmem_st8(tO, o);
}
__device__ __forceinline__ void scale_p(uint32_t tP, float down)
{
    uint32_t p[8];
    tmem_st_wait();
    tmem_ld8_wait(tP, p);
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = pack_bf16x2(bf16_lo(p[e]) * down, bf16_hi(p[e]) * down);
    tmem_st8(tP, p);
}

// Which piece of a 16-token group of an 8-bit cache lane `lane` holds: 16-byte piece `c` of rows
// `r`, r + 32 / (D / 16), ... (so that a warp reads 512 bytes at a time, and the eight lanes of
// a phase store to eight different chunk columns).
template <int D>
__device__ __forceinline__ void lane_piece(int lane, int *r, int *c)
{
    if (D == 128) {
        *c = (lane & 3) | ((lane >> 1) & 4);
        *r = ((lane >> 2) & 1) | ((lane >> 3) & 2);
    } else {
        *c = lane & 3;
        *r = lane >> 2;
    }
}

// A lane's pieces of a 16-token group as bf16 into its tile (dst: the group's first row).
template <int D>
__device__ __forceinline__ void store_codes(uint8_t *dst, const uint4 (&v)[D / 32], int r0, int piece, uint32_t base)
{
#pragma unroll
    for (int p = 0; p < D / 32; ++p) {
        const uint32_t c[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
        uint32_t x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) codes4_to_bf16(c[e], base, &x[2 * e], &x[2 * e + 1]);
        const int r = r0 + p * (512 / D);
        *reinterpret_cast<uint4 *>(dst + tile_off(r, 2 * piece)) = make_uint4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<uint4 *>(dst + tile_off(r, 2 * piece + 1)) = make_uint4(x[4], x[5], x[6], x[7]);
    }
}

// The infinities and NaN of V among a segment's tokens, to the rows that see them. pos: the row's
// position, -1: no row; finite: the row's weights are. A block of 8 columns where O is finite lacks
// what the loading warps took out; one where it is not is worked out from all tokens again.
template <int D, KvMode kMode>
__device__ __forceinline__ void add_bad(const KvDev &kv, const KvBatchDev &b, const Segment *w,
                                        int G, int window, int pos, bool finite, uint32_t tO)
{
    const int lane = threadIdx.x & 31;
    const int32_t *const table = b.table + (int64_t)w->seq * b.table_stride;
    const int2 seen = seen_by_all<kMode>(w, G, window);
    const int end = min(w->hi, w->lo + w->j1 * kKeys);
#pragma unroll 1
    for (int x = 0; x < D; x += 8) {
        uint32_t o[8];
        tmem_ld8_wait(tO + x, o);
        float zero = 0.0f, sum[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            zero = fmaf(__uint_as_float(o[e]), 0.0f, zero);
            sum[e] = 0.0f;
        }
        const bool all = __any_sync(0xffffffffu, finite && zero != 0.0f);
#pragma unroll 1
        for (int tok0 = w->lo + w->j0 * kKeys; tok0 < end; tok0 += 32) {  // a token a lane
            const int tok = tok0 + lane;
            uint32_t f[4] = {0, 0, 0, 0};
            if (tok < end && (all || edge_group(tok & ~15, seen))) {
                const int page = table[tok >> kv.page_shift];
                if (page >= 0 && page < kv.num_pages) {
                    const int64_t row =
                        (((int64_t)page * kv.H + w->head) << kv.page_shift) + (tok & ((1 << kv.page_shift) - 1));
                    const uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(kv.v) + row * D + x);
                    f[0] = v.x ^ finite_part(v.x);
                    f[1] = v.y ^ finite_part(v.y);
                    f[2] = v.z ^ finite_part(v.z);
                    f[3] = v.w ^ finite_part(v.w);
                }
            }
#pragma unroll 1
            for (uint32_t left = __ballot_sync(0xffffffffu, (f[0] | f[1] | f[2] | f[3]) != 0); left; left &= left - 1) {
                const int from = __ffs(left) - 1;
                const bool sees = tok0 + from <= pos && (window == 0 || tok0 + from > pos - window);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t u = __shfl_sync(0xffffffffu, f[e], from);
                    if (sees) {
                        sum[2 * e] += bf16_lo(u);
                        sum[2 * e + 1] += bf16_hi(u);
                    }
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = sum[e] == 0.0f ? o[e] : __float_as_uint(sum[e]);
        __syncwarp();
        tmem_st8(tO + x, o);
    }
    tmem_st_wait();
}

// Tile t of a segment's rows of Q on their way into shared memory, by 128 threads; rows past the chunk's last
// become zeros.
template <int D>
__device__ __forceinline__ void copy_q(const KvAttn &a, const Segment *w, int t, int tid, uint8_t *dst)
{
    constexpr int kLanes = D / 8, kRows = kTileRows / kLanes;
    const int G = a.G, rows = w->n * G, r = tid / kLanes, c = tid % kLanes;
    int q = w->tile * kBlockRows + t * kTileRows + r, i = div_g(a, q), g = q - i * G;  // row, its token and head
    const int step_i = div_g(a, kRows), step_g = kRows - step_i * G;
    const uint16_t *const src = a.Q + (int64_t)w->row0 * a.q_stride + (int64_t)w->head * G * D + c * 8;
#pragma unroll 4
    for (int x = 0; x < kTileRows / kRows; ++x) {
        const bool on = q < rows;
        cp_async16(smem_u32(dst + tile_off(r + x * kRows, c)), src + (on ? (int64_t)i * a.q_stride + g * D : 0),
                   on ? 16u : 0u);
        q += kRows;
        i += step_i;
        g += step_g;
        if (g >= G) {
            g -= G;
            ++i;
        }
    }
}
// The same threads' values with their signs as the scale's (sign: of a pair).
template <int D>
__device__ __forceinline__ void sign_q(int tid, uint8_t *tile, uint32_t sign)
{
    constexpr int kLanes = D / 8;
    if (sign == 0) return;
#pragma unroll 1
    for (int r = tid / kLanes; r < kTileRows; r += kTileRows / kLanes) {
        uint4 *const at = reinterpret_cast<uint4 *>(tile + tile_off(r, tid % kLanes));
        const uint4 u = *at;
        *at = make_uint4(u.x ^ sign, u.y ^ sign, u.z ^ sign, u.w ^ sign);
    }
}

template <int D, bool kInt8, KvMode kMode>
__global__ void __launch_bounds__(kThreads, 1)
    kv_prefill_kernel(KvDev kv, KvBatchDev b, KvAttn a, KvShareDev share, Plan plan)
{
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars &bars = *reinterpret_cast<Bars *>(smem + C::kBars);
    float *const scale_ring = reinterpret_cast<float *>(smem + C::kScales);
    __shared__ uint32_t tmem_slot;
    __shared__ uint32_t rest_flags[2][2];  // of the tiles' weights: a byte a warp, has it a second part?
    __shared__ volatile int abort_flag;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = a.G, window = kMode == kPlain ? a.window : 0;
    Segment *const segs = reinterpret_cast<Segment *>(smem + C::kSegs);
    // The first segment's Q comes by the softmax warps, which have nothing else to do then, while the loading warps
    // convert the first tokens' codes: 64 requests with one 8-bit prefix 56 us, not 58. (An unquantised cache's have
    // nothing to convert: 16 prompts of 16 answers 109 either way. In longer chunks what it does to the code costs
    // more: 512 tokens over 32000 8-bit 375, not 359.)
    constexpr bool kSoftQ = kMode == kPrefix && kInt8;
    const bool two_parts = kMode == kPrefix && share.two_parts;  // of every weight

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.q_full[i], kLoadWarps);
            mbar_init(&bars.q_empty[i], 1);
            for (int h = 0; h < 2; ++h) {
                mbar_init(&bars.s_full[i][h], 1);
                mbar_init(&bars.p_full[i][h], kTileRows / 32);
            }
            mbar_init(&bars.o_full[i], 1);
            mbar_init(&bars.pv_half[i], 1);
            mbar_init(&bars.drain[i], 1);
        }
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&bars.k_full[i], kLoadWarps / 2);
            mbar_init(&bars.k_empty[i], 2);
            mbar_init(&bars.v_full[i], kLoadWarps / 2);
            mbar_init(&bars.v_empty[i], 2);
        }
        for (int i = 0; i < C::kRing; ++i) mbar_init(&bars.sc_full[i], kLoadWarps);
        for (int i = 0; i < kSegments; ++i) {
            mbar_init(&bars.seg_full[i], 1);
            mbar_init(&bars.seg_empty[i], kSoftWarps + kLoadWarps + 2);
        }
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kSoftWarps + kLoadWarps) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    if constexpr (kMode == kPrefix) {
        // The groups are known once the kernel ahead has ended. Those behind may start then, so that they
        // too find what it wrote.
        pdl_wait_prior();
        pdl_launch_dependents();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = tmem_slot;

    // segment `k` of the share once it is there (a whole warp); null: no more, or a wait ran out
    auto segment = [&](int k) -> const Segment * {
        if (!warp_wait(&bars.seg_full[k % kSegments], (uint32_t)(k / kSegments) & 1u, &abort_flag, kv.err))
            return nullptr;
        const Segment *g = segs + k % kSegments;
        return g->j1 > 0 ? g : nullptr;
    };
    auto segment_done = [&](int k) {  // this warp has read all it needs of it
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.seg_empty[k % kSegments]);
    };

    if (warp < kSoftWarps) {
        // ---------------------------------------------------------------- softmax
        regs_up<kSoftRegs>();
        const int t = warp >> 2;                                   // the tile
        const int row_in_tile = threadIdx.x & 127;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 rows
        const uint32_t tS = lanes + t * 128, tO = lanes + C::kO + t * D;
        int it = 0;          // key tiles of the CTA,
        int ns = 0, nw = 0;  // key tiles and segments of this tile
        bool ok = true;
        for (int seg = 0; ok; ++seg) {
            const Segment *const w = segment(seg);
            if (!w) break;
            const int j0 = w->j0, j1 = w->j1;
            const int row_t = w->tile * kBlockRows + t * kTileRows;  // the tile's first row
            const int rows = w->n * G;
            if (row_t >= rows) {
                it += j1 - j0;
                segment_done(seg);
                continue;
            }
            if (kSoftQ && seg == 0) {
                uint8_t *const dst = smem + C::kQ + t * C::kTileBytes;
                copy_q<D>(a, w, t, row_in_tile, dst);
                cp_commit();
                cp_wait<0>();
                sign_q<D>(row_in_tile, dst, plan.q_sign);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.q_full[t]);
            }
            const int row = row_t + row_in_tile;
            const bool on = row < rows;
            const int i = on ? row / G : w->n - 1;
            const int pos = kMode == kPrefix ? w->L - 1 : w->L - w->n + i;
            const int tok_lo = w->lo;
            float m = -INFINITY, l = 0.0f;
            // raw score -> units of log2 (an 8-bit cache's keys' scales have that factor already)
            const uint64_t mul_2 = pack2(plan.scale_log2, plan.scale_log2);
            float thr = -INFINITY;  // a key above this may hold much of the row's weight so far
            for (int j = j0; j < j1; ++j, ++it, ++ns) {
                const int tok0 = tok_lo + j * kKeys;
                const int lim = pos - tok0;
                const int low = window > 0 ? pos - window - tok0 : -1;
                const bool mask = __any_sync(0xffffffffu, lim < kKeys - 1 || low >= 0);
                const int ring = it % C::kRing;
                const float *const sc = scale_ring + ring * 256;
                ok = warp_wait(&bars.s_full[t][0], (uint32_t)ns & 1u, &abort_flag, kv.err);
                // The scales second: a tile that skipped a segment has not followed sc_full, and a parity
                // tells a phase only from its neighbours. The MMA warp that made S of tile `it` has seen
                // v_full of tile it - 1, and a loading warp arrives at a tile's sc_full before it loads the
                // next: sc_full of every tile up to it - 2 is complete here.
                if (kInt8)
                    ok = ok && warp_wait(&bars.sc_full[ring], (uint32_t)(it / C::kRing) & 1u, &abort_flag, kv.err);
                if (!ok) break;
                tc_fence_after_sync();
                uint32_t s[kPart];
                tmem_ld32(tS, s);
                bool rest_half = false;
#pragma unroll 1
                for (int x = 0; x < 4; ++x) {  // 32 keys at a time
                    const int k0 = x * kPart;
                    uint64_t z[kPart / 2];
                    tmem_wait32(s);
                    float top = part_scores<kInt8>(s, sc + k0, mul_2, z);
                    if (mask) top = mask_scores(z, lim - k0, low - k0);
                    if (x == 1) {
                        ok = warp_wait(&bars.s_full[t][1], (uint32_t)ns & 1u, &abort_flag, kv.err);
                        if (!ok) break;
                        tc_fence_after_sync();
                    }
                    tmem_ld32(tS + (k0 + kPart) % kKeys, s);  // (the last one's is not used)
                    // two parts where a key may hold much of a row's weight; m is moved with the tile's
                    // first keys, and where it is far off
                    const bool rest = __any_sync(0xffffffffu, top > thr);
                    const bool far = top > m + 16.0f;
                    if (rest && (x == 0 || __any_sync(0xffffffffu, far))) {
                        const float m2 = x == 0 || far ? fmaxf(m, top) : m;
                        const float down = m == -INFINITY ? 0.0f : fast_exp2(m - m2);
                        m = m2;
                        l *= down;
                        // the product before these keys' is done
                        ok = x < 2 ? warp_wait(&bars.s_full[t][1], (uint32_t)ns & 1u, &abort_flag, kv.err)
                                   : warp_wait(&bars.pv_half[t], (uint32_t)ns & 1u, &abort_flag, kv.err);
                        if (!ok) break;
                        tc_fence_after_sync();
                        if (j > j0 || x > 1)
#pragma unroll 1
                            for (int y = 0; y < D; y += 8) scale_o(tO + y, down);
                        // weights of this half that no product has had: what another rounding takes
                        // from them is 2^-16 of less than 2^-8
                        if (x & 1)
#pragma unroll 1
                            for (int y = 0; y < kPart; y += 8) scale_p(tS + k0 - kPart + y, down);
                    }
                    const float mn = m == -INFINITY ? 0.0f : m;
                    l += kInt8 && mask ? part_weights<kInt8, kInt8>(z, tS + k0, sc + k0, mn, two_parts || rest)
                                       : part_weights<kInt8, false>(z, tS + k0, sc + k0, mn, two_parts || rest);
                    thr = mn + fminf(fast_log2(l) - 1.58496f, 16.0f);  // a third of what the row has
                    rest_half |= two_parts || rest;
                    if (x & 1) {
                        if (lane == 0)
                            reinterpret_cast<volatile uint8_t *>(&rest_flags[t][x >> 1])[warp & 3] = rest_half;
                        rest_half = false;
                        tmem_st_wait();
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars.p_full[t][x >> 1]);
                    }
                }
                tmem_wait32(s);
                if (!ok) break;
            }
            if (!ok) break;
            ok = warp_wait(&bars.o_full[t], (uint32_t)nw & 1u, &abort_flag, kv.err);
            ++nw;
            if (!ok) break;
            tc_fence_after_sync();
            const bool whole = w->whole;
            float inv = l == 0.0f ? 0.0f : 1.0f / l, prior = 0.0f;
            const int64_t out_t = w->row0 + i;
            const int h = w->head * G + (on ? row % G : 0);
            uint16_t *const dst = a.O + out_t * a.o_stride + (int64_t)h * D;
            const int first_own = w->first, w_tile = w->tile;
            const int64_t shared_row = out_t * a.Hq + h;  // of the prefix's arrays
            // the prefix's lse, kOwn
            const float P = kMode == kOwn && on && first_own > 0 ? share.lse2[shared_row] : -INFINITY;
            // A row's O is to be multiplied by join(m, l), which makes m, l the row's; the prefix's by *prior.
            auto join = [&](float &M, float &sum, float *prior) {
                float own = 1.0f;
                *prior = 0.0f;
                if constexpr (kMode == kOwn) {
                    const float top = fmaxf(M, P), ref = top == -INFINITY ? 0.0f : top;
                    const float wt = fast_exp2(P - ref);
                    own = fast_exp2(M - ref);
                    sum = fmaf(sum, own, wt);
                    M = top;
                    *prior = sum == 0.0f ? 0.0f : wt / sum;
                }
                return sum == 0.0f ? 0.0f : own / sum;
            };
            const bool joined = kMode == kOwn && first_own > 0;
            const float *const prior_o = share.O + shared_row * D;
            auto put_lse = [&](float M, float sum) {
                const float lse2 = sum == 0.0f ? -INFINITY : M + log2f(sum);
                if constexpr (kMode == kPrefix)
                    share.lse2[shared_row] = lse2;
                else if (a.lse)
                    a.lse[shared_row] = lse2 * kLn2;
            };
            if (kMode == kOwn && whole) inv = join(m, l, &prior);
            const int slot = w->slot, c0 = w->c0, c1 = w->c1;
            if constexpr (!kInt8) {
                // bad values of V: known from the loading warps, or seen in O, of which 0 O is then not 0
                // (looked for while O is written: 8 prompts of 2048 bf16 412 us, not 390)
                float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
                for (int x = 0; x < D; x += 32) {
                    uint32_t o[32];
                    tmem_ld32_wait(tO + x, o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) zero[e & 3] = fmaf(__uint_as_float(o[e]), 0.0f, zero[e & 3]);
                }
                const bool odd = on && l == l && (zero[0] + zero[1]) + (zero[2] + zero[3]) != 0.0f;
                if (__any_sync(0xffffffffu, odd || *const_cast<const volatile int *>(&w->bad)))
                    add_bad<D, kMode>(kv, b, w, G, window, on ? pos : -1, on && l == l, tO);
            }
            segment_done(seg);
            // a warp's rows of a piece: [D / 4][32][4], so that the warp writes 512 bytes at a time
            // (kPrefix: row by row, as the kernel behind reads them)
            constexpr int kPartStep = kMode == kPrefix ? 1 : 32;
            float *const all_parts = kMode == kPrefix ? share.part : plan.part;
            float *const part = all_parts + ((int64_t)slot * 8 + warp) * 32 * D + lane * (kMode == kPrefix ? D : 4);
            float2 *const part_ml =
                reinterpret_cast<float2 *>(all_parts + (int64_t)2 * gridDim.x * kBlockRows * D) + warp * 32 + lane;
            uint8_t *const out = smem + C::kOut + warp * 32 * kOutPitch;
            uint16_t *to[4];  // through shared memory (see below): the rows this lane writes a piece of
            bool to_on[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int r = y * 8 + (lane >> 2);
                to[y] = reinterpret_cast<uint16_t *>(__shfl_sync(0xffffffffu, (uint64_t)dst, r)) + (lane & 3) * 8;
                to_on[y] = row - lane + r < rows;
            }
#pragma unroll 2
            for (int x = 0; x < D; x += 32) {
                uint32_t o[32];
                tmem_ld32_wait(tO + x, o);
                if constexpr (kMode == kOwn) {
                    if (whole && on && joined) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 v = *reinterpret_cast<const float4 *>(prior_o + x + e);
                            const float u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const float mine = add_piece<kInt8>(inv, __uint_as_float(o[e + y]), 0.0f);
                                o[e + y] = __float_as_uint(add_piece<kInt8>(prior, u[y], mine));
                            }
                        }
                    } else if (whole) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
                    }
                }
                if (kMode == kPrefix && whole) {
                    if (on)
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(share.O + shared_row * D + x + e) =
                                make_float4(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv,
                                            __uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
                } else if (whole) {
                    const float mul = kMode == kOwn ? 1.0f : inv;
                    // a thread's own 16-byte stores would touch 32 rows at a time (6300 cycles a
                    // segment): four lanes a row write 64 bytes of each
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t v[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            v[y] = pack_bf16x2(__uint_as_float(o[e + 2 * y]) * mul, __uint_as_float(o[e + 2 * y + 1]) * mul);
                        *reinterpret_cast<uint4 *>(out + lane * kOutPitch + e * 2) = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint4 v =
                            *reinterpret_cast<const uint4 *>(out + (y * 8 + (lane >> 2)) * kOutPitch + (lane & 3) * 16);
                        if (to_on[y]) *reinterpret_cast<uint4 *>(to[y] + x) = v;
                    }
                    __syncwarp();
                } else if (on) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<uint4 *>(part + (x + e) * kPartStep) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
                __syncwarp();  // the next load is the whole warp's
            }
            tc_fence_before_sync();
            if (whole) {
                if (on) {
                    put_lse(m, l);
                    if constexpr (kMode == kPrefix) share.where[shared_row].x = kJoined;
                }
            } else if constexpr (kMode == kPrefix) {
                if (on) {
                    part_ml[slot * kBlockRows] = make_float2(m, l);
                    if (slot & 1)  // the first piece
                        share.where[shared_row] = make_uint2((uint32_t)c1 << 16 | (uint32_t)c0, row - w_tile * kBlockRows);
                }
            } else {
                if (on) part_ml[slot * kBlockRows] = make_float2(m, l);
                __threadfence();
                __syncwarp();
                int last = 0;
                if (lane == 0) {
                    int *const n = plan.count + c0 * 8 + warp;
                    last = atomicAdd(n, 1) == c1 - c0;
                    if (last) *n = 0;  // for the next call
                }
                last = __shfl_sync(0xffffffffu, last, 0);
                if (last && on) {
                    __threadfence();
                    float M = -INFINITY, sum = 0.0f;
#pragma unroll 4
                    for (int x = c0; x <= c1; ++x)
                        M = fmaxf(M, __ldcg(&part_ml[(2 * x + (x == c0 ? 1 : 0)) * kBlockRows].x));
                    const float Mx = M == -INFINITY ? 0.0f : M;
#pragma unroll 4
                    for (int x = c0; x <= c1; ++x) {
                        const float2 e = __ldcg(&part_ml[(2 * x + (x == c0 ? 1 : 0)) * kBlockRows]);
                        sum += fast_exp2(e.x - Mx) * e.y;
                    }
                    const float back = join(M, sum, &prior);
#pragma unroll 1
                    for (int d = 0; d < D; d += 8) {
                        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
                        for (int x = c0; x <= c1; ++x) {
                            const int sl = 2 * x + (x == c0 ? 1 : 0);
                            const float wt = fast_exp2(__ldcg(&part_ml[sl * kBlockRows].x) - Mx);
                            const float *src = plan.part + ((int64_t)sl * 8 + warp) * 32 * D + lane * 4 + d * 32;
                            const float4 v0 = __ldcg(reinterpret_cast<const float4 *>(src));
                            const float4 v1 = __ldcg(reinterpret_cast<const float4 *>(src + 128));
                            acc[0] = add_piece<kInt8>(wt, v0.x, acc[0]);
                            acc[1] = add_piece<kInt8>(wt, v0.y, acc[1]);
                            acc[2] = add_piece<kInt8>(wt, v0.z, acc[2]);
                            acc[3] = add_piece<kInt8>(wt, v0.w, acc[3]);
                            acc[4] = add_piece<kInt8>(wt, v1.x, acc[4]);
                            acc[5] = add_piece<kInt8>(wt, v1.y, acc[5]);
                            acc[6] = add_piece<kInt8>(wt, v1.z, acc[6]);
                            acc[7] = add_piece<kInt8>(wt, v1.w, acc[7]);
                        }
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            if constexpr (kMode == kOwn) {
                                acc[y] = add_piece<kInt8>(back, acc[y], 0.0f);
                                if (joined) acc[y] = add_piece<kInt8>(prior, prior_o[d + y], acc[y]);
                            } else {
                                acc[y] *= back;
                            }
                        }
                        *reinterpret_cast<uint4 *>(dst + d) =
                            make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                                       pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
                    }
                    put_lse(M, sum);
                }
                __syncwarp();
            }
        }
    } else if (warp < kSoftWarps + kLoadWarps) {
        // ------------------------------------------------- Q, K and V into shared memory
        regs_down<kLoadRegs>();
        // Warps 0 and 1 of these bring K, 2 and 3 V (the stages of the two come free at different
        // times): 64 tokens of every key tile as four 16-token groups, each of one page.
        constexpr int kGroups = 4;
        const int lw = warp - kSoftWarps;
        const bool is_v = lw >= 2;
        const int tid = threadIdx.x - kSoftWarps * 32;
        const uint32_t base = kv_opaque(0x43004300u);
        uint64_t *const full = is_v ? bars.v_full : bars.k_full, *const empty = is_v ? bars.v_empty : bars.k_empty;
        const void *const arena = is_v ? kv.v : kv.k;
        const uint16_t *const scales = is_v ? kv.vs : kv.ks;
        const float scale_mul = is_v ? 1.0f : plan.scale_log2;
        float *const scale_part = scale_ring + (is_v ? 128 : 0) + (lw & 1) * 64;
        uint8_t *const stages = smem + (is_v ? C::kV : C::kK) + (lw & 1) * 8192;
        int it = 0;
        uint32_t nq[2] = {0, 0};
        bool ok = true;
        int pr, pc;
        lane_piece<D>(lane, &pr, &pc);
        auto arrive = [&](uint64_t &bar) {  // the warp's part is in shared memory
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar);
        };

        for (int seg = 0; ok; ++seg) {
            const Segment *const w = segment(seg);
            if (!w) break;
            const int j0 = w->j0, j1 = w->j1, rows = w->n * G, head = w->head, hi = w->hi;
            const int lo = w->lo + (lw & 1) * 64;
            const int32_t *table = b.table + (int64_t)w->seq * b.table_stride;
            // cache row of the first token of the warp's group x of key tile j, and how many of the 16
            // there are
            auto group = [&](int j, int x, int *count) -> int64_t {
                const int tok = lo + j * kKeys + x * 16;
                *count = j < j1 ? min(16, max(0, hi - tok)) : 0;
                if (*count == 0) return 0;
                int page = table[tok >> kv.page_shift];
                if (page < 0 || page >= kv.num_pages) {
                    kv_flag_range(kv.err);
                    *count = 0;
                    page = 0;
                }
                return (((int64_t)page * kv.H + head) << kv.page_shift) + (tok & ((1 << kv.page_shift) - 1));
            };
            // the lane's pieces of a group of codes (zeros past its end)
            auto fetch = [&](int64_t row, int count, uint4 (&v)[D / 32]) {
                const uint8_t *src = static_cast<const uint8_t *>(arena) + (row + pr) * D + pc * 16;
#pragma unroll
                for (int p = 0; p < D / 32; ++p) {
                    v[p] = make_uint4(0, 0, 0, 0);
                    if (pr + p * (512 / D) < count) v[p] = *reinterpret_cast<const uint4 *>(src + p * 512);
                }
            };
            // bf16: straight into shared memory (rows past the end hold anything: zeros)
            auto copy = [&](uint8_t *dst, int64_t row, int count) {
                constexpr int kLanes = D / 8, kStep = 32 / kLanes;
                const uint8_t *src = static_cast<const uint8_t *>(arena) + row * (2 * D) + lane * 16;
#pragma unroll
                for (int p = 0; p < 16 / kStep; ++p) {
                    const int r = p * kStep + lane / kLanes;
                    cp_async16(smem_u32(dst + tile_off(r, lane % kLanes)), src + p * 512, r < count ? 16u : 0u);
                }
            };
            // Where not all rows see all tokens the infinities and NaN of V (bf16) become zeros: a weight
            // of 0 does not keep them out of a product.
            const int2 seen = is_v ? seen_by_all<kMode>(w, G, window) : make_int2(0, INT32_MAX);
            auto drop_bad = [&](uint8_t *dst, int j) {
                constexpr int kLanes = D / 8, kStep = 32 / kLanes;
#pragma unroll 1
                for (int x = 0; x < kGroups; ++x) {
                    const int tok0 = lo + j * kKeys + x * 16;
                    if (!edge_group(tok0, seen) || tok0 >= hi) continue;
                    auto at = [&](int p) {  // what this lane copied
                        return reinterpret_cast<uint4 *>(dst + x * 2048 +
                                                         tile_off(p * kStep + lane / kLanes, lane % kLanes));
                    };
                    uint32_t top = 0;  // a carry into a half's highest bit: an exponent of all ones
#pragma unroll
                    for (int p = 0; p < 16 / kStep; ++p) {
                        const uint4 u = *at(p);
                        top |= (u.x & 0x7F807F80u) + 0x00800080u;
                        top |= (u.y & 0x7F807F80u) + 0x00800080u;
                        top |= (u.z & 0x7F807F80u) + 0x00800080u;
                        top |= (u.w & 0x7F807F80u) + 0x00800080u;
                    }
                    if ((top & 0x80008000u) == 0) continue;
#pragma unroll 1
                    for (int p = 0; p < 16 / kStep; ++p) {
                        const uint4 u = *at(p);
                        *at(p) = make_uint4(finite_part(u.x), finite_part(u.y), finite_part(u.z), finite_part(u.w));
                    }
                    *const_cast<volatile int *>(&w->bad) = 1;
                }
            };
            int count[kGroups];
            int64_t row[kGroups];
#pragma unroll
            for (int x = 0; x < kGroups; ++x) row[x] = group(j0, x, &count[x]);
            uint4 v[kInt8 ? 2 : 1][kInt8 ? D / 32 : 1];
            if constexpr (kInt8) {
#pragma unroll
                for (int x = 0; x < 2; ++x) fetch(row[x], count[x], v[x]);
            } else {
                ok = warp_wait(&empty[it % C::kStages], ((uint32_t)(it / C::kStages) & 1u) ^ 1u, &abort_flag, kv.err);
                if (!ok) break;
                uint8_t *const dst = stages + (it % C::kStages) * C::kTileBytes;
#pragma unroll
                for (int x = 0; x < kGroups; ++x) copy(dst + x * 2048, row[x], count[x]);
                cp_commit();
            }

            // Q: copies of both tiles' rows first, so that they cost one latency
            const int nt = w->tile * kBlockRows + kTileRows < rows ? 2 : 1;
            for (int t = 0; t < nt && ok; ++t) {
                const uint32_t phase = nq[t]++;
                if (kSoftQ && seg == 0) continue;
                ok = warp_wait(&bars.q_empty[t], (phase & 1u) ^ 1u, &abort_flag, kv.err);
                if (ok) copy_q<D>(a, w, t, tid, smem + C::kQ + t * C::kTileBytes);
            }
            cp_commit();
            if (!ok) {
                cp_wait<0>();
                break;
            }
            if constexpr (!kInt8) {
                cp_wait<1>();
                drop_bad(stages + (it % C::kStages) * C::kTileBytes, j0);
                arrive(full[it % C::kStages]);
            }
            if (!kSoftQ || seg > 0) {
                cp_wait<0>();
                for (int t = 0; t < nt; ++t) {
                    sign_q<D>(tid, smem + C::kQ + t * C::kTileBytes, plan.q_sign);
                    arrive(bars.q_full[t]);
                }
            }
            segment_done(seg);
            if (!ok) break;

            for (int j = j0; j < j1; ++j, ++it) {
                const int s = it % C::kStages;
                const uint32_t ph = ((uint32_t)(it / C::kStages) & 1u) ^ 1u;
                uint8_t *const dst = stages + s * C::kTileBytes;
                if constexpr (kInt8) {
                    // scales of tokens 16 x + lane % 16, two groups at a time
                    const int x = lane >> 4, ring = it % C::kRing;
                    float sc[2];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int64_t r = x ? row[2 * y + 1] : row[2 * y];
                        sc[y] = 0.0f;
                        if ((lane & 15) < (x ? count[2 * y + 1] : count[2 * y]))
                            sc[y] = __uint_as_float((uint32_t)scales[r + (lane & 15)] << 16) * scale_mul;
                    }
                    // groups 0 and 1 of this tile are in registers; 2, 3 and the next tile's 0, 1
                    // are on their way while the two before them are converted
                    int64_t r0 = row[2], r1 = row[3];
                    int c0 = count[2], c1 = count[3];
#pragma unroll
                    for (int y = 0; y < kGroups; ++y) row[y] = group(j + 1, y, &count[y]);
                    ok = warp_wait(&empty[s], ph, &abort_flag, kv.err);
                    if (!ok) break;
#pragma unroll 1
                    for (int y = 0; y < 2; ++y) {
                        store_codes<D>(dst + y * 4096, v[0], pr, pc, base);
                        fetch(r0, c0, v[0]);
                        store_codes<D>(dst + y * 4096 + 2048, v[1], pr, pc, base);
                        fetch(r1, c1, v[1]);
                        r0 = row[0], r1 = row[1];
                        c0 = count[0], c1 = count[1];
                    }
                    scale_part[ring * 256 + lane] = sc[0];
                    scale_part[ring * 256 + 32 + lane] = sc[1];
                    arrive(full[s]);
                    if (lane == 0) mbar_arrive(&bars.sc_full[ring]);
                } else if (j > j0) {
#pragma unroll
                    for (int y = 0; y < kGroups; ++y) row[y] = group(j, y, &count[y]);
                    ok = warp_wait(&empty[s], ph, &abort_flag, kv.err);
                    if (!ok) break;
#pragma unroll
                    for (int y = 0; y < kGroups; ++y) copy(dst + y * 2048, row[y], count[y]);
                    cp_commit();
                    cp_wait<0>();
                    drop_bad(dst, j);
                    arrive(full[s]);
                }
            }
        }
        cp_wait<0>();  // (a wait that ran out may leave copies behind)
    } else {
        // -------------------------------------------------------------------- MMAs
        regs_down<kMmaRegs>();
        const int t = warp - kSoftWarps - kLoadWarps;
        if (t < 2) {
            // Tile t's products. An MMA is issued when the one before it has started, so what a warp
            // does between its MMAs (waiting for weights, commits: 600 cycles a key tile) idles the
            // tensor cores unless another warp issues meanwhile: a warp a tile.
            const uint32_t lead = lane == 0;
            const uint32_t id_s = idesc_bf16_f32(kTileRows, kHalf);
            const uint32_t id_o = idesc_bf16_f32(kTileRows, D) | (1u << 16);  // B: N along the row
            const uint64_t dq = sdesc_k_sw128(smem_u32(smem + C::kQ) + t * C::kTileBytes);
            const uint64_t dk = sdesc_k_sw128(smem_u32(smem + C::kK)), dv = sdesc_mn_sw128(smem_u32(smem + C::kV));
            constexpr uint32_t kTile16 = C::kTileBytes / 16;  // descriptors count 16-byte units
            const uint32_t tS = tmem + t * 128, tO = tmem + C::kO + t * D;
            uint32_t it = 0, np = 0, nq = 0;
            bool ok = true;
            auto commit = [&](uint64_t &bar) { commit_lead(lead, smem_u32(&bar)); };
            auto wait = [&](uint64_t &bar, uint32_t parity) {
                ok = ok && warp_wait(&bar, parity & 1u, &abort_flag, kv.err);
            };
            auto score = [&](uint32_t s, int h) {  // S = Q K^T of half h of the key tile in stage s
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint32_t off = (i >> 2) * 1024 + (i & 3) * 2;
                    mma_ss(lead, tS + h * kHalf, dq + off, dk + s * kTile16 + h * (kHalf * 8) + off, id_s, i > 0);
                }
                commit(bars.s_full[t][h]);
            };
            for (int seg = 0; ok; ++seg) {
                const Segment *const w = segment(seg);
                if (!w) break;
                const int n = __shfl_sync(0xffffffffu, w->j1 - w->j0, 0);
                const int nt = __shfl_sync(0xffffffffu, w->tile * kBlockRows + kTileRows < w->n * G ? 2 : 1, 0);
                segment_done(seg);
                if (t >= nt) {
                    // nothing to multiply: give the stages back as they fill
                    for (int j = 0; j < n && ok; ++j, ++it) {
                        const uint32_t s = it % C::kStages, ph = it / C::kStages;
                        wait(bars.k_full[s], ph);
                        if (ok && lead) mbar_arrive(&bars.k_empty[s]);
                        wait(bars.v_full[s], ph);
                        if (ok && lead) mbar_arrive(&bars.v_empty[s]);
                        __syncwarp();
                    }
                    continue;
                }
                wait(bars.k_full[it % C::kStages], it / C::kStages);
                wait(bars.q_full[t], nq++);
                if (!ok) break;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) score(it % C::kStages, h);
                commit(bars.k_empty[it % C::kStages]);
                if (n == 1) commit(bars.q_empty[t]);
#pragma unroll 1
                for (int j = 0; j < n; ++j, ++it, ++np) {
                    const uint32_t s = it % C::kStages, s1 = (it + 1) % C::kStages;
                    wait(bars.v_full[s], it / C::kStages);
                    if (j + 1 < n) wait(bars.k_full[s1], (it + 1) / C::kStages);
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        wait(bars.p_full[t][h], np);
                        if (!ok) break;
                        tc_fence_after_sync();
                        const uint32_t a = tS + h * kHalf;
                        const uint64_t b = dv + s * kTile16 + h * (kHalf * 8);
#pragma unroll
                        for (int i = 0; i < kHalf / 16; ++i) mma_ts(lead, tO, a + i * 16, b + i * 128, id_o, (j | h | i) != 0);
                        if (__any_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(&rest_flags[t][h]) != 0)) {
#pragma unroll 1
                            for (int i = 0; i < kHalf / 16; ++i)
                                mma_ts(lead, tO, a + 8 + i * 16, b + i * 128, id_o, 1);
                        }
                        if (h == 0) commit(bars.pv_half[t]);
                        if (j + 1 < n) score(s1, h);
                    }
                    if (!ok) break;
                    if (j + 1 < n) {
                        commit(bars.k_empty[s1]);
                        if (j + 2 == n) commit(bars.q_empty[t]);
                    } else {
                        commit(bars.o_full[t]);
                    }
                    commit(bars.v_empty[s]);
                    __syncwarp();
                }
            }
            // no MMA may be in flight when the tensor memory goes
            commit(bars.drain[t]);
            int unused = 0;
            small_wait(&bars.drain[t], 0, &unused, kv.err);
            __syncwarp();
        } else if (t == 2) {
            // ------------------------------------------- the share, segment by segment
            KvWork<kBlockRows, kKeys, kHeadUnits, kMode> w(kv, b, a, share, plan.min_rows, INT32_MAX, lane,
                                                           kMode != kPrefix);
            bool more = kMode == kPrefix ? w.take_begin(share.begins[blockIdx.x])
                                         : w.take_share(blockIdx.x, min((int64_t)gridDim.x, w.total));
            KvShareItem begun{-1, 0, 0, 0, 0, {0, 0, 0}};  // kPrefix: the item that begins here and ends elsewhere
            for (int seg = 0;; ++seg) {
                if (!warp_wait(&bars.seg_empty[seg % kSegments], ((uint32_t)(seg / kSegments) & 1u) ^ 1u, &abort_flag,
                               kv.err))
                    break;
                more = more && w.next();
                Segment g{};
                if (more) {
                    g.seq = kMode == kPrefix ? w.sh.lo : w.seq;
                    g.row0 = w.sh.row0;
                    g.n = w.sh.n;
                    g.L = w.sh.L;
                    g.tile = w.tile;
                    g.head = w.head;
                    g.lo = w.lo;
                    g.hi = w.hi;
                    g.j0 = w.j0;
                    g.j1 = w.j1;
                    g.whole = w.whole();
                    g.slot = 2 * blockIdx.x + (w.first() ? 1 : 0);
                    g.c0 = w.first_cta();
                    g.c1 = w.last_cta();
                    g.first = w.sh.lo;
                    if (kMode == kPrefix && !g.whole && w.first())
                        begun = KvShareItem{g.c1, g.row0, g.head, min(kBlockRows, g.n * G - g.tile * kBlockRows),
                                            g.tile * kBlockRows, {0, 0, 0}};
                }
                if (lane == 0) {
                    segs[seg % kSegments] = g;
                    mbar_arrive(&bars.seg_full[seg % kSegments]);
                }
                __syncwarp();
                if (!more) break;
            }
            if (kMode == kPrefix && lane == 0) share.items[blockIdx.x] = begun;
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kSoftWarps + kLoadWarps) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

template <KvMode kMode>
cudaError_t launch_kv_prefill_mode(const KvDev &kv, bool int8, const KvBatchDev &b, const KvAttn &a,
                                   const KvShareDev &share, int min_rows, float *part, int *count, int num_sms,
                                   cudaStream_t stream)
{
    auto launch = [&](int smem, auto *fn) {
        const cudaError_t e = ensure_smem_attr((const void *)fn, smem);
        if (e != cudaSuccess) return e;
        const Plan plan{min_rows, fabsf(a.scale) * 1.4426950408889634f, signbit(a.scale) ? 0x80008000u : 0u, part,
                        count};
        return kv_launch(kMode == kPrefix, fn, dim3(kv_prefill_grid(num_sms)), kThreads, smem, stream, kv, b, a, share,
                         plan);
    };
    if (kv.D == 128)
        return int8 ? launch(Cfg<128>::kSmem, kv_prefill_kernel<128, true, kMode>)
                    : launch(Cfg<128>::kSmem, kv_prefill_kernel<128, false, kMode>);
    return int8 ? launch(Cfg<64>::kSmem, kv_prefill_kernel<64, true, kMode>)
                : launch(Cfg<64>::kSmem, kv_prefill_kernel<64, false, kMode>);
}

}  // namespace
}  // namespace lora
