// kv_prefill.cu -- attention of longer chunks over the paged cache: the products on the tcgen05
// tensor cores.
//
// For a row (one query head of one new token) at position pos and its visible keys j:
//   z_j = scale <Q, K_j>,  m >= max z_j - 8,  l = sum 2^(z_j - m),  O = sum 2^(z_j - m) V_j / l
// (z in units of log2), over tiles of 128 keys in one pass. m is any number near the maximum: it
// cancels in O / l, so it is only moved, and O rescaled, when a score passes it by 2^8.
//
// A CTA works on 256 rows of one kv head: the G query heads that share it for 256 / G tokens, so
// K and V are read once for all of them, as two MMA tiles of 128 rows. Warps 0-3 and 4-7 do the
// softmax of one tile each (a thread holds a row), 8-11 bring K and V tiles into shared memory
// (8-bit codes become bf16 on the way), warp 12 issues the MMAs:
//   S_t = Q_t K^T  (both operands in shared memory, S in tensor memory, 128 columns a tile)
//   O_t += P_t V   (P, the bf16 weights, written by the softmax over S; O in tensor memory)
// in the order PV_0(j) S_0(j+1) PV_1(j) S_1(j+1): while one tile's softmax runs, the tensor cores
// do the other tile's products. MMAs of one thread execute in order, so S_t(j+1) overwrites
// P_t(j) only after PV_t(j) has read it, and the commit behind S_t(j+1) covers PV_t(j).
//
// The scales of an 8-bit cache stay outside the products: the codes are exact in bf16, a
// key's scale multiplies its column of S, a value's its weight.
//
// Work is shared out like the short-chunk kernel's: the grid's CTAs (one an SM) take equal
// contiguous runs of 128-token units over all items, pieces of an item go to scratch as
// (m, l, O), and the warp that finishes a piece of 32 rows last joins them in CTA order.
#include "kv_device.cuh"

namespace lora {
namespace {

constexpr int kBlockRows = 256, kTileRows = 128, kKeys = 128;
constexpr int kSoftWarps = 8, kLoadWarps = 4;
constexpr int kThreads = (kSoftWarps + kLoadWarps + 4) * 32;  // the MMA warp's group has three idle warps
// registers a thread of the softmax warps, the loading warps and the MMA warp's group: a block of
// 512 threads starts with 128 each, and 2 x 168 + 104 + 72 is 4 x 128
constexpr int kSoftRegs = 168, kLoadRegs = 104, kMmaRegs = 72;
static_assert(2 * kSoftRegs + kLoadRegs + kMmaRegs <= 4 * 128, "register split");
// rows that see fewer keys than this get weights in two bf16 parts (see below)
constexpr int kFewKeys = 128;

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
    static constexpr int kScales = kV + kStages * kTileBytes;  // float [2][kRing][128]
    static constexpr int kBars = kScales + 2 * kRing * 128 * 4;
    static constexpr int kSmem = kBars + 512 + 1024;           // and room to align to 1024
    static constexpr uint32_t kO = 256;                        // tensor memory column of O_0
};

struct Bars {
    uint64_t q_full[2], q_empty[2], k_full[4], k_empty[4], v_full[4], v_empty[4], sc_full[6], s_full[2],
        p_full[2], o_full[2], drain;
};
static_assert(sizeof(Bars) <= 512, "barriers");

struct Plan {
    int min_rows;
    float scale_log2;
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

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
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

// A wait of a whole warp: every lane waits (and so sees what the barrier released), and all
// agree on whether it ran out.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *err)
{
    return __all_sync(0xffffffffu, mbar_wait_inl(bar, parity, abort_flag, err));
}

// The scores of N keys of this thread's row: z in units of log2, -inf where the row does not see
// the key (columns above lim or up to low).
template <bool kInt8, int N>
__device__ __forceinline__ void chunk_z(const uint32_t *s, const float *sc, float c, bool mask, int lim, int low,
                                        int col0, float (&z)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        uint64_t c01, c23;
        if (kInt8) {
            const float4 f = *reinterpret_cast<const float4 *>(sc + col0 + i);
            c01 = pack2(f.x, f.y);
            c23 = pack2(f.z, f.w);
        } else {
            c01 = c23 = pack2(c, c);
        }
        unpack2(mul2(pack2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), c01), &z[i], &z[i + 1]);
        unpack2(mul2(pack2(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), c23), &z[i + 2], &z[i + 3]);
    }
    if (mask) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = col0 + i <= lim && col0 + i > low ? z[i] : -INFINITY;
    }
}

// z becomes the weights 2^(z - m) times the values' scales (0 for a key the row does not see,
// whatever its scale is); returns the weights' sum.
template <bool kInt8, int N>
__device__ __forceinline__ float chunk_w(float (&z)[N], float m, const float *vsc, bool mask, int col0)
{
    const uint64_t neg = pack2(-m, -m);
    uint64_t sum = 0;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        unpack2(add2(pack2(z[i], z[i + 1]), neg), &z[i], &z[i + 1]);
        z[i] = fast_exp2(z[i]);
        z[i + 1] = fast_exp2(z[i + 1]);
        sum = add2(sum, pack2(z[i], z[i + 1]));
    }
    if (kInt8) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(vsc + col0 + i);
            float v[4];
            unpack2(mul2(pack2(z[i], z[i + 1]), pack2(f.x, f.y)), &v[0], &v[1]);
            unpack2(mul2(pack2(z[i + 2], z[i + 3]), pack2(f.z, f.w)), &v[2], &v[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) z[i + e] = mask && z[i + e] == 0.0f ? 0.0f : v[e];
        }
    }
    float a, b;
    unpack2(sum, &a, &b);
    return a + b;
}

template <int D, bool kInt8>
__global__ void __launch_bounds__(kThreads, 1) kv_prefill_kernel(KvDev kv, KvBatchDev b, KvAttn a, Plan plan)
{
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars &bars = *reinterpret_cast<Bars *>(smem + C::kBars);
    float *const kscale = reinterpret_cast<float *>(smem + C::kScales);
    float *const vscale = kscale + C::kRing * 128;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = a.G;
    KvWork<kBlockRows, kKeys> w(kv, b, G, a.window, plan.min_rows, INT32_MAX, lane);
    if (!w.take_share(blockIdx.x, min((int64_t)gridDim.x, w.total))) return;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.q_full[i], kLoadWarps * 32);
            mbar_init(&bars.q_empty[i], 1);
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.p_full[i], kTileRows);
            mbar_init(&bars.o_full[i], 1);
        }
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&bars.k_full[i], kLoadWarps * 32);
            mbar_init(&bars.k_empty[i], 1);
            mbar_init(&bars.v_full[i], kLoadWarps * 32);
            mbar_init(&bars.v_empty[i], 1);
        }
        for (int i = 0; i < C::kRing; ++i) mbar_init(&bars.sc_full[i], kLoadWarps * 32);
        mbar_init(&bars.drain, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kSoftWarps + kLoadWarps) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = tmem_slot;

    if (warp < kSoftWarps) {
        // ---------------------------------------------------------------- softmax
        regs_up<kSoftRegs>();
        const int t = warp >> 2;                                   // the tile
        const int row_in_tile = threadIdx.x & 127;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 rows
        const uint32_t tS = lanes + t * 128, tO = lanes + C::kO + t * D;
        int it = 0, ns = 0, nw = 0;  // key tiles of all work, of this tile's, and its work
        bool ok = true;
        while (ok && w.next()) {
            const int j0 = (int)(w.u - w.item0), j1 = (int)(w.seg_end - w.item0);
            const int row_t = w.tile * kBlockRows + t * kTileRows;  // the tile's first row
            const int64_t rows = (int64_t)w.sh.n * G;
            if (row_t >= rows) {
                it += j1 - j0;
                continue;
            }
            const int row = row_t + row_in_tile;
            const bool on = row < rows;
            const int i = on ? row / G : w.sh.n - 1;
            const int pos = w.sh.L - w.sh.n + i;
            // Rows that see few keys: a weight rounded to bf16 is off by up to 2^-8, which shows
            // where few of them add up. Their weights go to the product as a rounded part and
            // the rest.
            const int first_pos = w.sh.L - w.sh.n + row_t / G;
            const bool few = first_pos + 1 < kFewKeys || (a.window > 0 && a.window < kFewKeys);
            float m = -INFINITY, l = 0.0f;
            for (int j = j0; j < j1; ++j, ++it, ++ns) {
                const int tok0 = w.lo + j * kKeys;
                const int lim = pos - tok0;
                const int low = a.window > 0 ? pos - a.window - tok0 : -1;
                const bool mask = __any_sync(0xffffffffu, lim < kKeys - 1 || low >= 0);
                const float *ksc = kscale + (it % C::kRing) * 128, *vsc = vscale + (it % C::kRing) * 128;
                if (kInt8)
                    ok = warp_wait(&bars.sc_full[it % C::kRing], (uint32_t)(it / C::kRing) & 1u, &abort_flag,
                                   kv.err);
                ok = ok && warp_wait(&bars.s_full[t], (uint32_t)ns & 1u, &abort_flag, kv.err);
                if (!ok) break;
                tc_fence_after_sync();
                uint32_t p[64];
                // the scores of the tile against m; where one passes it by 2^8 (always in a
                // piece's first tile): m moves, O and l follow, and once more
                bool again = j == j0 || few;
                float top = -INFINITY;
                if (again) {
#pragma unroll 1
                    for (int ch = 0; ch < 4; ++ch) {
                        uint32_t s[32];
                        float z[32];
                        tmem_ld32_wait(tS + ch * 32, s);
                        chunk_z<kInt8, 32>(s, ksc, plan.scale_log2, mask, lim, low, ch * 32, z);
#pragma unroll
                        for (int e = 0; e < 32; ++e) top = fmaxf(top, z[e]);
                    }
                }
                float add = 0.0f;
#pragma unroll 1
                for (;;) {
                    if (again) {
                        const float m2 = fmaxf(m, top);
                        const float down = m == -INFINITY ? 0.0f : fast_exp2(m - m2);
                        if (j > j0 && __any_sync(0xffffffffu, m2 > m)) {
                            l *= down;
#pragma unroll 1
                            for (int x = 0; x < D; x += 32) {
                                uint32_t o[32];
                                tmem_ld32_wait(tO + x, o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * down);
                                tmem_st16(tO + x, o);
                                tmem_st16(tO + x + 16, o + 16);
                            }
                            tmem_st_wait();
                        }
                        m = m2;
                    }
                    if (few) break;
                    const float mx = m == -INFINITY ? 0.0f : m;
                    add = 0.0f;
                    top = -INFINITY;
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch) {
                        uint32_t s[32];
                        float z[32];
                        tmem_ld32_wait(tS + ch * 32, s);
                        chunk_z<kInt8, 32>(s, ksc, plan.scale_log2, mask, lim, low, ch * 32, z);
#pragma unroll
                        for (int e = 0; e < 32; ++e) top = fmaxf(top, z[e]);
                        add += chunk_w<kInt8, 32>(z, mx, vsc, mask, ch * 32);
#pragma unroll
                        for (int e = 0; e < 16; ++e) p[ch * 16 + e] = pack_bf16x2(z[2 * e], z[2 * e + 1]);
                    }
                    again = __any_sync(0xffffffffu, top > m + 8.0f);
                    if (!again) break;
                }
                if (!few) {
#pragma unroll
                    for (int x = 0; x < 64; x += 16) tmem_st16(tS + x, p + x);
                } else {
                    // the rounded parts to columns 0..63, the rests to 64..127: the scores
                    // these overwrite are read first
                    const float mx = m == -INFINITY ? 0.0f : m;
                    uint32_t s[64];
                    tmem_ld32_wait(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(s));
                    tmem_ld32_wait(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
#pragma unroll
                    for (int ch = 0; ch < 8; ++ch) {
                        uint32_t x[16], hi[8], rest[8];
                        float z[16];
                        if (ch < 4) tmem_ld16_wait(tS + ch * 16, x);
                        chunk_z<kInt8, 16>(ch < 4 ? x : s + (ch & 3) * 16, ksc, plan.scale_log2, mask, lim, low, ch * 16,
                                           z);
                        add += chunk_w<kInt8, 16>(z, mx, vsc, mask, ch * 16);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            hi[e] = pack_bf16x2(z[2 * e], z[2 * e + 1]);
                            rest[e] = pack_bf16x2(z[2 * e] - bf16_lo(hi[e]), z[2 * e + 1] - bf16_hi(hi[e]));
                        }
                        tmem_st8(tS + ch * 8, hi);
                        tmem_st8(tS + 64 + ch * 8, rest);
                    }
                }
                l += add;
                tmem_st_wait();
                tc_fence_before_sync();
                mbar_arrive(&bars.p_full[t]);
            }
            if (!ok) break;
            ok = warp_wait(&bars.o_full[t], (uint32_t)nw & 1u, &abort_flag, kv.err);
            ++nw;
            if (!ok) break;
            tc_fence_after_sync();
            const bool whole = w.whole();
            const int64_t out_t = w.sh.row0 + i;
            const int h = w.head * G + (on ? row % G : 0);
            uint16_t *const dst = a.O + out_t * a.o_stride + (int64_t)h * D;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const int slot = 2 * blockIdx.x + (w.u == w.item0 ? 1 : 0);
            // a warp's rows of a piece: [D / 4][32][4], so that the warp writes 512 bytes at a time
            float *const part = plan.part + ((int64_t)slot * 8 + warp) * 32 * D + lane * 4;
            float2 *const part_ml =
                reinterpret_cast<float2 *>(plan.part + (int64_t)2 * gridDim.x * kBlockRows * D) + warp * 32 + lane;
#pragma unroll 1
            for (int x = 0; x < D; x += 32) {
                uint32_t o[32];
                tmem_ld32_wait(tO + x, o);
                if (whole) {
                    if (on) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint32_t v[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                v[y] = pack_bf16x2(__uint_as_float(o[e + 2 * y]) * inv,
                                                   __uint_as_float(o[e + 2 * y + 1]) * inv);
                            *reinterpret_cast<uint4 *>(dst + x + e) = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                    }
                } else if (on) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<uint4 *>(part + (x + e) * 32) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
            }
            tc_fence_before_sync();
            if (whole) {
                if (on && a.lse)
                    a.lse[out_t * a.Hq + h] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
            } else {
                if (on) part_ml[slot * kBlockRows] = make_float2(m, l);
                const int c0 = w.cta_of(w.item0), c1 = w.cta_of(w.item0 + w.nu - 1);
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
                    const float back = sum == 0.0f ? 0.0f : 1.0f / sum;
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
                            acc[0] = fmaf(wt, v0.x, acc[0]);
                            acc[1] = fmaf(wt, v0.y, acc[1]);
                            acc[2] = fmaf(wt, v0.z, acc[2]);
                            acc[3] = fmaf(wt, v0.w, acc[3]);
                            acc[4] = fmaf(wt, v1.x, acc[4]);
                            acc[5] = fmaf(wt, v1.y, acc[5]);
                            acc[6] = fmaf(wt, v1.z, acc[6]);
                            acc[7] = fmaf(wt, v1.w, acc[7]);
                        }
                        *reinterpret_cast<uint4 *>(dst + d) =
                            make_uint4(pack_bf16x2(acc[0] * back, acc[1] * back), pack_bf16x2(acc[2] * back, acc[3] * back),
                                       pack_bf16x2(acc[4] * back, acc[5] * back), pack_bf16x2(acc[6] * back, acc[7] * back));
                    }
                    if (a.lse) a.lse[out_t * a.Hq + h] = sum == 0.0f ? -INFINITY : (M + log2f(sum)) * kLn2;
                }
                __syncwarp();
            }
        }
    } else if (warp < kSoftWarps + kLoadWarps) {
        // ------------------------------------------------- Q, K and V into shared memory
        regs_down<kLoadRegs>();
        const int lw = warp - kSoftWarps;
        const int tid = threadIdx.x - kSoftWarps * 32;
        const uint32_t base = kv_opaque(0x43004300u);
        int it = 0, nw[2] = {0, 0};
        bool ok = true;
        // 8-bit: a thread holds 16 codes of a row (two chunks of bf16); bf16: one chunk
        constexpr int kRowLanes = kInt8 ? D / 16 : D / 8;
        constexpr int kPassRows = kLoadWarps * 32 / kRowLanes, kPasses = kKeys / kPassRows;
        int cl, rl;  // lane -> 16-byte piece of a row, row of the warp's: a phase of eight lanes
                     // stores to eight different chunk columns
        if (kInt8 && D == 128) {
            cl = (lane & 3) | ((lane >> 1) & 4);
            rl = ((lane >> 2) & 1) | ((lane >> 3) & 2);
        } else {
            cl = lane % kRowLanes;
            rl = lane / kRowLanes;
        }
        const int r0 = lw * (32 / kRowLanes) + rl;  // the thread's rows: r0 + kPassRows * pass

        while (ok && w.next()) {
            const int j0 = (int)(w.u - w.item0), j1 = (int)(w.seg_end - w.item0);
            const int64_t rows = (int64_t)w.sh.n * G;
            const int32_t *table = b.table + (int64_t)w.seq * b.table_stride;

            // lane i < 8: cache row of token 16 i of key tile j (head's), or -1
            auto group_rows = [&](int j) -> int64_t {
                const int tok = w.lo + j * kKeys + lane * 16;
                if (lane >= 8 || tok >= w.hi) return -1;
                const int page = table[tok >> kv.page_shift];
                if (page < 0 || page >= kv.num_pages) {
                    kv_flag_range(kv.err);
                    return -1;
                }
                return (((int64_t)page * kv.H + w.head) << kv.page_shift) + (tok & ((1 << kv.page_shift) - 1));
            };
            // cache row of row r of the tile, or -1 past the end
            auto cache_row = [&](int64_t groups, int j, int r) -> int64_t {
                const int64_t g0 = __shfl_sync(0xffffffffu, groups, r >> 4);
                return g0 < 0 || w.lo + j * kKeys + r >= w.hi ? -1 : g0 + (r & 15);
            };
            int64_t groups = group_rows(j0);

            // Q: the tiles' rows, 8 (D 64: 16) at a time
            for (int t = 0; t < 2 && ok; ++t) {
                const int row_t = w.tile * kBlockRows + t * kTileRows;
                if (row_t >= rows) break;
                ok = warp_wait(&bars.q_empty[t], ((uint32_t)nw[t] & 1u) ^ 1u, &abort_flag, kv.err);
                if (!ok) break;
                ++nw[t];
                constexpr int kLanesQ = D / 8, kRowsQ = 128 / kLanesQ;
#pragma unroll 8
                for (int x = 0; x < kTileRows / kRowsQ; ++x) {
                    const int r = x * kRowsQ + tid / kLanesQ, ch = tid % kLanesQ;
                    const int row = row_t + r;
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (row < rows)
                        v = ldg_nc_v4(a.Q + (int64_t)(w.sh.row0 + row / G) * a.q_stride +
                                      (int64_t)(w.head * G + row % G) * D + ch * 8);
                    *reinterpret_cast<uint4 *>(smem + C::kQ + t * C::kTileBytes + tile_off(r, ch)) = v;
                }
                fence_proxy_async_smem();
                mbar_arrive(&bars.q_full[t]);
            }
            if (!ok) break;

            // one operand's tile: `rows_of` its cache rows
            auto load_store = [&](const void *arena, uint8_t *dst, int64_t grp, int j) {
#pragma unroll
                for (int p0 = 0; p0 < kPasses; p0 += 8) {
                    uint4 v[8 < kPasses ? 8 : kPasses];
#pragma unroll
                    for (int p = 0; p < 8 && p < kPasses; ++p) {
                        const int64_t row = cache_row(grp, j, r0 + (p0 + p) * kPassRows);
                        v[p] = make_uint4(0, 0, 0, 0);
                        if (row >= 0)
                            v[p] = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(arena) +
                                                                    row * (D * (kInt8 ? 1 : 2)) + cl * 16);
                    }
                    if (p0 == 0) {
                        // the stage, once the MMAs that read it are done (the caller's barrier)
                        ok = ok && warp_wait(dst < smem + C::kV ? &bars.k_empty[it % C::kStages]
                                                                : &bars.v_empty[it % C::kStages],
                                             ((uint32_t)(it / C::kStages) & 1u) ^ 1u, &abort_flag, kv.err);
                        if (!ok) return;
                    }
#pragma unroll
                    for (int p = 0; p < 8 && p < kPasses; ++p) {
                        const int r = r0 + (p0 + p) * kPassRows;
                        if (kInt8) {
                            uint4 x, y;
                            codes4_to_bf16(v[p].x, base, &x.x, &x.y);
                            codes4_to_bf16(v[p].y, base, &x.z, &x.w);
                            codes4_to_bf16(v[p].z, base, &y.x, &y.y);
                            codes4_to_bf16(v[p].w, base, &y.z, &y.w);
                            *reinterpret_cast<uint4 *>(dst + tile_off(r, 2 * cl)) = x;
                            *reinterpret_cast<uint4 *>(dst + tile_off(r, 2 * cl + 1)) = y;
                        } else {
                            *reinterpret_cast<uint4 *>(dst + tile_off(r, cl)) = v[p];
                        }
                    }
                }
            };

            for (int j = j0; j < j1 && ok; ++j, ++it) {
                const int s = it % C::kStages;
                const int64_t ahead = j + 1 < j1 ? group_rows(j + 1) : -1;
                if (kInt8) {
                    const int64_t row = cache_row(groups, j, tid);
                    float ks = 0.0f, vs = 0.0f;
                    if (row >= 0) {
                        ks = __uint_as_float((uint32_t)kv.ks[row] << 16) * plan.scale_log2;
                        vs = __uint_as_float((uint32_t)kv.vs[row] << 16);
                    }
                    ok = warp_wait(&bars.k_empty[s], ((uint32_t)(it / C::kStages) & 1u) ^ 1u, &abort_flag, kv.err);
                    if (!ok) break;
                    kscale[(it % C::kRing) * 128 + tid] = ks;
                    vscale[(it % C::kRing) * 128 + tid] = vs;
                    mbar_arrive(&bars.sc_full[it % C::kRing]);
                }
                load_store(kv.k, smem + C::kK + s * C::kTileBytes, groups, j);
                if (!ok) break;
                fence_proxy_async_smem();
                mbar_arrive(&bars.k_full[s]);
                load_store(kv.v, smem + C::kV + s * C::kTileBytes, groups, j);
                if (!ok) break;
                fence_proxy_async_smem();
                mbar_arrive(&bars.v_full[s]);
                groups = ahead;
            }
        }
    } else {
        // -------------------------------------------------------------------- MMAs
        regs_down<kMmaRegs>();
        if (warp == kSoftWarps + kLoadWarps) {
        const uint32_t id_s = idesc_bf16_f32(kTileRows, kKeys);
        const uint32_t id_o = idesc_bf16_f32(kTileRows, D) | (1u << 16);  // B: N along the row
        const uint32_t sq = smem_u32(smem + C::kQ), sk = smem_u32(smem + C::kK), sv = smem_u32(smem + C::kV);
        int it = 0, np[2] = {0, 0}, nw[2] = {0, 0};
        bool ok = true;
        while (ok && w.next()) {
            const int n = (int)(w.seg_end - w.u);
            const int64_t rows = (int64_t)w.sh.n * G;
            const int nt = w.tile * (int64_t)kBlockRows + kTileRows < rows ? 2 : 1;
            bool few[2];
            for (int t = 0; t < 2; ++t) {
                const int first_pos = w.sh.L - w.sh.n + (w.tile * kBlockRows + t * kTileRows) / G;
                few[t] = first_pos + 1 < kFewKeys || (a.window > 0 && a.window < kFewKeys);
            }
            // S_t = Q_t K^T of key tile `at`
            auto scores = [&](int t, int at) {
                if (lane == 0) {
                    const int s = at % C::kStages;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_bf16_ss(tmem + t * 128,
                                    sdesc_k_sw128(sq + t * C::kTileBytes + (k >> 2) * 16384 + (k & 3) * 32),
                                    sdesc_k_sw128(sk + s * C::kTileBytes + (k >> 2) * 16384 + (k & 3) * 32), id_s, k > 0);
                    mma_commit(&bars.s_full[t]);
                }
                __syncwarp();
            };
            ok = warp_wait(&bars.k_full[it % C::kStages], (uint32_t)(it / C::kStages) & 1u, &abort_flag, kv.err);
            for (int t = 0; t < nt && ok; ++t) {
                ok = warp_wait(&bars.q_full[t], (uint32_t)nw[t] & 1u, &abort_flag, kv.err);
                if (!ok) break;
                tc_fence_after_sync();
                scores(t, it);
                if (n == 1 && lane == 0) mma_commit(&bars.q_empty[t]);
            }
            if (!ok) break;
            if (lane == 0) mma_commit(&bars.k_empty[it % C::kStages]);
            for (int j = 0; j < n && ok; ++j, ++it) {
                const int s = it % C::kStages;
                for (int t = 0; t < nt && ok; ++t) {
                    if (t == 0)
                        ok = warp_wait(&bars.v_full[s], (uint32_t)(it / C::kStages) & 1u, &abort_flag, kv.err);
                    ok = ok && warp_wait(&bars.p_full[t], (uint32_t)np[t] & 1u, &abort_flag, kv.err);
                    if (!ok) break;
                    ++np[t];
                    tc_fence_after_sync();
                    if (lane == 0) {
#pragma unroll
                        for (int k = 0; k < kKeys / 16; ++k)
                            mma_bf16_ts(tmem + C::kO + t * D, tmem + t * 128 + k * 8,
                                        sdesc_mn_sw128(sv + s * C::kTileBytes + k * 2048), id_o, (j | k) != 0);
                        if (few[t]) {
#pragma unroll
                            for (int k = 0; k < kKeys / 16; ++k)
                                mma_bf16_ts(tmem + C::kO + t * D, tmem + t * 128 + 64 + k * 8,
                                            sdesc_mn_sw128(sv + s * C::kTileBytes + k * 2048), id_o, 1);
                        }
                        if (t == nt - 1) mma_commit(&bars.v_empty[s]);
                        if (j == n - 1) mma_commit(&bars.o_full[t]);
                    }
                    __syncwarp();
                    if (j + 1 < n) {
                        const int s1 = (it + 1) % C::kStages;
                        if (t == 0) {
                            ok = warp_wait(&bars.k_full[s1], (uint32_t)((it + 1) / C::kStages) & 1u, &abort_flag, kv.err);
                            if (!ok) break;
                            tc_fence_after_sync();
                        }
                        scores(t, it + 1);
                        if (lane == 0) {
                            if (j + 2 == n) mma_commit(&bars.q_empty[t]);
                            if (t == nt - 1) mma_commit(&bars.k_empty[s1]);
                        }
                        __syncwarp();
                    }
                }
            }
            for (int t = 0; t < nt; ++t) ++nw[t];
        }
        // no MMA may be in flight when the tensor memory goes
        if (lane == 0) {
            mma_commit(&bars.drain);
            int unused = 0;
            mbar_wait_inl(&bars.drain, 0, &unused, kv.err);
        }
        __syncwarp();
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kSoftWarps + kLoadWarps) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

int kv_prefill_grid(int num_sms) { return num_sms; }

size_t kv_prefill_part_floats(int D, int num_sms)
{
    return (size_t)2 * kv_prefill_grid(num_sms) * kBlockRows * (D + 2);
}

cudaError_t launch_kv_prefill(const KvDev &kv, bool int8, const KvBatchDev &b, const KvAttn &a, int min_rows,
                              float *part, int *count, int num_sms, cudaStream_t stream)
{
    auto launch = [&](int smem, auto *fn) {
        const cudaError_t e = ensure_smem_attr((const void *)fn, smem);
        if (e != cudaSuccess) return e;
        const Plan plan{min_rows, a.scale * 1.4426950408889634f, part, count};
        fn<<<kv_prefill_grid(num_sms), kThreads, smem, stream>>>(kv, b, a, plan);
        return cudaGetLastError();
    };
    if (kv.D == 128)
        return int8 ? launch(Cfg<128>::kSmem, kv_prefill_kernel<128, true>)
                    : launch(Cfg<128>::kSmem, kv_prefill_kernel<128, false>);
    return int8 ? launch(Cfg<64>::kSmem, kv_prefill_kernel<64, true>)
                : launch(Cfg<64>::kSmem, kv_prefill_kernel<64, false>);
}

}  // namespace lora
