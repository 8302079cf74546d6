// kv_decode.cu -- attention of short chunks (single tokens above all) over the paged cache.
//
// For a row at position pos and its visible keys j:
//   z_j = scale <Q, K_j>,  m = max z_j,  l = sum exp(z_j - m),  O = sum exp(z_j - m) V_j / l,
// in one pass with a running m (z is kept in units of log2: exp(x) = 2^(x log2 e)). Sets of
// keys combine: (m, l, O) of two sets become M = max m, sums weighted by 2^(m - M); so the keys
// of one head are split over warps, and over CTAs, and joined at the end.
//
// What bounds it: HBM. A single-token step reads every cached byte once for G = Hq / Hkv query
// heads: 2 G flops a byte of an 8-bit cache. The products run as warp-level MMAs with the cache
// as the 16-row operand, S^T = K Q^T and O^T = V^T P^T, so that the G heads (times the chunk's
// tokens) fill tiles of 8 columns: half the instructions, accumulators and softmax of the other
// way round, where 4 heads would leave 12 of 16 rows idle. What is left is issue slots for
// turning codes into bf16, about half of all instructions with an 8-bit cache.
//
// Split: the work is the list of items (sequence, row tile, kv head), each a run of 64-token
// units; the grid's CTAs take equal contiguous shares of all units together, whatever the
// lengths, so no SM waits for the longest sequence. A CTA's share covers some whole items
// and up to two pieces; a piece's (m, l, O) goes to scratch, and the CTA that finishes an item
// last (a counter) joins its pieces in CTA order: the result does not depend on which one it is.
// Inside a CTA the four warps take 16-token steps in turn, each streaming its own codes through
// its own ring of shared memory with 16-byte asynchronous copies: no barrier until an item ends.
//
// Measured, calls one after another, 32 query heads on 8 kv heads of 128 values: 64 requests of one
// token over 17 to 8191 tokens, 8-bit, 100 us (5.5 TB/s); 256 requests over 500 to 4095, bf16, 366 us
// (6.6 TB/s, 98 % of the copy bandwidth); 32 requests of 3 to 6 tokens over 300 to 6000, 8-bit, 82 us
// (2.7 TB/s: three row tiles' accumulators leave 8 warps an SM, which wait for their own arithmetic); one
// request over 2047 tokens 11 us on the GPU (loads that depend on one another: lengths, pages, codes, then the
// join).
#include <climits>
#include <type_traits>

#include "kv_device.cuh"

namespace lora {
namespace {

constexpr int kWarps = 4;
constexpr int kStep = 16;            // tokens per warp step: never crosses a page (pages hold 16 k)
constexpr int kUnit = kWarps * kStep;
// An item's cost beside its units, in units: 32 8-bit drafts 85 us at 2, 81 at 3, 79 at 4, 64 requests of
// one token 99 at each.
constexpr int kHeadUnits = 4;
constexpr int kMinUnits = 2;         // one request, one token: 11.2 us at 1, 11.0 at 2, 11.6 at 4

constexpr int kMaxCtas = 4;    // CTAs an SM, of any variant
constexpr int kPartRows = 48;  // and the rows that those of one SM hold

// kN: tiles of 8 rows (a row: one query head of one new token) an item holds.
template <int D, bool kInt8, int kN>
struct Cfg {
    static constexpr int kRows = 8 * kN;
    static constexpr int kRowBytes = D * (kInt8 ? 1 : 2);
    static constexpr int kTile = kStep * kRowBytes;              // K or V of a step
    static constexpr int kStage = 2 * kTile + 4 * kStep;         // K, V, then both scales
    static constexpr bool kWide = kRowBytes == 256;
    // 4 CTAs of 50 KB an SM (3 of 66 KB where two row tiles take the registers, 2 for three, which
    // spill at 3: 104 us against 81 for 32 drafts; rows of 256 bytes: 2 of 98 KB): 100 to
    // 150 KB in flight beside the stages in use. (Two row tiles of an 8-bit cache, D = 128: 16 bytes a thread
    // spill; the others none.)
    static constexpr int kStages = kWide || kN == 1 ? 3 : 4;
    static constexpr int kCtas = kWide || kN == 3 ? 2 : kN == 1 ? 4 : 3;
    static constexpr int kRing = kStages * kStage;
    static constexpr int kSmem = kWarps * kRing;
    static constexpr int kLdO = D + 4;                           // fp32 row of O in shared memory
    static constexpr int kMaxGrid = kSmem / (4 * kRows);         // pieces whose weights fit the rings
    static_assert(kRing >= kRows * kLdO * 4, "O of a warp is parked in its ring");
    static_assert(kCtas * kRows <= kPartRows && kCtas <= kMaxCtas, "scratch of an SM's CTAs");
};

// Byte offset of 16-byte chunk c of row r in a tile. The chunks of a 128-byte line are permuted
// by the row so that the lanes of a phase of a shared load fall into different banks: for K two
// neighbouring rows with four chunks each, for V rows 2 c with two chunks each.
template <int kRowBytes>
__device__ __forceinline__ uint32_t swz(int r, int c)
{
    if (kRowBytes == 64)  // two rows a line
        return (uint32_t)((r >> 1) * 128 + (((((r & 1) << 2) + c) ^ (((r >> 1) & 3) << 1)) << 4));
    // rows of 256 bytes: two halves of 128-byte rows, one after the other
    return (uint32_t)((c >> 3) * (kStep * 128) + r * 128 + (((c & 7) ^ (((r & 1) << 2) | ((r >> 1) & 3))) << 4));
}

// V's chunk (of the 8 of a 128-byte row) that the lanes of group g read
__device__ __forceinline__ int v_chunk(int g) { return ((g & 1) << 2) + (g >> 1); }

// D += A B, 16 x 8 x 16, fp32 sums; bf16 operands (mma16816) or f16 ones (mma16816_f16)
__device__ __forceinline__ void mma16816_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit values, a row over four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

struct Plan {
    int max_rows;        // takes the sequences of at most this many rows (n G)
    float scale_log2;    // scale * log2(e)
    float *part;         // [2 grid][rows][D] + [2 grid][rows][2] (m, l)
    int *count;          // [grid] arrivals at the item that starts in that CTA and ends in another
};

// A warp's steps of an item, nk of them from token `tok`, for the first kT tiles of its rows, and
// then their O into the ring and (m, l) into sm_m and sm_l. issue() starts the copy of the next step.
// v_row(j): V of token j < tok_end, which the table names (for an unquantised cache's bad values).
template <int D, bool kInt8, int kN, int kT, class Issue, class Row>
__device__ __forceinline__ void run_steps(Issue &issue, Row &v_row, int nk, int tok, int tok_end, int window, int rows,
                                          int pos_min, int pos_max, uint32_t base, uint8_t *ring,
                                          const uint4 (&sm_q)[kN][D / 32][32], const float *sm_back, const int *sm_pos,
                                          float *sm_m, float *sm_l)
{
    using C = Cfg<D, kInt8, kN>;
    constexpr int kM = D / 16;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    // of the rows this lane has scores of: 8 t + 2 c, + 1
    float back_mul[kT][2];
#pragma unroll
    for (int t = 0; t < kT; ++t) {
        back_mul[t][0] = sm_back[8 * t + 2 * c];
        back_mul[t][1] = sm_back[8 * t + 2 * c + 1];
    }
    float o[kT][kM][4];
    float m[kT][2], l[kT][2];
#pragma unroll
    for (int t = 0; t < kT; ++t) {
#pragma unroll
        for (int i = 0; i < kM; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[t][i][e] = 0.0f;
        m[t][0] = m[t][1] = -INFINITY;
        l[t][0] = l[t][1] = 0.0f;
    }

    bool bad = false;  // V had an infinity or a NaN that was left out of the product
    int stage = 0;
    const int tok_first = tok;
    for (int k = 0; k < nk; ++k, tok += kStep * kWarps) {
        cp_wait<C::kStages - 2>();
        __syncwarp();
        const uint8_t *st = ring + stage * C::kStage;
        stage = stage + 1 == C::kStages ? 0 : stage + 1;

        // S^T = K Q^T: rows are tokens g and g + 8, columns the query rows
        float s[kT][4];
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[t][e] = 0.0f;
#pragma unroll
        for (int x = 0; x < C::kRowBytes / 64; ++x) {
            const uint4 w0 = *reinterpret_cast<const uint4 *>(st + swz<C::kRowBytes>(g, 4 * x + c));
            const uint4 w1 = *reinterpret_cast<const uint4 *>(st + swz<C::kRowBytes>(g + 8, 4 * x + c));
            const uint32_t u0[4] = {w0.x, w0.y, w0.z, w0.w}, u1[4] = {w1.x, w1.y, w1.z, w1.w};
            if constexpr (kInt8) {
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    uint32_t u[2][4];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        codes4_to_f16(u0[j + y], &u[y][0], &u[y][2]);
                        codes4_to_f16(u1[j + y], &u[y][1], &u[y][3]);
                    }
#pragma unroll
                    for (int t = 0; t < kT; ++t) {
                        const uint4 q = sm_q[t][2 * x + j / 2][lane];
                        mma16816_f16(s[t], u[0][0], u[0][1], u[0][2], u[0][3], q.x, q.y);
                        mma16816_f16(s[t], u[1][0], u[1][1], u[1][2], u[1][3], q.z, q.w);
                    }
                }
            } else {
#pragma unroll
                for (int t = 0; t < kT; ++t) {
                    const uint4 q = sm_q[t][x][lane];
                    mma16816(s[t], u0[0], u1[0], u0[1], u1[1], q.x, q.y);
                    mma16816(s[t], u0[2], u1[2], u0[3], u1[3], q.z, q.w);
                }
            }
        }

        // z in units of log2, masked; s[t][2 y + e]: token g + 8 y, row 8 t + 2 c + e
        float ks[2] = {1.0f, 1.0f}, vs[2] = {1.0f, 1.0f};
        if (kInt8) {
            const uint16_t *sc = reinterpret_cast<const uint16_t *>(st + 2 * C::kTile);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                ks[y] = __uint_as_float((uint32_t)sc[g + 8 * y] << 16);
                vs[y] = __uint_as_float((uint32_t)sc[16 + g + 8 * y] << 16);
            }
        }
        const bool edge = tok + kStep - 1 > pos_min || (window > 0 && tok <= pos_max - window);
        bool grow = false;
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    s[t][2 * y + e] *= back_mul[t][e];
                    if (kInt8) s[t][2 * y + e] *= ks[y];
                    if (edge) {
                        const int j = tok + g + 8 * y, p = sm_pos[8 * t + 2 * c + e];
                        const bool see = j <= p && (window == 0 || j > p - window);
                        s[t][2 * y + e] = see ? s[t][2 * y + e] : -INFINITY;
                    }
                }
                grow |= fmaxf(s[t][e], s[t][2 + e]) > m[t][e] + 8.0f;
            }

        // The maximum only has to be near the true one: O and l are rescaled when a key passes
        // it by 2^8 (weights then reach 256, which changes nothing about their precision).
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int t = 0; t < kT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = fmaxf(s[t][e], s[t][2 + e]);
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    v = fmaxf(v, m[t][e]);
                    const float down = m[t][e] == -INFINITY ? 0.0f : fast_exp2(m[t][e] - v);
                    m[t][e] = v;
                    l[t][e] *= down;
#pragma unroll
                    for (int i = 0; i < kM; ++i) {
                        o[t][i][e] *= down;
                        o[t][i][2 + e] *= down;
                    }
                }
        }
        // Weights: summed in fp32, and for the product with V a pair of bf16, the rounded weight
        // and the rest (together off by 2^-16 of it: one bf16 alone, 2^-8, shows in rows that see few
        // keys, and HBM leaves the tensor cores the time). An 8-bit cache's V scale is
        // multiplied in first; a masked key's weight is 0 whatever its scale is.
        uint32_t p[kT][2], p2[kT][2];
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float w[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float z = s[t][2 * y + e];
                    w[e] = fast_exp2(z - (m[t][e] == -INFINITY ? 0.0f : m[t][e]));
                    l[t][e] += w[e];
                    if (kInt8) w[e] = z == -INFINITY ? 0.0f : w[e] * vs[y];
                }
                const uint32_t top = pack_bf16x2(w[0], w[1]);
                p[t][y] = transpose8x8(top);
                p2[t][y] = transpose8x8(pack_bf16x2(w[0] - bf16_lo(top), w[1] - bf16_hi(top)));
            }

        // O^T += V^T P^T: a lane reads its dims of tokens 2 c, 2 c + 1, 2 c + 8, 2 c + 9; dims
        // 2 i and 2 i + 1 of them are rows g and g + 8 of MMA i
        const uint8_t *vt = st + C::kTile;
        if constexpr (kInt8) {
            uint32_t w[4][D / 32];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 2 * c + (r & 1) + 8 * (r >> 1);
                if constexpr (D == 128) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(vt + swz<C::kRowBytes>(row, v_chunk(g)));
                    w[r][0] = v.x;
                    w[r][1] = v.y;
                    w[r][2] = v.z;
                    w[r][3] = v.w;
                } else {
                    const uint2 v =
                        *reinterpret_cast<const uint2 *>(vt + swz<C::kRowBytes>(row, g >> 1) + (g & 1) * 8);
                    w[r][0] = v.x;
                    w[r][1] = v.y;
                }
            }
#pragma unroll
            for (int i = 0; i < kM; ++i) {
                const int x = i >> 1, y = 2 * (i & 1);
                const uint32_t a0 = codes_pair_to_bf16(w[0][x], w[1][x], y, base);
                const uint32_t a1 = codes_pair_to_bf16(w[0][x], w[1][x], y + 1, base);
                const uint32_t a2 = codes_pair_to_bf16(w[2][x], w[3][x], y, base);
                const uint32_t a3 = codes_pair_to_bf16(w[2][x], w[3][x], y + 1, base);
#pragma unroll
                for (int t = 0; t < kT; ++t) {
                    mma16816(o[t][i], a0, a1, a2, a3, p[t][0], p[t][1]);
                    mma16816(o[t][i], a0, a1, a2, a3, p2[t][0], p2[t][1]);
                }
            }
        } else {
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
                uint32_t w[4][4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 2 * c + (r & 1) + 8 * (r >> 1);
                    const uint4 v =
                        *reinterpret_cast<const uint4 *>(vt + swz<C::kRowBytes>(row, 8 * x + v_chunk(g)));
                    w[r][0] = v.x;
                    w[r][1] = v.y;
                    w[r][2] = v.z;
                    w[r][3] = v.w;
                }
                if (edge) {  // not all rows see all of these tokens
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t f = finite_part(w[r][i]);
                            bad |= f != w[r][i];
                            w[r][i] = f;
                        }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a0 = __byte_perm(w[0][i], w[1][i], 0x5410);
                    const uint32_t a1 = __byte_perm(w[0][i], w[1][i], 0x7632);
                    const uint32_t a2 = __byte_perm(w[2][i], w[3][i], 0x5410);
                    const uint32_t a3 = __byte_perm(w[2][i], w[3][i], 0x7632);
#pragma unroll
                    for (int t = 0; t < kT; ++t) {
                        mma16816(o[t][4 * x + i], a0, a1, a2, a3, p[t][0], p[t][1]);
                        mma16816(o[t][4 * x + i], a0, a1, a2, a3, p2[t][0], p2[t][1]);
                    }
                }
            }
        }
        __syncwarp();
        issue();
    }
    cp_wait<0>();
    __syncwarp();

#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 4);
            l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 8);
            l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 16);
        }
    if constexpr (!kInt8) {
        // 0 O is 0 for a finite O; a row whose weights are NaN is NaN as it is
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float zero = 0.0f;
#pragma unroll
                for (int i = 0; i < kM; ++i) zero = fmaf(o[t][i][e], 0.0f, fmaf(o[t][i][2 + e], 0.0f, zero));
                bad |= zero != 0.0f && l[t][e] == l[t][e];
            }
        if (__any_sync(0xffffffffu, bad)) {
            // once to clear what the product made of them, once to add them up
#pragma unroll 1
            for (int pass = 0; pass < 2; ++pass)
#pragma unroll 1
                for (int y = 0; y < nk * kStep; ++y) {
                    const int j = tok_first + y % kStep + y / kStep * (kStep * kWarps);
                    if (j >= tok_end) break;
                    const uint16_t *const row = v_row(j);
#pragma unroll
                    for (int x = 0; x < D / 64; ++x) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(row + 64 * x + 8 * v_chunk(g));
                        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int t = 0; t < kT; ++t)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int p = sm_pos[8 * t + 2 * c + e];
                                if (j > p || (window > 0 && j <= p - window)) continue;
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const uint32_t f = u[i] ^ finite_part(u[i]);
                                    float &lo = o[t][4 * x + i][e], &hi = o[t][4 * x + i][2 + e];
                                    if (f & 0xFFFFu) lo = pass == 0 ? 0.0f : lo + bf16_lo(f);
                                    if (f >> 16) hi = pass == 0 ? 0.0f : hi + bf16_hi(f);
                                }
                            }
                    }
                }
        }
    }

    // ---- join the warps: O in the warp's ring, (m, l) beside it
    float *so = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 8 * t + 2 * c + e;
            if (g == 0) {
                sm_m[r] = m[t][e];
                sm_l[r] = l[t][e];
            }
            // MMA i, rows g and g + 8: dims d + 2 i and d + 2 i + 1 (bf16: of each 64-dim half)
            if (r < rows)
#pragma unroll
                for (int i = 0; i < kM; i += 2) {
                    const int d = kInt8 ? (D == 128 ? 16 * v_chunk(g) : 8 * g) + 2 * i
                                        : 64 * (i / 4) + 8 * v_chunk(g) + 2 * (i % 4);
                    *reinterpret_cast<float4 *>(so + r * C::kLdO + d) =
                        make_float4(o[t][i][e], o[t][i][2 + e], o[t][i + 1][e], o[t][i + 1][2 + e]);
                }
        }
}

template <int D, bool kInt8, int kN>
__global__ void __launch_bounds__(kWarps * 32, Cfg<D, kInt8, kN>::kCtas)
    kv_decode_kernel(KvDev kv, KvBatchDev b, KvAttn a, Plan plan)
{
    using C = Cfg<D, kInt8, kN>;
    constexpr int R = C::kRows;
    constexpr int kM = D / 16;                    // MMAs of 16 dimensions
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float sm_m[kWarps][R], sm_l[kWarps][R], sm_w[kWarps][R], sm_lse[R];
    __shared__ float sm_back[R];
    __shared__ int sm_pos[R];
    __shared__ uint4 sm_q[kN][kM / 2][32];  // [tile][pair of MMAs][lane]: the same for all warps
    __shared__ int sm_last;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int G = a.G;

    KvWork<R, kUnit, kHeadUnits> w(kv, b, a, 0, plan.max_rows, lane);
    // a CTA takes kMinUnits units at least: more pieces of an item cost more to join than
    // they save
    if (!w.take_share(blockIdx.x, min((int64_t)gridDim.x, (w.total + kMinUnits - 1) / kMinUnits))) return;

    const uint32_t base = kv_opaque(0x43004300u);
    uint8_t *const ring = smem + warp * C::kRing;
    const uint32_t ring_addr = smem_u32(ring);
    // this lane's part of a copy: chunks lane + 32 x of a tile
    constexpr int kChunks = C::kRowBytes / 16, kCopies = C::kTile / 512;
    uint32_t dst[kCopies];
#pragma unroll
    for (int x = 0; x < kCopies; ++x)
        dst[x] = ring_addr + swz<C::kRowBytes>((lane + 32 * x) / kChunks, (lane + 32 * x) % kChunks);

    while (w.next()) {
        const KvSeq &sh = w.sh;
        const int seq = w.seq, tile = w.tile, head = w.head;
        const int tok0 = w.lo + w.j0 * kUnit, tok1 = min(w.hi, w.lo + w.j1 * kUnit);
        const int rows = min(R, sh.n * G - tile * R);

        // ---- this warp's steps: tokens tok0 + 16 (warp + 4 k)
        const int nk = max(0, (tok1 - tok0 + kStep - 1) / kStep - warp + kWarps - 1) / kWarps;
        int page_cache = 0;  // lane i: the page of step (k & ~31) + i
        const int32_t *table = b.table + (int64_t)seq * b.table_stride;
        int fill_k = 0, fill_stage = 0;  // the next step to copy and its stage
        auto issue = [&]() {
            const int k = fill_k++;
            if (k < nk) {
                if ((k & 31) == 0) {
                    page_cache = 0;
                    if (k + lane < nk) {
                        page_cache = table[(tok0 + kStep * (warp + kWarps * (k + lane))) >> kv.page_shift];
                        if (page_cache < 0 || page_cache >= kv.num_pages) {
                            kv_flag_range(kv.err);
                            page_cache = 0;
                        }
                    }
                }
                const int page = __shfl_sync(0xffffffffu, page_cache, k & 31);
                const int tok = tok0 + kStep * (warp + kWarps * k);
                const int64_t row = (((int64_t)page * kv.H + head) << kv.page_shift) +
                                    (tok & ((1 << kv.page_shift) - 1));
                const uint32_t st = fill_stage * C::kStage;
                const uint8_t *ksrc = static_cast<const uint8_t *>(kv.k) + row * C::kRowBytes + lane * 16;
                const uint8_t *vsrc = static_cast<const uint8_t *>(kv.v) + row * C::kRowBytes + lane * 16;
                if (tok + kStep <= sh.L) {
#pragma unroll
                    for (int x = 0; x < kCopies; ++x) {
                        cp_async16(dst[x] + st, ksrc + x * 512, 16u);
                        cp_async16(dst[x] + st + C::kTile, vsrc + x * 512, 16u);
                    }
                } else {
                    // rows past the sequence's end hold anything: zeros in their place
#pragma unroll
                    for (int x = 0; x < kCopies; ++x) {
                        const uint32_t bytes = tok + (lane + 32 * x) / kChunks < sh.L ? 16u : 0u;
                        cp_async16(dst[x] + st, ksrc + x * 512, bytes);
                        cp_async16(dst[x] + st + C::kTile, vsrc + x * 512, bytes);
                    }
                }
                if (kInt8 && lane < 4)
                    cp_async16(ring_addr + st + 2 * C::kTile + lane * 16,
                               reinterpret_cast<const uint8_t *>((lane < 2 ? kv.ks : kv.vs) + row) + (lane & 1) * 16,
                               16u);
                fill_stage = fill_stage + 1 == C::kStages ? 0 : fill_stage + 1;
            }
            cp_commit();
        };
        auto v_row = [&](int j) {  // (a bad page: the same stand-in as above)
            int page = table[j >> kv.page_shift];
            if (page < 0 || page >= kv.num_pages) page = 0;
            return static_cast<const uint16_t *>(kv.v) +
                   ((((int64_t)page * kv.H + head) << kv.page_shift) + (j & ((1 << kv.page_shift) - 1))) * D;
        };
#pragma unroll
        for (int k = 0; k < C::kStages - 1; ++k) issue();

        // Q as the 8-column operand, a tile a warp: lane (g, c) holds row g of it; its dims of MMA i
        // are those its K words hold (8-bit: 64-dim blocks of 16 dims a lane; bf16: 32-dim blocks of 8)
        static_assert(kN <= kWarps, "a tile a warp");
        if (warp < kN) {
            const int row = tile * R + 8 * warp + g;
            const bool on = 8 * warp + g < rows;
            const int i = row / G;
            const uint16_t *src = a.Q + (int64_t)(sh.row0 + i) * a.q_stride + (int64_t)(head * G + row % G) * D;
            constexpr int kBlock = kInt8 ? 64 : 32, kLane = kBlock / 4;
            uint4 q[kM / 2];
#pragma unroll
            for (int x = 0; x < kM / 2; ++x) {
                q[x] = make_uint4(0, 0, 0, 0);
                if (on) q[x] = ldg_nc_v4(src + (x / (kLane / 8)) * kBlock + c * kLane + (x % (kLane / 8)) * 8);
            }
            // An 8-bit cache's codes become f16 in two thirds of the instructions bf16 takes, so Q
            // becomes f16 too, its row scaled by the power of two that puts the largest magnitude
            // into [2^14, 2^15): values down to 2^-28 of that keep all their bits, and the
            // rest are off by at most 2^-39 of it.
            float back = 1.0f;
            if (kInt8) {
                uint32_t top = 0;
#pragma unroll
                for (int x = 0; x < kM / 2; ++x) {
                    const uint32_t v[4] = {q[x].x, q[x].y, q[x].z, q[x].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = max(top, max(v[e] & 0x7FFFu, (v[e] >> 16) & 0x7FFFu));
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int up = min(14 + 127 - (int)(top >> 7), 126);  // bf16's exponent field
                const float mul = __uint_as_float((uint32_t)(127 + up) << 23);
                back = __uint_as_float((uint32_t)(127 - up) << 23);
                auto f16 = [&](uint32_t v) {
                    const __half2 h = __floats2half2_rn(bf16_lo(v) * mul, bf16_hi(v) * mul);
                    return *reinterpret_cast<const uint32_t *>(&h);
                };
#pragma unroll
                for (int x = 0; x < kM / 2; ++x) q[x] = make_uint4(f16(q[x].x), f16(q[x].y), f16(q[x].z), f16(q[x].w));
            }
#pragma unroll
            for (int x = 0; x < kM / 2; ++x) sm_q[warp][x][lane] = q[x];
            if (c == 0) {
                sm_back[8 * warp + g] = back * plan.scale_log2;  // to units of log2
                // rows beyond the tile: any position, not written
                sm_pos[8 * warp + g] = on ? sh.L - sh.n + i : sh.L - 1;
            }
        }
        __syncthreads();
        const int pos_min = sh.L - sh.n + tile * R / G, pos_max = sh.L - sh.n + (tile * R + rows - 1) / G;
        // one tile where the item's rows fit it (40 requests of 7 heads, 37 of them of one token: 99 us
        // with all tiles, 93 with one)
        auto run = [&](auto tiles) {
            run_steps<D, kInt8, kN, decltype(tiles)::value>(issue, v_row, nk, tok0 + kStep * warp, tok1, a.window, rows,
                                                            pos_min, pos_max, base, ring, sm_q, sm_back, sm_pos,
                                                            sm_m[warp], sm_l[warp]);
        };
        if (rows <= 8)
            run(std::integral_constant<int, 1>());
        else
            run(std::integral_constant<int, kN>());
        __syncthreads();
        const bool whole = w.whole();
        const int slot = 2 * blockIdx.x + (w.first() ? 1 : 0);
        float *part_o = plan.part + (int64_t)slot * R * D;
        float *part_ml = plan.part + (int64_t)2 * gridDim.x * R * D + slot * 2 * R;
        if (threadIdx.x < R) {
            const int r = threadIdx.x;
            float M = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int x = 0; x < kWarps; ++x) M = fmaxf(M, sm_m[x][r]);
            const float Mx = M == -INFINITY ? 0.0f : M;
#pragma unroll
            for (int x = 0; x < kWarps; ++x) {
                const float wt = fast_exp2(sm_m[x][r] - Mx);
                sm_w[x][r] = wt;
                sum += wt * sm_l[x][r];
            }
            if (whole) {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
                for (int x = 0; x < kWarps; ++x) sm_w[x][r] *= inv;
                sm_lse[r] = sum == 0.0f ? -INFINITY : (M + log2f(sum)) * kLn2;
            } else {
                part_ml[2 * r] = M;
                part_ml[2 * r + 1] = sum;
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < rows * (D / 4); i += kWarps * 32) {
            const int r = i / (D / 4), d = (i % (D / 4)) * 4;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int x = 0; x < kWarps; ++x) {
                const float4 v = *reinterpret_cast<const float4 *>(
                    reinterpret_cast<const float *>(smem + x * C::kRing) + r * C::kLdO + d);
                const float wt = sm_w[x][r];
                acc.x = add_piece<kInt8>(wt, v.x, acc.x);
                acc.y = add_piece<kInt8>(wt, v.y, acc.y);
                acc.z = add_piece<kInt8>(wt, v.z, acc.z);
                acc.w = add_piece<kInt8>(wt, v.w, acc.w);
            }
            if (whole) {
                const int row = tile * R + r;
                const int64_t t = sh.row0 + row / G;
                const int h = head * G + row % G;
                *reinterpret_cast<uint2 *>(a.O + t * a.o_stride + (int64_t)h * D + d) =
                    make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
                if (d == 0 && a.lse) a.lse[t * a.Hq + h] = sm_lse[r];
            } else {
                *reinterpret_cast<float4 *>(part_o + r * D + d) = acc;
            }
        }

        // ---- a piece of an item: the last CTA to arrive joins the pieces
        if (!whole) {
            const int c0 = w.first_cta(), c1 = w.last_cta();
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) {
                const int n = atomicAdd(&plan.count[c0], 1);
                sm_last = n == c1 - c0;
                if (sm_last) plan.count[c0] = 0;  // for the next call
            }
            __syncthreads();
            if (sm_last) {
                __threadfence();
                // the pieces' weights first (into the rings), then their O: two rounds of
                // independent loads, not one load after another
                const float *ml = plan.part + (int64_t)2 * gridDim.x * R * D;
                float *wt = reinterpret_cast<float *>(smem);  // [piece][R]
                const int n = c1 - c0 + 1;                    // at most kMaxGrid
                for (int i = threadIdx.x; i < n * R; i += kWarps * 32) {
                    const int x = i / R, r = i % R;
                    wt[i] = __ldcg(ml + (2 * (c0 + x) + (x == 0 ? 1 : 0)) * 2 * R + 2 * r);
                }
                __syncthreads();
                // a row's maximum and weights by one warp: rows warp, warp + 4, ...
                for (int r = warp; r < R; r += kWarps) {
                    float M = -INFINITY, sum = 0.0f;
                    for (int x = lane; x < n; x += 32) M = fmaxf(M, wt[x * R + r]);
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
                    const float Mx = M == -INFINITY ? 0.0f : M;
                    for (int x = lane; x < n; x += 32) {
                        const float w = fast_exp2(wt[x * R + r] - Mx);
                        sum += w * __ldcg(ml + (2 * (c0 + x) + (x == 0 ? 1 : 0)) * 2 * R + 2 * r + 1);
                        wt[x * R + r] = w;
                    }
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                    if (lane == 0) {
                        sm_w[0][r] = sum == 0.0f ? 0.0f : 1.0f / sum;
                        sm_lse[r] = sum == 0.0f ? -INFINITY : (M + log2f(sum)) * kLn2;
                    }
                }
                __syncthreads();
                for (int i = threadIdx.x; i < rows * (D / 4); i += kWarps * 32) {
                    const int r = i / (D / 4), d = (i % (D / 4)) * 4;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    const float *src = plan.part + r * D + d;
#pragma unroll 8
                    for (int x = 0; x < n; ++x) {
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(
                            src + (int64_t)(2 * (c0 + x) + (x == 0 ? 1 : 0)) * R * D));
                        const float w = wt[x * R + r];
                        acc.x = add_piece<kInt8>(w, v.x, acc.x);
                        acc.y = add_piece<kInt8>(w, v.y, acc.y);
                        acc.z = add_piece<kInt8>(w, v.z, acc.z);
                        acc.w = add_piece<kInt8>(w, v.w, acc.w);
                    }
                    const float inv = sm_w[0][r];
                    const int row = tile * R + r;
                    const int64_t t = sh.row0 + row / G;
                    const int h = head * G + row % G;
                    *reinterpret_cast<uint2 *>(a.O + t * a.o_stride + (int64_t)h * D + d) =
                        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
                    if (d == 0 && a.lse) a.lse[t * a.Hq + h] = sm_lse[r];
                }
            }
        }
        __syncthreads();  // the rings and the small arrays are free again
    }
}

}  // namespace

int kv_decode_grid(int num_sms) { return kMaxCtas * num_sms; }

// two pieces a CTA
size_t kv_decode_part_floats(int D, int num_sms) { return (size_t)2 * kPartRows * num_sms * (D + 2); }

cudaError_t launch_kv_decode(const KvDev &kv, bool int8, const KvBatchDev &b, const KvAttn &a, int max_new,
                             int max_rows, float *part, int *count, int num_sms, cudaStream_t stream)
{
    auto launch = [&](auto cfg, auto *fn) {
        using C = decltype(cfg);
        const cudaError_t e = ensure_smem_attr((const void *)fn, C::kSmem);
        if (e != cudaSuccess) return e;
        const Plan plan{max_rows, a.scale * 1.4426950408889634f, part, count};
        fn<<<min(C::kCtas * num_sms, C::kMaxGrid), kWarps * 32, C::kSmem, stream>>>(kv, b, a, plan);
        return cudaGetLastError();
    };
    const int64_t rows = (int64_t)max_new * a.G;
    auto pick = [&](auto d, auto i8) {
        constexpr int D = decltype(d)::value;
        constexpr bool kInt8 = decltype(i8)::value;
        if (rows <= 8) return launch(Cfg<D, kInt8, 1>(), kv_decode_kernel<D, kInt8, 1>);
        if (rows <= 16) return launch(Cfg<D, kInt8, 2>(), kv_decode_kernel<D, kInt8, 2>);
        return launch(Cfg<D, kInt8, 3>(), kv_decode_kernel<D, kInt8, 3>);
    };
    using std::integral_constant;
    if (kv.D == 128)
        return int8 ? pick(integral_constant<int, 128>(), std::true_type())
                    : pick(integral_constant<int, 128>(), std::false_type());
    return int8 ? pick(integral_constant<int, 64>(), std::true_type())
                : pick(integral_constant<int, 64>(), std::false_type());
}

}  // namespace lora
