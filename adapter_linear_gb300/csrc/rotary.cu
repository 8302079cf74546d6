// rotary.cu -- rotary positions: frequencies (host), and the kernel that rotates tensors of tokens.
//
// Pair i of a head at position p turns by the angle p f_i: (x, y) -> g (x cos - y sin, x sin + y cos), g the scaling's
// factor; the other way round (inverse) with -sin. In fp32, each result rounded once to bf16.
//
// What bounds it: many tokens, HBM: a value is read and written once, and a token's angles are worked out once for all
// its heads by the lanes that hold them. Few tokens: a launch and two loads that depend on nothing but the
// position. Measured: 30011 tokens of 24 + 8 heads of 128 values, 64 of them rotated, out of a fused projection, 81 us
// (6.0 TB/s, 89 % of the copy bandwidth; before lanes' runs filled sectors and L1 was given room 95); 64 tokens
// of 32 + 8 heads 3.3 us.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "pool_state.h"
#include "launch_stream.h"
#include "rotary_device.cuh"

using namespace lora;

namespace {

struct Tensors {
    const uint16_t *in[LORA_ROTARY_MAX_TENSORS];
    uint16_t *out[LORA_ROTARY_MAX_TENSORS];
    int64_t in_stride[LORA_ROTARY_MAX_TENSORS], out_stride[LORA_ROTARY_MAX_TENSORS];
    int heads[LORA_ROTARY_MAX_TENSORS];
    int n;
};

constexpr int kBatch = 4;  // blocks loaded before any is stored

// A row is one head of one token; head_dim / 16 lanes hold one, a block is the 32 / (head_dim / 16) rows of one
// tensor that a warp holds at a time. A warp takes a chunk of tokens, or a part of one token's blocks; its lanes'
// eight angles serve all its rows of a token.
template <bool kHalf>
__global__ void __launch_bounds__(RotaryGrid::kWarps * 32, RotaryGrid::kCtas)
    rotary_kernel(const __grid_constant__ RotaryDev rot, const __grid_constant__ Tensors x, int head_dim,
                  const int32_t *positions, int T, int inverse, int parts)
{
    // Its start overlaps the end of the kernel ahead (many tokens, call after call, 84 us, so 81.5), whose results are there
    // from here on. They may be the positions, so these are not __restrict__: that would let them be read as memory that
    // nothing writes while this kernel runs.
    pdl_wait_prior();
    const int lane = threadIdx.x & 31;
    const int lanes = head_dim / 16, per = 32 / lanes;  // lanes of a row, rows of a block
    const int sub = lane / lanes, c = lane - sub * lanes;
    int all = 0;
    for (int k = 0; k < x.n; ++k) all += (x.heads[k] + per - 1) / per;
    const RotaryShare me(T, all, parts);
    int d0, d1;
    rotary_runs(rot, head_dim, c, &d0, &d1);
    const bool turns = 16 * c < rot.dim;
#pragma unroll 1
    for (int t = me.t0; t < me.t1; t += me.step) {
        Turn8 turn;
        if (turns) turn = rotary_turn<kHalf>(rot, c, positions[t], inverse);
        int first = 0;  // the tensor's first block
#pragma unroll 1
        for (int k = 0; k < x.n; ++k) {
            const int heads = x.heads[k], blocks = (heads + per - 1) / per;
            const int from = max(me.b0 - first, 0) * per, to = min((me.b1 - first) * per, heads);
            first += blocks;
            // (in place: what is not rotated is there)
            const uint16_t *const src = x.in[k] + (int64_t)t * x.in_stride[k];
            uint16_t *const dst = x.out[k] + (int64_t)t * x.out_stride[k];
            const bool on = sub < per && (turns || src != dst);
#pragma unroll 1
            for (int r0 = from + sub; r0 < to; r0 += kBatch * per) {
                uint4 v[kBatch][2];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int at = (r0 + i * per) * head_dim;
                    if (!on || r0 + i * per >= to) continue;
                    v[i][0] = *reinterpret_cast<const uint4 *>(src + at + d0);
                    v[i][1] = *reinterpret_cast<const uint4 *>(src + at + d1);
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int at = (r0 + i * per) * head_dim;
                    if (!on || r0 + i * per >= to) continue;
                    if (turns) {
                        float f[16];
                        unpack16(v[i], f);
                        rotary_pairs<kHalf>(turn, f);
                        v[i][0] = pack8(f);
                        v[i][1] = pack8(f + 8);
                    }
                    *reinterpret_cast<uint4 *>(dst + at + d0) = v[i][0];
                    *reinterpret_cast<uint4 *>(dst + at + d1) = v[i][1];
                }
            }
        }
    }
}

bool positive(double x) { return std::isfinite(x) && x > 0.0; }

constexpr double kTwoPi = 6.283185307179586476925;

}  // namespace

extern "C" {

lora_status lora_rotary_frequencies(int rotary_dim, double base, int scaling, double scale, double trained,
                                    const double *options, double *freq, double *factor)
{
    if (!freq || !factor || !positive(base)) return LORA_ERR_ARG;
    if (scaling < LORA_ROTARY_PLAIN || scaling > LORA_ROTARY_BANDS) return LORA_ERR_ARG;
    if (rotary_dim < 16 || rotary_dim > LORA_ROTARY_MAX_DIM || rotary_dim % 16 != 0) return LORA_ERR_SHAPE;
    if (scaling != LORA_ROTARY_PLAIN && !positive(scale)) return LORA_ERR_ARG;
    const bool yarn = scaling == LORA_ROTARY_YARN, bands = scaling == LORA_ROTARY_BANDS;
    double o0 = yarn ? 32.0 : 1.0, o1 = yarn ? 1.0 : 4.0;
    if (yarn || bands) {
        if (!positive(trained)) return LORA_ERR_ARG;
        if (options) {
            o0 = options[0];
            o1 = options[1];
        }
        if (!positive(o0) || !positive(o1) || (yarn ? o0 <= o1 : o0 >= o1)) return LORA_ERR_ARG;
        if (yarn && base <= 1.0) return LORA_ERR_ARG;
    }
    const int R = rotary_dim;
    if (scaling == LORA_ROTARY_NTK) base *= std::pow(scale, (double)R / (R - 2));
    // pair at which a model of this base turns `turns` times over the trained context
    auto pair_of = [&](double turns) { return R * std::log(trained / (kTwoPi * turns)) / (2.0 * std::log(base)); };
    double low = 0.0, high = 0.0;
    if (yarn) {
        low = std::fmax(std::floor(pair_of(o0)), 0.0);
        high = std::fmin(std::ceil(pair_of(o1)), R - 1.0);
        if (high <= low) high = low + 0.001;
    }
    *factor = yarn && scale > 1.0 ? 0.1 * std::log(scale) + 1.0 : 1.0;
    for (int i = 0; i < R / 2; ++i) {
        double f = std::pow(base, -2.0 * i / R);
        if (scaling == LORA_ROTARY_LINEAR) f /= scale;
        if (yarn) {
            const double far = std::fmin(std::fmax((i - low) / (high - low), 0.0), 1.0);
            f = f / scale * far + f * (1.0 - far);
        }
        if (bands) {
            const double turns = trained * f / kTwoPi;
            const double near = std::fmin(std::fmax((turns - o0) / (o1 - o0), 0.0), 1.0);
            f = f / scale * (1.0 - near) + f * near;
        }
        freq[i] = f;
    }
    return LORA_OK;
}

lora_status lora_rotary_init(int rotary_dim, int layout, const double *freq, double factor, lora_rotary *out)
{
    if (!freq || !out || !std::isfinite(factor) || !std::isfinite((float)factor)) return LORA_ERR_ARG;
    if (layout != LORA_ROTARY_HALF && layout != LORA_ROTARY_INTERLEAVED) return LORA_ERR_ARG;
    if (rotary_dim < 16 || rotary_dim > LORA_ROTARY_MAX_DIM || rotary_dim % 16 != 0) return LORA_ERR_SHAPE;
    for (int i = 0; i < rotary_dim / 2; ++i)
        if (!std::isfinite(freq[i])) return LORA_ERR_ARG;
    lora_rotary r = {};
    r.rotary_dim = rotary_dim;
    r.layout = layout;
    r.factor = (float)factor;
    for (int i = 0; i < rotary_dim / 2; ++i) {
        // (of the magnitude, whose fraction is exact: that of a small negative number would lose its last bits beside 1)
        double turns = std::fabs(freq[i]) / kTwoPi;
        turns -= std::floor(turns);
        const uint64_t step = (uint64_t)std::ldexp(turns, 64);
        r.step[i] = freq[i] < 0.0 ? 0 - step : step;
    }
    *out = r;
    return LORA_OK;
}

lora_status lora_rotary_apply(const lora_rotary *rotary, int n, const lora_rotary_tensor *tensors, int head_dim,
                              const int32_t *positions, int T, int inverse, lora_stream_t stream)
{
    if (!rotary_ok(rotary) || !tensors || n < 1 || n > LORA_ROTARY_MAX_TENSORS || T < 0 || T > (1 << 30))
        return LORA_ERR_ARG;
    if (head_dim < rotary->rotary_dim || head_dim > LORA_ROTARY_MAX_DIM || head_dim % 16 != 0) return LORA_ERR_SHAPE;
    Tensors x = {};
    for (int i = 0; i < LORA_ROTARY_MAX_TENSORS; ++i) {
        if (i < n) {
            const lora_rotary_tensor &a = tensors[i];
            if (a.heads < 1 || a.heads > 65536) return LORA_ERR_ARG;
            const int64_t row = (int64_t)a.heads * head_dim;
            if (T > 0 && (!a.in || !a.out)) return LORA_ERR_ARG;
            if ((reinterpret_cast<uintptr_t>(a.in) | reinterpret_cast<uintptr_t>(a.out)) & 15) return LORA_ERR_ARG;
            if (a.in_stride < row || a.out_stride < row || a.in_stride % 8 != 0 || a.out_stride % 8 != 0)
                return LORA_ERR_ARG;
            if (a.in == a.out && a.in_stride != a.out_stride) return LORA_ERR_ARG;
            x.in[i] = static_cast<const uint16_t *>(a.in);
            x.out[i] = static_cast<uint16_t *>(a.out);
            x.in_stride[i] = a.in_stride;
            x.out_stride[i] = a.out_stride;
            x.heads[i] = a.heads;
        }
    }
    x.n = n;
    if (T == 0) return LORA_OK;
    if (!positions || (reinterpret_cast<uintptr_t>(positions) & 3)) return LORA_ERR_ARG;
    int dev = 0;
    CUDA_TRY(cudaGetDevice(&dev));
    // multiprocessors of the devices asked about so far; -1: not a device of ours
    static std::atomic<int> known[64];
    int sms = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (sms == 0) {
        int major = 0, minor = 0;
        CUDA_TRY(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev));
        CUDA_TRY(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev));
        CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
        if (major != 10 || minor != 3) sms = -1;
        if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
    }
    if (sms < 0) return LORA_ERR_UNSUPPORTED;
    auto *const fn = rotary->layout == LORA_ROTARY_HALF ? rotary_kernel<true> : rotary_kernel<false>;
    const int per = 32 / (head_dim / 16);
    int64_t all = 0;  // blocks of a token
    for (int i = 0; i < n; ++i) all += (x.heads[i] + per - 1) / per;
    const RotaryGrid g(T, all, sms);
    CUDA_TRY(launch_stream(g.streams, true, fn, g.ctas, RotaryGrid::kWarps * 32, stream, rotary_view(rotary), x, head_dim,
                           positions, T, (int)(inverse != 0), g.parts));
    return LORA_OK;
}

}  // extern "C"
