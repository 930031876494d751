// Rotary positions on rows of heads, and the frequency tables they use.
//
// Pair (a, b) number i of a head at position p turns by the angle p f_i:
//   y_a = g (x_a cos - x_b sin),  y_b = g (x_b cos + x_a sin),
// the backward by the opposite angle (the transpose of the same map).
//
// Angles.  p f_i reaches 10^6 radians and more, where a float32 product is off
// by 0.06 radians.  The table therefore holds f_i / (2 pi), the turns per
// position, as a 64-bit binary fraction of a turn; p times that, modulo 2^64,
// is the exact angle of the rounded frequency modulo whole turns (whole turns
// fall off the top), off by at most p 2^-65 turns.  Its upper 32 bits, as a
// signed fraction of half a turn, go to sincospif.
#include <algorithm>
#include <cmath>

#include "chained.cuh"
#include "checks.h"
#include "device_common.cuh"
#include "operators.h"

namespace zbk {

namespace {

constexpr int kRotThreads = 128;
constexpr int kRotMaxPairs = 512;
constexpr int kRotUnroll = 4;  // heads whose loads a thread issues together
constexpr int kRotHeads = 8;   // heads a thread takes, about

struct RotaryArgs {
    const uint16_t* x;
    uint16_t* y;
    int64_t ld_x, ld_y;
    const int32_t* positions;
    const uint64_t* turns;
    float magnitude;
    int tokens, n_heads, head_dim, rot;
    int columns, groups;  // 16-element columns of a head; threads that share a column's heads
    int64_t threads;
    float sign;  // +1 forward, -1 backward
};

__device__ __forceinline__ void rotate2(uint32_t& a, uint32_t& b, float2 cs0, float2 cs1) {
    const float a0 = bf16_lo(a), a1 = bf16_hi(a), b0 = bf16_lo(b), b1 = bf16_hi(b);
    a = pack_bf16x2(a0 * cs0.x - b0 * cs0.y, a1 * cs1.x - b1 * cs1.y);
    b = pack_bf16x2(b0 * cs0.x + a0 * cs0.y, b1 * cs1.x + a1 * cs1.y);
}

// The pair (low, high) of one word.
__device__ __forceinline__ uint32_t rotate1(uint32_t w, float2 cs) {
    const float a = bf16_lo(w), b = bf16_hi(w);
    return pack_bf16x2(a * cs.x - b * cs.y, b * cs.x + a * cs.y);
}

// One thread takes one 16-element column of one token (8 elements from each half
// of the rotated part with kHalf, or 16 consecutive ones; behind the rotated part
// a column is copied) and every groups-th head.  It issues the loads of its first
// heads, forms the column's 8 cosines and sines while they fly, and keeps those in
// registers.  Neighbouring threads take neighbouring columns, then neighbouring
// heads: a warp's accesses cover whole heads.  Every head is read and written once;
// the kernel is bound by HBM: 72 heads of 128, half of each turned, 16384 tokens in 89
// us, the measured copy rate; 40 heads, 4096 tokens in 15.
template <bool kHalf>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotaryArgs p) {
    const int64_t id = static_cast<int64_t>(blockIdx.x) * kRotThreads + threadIdx.x;
    if (id >= p.threads) return;
    const int per_token = p.columns * p.groups;
    const int t = static_cast<int>(id / per_token);
    const int r = static_cast<int>(id - static_cast<int64_t>(t) * per_token);
    const int group = r / p.columns, c = r - group * p.columns;
    const bool turned = 16 * c < p.rot;
    const int at = kHalf && turned ? 8 * c : 16 * c;
    const int second = kHalf && turned ? p.rot >> 1 : 8;
    const bool both = turned || at + second < p.head_dim;  // the last copied column may be 8 elements
    const uint16_t* src = p.x + t * p.ld_x + at;
    uint16_t* dst = p.y + t * p.ld_y + at;
    uint4 u[kRotUnroll], v[kRotUnroll];
    auto load = [&](int h0) {
#pragma unroll
        for (int i = 0; i < kRotUnroll; ++i) {
            const int h = h0 + i * p.groups;
            if (h < p.n_heads) {
                u[i] = *reinterpret_cast<const uint4*>(src + h * p.head_dim);
                if (both) v[i] = *reinterpret_cast<const uint4*>(src + h * p.head_dim + second);
            }
        }
    };
    wait_for_previous();
    load(group);
    float2 cs[8];
    if (turned) {
        const int64_t pos = p.positions ? p.positions[t] : t;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint64_t frac = static_cast<uint64_t>(pos) * p.turns[8 * c + k];
            // the upper 32 bits as a signed number of half turns in [-1, 1)
            float sn, cn;
            sincospif(static_cast<float>(static_cast<int32_t>(frac >> 32)) * 0x1p-31f, &sn, &cn);
            cs[k] = make_float2(cn * p.magnitude, sn * p.magnitude * p.sign);
        }
    }
    for (int h0 = group;;) {
#pragma unroll
        for (int i = 0; i < kRotUnroll; ++i) {
            const int h = h0 + i * p.groups;
            if (h >= p.n_heads) break;
            if (turned) {
                if (kHalf) {
                    rotate2(u[i].x, v[i].x, cs[0], cs[1]);
                    rotate2(u[i].y, v[i].y, cs[2], cs[3]);
                    rotate2(u[i].z, v[i].z, cs[4], cs[5]);
                    rotate2(u[i].w, v[i].w, cs[6], cs[7]);
                } else {
                    u[i] = make_uint4(rotate1(u[i].x, cs[0]), rotate1(u[i].y, cs[1]), rotate1(u[i].z, cs[2]), rotate1(u[i].w, cs[3]));
                    v[i] = make_uint4(rotate1(v[i].x, cs[4]), rotate1(v[i].y, cs[5]), rotate1(v[i].z, cs[6]), rotate1(v[i].w, cs[7]));
                }
            }
            *reinterpret_cast<uint4*>(dst + h * p.head_dim) = u[i];
            if (both) *reinterpret_cast<uint4*>(dst + h * p.head_dim + second) = v[i];
        }
        h0 += kRotUnroll * p.groups;
        if (h0 >= p.n_heads) break;
        load(h0);
    }
}

zb_status rotary(const void* x, int64_t ld_x, void* y, int64_t ld_y, const int32_t* positions, const uint64_t* turns,
                 float magnitude, int32_t tokens, int32_t n_heads, int32_t head_dim, int32_t rotary_dim, int32_t pairs,
                 void* stream, float sign) {
    if (pairs != ZB_ROTARY_HALF && pairs != ZB_ROTARY_INTERLEAVED) return ZB_ERR_ARG;
    if (!tokens_ok(tokens) || n_heads <= 0 || head_dim <= 0 || head_dim % 8 != 0 || n_heads > kMaxFeature / head_dim ||
        !feature_ok(n_heads * head_dim) || rotary_dim < 16 || rotary_dim > head_dim || rotary_dim % 16 != 0 ||
        rotary_dim / 2 > kRotMaxPairs)
        return ZB_ERR_SHAPE;
    if (ld_x < n_heads * head_dim || ld_y < n_heads * head_dim || ld_x % 8 != 0 || ld_y % 8 != 0) return ZB_ERR_SHAPE;
    if (!rows_ok(x, tokens) || !rows_ok(y, tokens) || (positions && (reinterpret_cast<uintptr_t>(positions) & 3u)) ||
        !fixed_ok(turns) || !(std::fabs(magnitude) <= 3.4e38f) || (x == y && ld_x != ld_y))
        return ZB_ERR_ARG;
    ZB_TRY(device_ok());
    if (tokens == 0) return ZB_OK;
    return cuda_status(launch_rotary(x, ld_x, y, ld_y, positions, turns, magnitude, tokens, n_heads, head_dim, rotary_dim,
                                     pairs == ZB_ROTARY_HALF, sign, as_stream(stream)));
}

}  // namespace

cudaError_t launch_rotary(const void* x, int64_t ld_x, void* y, int64_t ld_y, const int32_t* positions,
                          const uint64_t* turns, float magnitude, int tokens, int n_heads, int head_dim, int rotary_dim,
                          bool half, float sign, cudaStream_t stream) {
    if (tokens <= 0) return cudaSuccess;
    RotaryArgs p{};
    p.x = static_cast<const uint16_t*>(x);
    p.y = static_cast<uint16_t*>(y);
    p.ld_x = ld_x;
    p.ld_y = ld_y;
    p.positions = positions;
    p.turns = turns;
    p.magnitude = magnitude;
    p.tokens = tokens;
    p.n_heads = n_heads;
    p.head_dim = head_dim;
    p.rot = rotary_dim;
    p.sign = sign;
    // in place, what lies behind the rotated part stays as it is
    p.columns = (rotary_dim >> 4) + (x == y ? 0 : (head_dim - rotary_dim + 15) >> 4);
    p.groups = (n_heads + kRotHeads - 1) / kRotHeads;
    p.threads = static_cast<int64_t>(tokens) * p.columns * p.groups;
    const unsigned grid = static_cast<unsigned>((p.threads + kRotThreads - 1) / kRotThreads);
    return half ? launch_chained(rotary_kernel<true>, grid, kRotThreads, 0, stream, p)
                : launch_chained(rotary_kernel<false>, grid, kRotThreads, 0, stream, p);
}

}  // namespace zbk

extern "C" zb_status zb_op_rotary_forward(const void* x, int64_t ld_x, void* y, int64_t ld_y, const int32_t* positions,
                                          const uint64_t* turns, float magnitude, int32_t tokens, int32_t n_heads,
                                          int32_t head_dim, int32_t rotary_dim, int32_t pairs, void* stream) {
    return zbk::rotary(x, ld_x, y, ld_y, positions, turns, magnitude, tokens, n_heads, head_dim, rotary_dim, pairs, stream,
                       1.f);
}

extern "C" zb_status zb_op_rotary_backward(const void* dy, int64_t ld_dy, void* dx, int64_t ld_dx, const int32_t* positions,
                                           const uint64_t* turns, float magnitude, int32_t tokens, int32_t n_heads,
                                           int32_t head_dim, int32_t rotary_dim, int32_t pairs, void* stream) {
    return zbk::rotary(dy, ld_dy, dx, ld_dx, positions, turns, magnitude, tokens, n_heads, head_dim, rotary_dim, pairs,
                       stream, -1.f);
}

extern "C" zb_status zb_rotary_frequencies(const zb_rotary_config* cfg, uint64_t* turns, float* magnitude) {
    if (!cfg || !turns || !magnitude) return ZB_ERR_ARG;
    const int rot = cfg->rotary_dim;
    if (rot < 16 || rot % 16 != 0 || rot / 2 > zbk::kRotMaxPairs) return ZB_ERR_SHAPE;
    const double two_pi = 6.283185307179586476925286766559;
    double base = cfg->base;
    const double factor = cfg->factor, context = cfg->context;
    if (!(base > 1.0) || !std::isfinite(base)) return ZB_ERR_ARG;
    if (cfg->scaling < ZB_ROTARY_SCALE_NONE || cfg->scaling > ZB_ROTARY_SCALE_BANDED) return ZB_ERR_ARG;
    if (cfg->scaling != ZB_ROTARY_SCALE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return ZB_ERR_ARG;
    if (cfg->scaling >= ZB_ROTARY_SCALE_YARN &&
        (!(context >= 1.0) || !std::isfinite(context) || !(cfg->low > 0.0) || !(cfg->high > cfg->low) || !std::isfinite(cfg->high)))
        return ZB_ERR_ARG;
    double mag = 1.0, ramp_low = 0.0, ramp_end = 1.0;
    if (cfg->scaling == ZB_ROTARY_SCALE_NTK) base *= std::pow(factor, rot / (rot - 2.0));
    if (!std::isfinite(base)) return ZB_ERR_ARG;
    if (cfg->scaling == ZB_ROTARY_SCALE_YARN) {
        // the pair that makes `turns` turns over the original context
        auto at = [&](double n) { return rot * std::log(context / (n * two_pi)) / (2.0 * std::log(base)); };
        ramp_low = std::max(std::floor(at(cfg->high)), 0.0);
        ramp_end = std::min(std::ceil(at(cfg->low)), rot - 1.0);
        mag = 0.1 * std::log(factor) + 1.0;
    }
    for (int i = 0; i < rot / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot);
        if (cfg->scaling == ZB_ROTARY_SCALE_LINEAR) f /= factor;
        if (cfg->scaling == ZB_ROTARY_SCALE_YARN) {
            // (a context of a few tokens: no pair makes `low` turns, and the ramp ends before it starts)
            const double r = ramp_end > ramp_low ? std::min(1.0, std::max(0.0, (i - ramp_low) / (ramp_end - ramp_low)))
                                                 : i >= ramp_end ? 1.0 : 0.0;
            f = f / factor * r + f * (1.0 - r);
        }
        if (cfg->scaling == ZB_ROTARY_SCALE_BANDED) {
            const double n = context * f / two_pi;  // turns over the original context
            const double keep = std::min(1.0, std::max(0.0, (n - cfg->low) / (cfg->high - cfg->low)));
            f = f * keep + f / factor * (1.0 - keep);
        }
        // f <= 1 radian, so f / (2 pi) is below a quarter turn and fits
        turns[i] = static_cast<uint64_t>(std::floor(std::ldexp(f / two_pi, 64) + 0.5));
    }
    *magnitude = static_cast<float>(mag);
    return ZB_OK;
}
