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

#include "checks.h"
#include "device_common.cuh"
#include "operators.h"

namespace zbk {

namespace {

constexpr int kRotThreads = 256;
// A block computes the sines of kRotPairs (token, pair) entries into shared
// memory, then applies them to every head of those tokens.
constexpr int kRotPairs = 512;

struct RotaryArgs {
    const uint16_t* x;
    uint16_t* y;
    int64_t ld_x, ld_y;
    const int32_t* positions;
    const uint64_t* turns;
    float magnitude;
    int tokens, n_heads, head_dim, rot;
    int tokens_per_block;
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

// One item is 16 elements of one head of one token: 8 from each half of the
// rotated part (kHalf), or 16 consecutive ones.
template <bool kHalf>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotaryArgs p) {
    __shared__ float2 table[kRotPairs];
    const int pairs = p.rot >> 1;
    const int t0 = blockIdx.x * p.tokens_per_block;
    const int nt = min(p.tokens_per_block, p.tokens - t0);
    for (int e = threadIdx.x; e < nt * pairs; e += kRotThreads) {
        const int t = e / pairs, i = e - t * pairs;
        const int64_t pos = p.positions ? p.positions[t0 + t] : t0 + t;
        const uint64_t frac = static_cast<uint64_t>(pos) * p.turns[i];
        // the upper 32 bits as a signed number of half turns in [-1, 1)
        float s, c;
        sincospif(static_cast<float>(static_cast<int32_t>(frac >> 32)) * 0x1p-31f, &s, &c);
        table[e] = make_float2(c * p.magnitude, s * p.magnitude * p.sign);
    }
    __syncthreads();
    const int per_head = p.rot >> 4;
    const int per_token = p.n_heads * per_head;
    for (int e = threadIdx.x; e < nt * per_token; e += kRotThreads) {
        const int t = e / per_token, r = e - t * per_token;
        const int h = r / per_head, c = r - h * per_head;
        const int64_t at = static_cast<int64_t>(h) * p.head_dim + (kHalf ? 8 * c : 16 * c);
        const uint16_t* src = p.x + (t0 + t) * p.ld_x + at;
        uint16_t* dst = p.y + (t0 + t) * p.ld_y + at;
        const int second = kHalf ? pairs : 8;
        uint4 u = *reinterpret_cast<const uint4*>(src), v = *reinterpret_cast<const uint4*>(src + second);
        const float2* cs = table + t * pairs + 8 * c;
        if (kHalf) {
            rotate2(u.x, v.x, cs[0], cs[1]);
            rotate2(u.y, v.y, cs[2], cs[3]);
            rotate2(u.z, v.z, cs[4], cs[5]);
            rotate2(u.w, v.w, cs[6], cs[7]);
        } else {
            u = make_uint4(rotate1(u.x, cs[0]), rotate1(u.y, cs[1]), rotate1(u.z, cs[2]), rotate1(u.w, cs[3]));
            v = make_uint4(rotate1(v.x, cs[4]), rotate1(v.y, cs[5]), rotate1(v.z, cs[6]), rotate1(v.w, cs[7]));
        }
        *reinterpret_cast<uint4*>(dst) = u;
        *reinterpret_cast<uint4*>(dst + second) = v;
    }
    // the part of a head behind the rotated one, when y is not x
    const int tail = (p.head_dim - p.rot) >> 3;
    if (tail == 0 || p.x == p.y) return;
    const int tail_token = p.n_heads * tail;
    for (int e = threadIdx.x; e < nt * tail_token; e += kRotThreads) {
        const int t = e / tail_token, r = e - t * tail_token;
        const int h = r / tail, c = r - h * tail;
        const int64_t at = static_cast<int64_t>(h) * p.head_dim + p.rot + 8 * c;
        *reinterpret_cast<uint4*>(p.y + (t0 + t) * p.ld_y + at) =
            *reinterpret_cast<const uint4*>(p.x + (t0 + t) * p.ld_x + at);
    }
}

zb_status rotary(const void* x, int64_t ld_x, void* y, int64_t ld_y, const int32_t* positions, const uint64_t* turns,
                 float magnitude, int32_t tokens, int32_t n_heads, int32_t head_dim, int32_t rotary_dim, int32_t pairs,
                 void* stream, float sign) {
    if (pairs != ZB_ROTARY_HALF && pairs != ZB_ROTARY_INTERLEAVED) return ZB_ERR_ARG;
    if (!tokens_ok(tokens) || n_heads <= 0 || head_dim <= 0 || head_dim % 8 != 0 || n_heads > kMaxFeature / head_dim ||
        !feature_ok(n_heads * head_dim) || rotary_dim < 16 || rotary_dim > head_dim || rotary_dim % 16 != 0 ||
        rotary_dim / 2 > kRotPairs)
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
    p.tokens_per_block = std::max(1, kRotPairs / (rotary_dim / 2));
    const unsigned grid = static_cast<unsigned>((tokens + p.tokens_per_block - 1) / p.tokens_per_block);
    if (half)
        rotary_kernel<true><<<grid, kRotThreads, 0, stream>>>(p);
    else
        rotary_kernel<false><<<grid, kRotThreads, 0, stream>>>(p);
    return cudaGetLastError();
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
    if (rot < 16 || rot % 16 != 0 || rot / 2 > zbk::kRotPairs) return ZB_ERR_SHAPE;
    const double two_pi = 6.283185307179586476925286766559;
    double base = cfg->base;
    const double factor = cfg->factor, context = cfg->context;
    if (!(base > 1.0) || !std::isfinite(base)) return ZB_ERR_ARG;
    if (cfg->scaling < ZB_ROTARY_SCALE_NONE || cfg->scaling > ZB_ROTARY_SCALE_BANDED) return ZB_ERR_ARG;
    if (cfg->scaling != ZB_ROTARY_SCALE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return ZB_ERR_ARG;
    if (cfg->scaling >= ZB_ROTARY_SCALE_YARN &&
        (!(context >= 1.0) || !std::isfinite(context) || !(cfg->low > 0.0) || !(cfg->high > cfg->low) || !std::isfinite(cfg->high)))
        return ZB_ERR_ARG;
    double mag = 1.0, ramp_low = 0.0, ramp_span = 1.0;
    if (cfg->scaling == ZB_ROTARY_SCALE_NTK) base *= std::pow(factor, rot / (rot - 2.0));
    if (!std::isfinite(base)) return ZB_ERR_ARG;
    if (cfg->scaling == ZB_ROTARY_SCALE_YARN) {
        // the pair that makes `turns` turns over the original context
        auto at = [&](double n) { return rot * std::log(context / (n * two_pi)) / (2.0 * std::log(base)); };
        ramp_low = std::max(std::floor(at(cfg->high)), 0.0);
        ramp_span = std::max(std::min(std::ceil(at(cfg->low)), rot - 1.0) - ramp_low, 1e-3);
        mag = 0.1 * std::log(factor) + 1.0;
    }
    for (int i = 0; i < rot / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot);
        if (cfg->scaling == ZB_ROTARY_SCALE_LINEAR) f /= factor;
        if (cfg->scaling == ZB_ROTARY_SCALE_YARN) {
            const double r = std::min(1.0, std::max(0.0, (i - ramp_low) / ramp_span));
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
