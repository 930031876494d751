// Activations in 8 bits: one scale byte per 32 consecutive columns of a row, and per
// element a sign and a magnitude up to 127 in units of the block's power of two.
//
// With a block's largest value in [63.75, 127.5) units, the error is half a unit, at most
// 2^-7 of that value.  The unit is a power of two, so that 127 units are a bf16 number
// exactly: what the codes stand for passes through bf16 kernels without another rounding
// (a unit of largest / 127 would halve the worst error and lose that).  Integers rather
// than a small float: over 32 normally distributed values the mean error is a quarter of
// what 3 mantissa bits leave.
#pragma once

#include <cstdint>

#include "device_common.cuh"

namespace zbk {

constexpr int kPackBlock = 32;
constexpr uint32_t kPackNotFinite = 255;  // scale byte of a block that held a value that is not finite

// The largest magnitude's bf16 bits of two pairs of bf16 numbers, per half.
__device__ __forceinline__ uint32_t pack_top2(uint32_t top, uint32_t w) { return __vmaxu2(top, w & 0x7fff7fffu); }

// The scale byte of a block from the bf16 bits of its largest magnitude: the exponent
// less 6, one more where all seven mantissa bits are set (127.5 units, which round to 128).
__device__ __forceinline__ uint32_t pack_scale(uint32_t top) {
    if (top >= 0x7f80u) return kPackNotFinite;
    const int s = static_cast<int>((top + 1u) >> 7) - 6;
    return static_cast<uint32_t>(min(max(s, 1), 248));
}

// 2^(127 - scale), which takes magnitudes to units.
__device__ __forceinline__ float pack_factor(uint32_t scale) { return __uint_as_float((254u - min(scale, 253u)) << 23); }

// Four codes from two pairs of bf16 numbers.  |x| factor + 1.5 2^23 rounds to the nearest
// even unit in its last bits; only the largest bf16 number would pass 127 (scale 248).
__device__ __forceinline__ uint32_t pack_codes(uint32_t w0, uint32_t w1, float factor) {
    constexpr float kBig = 12582912.f;
    const float a = fminf(fmaf(fabsf(bf16_lo(w0)), factor, kBig), kBig + 127.f);
    const float b = fminf(fmaf(fabsf(bf16_hi(w0)), factor, kBig), kBig + 127.f);
    const float c = fminf(fmaf(fabsf(bf16_lo(w1)), factor, kBig), kBig + 127.f);
    const float d = fminf(fmaf(fabsf(bf16_hi(w1)), factor, kBig), kBig + 127.f);
    const uint32_t ab = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040);
    const uint32_t cd = __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040);
    const uint32_t mags = __byte_perm(ab, cd, 0x5410);
    return (mags & 0x7f7f7f7fu) | (__byte_perm(w0, w1, 0x7531) & 0x80808080u);
}

// One whole block: 16 words of bf16 pairs to 8 words of codes; returns the scale byte.
__device__ __forceinline__ uint32_t pack_block(const uint32_t (&w)[16], uint4& lo, uint4& hi) {
    uint32_t top2 = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top2 = pack_top2(top2, w[i]);
    const uint32_t scale = pack_scale(max(top2 & 0xffffu, top2 >> 16));
    const float f = pack_factor(scale);
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = scale == kPackNotFinite ? 0u : pack_codes(w[2 * i], w[2 * i + 1], f);
    lo = make_uint4(c[0], c[1], c[2], c[3]);
    hi = make_uint4(c[4], c[5], c[6], c[7]);
    return scale;
}

// The unit 2^(scale - 127) of a block; NaN for one that was not finite.  A scale of 0 (which
// packing never writes) stands for 0.
__device__ __forceinline__ float unpack_unit(uint32_t scale) {
    return scale == kPackNotFinite ? __uint_as_float(0x7fffffffu) : __uint_as_float(scale << 23);
}

// Four codes as float32 values.
__device__ __forceinline__ void unpack_codes(uint32_t c, float unit, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t byte = (c >> (8 * i)) & 0xffu;
        const float mag = __uint_as_float(0x4b000000u | (byte & 0x7fu)) - 8388608.f;
        v[i] = __uint_as_float(__float_as_uint(mag * unit) ^ ((byte & 0x80u) << 24));
    }
}

}  // namespace zbk
