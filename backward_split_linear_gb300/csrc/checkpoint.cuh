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

// The larger magnitudes of two pairs of bf16 numbers, per half, with any sign; a NaN stays one.
__device__ __forceinline__ uint32_t pack_top2(uint32_t top, uint32_t w) {
    uint32_t d;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(top), "r"(w));
    return d;
}

// The larger magnitude's bits of a pair.
__device__ __forceinline__ uint32_t pack_top(uint32_t top2) { return max(top2 & 0x7fffu, (top2 >> 16) & 0x7fffu); }

// The scale byte of a block from the bf16 bits of its largest magnitude: the exponent
// less 6, one more where all seven mantissa bits are set (127.5 units, which round to 128).
__device__ __forceinline__ uint32_t pack_scale(uint32_t top) {
    if (top >= 0x7f80u) return kPackNotFinite;
    const int s = static_cast<int>((top + 1u) >> 7) - 6;
    return static_cast<uint32_t>(min(max(s, 1), 248));
}

// 2^(127 - scale), which takes magnitudes to units, as a pair of bf16 numbers.
__device__ __forceinline__ uint32_t pack_factor(uint32_t scale) { return ((254u - min(scale, 253u)) << 7) * 0x00010001u; }

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// Four codes from two pairs of bf16 numbers.  From 128 to 256 a bf16 number is a whole one,
// so |x| factor + 128 rounds to the nearest even unit, with the magnitude in its seven
// mantissa bits.  Blocks without the largest bf16 number and without what is not finite.
__device__ __forceinline__ uint32_t pack_codes(uint32_t w0, uint32_t w1, uint32_t factor) {
    const uint32_t a = fma_bf16x2(w0 & 0x7fff7fffu, factor, 0x43004300u);
    const uint32_t b = fma_bf16x2(w1 & 0x7fff7fffu, factor, 0x43004300u);
    return __byte_perm(a, b, 0x6420) | (__byte_perm(w0, w1, 0x7531) & 0x80808080u);
}

// The others: the largest number would take 127.5 units and takes 127; codes are 0 in a
// block with a value that is not finite.
constexpr uint32_t kPackLargest = 0x7f7f;
__device__ __forceinline__ uint32_t pack_codes_slow(uint32_t w0, uint32_t w1, uint32_t factor, uint32_t scale) {
    if (scale == kPackNotFinite) return 0u;
    const uint32_t m0 = __vminu2(w0 & 0x7fff7fffu, 0x7f7e7f7eu), m1 = __vminu2(w1 & 0x7fff7fffu, 0x7f7e7f7eu);
    return pack_codes(m0 | (w0 & 0x80008000u), m1 | (w1 & 0x80008000u), factor);
}

// One whole block: 16 words of bf16 pairs to 8 words of codes; returns the scale byte.
__device__ __forceinline__ uint32_t pack_block(const uint32_t (&w)[16], uint4& lo, uint4& hi) {
    uint32_t top2 = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top2 = pack_top2(top2, w[i]);
    const uint32_t top = pack_top(top2), scale = pack_scale(top);
    const uint32_t f = pack_factor(scale);
    uint32_t c[8];
    if (top < kPackLargest) {
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = pack_codes(w[2 * i], w[2 * i + 1], f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = pack_codes_slow(w[2 * i], w[2 * i + 1], f, scale);
    }
    lo = make_uint4(c[0], c[1], c[2], c[3]);
    hi = make_uint4(c[4], c[5], c[6], c[7]);
    return scale;
}

// The unit 2^(scale - 127) of a block, as a pair of bf16 numbers; NaN for one that was not
// finite.  A scale of 0 (which packing never writes) stands for 0.
__device__ __forceinline__ uint32_t unpack_unit(uint32_t scale) {
    return scale == kPackNotFinite ? 0x7fff7fffu : (scale << 7) * 0x00010001u;
}

// Codes 2 kHalf and 2 kHalf + 1 of the four in `c` as a pair of bf16 numbers: 128 + m from the
// bits, less 128, times the unit, all exact.
template <int kHalf>
__device__ __forceinline__ uint32_t unpack_pair(uint32_t c, uint32_t unit) {
    const uint32_t m = __byte_perm(c & 0x7f7f7f7fu, 0x43434343u, kHalf ? 0x4342 : 0x4140);
    const uint32_t v = fma_bf16x2(fma_bf16x2(m, 0x3f803f80u, 0xc300c300u), unit, 0x80008000u);
    return v ^ (__byte_perm(c, 0u, kHalf ? 0x3424 : 0x1404) & 0x80008000u);
}

}  // namespace zbk
