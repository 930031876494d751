// Linear layers with a bias, an activation and a residual, forward and split backward:
//   F   z = x w^T + bias, y = act(z) + residual, and z and y as checkpoints (bf16 or 8 bits)
//   B   dz = (dy w) act'(z), and the bias gradient sum_t dz of the layer that made z
//   W   dw += dy^T x from an 8-bit checkpoint of x
//
// One kernel for all three: a CTA pair computes 256 x 256 tiles with tcgen05.mma
// (cta_group::2, bf16 in, float32 in tensor memory), operands by TMA through a ring of six
// 64-deep stages, two accumulators, one persistent pair per two SMs.  Warp 0 loads, warp 1
// issues the MMAs (2 and 3 only fill their warpgroup), warps 4-11 are the epilogue: warp w
// reads the 32 tensor-memory lanes 32 (w % 4) ... and one half of the columns.  Eight epilogue warps
// rather than the four of the plain GEMM because an epilogue here costs up to 3500 cycles per 32 x 32 block (gelu, two 8-bit
// blocks), which has to stay below the tile's MMAs.
//
// Sums.  The tensor core drops what falls below its accumulator's last bit, always towards
// zero: over 4096 terms a sum of products comes out 4e-6 short, over 16384 1.9e-5 (measured
// against float64), where float32 sums that round to nearest stay below 1e-6.  bf16 results do not
// show that, float32 gradients and the borders of 8-bit codes do.  So an accumulator holds few terms, fewest where
// results are float32 sums or codes (W, B with a bias gradient, F with an 8-bit output): the epilogue warps add it to sums
// in their registers, while the MMAs fill the other accumulator.
//
// GB300, 4096 rows of an 8B-shaped layer (4096 x 14336; 252.5 us at the measured peak of 1905
// TFLOP/s): F with gelu, z and y in 8 bits 281 us, B with gelu from 8 bits and a bias gradient 267, W 260
// (and 9 for its operand's unpacking); 318, 307 and 298 once the power cap holds the clocks, where
// a plain F takes 270 and a plain W 304.  While an epilogue computes, its MMAs take 630 to 740 cycles
// for 64 terms, with the arithmetic alone, and 505 otherwise.
#include <algorithm>
#include <mutex>

#include "chained.cuh"
#include "checkpoint.cuh"
#include "checks.h"
#include "device_common.cuh"
#include "gemm_common.h"
#include "operators.h"

namespace zbk {

namespace {

constexpr int kLinThreads = 384;
constexpr int kLinFirstWarps = 4;  // loads, MMAs, two idle
constexpr int kLinEpiWarps = 8;
constexpr int kLinStages = 6;
constexpr int kLinTile = 256;  // rows and columns of a pair's tile
constexpr int kLinHalf = 128;  // rows (A) and columns (B) that each CTA loads
constexpr int kLinBK = 64;
constexpr uint32_t kLinOperand = kLinHalf * kLinBK * 2;  // 16 KiB
constexpr uint32_t kLinMnBlock = 64 * kLinBK * 2;        // a 64-wide block of an MN-major tile
constexpr uint32_t kLinStaging = 32768;                  // of all epilogue warps
constexpr uint32_t kLinTmemCols = 512;
constexpr int kLinBars = 2 * kLinStages + 5 + 2 * kLinEpiWarps;
constexpr size_t kLinSmem = 1024 + kLinStages * 2 * kLinOperand + kLinStaging + kLinBars * 8 + 16;
static_assert(kLinSmem <= 232448, "shared memory");
// Registers a thread: 384 x 168 at launch, of which 128 x 64 + 256 x 216 are used.
constexpr int kLinFewRegs = 64, kLinManyRegs = 216;

enum : int { kLinForward = 0, kLinActivationBackward = 1, kLinAccumulate = 2 };

// k blocks (of 64 terms) that an accumulator in tensor memory holds: `first` in a tile's first two,
// `later` in the others.  Where the epilogue is long the first two hold more: while its warps work on the tile
// before, the MMAs get that far and no further.
struct LinSums {
    int first, later;
};

// W, and F and B where they make codes or a bias gradient (`fine`): as near to float64 as float32 additions one after
// another.  Those are nearer the smaller K is, so that sums are shorter there; below 256 terms in F, 512 in B and 1500 in
// W they are the nearer ones (K = 192: 0.9e-7 against 1.7e-7 in B; 522 rows: 0.6e-7 against 1.0e-7 in W, the widest gaps).
// F with gelu, z and y in 8 bits, the error of z's values (float32 arithmetic's), first blocks in front:
//   K = 4096: 16 1.33e-4, 12 1.05e-4, 11 0.99e-4 (1.02e-4); 2112: 11 1.23e-4, 6 0.83e-4 (1.00e-4);
//   1024: 5 0.76e-4, 3 0.60e-4 (0.75e-4); 640: 4 0.66e-4, 2 0.51e-4 (0.53e-4)
// and what it costs: 8B-shaped 274 us with 16 and 293 with 11, 4096 rows of K = 2048 to 4096 columns 58.5 and 64.8.
// B with gelu from 8 bits, the error of the bias gradient (float32 arithmetic's):
//   4096: 14 6.1e-7 (6.2e-7), 6.7e-7 with 8 blocks in later ones; 2112: 11 5.9e-7, 8 3.7e-7 (4.2e-7);
//   1024: 8 4.8e-7, 4 2.5e-7 (2.7e-7); 640: 8 4.3e-7, 3 2.0e-7 (2.3e-7)
// and what it costs: nothing 8B-shaped (277 us), 58.5 -> 62.6 at K = 2048.
// W: 8 throughout, 1.1e-7 with 4096 rows (1.9e-7).
// bf16 results alone: 16.  Their last bit is 2^13 times what those sums drop, and nothing is kept of them in float32; all
// of K in one accumulator took 0.3 to 2 % less time, but with K = 14336 results differed from those of float32 arithmetic by
// 2.2e-4, with 16 blocks by 0.7e-4.
constexpr int kLinSumBlocks = 8, kLinPlainBlocks = 16;

inline LinSums lin_sums(int epi, bool fine, int k_blocks) {
    if (epi == kLinAccumulate) return {kLinSumBlocks, kLinSumBlocks};
    if (!fine) return {kLinPlainBlocks, kLinPlainBlocks};
    const int first = epi == kLinForward ? std::max(2, std::min(11, k_blocks / 5)) : std::max(3, std::min(14, k_blocks / 4));
    return {first, std::min(first, 4)};
}

// W pauses before each box of dw.  All SMs finish their tiles at about the same time, and the next
// tile's loads waited 4000 cycles, instead of 1200, behind 20 MB of additions; spread over the time of
// two accumulators these let them through.  14336 x 4096 weights, with the operand's unpacking: 286 -> 272 us
// with 4096 rows (277 with 100 ns; 600 gain 1 %), 172 -> 161 with 2048, 124 -> 116 with 1024.  Not where a
// tile has fewer than two accumulators (512 rows: 108 -> 110) and not on a pair's last tile.
constexpr unsigned kLinPauseNs = 300;

struct LinParams {
    int m, n, k_blocks;
    LinSums sums;
    int tiles_m, tiles_n, group, group_m;
    int tile_n;  // columns of a tile: 256, or fewer where that fills a single wave
    // tiles from narrow_from on (a short last wave) are `parts` units of 256 / parts columns each;
    // with K split, the pairs of a unit
    int narrow_from, parts, num_units;
    uint32_t a_bytes;  // of one CTA's A tile: few rows have a box of as many (rounded up to 8)
    int act;
    bool wide;                 // z, residual and codes start at 32-byte boundaries
    const float* bias;         // F: [n] or NULL
    const uint16_t* residual;  // F: [m, n] or NULL
    uint16_t* z;               // F: written, B: read; [m, n] or NULL
    uint8_t* z_codes;          // the same in 8 bits: [m, n] and [m, n / 32]
    uint8_t* z_scales;
    uint8_t* y_codes;          // F: y in 8 bits
    uint8_t* y_scales;
    float* col_sums;           // B: [ceil(m / 32)][n] sums of dz over 32 rows each, or NULL
    int* status;
};

struct LinUnit {
    int tile, part;
    int cols;  // tile_n, 128 or 64
};

__device__ __forceinline__ LinUnit lin_unit(const LinParams& p, int u) {
    if (u < p.narrow_from) return LinUnit{u, 0, p.tile_n};
    const int v = u - p.narrow_from, shift = p.parts >> 1;  // 1, 2 or 4 parts
    return LinUnit{p.narrow_from + (v >> shift), v & (p.parts - 1), kLinTile >> shift};
}

__device__ __forceinline__ void lin_tile(const LinParams& p, int tile, int& tm, int& tn) {
    const int across = p.group_m ? p.tiles_n : p.tiles_m, along = p.group_m ? p.tiles_m : p.tiles_n;
    const int g = tile / (p.group * across), in = tile - g * p.group * across;
    const int size = min(p.group, along - g * p.group);
    const int a = g * p.group + in % size, b = in / size;
    tm = p.group_m ? a : b;
    tn = p.group_m ? b : a;
}

// Which of a unit's operand boxes CTA `rank` loads: none of rows past M or columns past N.  What
// its tiles then hold reaches rows and columns of the result that are not stored.
struct LinBoxes {
    bool a;
    int b;  // boxes of 64 columns
    uint32_t bytes;
};

__device__ __forceinline__ LinBoxes lin_boxes(const LinParams& p, int tm, int col0, int cols, int rank) {
    LinBoxes x;
    x.a = tm * kLinTile + rank * kLinHalf < p.m;
    const int n0 = col0 + rank * (cols / 2);
    x.b = n0 >= p.n ? 0 : cols > kLinHalf && n0 + 64 < p.n ? 2 : 1;
    x.bytes = (x.a ? p.a_bytes : 0u) + static_cast<uint32_t>(x.b) * kLinMnBlock;
    return x;
}

// ---------------------------------------------------------------- activations
//
// Two values at a time, for the packed float32 instructions.  gelu goes through the normal
// distribution's tail and gelu_tanh through the logistic function (0.5 (1 + tanh u) =
// 1 / (1 + exp(-2 u))): neither cancels where the activation is small.  A NaN stays one.

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ float2 exp2_fast(float2 x) {
    float2 r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(x.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(x.y));
    return r;
}

__device__ __forceinline__ float2 reciprocal_fast(float2 x) {
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(x.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(x.y));
    return r;
}

// The smaller (larger) of two numbers; a NaN stays one.
__device__ __forceinline__ float min_nan(float x, float y) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

// Behind +-30 an activation's slope is 0 or 1 to the last bit, and its terms would pass the range.
constexpr float kActMost = 30.f;
__device__ __forceinline__ float2 act_clamp(float2 z) {
    return make_float2(max_nan(min_nan(z.x, kActMost), -kActMost), max_nan(min_nan(z.y, kActMost), -kActMost));
}

// The standard normal distribution's tail beyond a >= 0, and exp(-a^2 / 2).  The tail is
// 0.5 exp(-x^2) erfcx(x), x = a / sqrt(2), with the scaled function erfcx(x) as t Q(t), t = 1 / (1 +
// 0.42 x) (the form of Hastings, "Approximations for Digital Computers", with a Q of degree
// 7 fitted here to erfcx over 0 <= x <= 9.6: off by 1.8e-7 of it at most; the float32
// steps add 1e-6 for a up to 5).  With erfcf and expf the epilogue bounded B: 431 us for the 8B-shaped
// down projection with a bias gradient, 354 with this in scalar steps.
__device__ __forceinline__ float2 normal_tail(float2 a, float2& e) {
    const float2 t = reciprocal_fast(__ffma2_rn(both(0.29698485f), a, both(1.0f)));
    e = exp2_fast(__fmul2_rn(__fmul2_rn(a, a), both(-0.72134752f)));
    float2 q = both(0.03501970320940018f);
    q = __ffma2_rn(q, t, both(-0.1597243994474411f));
    q = __ffma2_rn(q, t, both(0.21963188052177429f));
    q = __ffma2_rn(q, t, both(-0.06460575759410858f));
    q = __ffma2_rn(q, t, both(0.13401812314987183f));
    q = __ffma2_rn(q, t, both(0.0974719300866127f));
    q = __ffma2_rn(q, t, both(0.11977513879537582f));
    q = __ffma2_rn(q, t, both(0.1184132993221283f));
    return __fmul2_rn(__fmul2_rn(q, t), e);
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTanhA = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;

// 1 / (1 + exp(-z w)), with w' = -w log2(e)
__device__ __forceinline__ float2 logistic(float2 z, float2 w) {
    return reciprocal_fast(__fadd2_rn(exp2_fast(__fmul2_rn(z, w)), both(1.0f)));
}

__device__ __forceinline__ float2 tanh_weight(float2 z) {
    return __ffma2_rn(__fmul2_rn(z, z), both(-kTanhA * kTanhB * kLog2e), both(-kTanhA * kLog2e));
}

template <int kAct>
__device__ __forceinline__ float2 act_value(float2 z) {
    if constexpr (kAct == ZB_ACT_RELU) return make_float2(max_nan(z.x, 0.f), max_nan(z.y, 0.f));
    if constexpr (kAct == ZB_ACT_RELU2) {
        const float2 m = make_float2(max_nan(z.x, 0.f), max_nan(z.y, 0.f));
        return __fmul2_rn(m, m);
    }
    if constexpr (kAct == ZB_ACT_GELU) {  // max(z, 0) - |z| tail(|z|)
        const float2 a = make_float2(min_nan(fabsf(z.x), kActMost), min_nan(fabsf(z.y), kActMost));
        float2 e;
        const float2 tail = normal_tail(a, e);
        return __ffma2_rn(make_float2(-a.x, -a.y), tail, make_float2(fmaxf(z.x, 0.f), fmaxf(z.y, 0.f)));
    }
    if constexpr (kAct == ZB_ACT_GELU_TANH) return __fmul2_rn(z, logistic(z, tanh_weight(z)));
    if constexpr (kAct == ZB_ACT_SILU) return __fmul2_rn(z, logistic(z, both(-kLog2e)));
    return z;
}

template <int kAct>
__device__ __forceinline__ float2 act_slope(float2 z) {
    if constexpr (kAct == ZB_ACT_RELU)
        return make_float2(z.x > 0.f ? 1.f : (z.x <= 0.f ? 0.f : z.x), z.y > 0.f ? 1.f : (z.y <= 0.f ? 0.f : z.y));
    if constexpr (kAct == ZB_ACT_RELU2) return __fmul2_rn(make_float2(max_nan(z.x, 0.f), max_nan(z.y, 0.f)), both(2.f));
    const float2 c = act_clamp(z);
    if constexpr (kAct == ZB_ACT_GELU) {  // 1/2 +- (1/2 - tail) + z phi(z)
        float2 e;
        const float2 tail = normal_tail(make_float2(fabsf(c.x), fabsf(c.y)), e);
        float2 body = __ffma2_rn(tail, both(-1.f), both(0.5f));
        body = make_float2(copysignf(body.x, c.x), copysignf(body.y, c.y));
        return __fadd2_rn(__ffma2_rn(__fmul2_rn(c, both(0.3989422804014327f)), e, body), both(0.5f));
    }
    if constexpr (kAct == ZB_ACT_GELU_TANH) {  // s + c s (1 - s) 2u', 2u' = A (1 + 3 B c^2)
        const float2 s = logistic(c, tanh_weight(c));
        const float2 left = __ffma2_rn(s, make_float2(-s.x, -s.y), s);  // s - s^2
        const float2 du = __ffma2_rn(__fmul2_rn(c, c), both(3.f * kTanhA * kTanhB), both(kTanhA));
        return __ffma2_rn(__fmul2_rn(c, left), du, s);
    }
    if constexpr (kAct == ZB_ACT_SILU) {  // s + c s (1 - s)
        const float2 s = logistic(c, both(-kLog2e));
        return __ffma2_rn(c, __ffma2_rn(s, make_float2(-s.x, -s.y), s), s);
    }
    return both(1.f);
}

template <int kAct, int N>
__device__ __forceinline__ void act_values_of(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 y = act_value<kAct>(make_float2(v[i], v[i + 1]));
        v[i] = y.x;
        v[i + 1] = y.y;
    }
}

template <int N>
__device__ __forceinline__ void act_values(int act, float (&v)[N]) {
    switch (act) {
        case ZB_ACT_RELU: act_values_of<ZB_ACT_RELU>(v); break;
        case ZB_ACT_GELU: act_values_of<ZB_ACT_GELU>(v); break;
        case ZB_ACT_GELU_TANH: act_values_of<ZB_ACT_GELU_TANH>(v); break;
        case ZB_ACT_SILU: act_values_of<ZB_ACT_SILU>(v); break;
        case ZB_ACT_RELU2: act_values_of<ZB_ACT_RELU2>(v); break;
        default: break;
    }
}

// d[i] *= act'(z[i])
template <int kAct, int N>
__device__ __forceinline__ void act_slopes_of(float (&d)[N], const float (&z)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 y = __fmul2_rn(make_float2(d[i], d[i + 1]), act_slope<kAct>(make_float2(z[i], z[i + 1])));
        d[i] = y.x;
        d[i + 1] = y.y;
    }
}

template <int N>
__device__ __forceinline__ void act_slopes(int act, float (&d)[N], const float (&z)[N]) {
    switch (act) {
        case ZB_ACT_RELU: act_slopes_of<ZB_ACT_RELU>(d, z); break;
        case ZB_ACT_GELU: act_slopes_of<ZB_ACT_GELU>(d, z); break;
        case ZB_ACT_GELU_TANH: act_slopes_of<ZB_ACT_GELU_TANH>(d, z); break;
        case ZB_ACT_SILU: act_slopes_of<ZB_ACT_SILU>(d, z); break;
        case ZB_ACT_RELU2: act_slopes_of<ZB_ACT_RELU2>(d, z); break;
        default: break;
    }
}

// ---------------------------------------------------------------- epilogue of 32 columns of a row

__device__ __forceinline__ void to_words(const float (&v)[32], uint32_t (&w)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
}

// A box of 32 rows x 32 bf16 columns, 64 bytes a row, in the 64-byte TMA swizzle (16-byte
// word j of row r at word j ^ ((r >> 1) & 3)).
__device__ __forceinline__ void words_to_box(uint32_t box, int lane, const uint32_t (&w)[16]) {
    const uint32_t row = box + static_cast<uint32_t>(lane) * 64u, sw = (static_cast<uint32_t>(lane) >> 1) & 3u;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j)
        st_shared_v4(row + ((j ^ sw) << 4), make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]));
}

// 32 bytes of a row, a whole sector in one access where the tensor starts at one (`wide`).
// In two of 16 every sector went to L2 twice: 348 against 325 us for an 8B-shaped layer with z and y in 8 bits
// (sustained clocks).
__device__ __forceinline__ void store_sector(void* p, bool wide, const uint4& a, const uint4& b) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
                     "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                     : "memory");
    } else {
        static_cast<uint4*>(p)[0] = a;
        static_cast<uint4*>(p)[1] = b;
    }
}

__device__ __forceinline__ void load_sector(const void* p, bool wide, uint4& a, uint4& b) {
    if (wide) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                     : "l"(p)
                     : "memory");
    } else {
        a = static_cast<const uint4*>(p)[0];
        b = static_cast<const uint4*>(p)[1];
    }
}

// Scale bytes of consecutive 32-column blocks leave two at a time: a row of n / 32 bytes
// keeps no more than 2-byte alignment (n is a multiple of 64, so blocks come in pairs).
struct ScalePair {
    uint32_t first;
    bool alone;  // the warp has one block of the row
    __device__ __forceinline__ void put(uint8_t* scales, int64_t at, int c, uint32_t scale, bool ok) {
        if (alone) {
            if (ok) scales[at] = static_cast<uint8_t>(scale);
        } else if ((c & 1) == 0)
            first = scale;
        else if (ok)
            *reinterpret_cast<uint16_t*>(scales + at - 1) = static_cast<uint16_t>(first | (scale << 8));
    }
};

struct LinRow {
    ScalePair z, y;
};

// F.  `v` is the product on entry.  Writes z and the 8-bit checkpoints and leaves y's words in `yw`.
__device__ __forceinline__ void forward_chunk(const LinParams& p, LinRow& row, float (&v)[32], int m, int n, int c, bool ok,
                                              uint32_t (&yw)[16]) {
    const int64_t at = static_cast<int64_t>(m) * p.n + n;
    uint4 res[4];
    if (p.residual && ok) {
        load_sector(p.residual + at, p.wide, res[0], res[1]);
        load_sector(p.residual + at + 16, p.wide, res[2], res[3]);
    }
    if (p.bias) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float4 b = reinterpret_cast<const float4*>(p.bias + n)[j];
            const float2 lo = __fadd2_rn(make_float2(v[4 * j], v[4 * j + 1]), make_float2(b.x, b.y));
            const float2 hi = __fadd2_rn(make_float2(v[4 * j + 2], v[4 * j + 3]), make_float2(b.z, b.w));
            v[4 * j] = lo.x;
            v[4 * j + 1] = lo.y;
            v[4 * j + 2] = hi.x;
            v[4 * j + 3] = hi.y;
        }
    }
    if (p.z || p.z_codes) {
        uint32_t zw[16];
        to_words(v, zw);
        if (p.z) {
            if (ok) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    store_sector(p.z + at + 16 * j, p.wide, make_uint4(zw[8 * j], zw[8 * j + 1], zw[8 * j + 2], zw[8 * j + 3]),
                                 make_uint4(zw[8 * j + 4], zw[8 * j + 5], zw[8 * j + 6], zw[8 * j + 7]));
            }
        }
        if (p.z_codes) {
            uint4 lo, hi;
            const uint32_t scale = pack_block(zw, lo, hi);
            if (ok) store_sector(p.z_codes + at, p.wide, lo, hi);
            row.z.put(p.z_scales, at >> 5, c, scale, ok);
        }
    }
    act_values(p.act, v);
    if (p.residual && ok) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t rw[4] = {res[j].x, res[j].y, res[j].z, res[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[8 * j + 2 * e] += bf16_lo(rw[e]);
                v[8 * j + 2 * e + 1] += bf16_hi(rw[e]);
            }
        }
    }
    to_words(v, yw);
    if (p.y_codes) {
        uint4 lo, hi;
        const uint32_t scale = pack_block(yw, lo, hi);
        if (ok) store_sector(p.y_codes + at, p.wide, lo, hi);
        row.y.put(p.y_scales, at >> 5, c, scale, ok);
    }
}

// The words that hold 32 values of z: 16 (bf16), or 8 and a scale.
struct ZWords {
    uint4 w[4];
    uint32_t scale;
};

// A lane's row of a box of z, as TMA loaded it: 64 bytes in the 64-byte swizzle, or 32 of codes.
__device__ __forceinline__ void box_to_z(uint32_t box, int lane, bool packed, ZWords& z) {
    const uint32_t l = static_cast<uint32_t>(lane);
    if (packed) {
        z.w[0] = ld_shared_v4(box + 32u * l);
        z.w[1] = ld_shared_v4(box + 32u * l + 16u);
    } else {
        const uint32_t sw = (l >> 1) & 3u;
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) z.w[j] = ld_shared_v4(box + 64u * l + ((j ^ sw) << 4));
    }
}

// d[i] *= act'(z[i]), four words' values at a time
template <int kAct>
__device__ __forceinline__ void slopes_of(const ZWords& z, bool packed, float (&d)[32]) {
    auto pair = [&](int i, uint32_t w) {
        const float2 y = __fmul2_rn(make_float2(d[i], d[i + 1]), act_slope<kAct>(make_float2(bf16_lo(w), bf16_hi(w))));
        d[i] = y.x;
        d[i + 1] = y.y;
    };
    if (packed) {
        const uint32_t unit = unpack_unit(z.scale);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t w[4] = {z.w[j].x, z.w[j].y, z.w[j].z, z.w[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                pair(16 * j + 4 * e, unpack_pair<0>(w[e], unit));
                pair(16 * j + 4 * e + 2, unpack_pair<1>(w[e], unit));
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t w[4] = {z.w[j].x, z.w[j].y, z.w[j].z, z.w[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) pair(8 * j + 2 * e, w[e]);
        }
    }
}

__device__ __forceinline__ void slopes(int act, const ZWords& z, bool packed, float (&d)[32]) {
    switch (act) {
        case ZB_ACT_RELU: slopes_of<ZB_ACT_RELU>(z, packed, d); break;
        case ZB_ACT_GELU: slopes_of<ZB_ACT_GELU>(z, packed, d); break;
        case ZB_ACT_GELU_TANH: slopes_of<ZB_ACT_GELU_TANH>(z, packed, d); break;
        case ZB_ACT_SILU: slopes_of<ZB_ACT_SILU>(z, packed, d); break;
        case ZB_ACT_RELU2: slopes_of<ZB_ACT_RELU2>(z, packed, d); break;
        default: break;
    }
}

// Sums over the warp's 32 lanes (rows) of 32 columns; lane l gets column l's.  Five rounds
// of a transposing reduction (31 shuffles), in a fixed order.
__device__ __forceinline__ float column_sums(float (&v)[32], int lane) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const bool upper = (lane & off) != 0;
#pragma unroll
        for (int i = 0; i < off; ++i) {
            const float keep = upper ? v[i + off] : v[i];
            const float send = upper ? v[i] : v[i + off];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
    }
    return v[0];
}

// B's column sums of a chunk of dz.
__device__ __forceinline__ void add_columns(const LinParams& p, float (&v)[32], int n, int row0, int lane, bool ok) {
    if (!ok) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.f;
    }
    p.col_sums[static_cast<int64_t>(row0 >> 5) * p.n + n + lane] = column_sums(v, lane);
}

// ---------------------------------------------------------------- kernel

// An epilogue warp is done with an accumulator: its loads from tensor memory have returned
// (tcgen05.wait::ld), and tcgen05 fences on both sides order them ahead of the next MMAs' writes, which
// needs no release, only that the arrival comes before the wait's end: the PTX manual's pattern for tensor memory that passes
// between threads, a relaxed arrival and a wait at cluster scope.  No other memory is meant.  A release would wait until the
// warp's stores of the tile before are out, a thousand cycles a warp and one warp after another, with the MMAs waiting
// for all of them: 283 us against 272 for F with two 8-bit outputs, 281 against 269 for B with a bias gradient (with
// first accumulators of 16 and 14 blocks).
// All waits on barriers that the other CTA arrives on, or whose bytes its loads bring, are at cluster scope (1 us of 270).
__device__ __forceinline__ void arrive_empty(uint32_t caddr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(caddr) : "memory");
}

// kSums: a tile has several accumulators, which are added up in registers.  Where one holds all of K, its columns go
// through the epilogue 32 at a time (K = 1024, 4096 rows, 4096 columns: 27.2 us against 30.2).
template <bool A_MN, bool B_MN, int EPI, bool kSums>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kLinThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                  const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_z,
                  const __grid_constant__ LinParams p) {
    constexpr int kChunks = 4;  // 32-column chunks of a warp in a whole tile
    constexpr uint32_t kBox = kLinStaging / kLinEpiWarps;
    constexpr uint32_t kOutBox = EPI == kLinAccumulate ? 4096 : 2048;
    constexpr int kBoxes = kBox / kOutBox;    // used in turn
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t s_a = base, s_b = base + kLinStages * kLinOperand;
    const uint32_t s_out = s_b + kLinStages * kLinOperand;
    const uint32_t bars = s_out + kLinStaging;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (kLinStages + s); };
    auto tfull_bar = [&](int a) { return bars + 8u * (2 * kLinStages + a); };
    auto tempty_bar = [&](int a) { return bars + 8u * (2 * kLinStages + 2 + a); };
    const uint32_t drain_bar = bars + 8u * (2 * kLinStages + 4);
    const uint32_t side_bars = drain_bar + 8u;  // B: two of each epilogue warp, for its boxes of z
    const uint32_t tmem_slot = bars + 8u * kLinBars;
    volatile uint32_t* tmem_slot_ptr = reinterpret_cast<volatile uint32_t*>(smem_raw + (tmem_slot - raw));

    int* const status = p.status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    // k blocks of the accumulator that starts at block kc
    auto chunk_at = [&](int kc) {
        if (!kSums) return p.k_blocks;
        return kc < 2 * p.sums.first ? p.sums.first : p.sums.later;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < kLinStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), 2 * kLinEpiWarps);  // one lane of each epilogue warp of the pair
        }
        mbar_init(drain_bar, 1);
        for (int i = 0; i < 2 * kLinEpiWarps; ++i) mbar_init(side_bars + 8u * i, 1);
        mbar_fence_init();
        tma_prefetch_map(&map_a);
        tma_prefetch_map(&map_b);
        tma_prefetch_map(&map_out);
    }
    if (warp == 1) tmem_alloc_pair(tmem_slot, kLinTmemCols);
    tc_fence_before();
    cluster_sync_all();  // barriers of both CTAs initialised, tensor memory allocated
    release_next();
    wait_for_previous();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot_ptr;
    const uint32_t peer_base = ld_shared_cluster_u32(map_to_cta(tmem_slot, rank ^ 1u));
    const bool usable = peer_base == tmem_base;  // both CTAs must hold the accumulators at the same columns
    if (!usable && threadIdx.x == 0) atomicCAS(status, 0, kSitePairTmem);

    if (warp < kLinFirstWarps) {
        registers_release<kLinFewRegs>();
        if (usable && warp == 0) {
            if (lane == 0) {
                // ---------------- TMA producer (both CTAs)
                uint32_t n_fills = 0;
                int stage = 0;
                uint32_t phase = 0;
                bool ok = true;
                for (int u = pair; ok && u < p.num_units; u += npairs) {
                    const LinUnit w = lin_unit(p, u);
                    int tm, tn;
                    lin_tile(p, w.tile, tm, tn);
                    const int m0 = tm * kLinTile + static_cast<int>(rank) * kLinHalf;
                    // each CTA loads half of a unit's columns: two boxes of 64, or one, of which a
                    // unit of 64 columns reads half
                    const int col0 = tn * p.tile_n + w.part * w.cols;
                    const int n0 = col0 + static_cast<int>(rank) * (w.cols / 2);
                    const LinBoxes boxes = lin_boxes(p, tm, col0, w.cols, static_cast<int>(rank));
                    const uint32_t bytes = boxes.bytes + lin_boxes(p, tm, col0, w.cols, static_cast<int>(rank ^ 1u)).bytes;
                    for (int kb = 0; kb < p.k_blocks; ++kb) {
                        if (!mbar_wait_cluster(empty_bar(stage), phase ^ 1u, status, kSiteProducerEmpty)) {
                            ok = false;
                            break;
                        }
                        const uint32_t fb_local = full_bar(stage);
                        if (leader) mbar_arrive_expect_tx(fb_local, bytes);
                        const uint32_t fb = map_to_cta(fb_local, 0);
                        const int k0 = kb * kLinBK;
                        const uint32_t a_dst = s_a + stage * kLinOperand, b_dst = s_b + stage * kLinOperand;
                        if (boxes.a) {
                            if constexpr (A_MN) {
                                tma_load_2d_pair(a_dst, &map_a, fb, m0, k0);
                                tma_load_2d_pair(a_dst + kLinMnBlock, &map_a, fb, m0 + 64, k0);
                            } else {
                                tma_load_2d_pair(a_dst, &map_a, fb, k0, m0);
                            }
                        }
                        for (int j = 0; j < boxes.b; ++j) {
                            if constexpr (B_MN)
                                tma_load_2d_pair(b_dst + j * kLinMnBlock, &map_b, fb, n0 + 64 * j, k0);
                            else
                                tma_load_2d_pair(b_dst + j * kLinMnBlock, &map_b, fb, k0, n0 + 64 * j);
                        }
                        ++n_fills;
                        if (++stage == kLinStages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
                // Loads must land before shared memory goes away: rank 0 sees its full
                // barriers complete; rank 1 sees the MMA release each stage.
                for (int s = 0; s < kLinStages; ++s) {
                    const uint32_t uses = ring_uses(n_fills, kLinStages, s);
                    if (uses > 0) {
                        if (leader)
                            mbar_wait_cluster(full_bar(s), (uses - 1u) & 1u, status, kSiteDrain, kWaitLimitNs);
                        else
                            mbar_wait_cluster(empty_bar(s), (uses - 1u) & 1u, status, kSiteDrain, kWaitLimitNs);
                    }
                }
            }
        } else if (usable && warp == 1) {
            if (leader) {
                // ---------------- MMA issuer (rank 0): a converged warp, its elected lane carries each instruction
                const uint32_t issuer = elect_one_sync();
                int stage = 0;
                uint32_t phase = 0;
                uint32_t it = 0;
                bool ok = true;
                for (int u = pair; ok && u < p.num_units; u += npairs) {
                    const uint32_t idesc = mma_idesc_bf16(kLinTile, lin_unit(p, u).cols, A_MN, B_MN);
                    for (int kc = 0; ok && kc < p.k_blocks; kc += chunk_at(kc), ++it) {
                        const uint32_t acc = it & 1u, aph = (it >> 1) & 1u;
                        if (!__all_sync(0xffffffffu, mbar_wait_cluster_fast(tempty_bar(acc), aph ^ 1u, status, kSiteMmaTmemEmpty))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t d = tmem_base + acc * kLinTile;
                        const int kb1 = min(kc + chunk_at(kc), p.k_blocks);
                        for (int kb = kc; kb < kb1; ++kb) {
                            if (!__all_sync(0xffffffffu, mbar_wait_cluster_fast(full_bar(stage), phase, status, kSiteMmaFull))) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            const uint32_t a0 = s_a + stage * kLinOperand, b0 = s_b + stage * kLinOperand;
#pragma unroll
                            for (int k = 0; k < kLinBK / 16; ++k) {
                                const uint64_t ad = A_MN ? smem_desc_sw128(a0 + k * 2048, kLinMnBlock, 1024)
                                                         : smem_desc_sw128(a0 + k * 32, 16, 1024);
                                const uint64_t bd = B_MN ? smem_desc_sw128(b0 + k * 2048, kLinMnBlock, 1024)
                                                         : smem_desc_sw128(b0 + k * 32, 16, 1024);
                                umma_bf16_pair_elected(issuer, d, ad, bd, idesc, (kb != kc || k != 0) ? 1u : 0u);
                            }
                            umma_commit_pair_elected(issuer, empty_bar(stage), 0x3);
                            if (++stage == kLinStages) {
                                stage = 0;
                                phase ^= 1u;
                            }
                        }
                        if (ok) umma_commit_pair_elected(issuer, tfull_bar(acc), 0x3);
                    }
                }
                umma_commit_pair_elected(issuer, drain_bar, 0x1);
                mbar_wait(drain_bar, 0, status, kSiteDrain, kWaitLimitNs);
            }
        }
    } else {
        registers_claim<kLinManyRegs>();
        if (usable) {
            // ---------------- epilogue (both CTAs)
            const int q = warp & 3, half = (warp - kLinFirstWarps) >> 2;
            const int warp_at = warp - kLinFirstWarps;
            const uint32_t box0 = s_out + static_cast<uint32_t>(warp_at) * kBox;
            const uint32_t tlane = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
            uint32_t n_stored = 0, it = 0;
            uint32_t asked = 0, done = 0;  // boxes of z requested (lane 0) and used
            bool alive = true;
            auto acquire = [&]() {  // one verdict per warp: the tensor-memory loads are warp-wide
                alive = __all_sync(0xffffffffu, mbar_wait_cluster(tfull_bar(it & 1u), (it >> 1) & 1u, status, kSiteEpiTmemFull));
                tc_fence_after();
                return alive;
            };
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    arrive_empty(map_to_cta(tempty_bar(it & 1u), 0));
                }
                ++it;
            };
            // B's z comes by TMA into the box that dz leaves from, one chunk ahead: loads into
            // registers waited for the memory although their results were not used yet (a warp
            // has six scoreboards, and the activations take them all).
            const bool reads_z = EPI == kLinActivationBackward && p.act != ZB_ACT_NONE;
            auto row0_of = [&](int tm) { return tm * kLinTile + static_cast<int>(rank) * kLinHalf + q * 32; };
            auto ask_z = [&](int n, int row0) {
                const uint32_t bar = side_bars + 8u * (2 * warp_at + (asked & 1u));
                mbar_arrive_expect_tx(bar, p.z_codes ? 1024u : 2048u);
                tma_load_2d(box0 + (asked & 1u) * kOutBox, &map_z, bar, n, row0);
                ++asked;
            };
            auto first_columns = [](const LinUnit& w) { return (w.cols / 32 + 1) / 2 * 32; };  // of half 0
            auto columns_of = [&](const LinUnit& w, int tn) {  // a warp's first column
                return tn * p.tile_n + w.part * w.cols + half * first_columns(w);
            };
            LinUnit next = lin_unit(p, pair);
            int next_tm, next_tn;
            lin_tile(p, next.tile, next_tm, next_tn);
            if (reads_z && lane == 0) ask_z(columns_of(next, next_tn), row0_of(next_tm));
            for (int u = pair; alive && u < p.num_units; u += npairs) {
                const LinUnit w = next;
                const int tm = next_tm, tn = next_tn;
                const int row0 = row0_of(tm);  // first of this warp's rows
                const int m = row0 + lane;
                const bool row_ok = m < p.m;
                // this warp's columns: half of the unit's, 32 at a time
                const int cols = half == 0 ? first_columns(w) : w.cols - first_columns(w);
                const int col0 = half * first_columns(w);
                const int n_base = columns_of(w, tn);
                LinRow row;
                row.z.alone = row.y.alone = (cols | n_base) % 64 != 0;
                uint32_t scales = 0;  // B: of this row's blocks, a byte each
                // What a unit needs besides its sums, while its MMAs run: z's scales, and the place of
                // the next unit.
                auto look_ahead = [&]() {
                    if constexpr (EPI == kLinActivationBackward) {
                        if (reads_z && p.z_codes) {
                            const uint8_t* at = p.z_scales + ((static_cast<int64_t>(min(m, p.m - 1)) * p.n + n_base) >> 5);
#pragma unroll
                            for (int c = 0; c < kChunks; ++c)
                                if (32 * c < cols && n_base + 32 * c < p.n) scales |= static_cast<uint32_t>(at[c]) << (8 * c);
                        }
                    }
                    next = lin_unit(p, min(u + npairs, p.num_units - 1));
                    lin_tile(p, next.tile, next_tm, next_tn);
                };
                // What remains of a chunk once its product `v` is in registers.
                auto finish = [&](float (&v)[32], int c) {
                    if (!alive) return;
                    const int n = n_base + 32 * c;
                    const bool ok = row_ok && n < p.n;
                    const bool inside = row0 < p.m && n < p.n;  // warp-uniform: some of the box is
                    const uint32_t at = reads_z ? done : n_stored;
                    const uint32_t box = box0 + (at % kBoxes) * kOutBox;
                    uint32_t out[16];
                    if (reads_z) {
                        if (lane == 0) {
                            bulk_wait_group_read<0>();  // the other box's store has read it
                            if (32 * (c + 1) < cols)
                                ask_z(n + 32, row0);
                            else if (u + npairs < p.num_units)
                                ask_z(columns_of(next, next_tn), row0_of(next_tm));
                        }
                        __syncwarp();
                        alive = __all_sync(0xffffffffu, mbar_wait(side_bars + 8u * (2 * warp_at + (done & 1u)), (done >> 1) & 1u,
                                                                  status, kSiteEpiSideInput));
                        if (!alive) return;
                        ++done;
                    }
                    if (!inside) return;
                    if constexpr (EPI == kLinForward) forward_chunk(p, row, v, m, n, c, ok, out);
                    if constexpr (EPI == kLinActivationBackward) {
                        ZWords zw{};
                        if (reads_z) {
                            box_to_z(box, lane, p.z_codes != nullptr, zw);
                            zw.scale = (scales >> (8 * c)) & 0xffu;
                        }
                        slopes(p.act, zw, p.z_codes != nullptr, v);
                        to_words(v, out);
                    }
                    // the box's last store has read it, its z is in registers
                    if (!reads_z && lane == 0) {
                        bulk_wait_group_read<kBoxes - 1>();
                        if (EPI == kLinAccumulate && u + npairs < p.num_units && p.k_blocks >= 2 * p.sums.first) __nanosleep(kLinPauseNs);
                    }
                    __syncwarp();
                    if constexpr (EPI == kLinAccumulate) {
                        const uint32_t to = box + static_cast<uint32_t>(lane) * 128u;
#pragma unroll
                        for (uint32_t j = 0; j < 8; ++j)
                            st_shared_v4(to + ((j ^ (static_cast<uint32_t>(lane) & 7u)) << 4),
                                         make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                                                    __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3])));
                    } else {
                        words_to_box(box, lane, out);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {  // rows past M and columns past N are dropped
                        if constexpr (EPI == kLinAccumulate)
                            tma_reduce_add_2d(&map_out, box, n, row0);
                        else
                            tma_store_2d(&map_out, box, n, row0);
                        bulk_commit_group();
                    }
                    ++n_stored;
                    // last: the box's store, which the next chunk waits for, runs meanwhile
                    if constexpr (EPI == kLinActivationBackward) {
                        if (p.col_sums) add_columns(p, v, n, row0, lane, ok);
                    }
                };
                // the bias's 128 bytes of each chunk into L1, ahead of the loads that every lane makes
                if constexpr (EPI == kLinForward) {
                    if (p.bias && 32 * lane < cols && n_base + 32 * lane < p.n)
                        asm volatile("prefetch.global.L1 [%0];" ::"l"(p.bias + n_base + 32 * lane));
                }
                if constexpr (kSums) {
                    float sum[kChunks][32];
                    // The first accumulator without a wait between its columns, and what can wait
                    // behind it: the MMAs may stand still for it, after a tile whose epilogue was longer
                    // than two accumulators (F 272 -> 266 us, B 284 -> 279, with 16 and 14 blocks in the first two).
                    if (!acquire()) break;
                    {
                        const uint32_t t0 = tlane + (it & 1u) * kLinTile + static_cast<uint32_t>(col0);
                        uint32_t r[kChunks][32];
#pragma unroll
                        for (int c = 0; c < kChunks; ++c) tmem_load_32(t0 + 32u * c, r[c]);  // of narrow units too many
                        tmem_wait_load();
                        release();
#pragma unroll
                        for (int c = 0; c < kChunks; ++c)
#pragma unroll
                            for (int i = 0; i < 32; ++i) sum[c][i] = __uint_as_float(r[c][i]);
                    }
                    look_ahead();
                    for (int kc = chunk_at(0); alive && kc < p.k_blocks; kc += chunk_at(kc)) {
                        if (!acquire()) break;
                        const uint32_t t0 = tlane + (it & 1u) * kLinTile + static_cast<uint32_t>(col0);
#pragma unroll
                        for (int c = 0; c < kChunks; ++c) {
                            if (32 * c < cols) {
                                uint32_t r[32];
                                tmem_load_32(t0 + 32u * c, r);
                                tmem_wait_load();
#pragma unroll
                                for (int i = 0; i < 32; i += 2) {
                                    const float2 t = __fadd2_rn(make_float2(sum[c][i], sum[c][i + 1]),
                                                                make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])));
                                    sum[c][i] = t.x;
                                    sum[c][i + 1] = t.y;
                                }
                            }
                        }
                        release();
                    }
                    if (!alive) break;
                    if constexpr (EPI == kLinAccumulate) {
#pragma unroll
                        for (int c = 0; c < kChunks; ++c)
                            if (32 * c < cols) finish(sum[c], c);
                    } else {
                        // two copies of the long code rather than four: the sums move down
#pragma unroll 1
                        for (int c = 0; 32 * c < cols; c += 2) {
                            finish(sum[0], c);
                            if (32 * (c + 1) < cols) finish(sum[1], c + 1);
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                sum[0][i] = sum[2][i];
                                sum[1][i] = sum[3][i];
                            }
                        }
                    }
                } else {
                    look_ahead();
                    if (!acquire()) break;
                    const uint32_t t0 = tlane + (it & 1u) * kLinTile + static_cast<uint32_t>(col0);
#pragma unroll 1
                    for (int c = 0; 32 * c < cols; ++c) {
                        uint32_t r[32];
                        tmem_load_32(t0 + 32u * c, r);
                        tmem_wait_load();
                        if (32 * (c + 1) >= cols) release();
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
                        finish(v, c);
                    }
                }
            }
            // the boxes must stay until the last stores have read them; a box of z still in
            // flight (a wait gave up) must land
            if (lane == 0) {
                bulk_wait_group_read<0>();
                for (; done < asked; ++done) mbar_drain(side_bars + 8u * (2 * warp_at + (done & 1)), (done >> 1) & 1u, kWaitLimitNs);
            }
        }
    }

    tc_fence_before();
    cluster_sync_all();  // neither CTA leaves while the other may still signal it
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, kLinTmemCols);
    }
}

// ---------------------------------------------------------------- few tiles: K split in a cluster
//
// Outputs of so few tiles that most SMs would idle, over a long K (a pair takes 0.2 us for every 64
// terms, however few rows and columns there are).  A cluster of 2 or 4 CTA pairs computes one 256 x
// 128 unit, each pair over its share of K.  The partial sums go to shared memory, where the
// operands were, and every CTA finishes some of the unit's 32 x 32 blocks from all pairs' partial
// sums, added in the order of the pairs.  11 rows, K = 6720, 64 columns: 24.1 us on one pair, 13.0 on two, 10.0
// on four, 10.1 on eight; 185 rows, K = 11520, 1088 columns: 39.3, 21.5, 20.1 (20.9 with its sums of 1024 terms
// at a time, 22.6 with 8-bit outputs).  At K = 1024 it loses (256 rows,
// 1024 columns: 8.2 against 9.3), at 2048 it gains (64 rows, 2048 columns: 10.6 against 9.1).

constexpr int kSplitUnit = 128;       // columns of a unit
constexpr int kSplitTasks = 4 * 4;    // 32 x 32 blocks of a CTA's 128 x 128
constexpr int kSplitMinBlocks = 32;   // k blocks from which a split pays

__device__ __forceinline__ float4 ld_shared_cluster_f4(uint32_t caddr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(caddr)
                 : "memory");
    return v;
}

// 16-byte word j of row r of a 128 x 128 float32 block: eight consecutive rows cover all banks.
__device__ __forceinline__ uint32_t partial_at(uint32_t base, int r, uint32_t j) {
    return base + static_cast<uint32_t>(r) * 512u + ((j ^ (static_cast<uint32_t>(r) & 31u)) << 4);
}

template <bool A_MN, bool B_MN, int EPI>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_split_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                        const __grid_constant__ CUtensorMap map_out, const __grid_constant__ LinParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t s_a = base, s_b = base + kLinStages * kLinOperand;
    const uint32_t s_out = s_b + kLinStages * kLinOperand;
    const uint32_t bars = s_out + kLinStaging;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (kLinStages + s); };
    auto tfull_bar = [&](int a) { return bars + 8u * (2 * kLinStages + a); };
    auto tempty_bar = [&](int a) { return bars + 8u * (2 * kLinStages + 2 + a); };
    const uint32_t drain_bar = bars + 8u * (2 * kLinStages + 4);
    const uint32_t tmem_slot = bars + 8u * kLinBars;
    const uint32_t gave_up = tmem_slot + 4u;  // not 0: a warp of this CTA has no partial sums to give
    volatile uint32_t* gave_up_ptr = reinterpret_cast<volatile uint32_t*>(smem_raw + (gave_up - raw));
    volatile uint32_t* tmem_slot_ptr = reinterpret_cast<volatile uint32_t*>(smem_raw + (tmem_slot - raw));

    int* const status = p.status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t cta = cluster_ctarank(), rank = cta & 1u, first = cta & ~1u;  // first: the pair's rank 0
    const bool leader = rank == 0;
    const int split = static_cast<int>(cta >> 1), splits = p.parts;
    const int unit = static_cast<int>(blockIdx.x) / (2 * splits);
    const int tm = unit % p.tiles_m, tn = unit / p.tiles_m;
    const int kb0 = static_cast<int>(static_cast<int64_t>(split) * p.k_blocks / splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(split + 1) * p.k_blocks / splits);
    // k blocks of the accumulator that starts at block kc
    auto chunk_end = [&](int kc) { return min(kc + p.sums.later, kb1); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < kLinStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), 2 * kLinEpiWarps);
        }
        mbar_init(drain_bar, 1);
        *gave_up_ptr = 0u;
        mbar_fence_init();
        tma_prefetch_map(&map_a);
        tma_prefetch_map(&map_b);
        tma_prefetch_map(&map_out);
    }
    if (warp == 1) tmem_alloc_pair(tmem_slot, kLinTmemCols);
    tc_fence_before();
    cluster_sync_all();
    release_next();
    wait_for_previous();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot_ptr;
    const uint32_t peer_base = ld_shared_cluster_u32(map_to_cta(tmem_slot, cta ^ 1u));
    const bool usable = peer_base == tmem_base;
    if (!usable && threadIdx.x == 0) atomicCAS(status, 0, kSitePairTmem);
    bool alive = usable;

    if (usable && warp == 0) {
        if (lane == 0) {
            uint32_t n_fills = 0;
            int stage = 0;
            uint32_t phase = 0;
            const int m0 = tm * kLinTile + static_cast<int>(rank) * kLinHalf;
            const int col0 = tn * kSplitUnit, n0 = col0 + static_cast<int>(rank) * (kSplitUnit / 2);
            const LinBoxes boxes = lin_boxes(p, tm, col0, kSplitUnit, static_cast<int>(rank));
            const uint32_t bytes = boxes.bytes + lin_boxes(p, tm, col0, kSplitUnit, static_cast<int>(rank ^ 1u)).bytes;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait_cluster(empty_bar(stage), phase ^ 1u, status, kSiteProducerEmpty)) break;
                if (leader) mbar_arrive_expect_tx(full_bar(stage), bytes);
                const uint32_t fb = map_to_cta(full_bar(stage), first);
                const int k0 = kb * kLinBK;
                const uint32_t a_dst = s_a + stage * kLinOperand, b_dst = s_b + stage * kLinOperand;
                if (boxes.a) {
                    if constexpr (A_MN) {
                        tma_load_2d_pair(a_dst, &map_a, fb, m0, k0);
                        tma_load_2d_pair(a_dst + kLinMnBlock, &map_a, fb, m0 + 64, k0);
                    } else {
                        tma_load_2d_pair(a_dst, &map_a, fb, k0, m0);
                    }
                }
                if (boxes.b) {
                    if constexpr (B_MN)
                        tma_load_2d_pair(b_dst, &map_b, fb, n0, k0);
                    else
                        tma_load_2d_pair(b_dst, &map_b, fb, k0, n0);
                }
                ++n_fills;
                if (++stage == kLinStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            for (int s = 0; s < kLinStages; ++s) {
                const uint32_t uses = ring_uses(n_fills, kLinStages, s);
                if (uses > 0) mbar_wait_cluster(leader ? full_bar(s) : empty_bar(s), (uses - 1u) & 1u, status, kSiteDrain);
            }
        }
    } else if (usable && warp == 1) {
        if (leader) {
            const uint32_t issuer = elect_one_sync();
            constexpr uint32_t idesc = mma_idesc_bf16(kLinTile, kSplitUnit, A_MN, B_MN);
            const uint16_t both_ctas = static_cast<uint16_t>(3u << first);
            int stage = 0;
            uint32_t phase = 0, it = 0;
            bool ok = true;
            for (int kc = kb0; ok && kc < kb1; kc = chunk_end(kc), ++it) {
                const uint32_t acc = it & 1u, aph = (it >> 1) & 1u;
                if (!__all_sync(0xffffffffu, mbar_wait_cluster_fast(tempty_bar(acc), aph ^ 1u, status, kSiteMmaTmemEmpty))) break;
                tc_fence_after();
                const uint32_t d = tmem_base + acc * kLinTile;
                for (int kb = kc; kb < chunk_end(kc); ++kb) {
                    if (!__all_sync(0xffffffffu, mbar_wait_cluster_fast(full_bar(stage), phase, status, kSiteMmaFull))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a0 = s_a + stage * kLinOperand, b0 = s_b + stage * kLinOperand;
#pragma unroll
                    for (int k = 0; k < kLinBK / 16; ++k) {
                        const uint64_t ad = A_MN ? smem_desc_sw128(a0 + k * 2048, kLinMnBlock, 1024)
                                                 : smem_desc_sw128(a0 + k * 32, 16, 1024);
                        const uint64_t bd = B_MN ? smem_desc_sw128(b0 + k * 2048, kLinMnBlock, 1024)
                                                 : smem_desc_sw128(b0 + k * 32, 16, 1024);
                        umma_bf16_pair_elected(issuer, d, ad, bd, idesc, (kb != kc || k != 0) ? 1u : 0u);
                    }
                    umma_commit_pair_elected(issuer, empty_bar(stage), both_ctas);
                    if (++stage == kLinStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (ok) umma_commit_pair_elected(issuer, tfull_bar(acc), both_ctas);
            }
            umma_commit_pair_elected(issuer, drain_bar, static_cast<uint16_t>(1u << first));
            mbar_wait(drain_bar, 0, status, kSiteDrain, kWaitLimitNs);
        }
    } else if (usable && warp >= kLinFirstWarps) {
        // this pair's sums of 32 rows and 64 columns into the CTA's 128 x 128 block
        const int q = warp & 3, half = (warp - kLinFirstWarps) >> 2;
        const uint32_t tlane = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(64 * half);
        float sum[2][32];
        uint32_t it = 0;
        for (int kc = kb0; kc < kb1; kc = chunk_end(kc), ++it) {
            const uint32_t acc = it & 1u;
            alive = __all_sync(0xffffffffu, mbar_wait_cluster(tfull_bar(acc), (it >> 1) & 1u, status, kSiteEpiTmemFull));
            if (!alive) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t r[32];
                tmem_load_32(tlane + acc * kLinTile + 32u * c, r);
                tmem_wait_load();
#pragma unroll
                for (int i = 0; i < 32; ++i) sum[c][i] = kc == kb0 ? __uint_as_float(r[i]) : sum[c][i] + __uint_as_float(r[i]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                arrive_empty(map_to_cta(tempty_bar(acc), first));
            }
        }
        // the MMAs that read the operands are done with them in both CTAs of the pair
        if (alive) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j)
                    st_shared_v4(partial_at(s_a, q * 32 + lane, 16u * half + 8u * c + j),
                                 make_uint4(__float_as_uint(sum[c][4 * j]), __float_as_uint(sum[c][4 * j + 1]),
                                            __float_as_uint(sum[c][4 * j + 2]), __float_as_uint(sum[c][4 * j + 3])));
        }
    }

    if (warp >= kLinFirstWarps && !alive && lane == 0) *gave_up_ptr = 1u;
    cluster_sync_all();  // every pair's partial sums are there, or its word says that they are not
    const int per_cta = kSplitTasks / splits;
    const int warp_at = warp - kLinFirstWarps;
    bool finishes = warp_at >= 0 && warp_at < per_cta;
    // a block that misses a pair's sums is left alone: in W it holds those of earlier calls
    for (int s = 0; finishes && s < splits; ++s) finishes = ld_shared_cluster_u32(map_to_cta(gave_up, 2u * s + rank)) == 0u;
    if (finishes) {
        const int task = split * per_cta + warp_at, q = task & 3, c = task >> 2;
        const int row0 = tm * kLinTile + static_cast<int>(rank) * kLinHalf + q * 32, m = row0 + lane;
        const int n = tn * kSplitUnit + 32 * c;
        if (row0 < p.m && n < p.n) {
            const bool ok = m < p.m;
            float v[32];
            for (int s = 0; s < splits; ++s) {
                const uint32_t from = map_to_cta(s_a, 2u * s + rank);
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) {
                    const float4 t = ld_shared_cluster_f4(partial_at(from, q * 32 + lane, 8u * c + j));
                    v[4 * j] = s == 0 ? t.x : v[4 * j] + t.x;
                    v[4 * j + 1] = s == 0 ? t.y : v[4 * j + 1] + t.y;
                    v[4 * j + 2] = s == 0 ? t.z : v[4 * j + 2] + t.z;
                    v[4 * j + 3] = s == 0 ? t.w : v[4 * j + 3] + t.w;
                }
            }
            const uint32_t box = s_out + static_cast<uint32_t>(warp_at) * (kLinStaging / kLinEpiWarps);
            uint32_t out[16];
            if constexpr (EPI == kLinForward) {
                LinRow row;
                row.z.alone = row.y.alone = true;
                forward_chunk(p, row, v, m, n, 0, ok, out);
            }
            if constexpr (EPI == kLinActivationBackward) {
                if (p.act != ZB_ACT_NONE) {
                    ZWords zw{};
                    const int64_t at = static_cast<int64_t>(min(m, p.m - 1)) * p.n + n;
                    if (p.z_codes) {
                        load_sector(p.z_codes + at, p.wide, zw.w[0], zw.w[1]);
                        zw.scale = p.z_scales[at >> 5];
                    } else {
                        load_sector(p.z + at, p.wide, zw.w[0], zw.w[1]);
                        load_sector(p.z + at + 16, p.wide, zw.w[2], zw.w[3]);
                    }
                    slopes(p.act, zw, p.z_codes != nullptr, v);
                }
                to_words(v, out);
            }
            if constexpr (EPI == kLinAccumulate) {
                const uint32_t to = box + static_cast<uint32_t>(lane) * 128u;
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j)
                    st_shared_v4(to + ((j ^ (static_cast<uint32_t>(lane) & 7u)) << 4),
                                 make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                                            __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3])));
            } else {
                words_to_box(box, lane, out);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if constexpr (EPI == kLinAccumulate)
                    tma_reduce_add_2d(&map_out, box, n, row0);
                else
                    tma_store_2d(&map_out, box, n, row0);
                bulk_commit_group();
            }
            if constexpr (EPI == kLinActivationBackward) {
                if (p.col_sums) add_columns(p, v, n, row0, lane, ok);
            }
            if (lane == 0) bulk_wait_group_read<0>();
        }
    }

    tc_fence_before();
    cluster_sync_all();  // no CTA leaves while another may still read its partial sums
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, kLinTmemCols);
    }
}

// ---------------------------------------------------------------- bias gradient
//
// dbias[j] += sum over rows.  Two passes in a fixed order: sums over parts of the rows
// ([parts][n] float32), then their sum.  B's epilogue writes the first (parts of 32 rows);
// a bias without an activation behind it has column_parts_kernel.

constexpr int kColThreads = 256;
constexpr int kColGroups = 8;  // row groups of a block; a thread takes 8 columns
constexpr int kColUnroll = 4;
constexpr int kColTargetBlocks = 1216;  // 8 blocks of 256 threads on each of 152 SMs
constexpr int kColMostParts = 152;      // the second pass is short where the first has few columns

int column_parts(int tokens, int width) {
    const int across = (width + 255) / 256;
    return std::max(1, std::min({kColTargetBlocks / across, kColMostParts, (tokens + kColGroups - 1) / kColGroups}));
}

// Block x + y across: columns 256 x ..., the y-th part of the rows.  Bound by HBM.
__global__ void __launch_bounds__(kColThreads) column_parts_kernel(const uint16_t* dy, float* parts, int tokens, int width,
                                                                   int n_parts) {
    __shared__ float sums[kColGroups][256];
    release_next();
    wait_for_previous();
    const int across = (width + 255) / 256, bx = blockIdx.x % across, by = blockIdx.x / across;
    const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
    const int col = bx * 256 + 8 * lane;
    const int per = (tokens + n_parts - 1) / n_parts;
    const int t0 = by * per, t1 = min(tokens, t0 + per);
    float acc[8] = {};
    if (col < width) {
        for (int tb = t0 + group; tb < t1; tb += kColGroups * kColUnroll) {
            uint4 v[kColUnroll];
#pragma unroll
            for (int i = 0; i < kColUnroll; ++i) {
                const int t = tb + i * kColGroups;
                v[i] = t < t1 ? *reinterpret_cast<const uint4*>(dy + static_cast<int64_t>(t) * width + col) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < kColUnroll; ++i) {
                const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[2 * e] += bf16_lo(w[e]);
                    acc[2 * e + 1] += bf16_hi(w[e]);
                }
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[group][8 * lane + e] = acc[e];
    __syncthreads();
    const int j = bx * 256 + threadIdx.x;
    if (j < width) {
        float s = 0.f;
#pragma unroll
        for (int g = 0; g < kColGroups; ++g) s += sums[g][threadIdx.x];
        parts[static_cast<int64_t>(by) * width + j] = s;
    }
}

// A block finishes 32 columns: thread (c, g) adds the parts g, g + 8, ... of column c.
__global__ void __launch_bounds__(256) column_sum_kernel(const float* parts, float* out, int n_parts, int width) {
    __shared__ float sums[8][32];
    release_next();
    wait_for_previous();
    const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int j = blockIdx.x * 32 + c;
    float s = 0.f;
    for (int q0 = g; q0 < n_parts; q0 += 128) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = q0 + 8 * i < n_parts ? parts[static_cast<int64_t>(q0 + 8 * i) * width + j] : 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) s += v[i];
    }
    sums[g][c] = s;
    __syncthreads();
    if (g == 0) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) t += sums[k][c];
        out[j] += t;
    }
}

cudaError_t launch_column_sum(const float* parts, float* out, int n_parts, int width, cudaStream_t stream) {
    return launch_chained(column_sum_kernel, static_cast<unsigned>(width / 32), 256, 0, stream, parts, out, n_parts, width);
}

// ---------------------------------------------------------------- the activation alone

// dz = dy act'(z), 8 elements a thread.  Bound by HBM.
__global__ void __launch_bounds__(256) activation_backward_kernel(const uint16_t* dy, const uint16_t* z,
                                                                  const uint8_t* codes,
                                                                  const uint8_t* scales, uint16_t* dz,
                                                                  int64_t chunks, int act) {
    release_next();
    wait_for_previous();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= chunks) return;
    const uint4 dv = reinterpret_cast<const uint4*>(dy)[i];
    const uint32_t dw[4] = {dv.x, dv.y, dv.z, dv.w};
    float d[8], x[8];
    if (act == ZB_ACT_NONE) {
        reinterpret_cast<uint4*>(dz)[i] = dv;
        return;
    }
    if (codes) {
        const uint2 c = reinterpret_cast<const uint2*>(codes)[i];
        const uint32_t unit = unpack_unit(scales[i >> 2]);
        const uint32_t w[4] = {unpack_pair<0>(c.x, unit), unpack_pair<1>(c.x, unit), unpack_pair<0>(c.y, unit),
                               unpack_pair<1>(c.y, unit)};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = bf16_lo(w[e]);
            x[2 * e + 1] = bf16_hi(w[e]);
        }
    } else {
        const uint4 zv = reinterpret_cast<const uint4*>(z)[i];
        const uint32_t zw[4] = {zv.x, zv.y, zv.z, zv.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = bf16_lo(zw[e]);
            x[2 * e + 1] = bf16_hi(zw[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        d[2 * e] = bf16_lo(dw[e]);
        d[2 * e + 1] = bf16_hi(dw[e]);
    }
    act_slopes(act, d, x);
    reinterpret_cast<uint4*>(dz)[i] = make_uint4(pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3]), pack_bf16x2(d[4], d[5]),
                                                 pack_bf16x2(d[6], d[7]));
}

// ---------------------------------------------------------------- launches

// How many CTA pairs of a kernel fit on the current device at once, and how many clusters of 2
// and 4 pairs of its split form.
struct LinFit {
    int pairs;
    int clusters[2];
};

// (its forms with one accumulator and with several take the same registers and shared memory)
cudaError_t lin_fit(const void* kern, const void* one_kern, const void* split_kern, LinFit* fit) {
    LinFit f{};
    for (const void* k : {kern, one_kern, split_kern}) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kLinSmem));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sm_count()));
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = kLinSmem;
    cudaError_t e = cudaOccupancyMaxActiveClusters(&f.pairs, kern, &cfg);
    if (e != cudaSuccess) return e;
    if (f.pairs < 1) return cudaErrorInvalidConfiguration;
    for (int i = 0; i < 2; ++i) {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {4u << i, 1, 1};
        cfg.gridDim = dim3(static_cast<unsigned>(sm_count()) / (4u << i) * (4u << i));
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&f.clusters[i], split_kern, &cfg);
        if (e != cudaSuccess) return e;
    }
    *fit = f;
    return cudaSuccess;
}

// Columns of a tile: 256, or the fewest of 224, 192 and 160 with which a single wave that holds over
// half of the pairs still is one.  1000 rows, K = 14336, 4096 columns: 64 tiles of 256 columns in 71.7 us,
// 76 of 224 in 69.1 (in a burst; 81 under the power cap); 1024 rows, K = 4096: 26.8 and 25.4.  (Two waves lose: 1533 rows, K = 3264, 4800 columns
// take 32.6 us in 114 tiles of 256 columns and 35.2 in 150 of 192.)
int lin_tile_columns(int tiles_m, int n, int pairs) {
    auto tiles = [&](int w) { return static_cast<int64_t>(tiles_m) * ((n + w - 1) / w); };
    if (tiles(kLinTile) > pairs || 2 * tiles(kLinTile) <= pairs) return kLinTile;
    for (int w : {160, 192, 224})
        if (tiles(w) <= pairs) return w;
    return kLinTile;
}

// A chained launch in clusters of a size given here.
template <typename... P, typename... A>
cudaError_t launch_clusters(void (*kernel)(P...), unsigned grid, unsigned cluster, cudaStream_t stream, A&&... args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {cluster, 1, 1};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = kLinSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

template <bool A_MN, bool B_MN, int EPI>
cudaError_t launch_linear(const void* a, const void* b, void* out, LinParams& p, int k, cudaStream_t stream) try {
    constexpr auto kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    constexpr auto k128 = CU_TENSOR_MAP_SWIZZLE_128B;
    CUtensorMap ma, mb, mo;
    const uint32_t a_rows = A_MN ? kLinHalf : static_cast<uint32_t>(std::min(kLinHalf, (p.m + 7) / 8 * 8));
    p.a_bytes = a_rows * kLinBK * 2;
    bool ok = A_MN ? gemm_encode_map(&ma, a, k, p.m, p.m, 64, kLinBK, k128, kBf16)
                   : gemm_encode_map(&ma, a, p.m, k, k, 64, a_rows, k128, kBf16);
    ok = ok && (B_MN ? gemm_encode_map(&mb, b, k, p.n, p.n, 64, kLinBK, k128, kBf16)
                     : gemm_encode_map(&mb, b, p.n, k, k, 64, kLinHalf / 2, k128, kBf16));
    ok = ok && (EPI == kLinAccumulate
                    ? gemm_encode_map(&mo, out, p.m, p.n, p.n, 32, 32, k128, CU_TENSOR_MAP_DATA_TYPE_FLOAT32)
                    : gemm_encode_map(&mo, out, p.m, p.n, p.n, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B, kBf16));
    // B: boxes of z, or a map that nothing reads through
    CUtensorMap mz = ma;
    if (EPI == kLinActivationBackward && p.act != ZB_ACT_NONE)
        ok = ok && (p.z_codes ? gemm_encode_map(&mz, p.z_codes, p.m, p.n, p.n, 32, 32, CU_TENSOR_MAP_SWIZZLE_NONE,
                                                CU_TENSOR_MAP_DATA_TYPE_UINT8)
                              : gemm_encode_map(&mz, p.z, p.m, p.n, p.n, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B, kBf16));
    if (!ok) return cudaErrorInvalidValue;
    p.status = status_word();
    if (!p.status) return cudaErrorInvalidDevice;
    const uintptr_t starts = reinterpret_cast<uintptr_t>(p.residual) | reinterpret_cast<uintptr_t>(p.z) |
                             reinterpret_cast<uintptr_t>(p.z_codes) | reinterpret_cast<uintptr_t>(p.y_codes);
    p.wide = starts % 32 == 0;

    p.k_blocks = (k + kLinBK - 1) / kLinBK;
    const bool fine = p.col_sums || (EPI == kLinForward && (p.z_codes || p.y_codes));
    p.sums = lin_sums(EPI, fine, p.k_blocks);
    auto sums_kern = linear_kernel<A_MN, B_MN, EPI, true>;
    auto one_kern = linear_kernel<A_MN, B_MN, EPI, EPI == kLinAccumulate>;  // W's epilogue is short either way
    auto split_kern = linear_split_kernel<A_MN, B_MN, EPI>;
    static std::mutex mu;
    static LinFit fits[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    LinFit fit;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!fits[dev].pairs) {
            const cudaError_t e = lin_fit(reinterpret_cast<const void*>(sums_kern), reinterpret_cast<const void*>(one_kern),
                                          reinterpret_cast<const void*>(split_kern), &fits[dev]);
            if (e != cudaSuccess) return e;
        }
        fit = fits[dev];
    }
    const int pairs = fit.pairs;
    p.tiles_m = (p.m + kLinTile - 1) / kLinTile;
    // K split: the most pairs a unit for which all units run at once.
    const int units = p.tiles_m * ((p.n + kSplitUnit - 1) / kSplitUnit);
    for (int i = 1; i >= 0; --i) {
        const int splits = 2 << i;
        if (units > fit.clusters[i] || p.k_blocks < kSplitMinBlocks) continue;
        p.parts = splits;
        // 4 left the bias gradient 2.5e-7 off (185 rows, K = 11520), float32 arithmetic 2.3e-7, 3 leave it 2.1e-7
        if (fine) p.sums.later = std::min(p.sums.later, 3);
        return launch_clusters(split_kern, static_cast<unsigned>(units * 2 * splits), 2u * splits, stream, ma, mb, mo, p);
    }

    p.tile_n = lin_tile_columns(p.tiles_m, p.n, pairs);
    p.tiles_n = (p.n + p.tile_n - 1) / p.tile_n;
    const int tiles = p.tiles_m * p.tiles_n;
    bool group_m = false;
    p.group = gemm_raster(p.tiles_m, p.tiles_n, kLinTile, p.tile_n, k, std::min(tiles, pairs), &group_m);
    p.group_m = group_m ? 1 : 0;
    // A last wave that would keep at most half (a quarter) of the pairs busy runs as units of
    // half (a quarter) of a tile's columns on twice (four times) as many: each output element
    // takes the same steps.
    const int rem = p.tile_n == kLinTile ? tiles % pairs : 0;
    p.parts = rem == 0 || 2 * rem > pairs ? 1 : 4 * rem > pairs ? 2 : 4;
    p.narrow_from = p.parts == 1 ? tiles : tiles - rem;
    p.num_units = p.narrow_from + p.parts * (tiles - p.narrow_from);
    return launch_chained(p.k_blocks <= p.sums.first ? one_kern : sums_kern, 2u * static_cast<unsigned>(std::min(p.num_units, pairs)), kLinThreads, kLinSmem, stream, ma, mb, mo,
                          mz, p);
} catch (...) {  // the tile order is kept in a map, which may not get its memory
    return cudaErrorMemoryAllocation;
}

bool activation_ok(int32_t act) { return act >= ZB_ACT_NONE && act <= ZB_ACT_RELU2; }

// Codes and scales of a checkpoint with `tokens` rows.
bool checkpoint_ok(const zb_checkpoint* c, int32_t tokens) {
    return c && rows_ok(c->codes, tokens) && rows_ok(c->scales, tokens);
}

}  // namespace

}  // namespace zbk

extern "C" zb_status zb_op_linear_activation_forward(const void* x, const void* w, const float* bias, const void* residual,
                                                     void* y, void* z, const zb_checkpoint* z_packed,
                                                     const zb_checkpoint* y_packed, int32_t tokens, int32_t in_features,
                                                     int32_t out_features, int32_t activation, void* stream) {
    using namespace zbk;
    if (!activation_ok(activation) || (z && z_packed)) return ZB_ERR_ARG;
    if (!tokens_ok(tokens) || !feature_ok(in_features) || !feature_ok(out_features)) return ZB_ERR_SHAPE;
    if (!rows_ok(x, tokens) || !fixed_ok(w) || !rows_ok(y, tokens) || (bias && !aligned16(bias)) ||
        (residual && !aligned16(residual)) || (z && !aligned16(z)) || (z_packed && !checkpoint_ok(z_packed, tokens)) ||
        (y_packed && !checkpoint_ok(y_packed, tokens)))
        return ZB_ERR_ARG;
    ZB_TRY(device_ok());
    if (tokens == 0) return ZB_OK;
    LinParams p{};
    p.m = tokens;
    p.n = out_features;
    p.act = activation;
    p.bias = bias;
    p.residual = static_cast<const uint16_t*>(residual);
    p.z = static_cast<uint16_t*>(z);
    if (z_packed) {
        p.z_codes = static_cast<uint8_t*>(z_packed->codes);
        p.z_scales = static_cast<uint8_t*>(z_packed->scales);
    }
    if (y_packed) {
        p.y_codes = static_cast<uint8_t*>(y_packed->codes);
        p.y_scales = static_cast<uint8_t*>(y_packed->scales);
    }
    return cuda_status(launch_linear<false, false, kLinForward>(x, w, y, p, in_features, as_stream(stream)));
}

extern "C" size_t zb_op_backward_input_activation_scratch_bytes(int32_t tokens, int32_t in_features) {
    if (!zbk::tokens_ok(tokens) || !zbk::feature_ok(in_features)) return 0;
    return static_cast<size_t>((tokens + 31) / 32) * static_cast<size_t>(in_features) * sizeof(float);
}

extern "C" zb_status zb_op_backward_input_activation(const void* dy, const void* w, const void* z,
                                                     const zb_checkpoint* z_packed, void* dz, float* dbias, int32_t tokens,
                                                     int32_t in_features, int32_t out_features, int32_t activation,
                                                     void* scratch, size_t scratch_bytes, void* stream) {
    using namespace zbk;
    if (!activation_ok(activation) || (z && z_packed)) return ZB_ERR_ARG;
    if (!tokens_ok(tokens) || !feature_ok(in_features) || !feature_ok(out_features)) return ZB_ERR_SHAPE;
    if (!rows_ok(dy, tokens) || !fixed_ok(w) || !rows_ok(dz, tokens) || (z && !aligned16(z)) ||
        (z_packed && !checkpoint_ok(z_packed, tokens)) || (dbias && !aligned16(dbias)) ||
        (tokens > 0 && activation != ZB_ACT_NONE && !z && !z_packed))
        return ZB_ERR_ARG;
    if (dbias && tokens > 0 &&
        (!fixed_ok(scratch) || scratch_bytes < zb_op_backward_input_activation_scratch_bytes(tokens, in_features)))
        return ZB_ERR_WORKSPACE;
    ZB_TRY(device_ok());
    if (tokens == 0) return ZB_OK;
    LinParams p{};
    p.m = tokens;
    p.n = in_features;
    p.act = activation;
    p.z = static_cast<uint16_t*>(const_cast<void*>(z));
    if (z_packed) {
        p.z_codes = static_cast<uint8_t*>(z_packed->codes);
        p.z_scales = static_cast<uint8_t*>(z_packed->scales);
    }
    cudaStream_t s = as_stream(stream);
    if (dbias) p.col_sums = static_cast<float*>(scratch);
    ZB_TRY(cuda_status(launch_linear<false, true, kLinActivationBackward>(dy, w, dz, p, out_features, s)));
    if (!dbias) return ZB_OK;
    return cuda_status(launch_column_sum(p.col_sums, dbias, (tokens + 31) / 32, in_features, s));
}

extern "C" zb_status zb_op_activation_backward(const void* dy, const void* z, const zb_checkpoint* z_packed, void* dz,
                                               int32_t tokens, int32_t width, int32_t activation, void* stream) {
    using namespace zbk;
    if (!activation_ok(activation) || (z && z_packed)) return ZB_ERR_ARG;
    if (!tokens_ok(tokens) || !feature_ok(width)) return ZB_ERR_SHAPE;
    if (!rows_ok(dy, tokens) || !rows_ok(dz, tokens) || (z && !aligned16(z)) ||
        (z_packed && !checkpoint_ok(z_packed, tokens)) || (tokens > 0 && activation != ZB_ACT_NONE && !z && !z_packed))
        return ZB_ERR_ARG;
    ZB_TRY(device_ok());
    if (tokens == 0) return ZB_OK;
    const int64_t chunks = static_cast<int64_t>(tokens) * (width / 8);
    const int64_t grid = (chunks + 255) / 256;
    if (grid > 0x7fffffff) return ZB_ERR_SHAPE;
    return cuda_status(launch_chained(
        activation_backward_kernel, static_cast<unsigned>(grid), 256, 0, as_stream(stream), static_cast<const uint16_t*>(dy),
        static_cast<const uint16_t*>(z), z_packed ? static_cast<const uint8_t*>(z_packed->codes) : nullptr,
        z_packed ? static_cast<const uint8_t*>(z_packed->scales) : nullptr, static_cast<uint16_t*>(dz), chunks, activation));
}

extern "C" size_t zb_op_backward_bias_scratch_bytes(int32_t tokens, int32_t out_features) {
    if (!zbk::tokens_ok(tokens) || !zbk::feature_ok(out_features)) return 0;
    return static_cast<size_t>(zbk::column_parts(tokens, out_features)) * static_cast<size_t>(out_features) * sizeof(float);
}

extern "C" zb_status zb_op_backward_bias(const void* dy, float* dbias, int32_t tokens, int32_t out_features, void* scratch,
                                         size_t scratch_bytes, void* stream) {
    using namespace zbk;
    if (!tokens_ok(tokens) || !feature_ok(out_features)) return ZB_ERR_SHAPE;
    if (!rows_ok(dy, tokens) || !fixed_ok(dbias)) return ZB_ERR_ARG;
    if (tokens > 0 && (!fixed_ok(scratch) || scratch_bytes < zb_op_backward_bias_scratch_bytes(tokens, out_features)))
        return ZB_ERR_WORKSPACE;
    ZB_TRY(device_ok());
    if (tokens == 0) return ZB_OK;
    const int parts = column_parts(tokens, out_features);
    cudaStream_t s = as_stream(stream);
    const unsigned grid = static_cast<unsigned>((out_features + 255) / 256 * parts);
    ZB_TRY(cuda_status(launch_chained(column_parts_kernel, grid, kColThreads, 0, s, static_cast<const uint16_t*>(dy),
                                      static_cast<float*>(scratch), tokens, out_features, parts)));
    return cuda_status(launch_column_sum(static_cast<const float*>(scratch), dbias, parts, out_features, s));
}

extern "C" size_t zb_op_backward_weight_checkpoint_scratch_bytes(int32_t tokens, int32_t in_features) {
    if (!zbk::tokens_ok(tokens) || !zbk::feature_ok(in_features)) return 0;
    return static_cast<size_t>(tokens) * static_cast<size_t>(in_features) * 2;
}

extern "C" zb_status zb_op_backward_weight_checkpoint(const void* dy, const zb_checkpoint* x, float* dw, int32_t tokens,
                                                      int32_t in_features, int32_t out_features, void* scratch,
                                                      size_t scratch_bytes, void* stream) {
    using namespace zbk;
    if (!tokens_ok(tokens) || !feature_ok(in_features) || !feature_ok(out_features)) return ZB_ERR_SHAPE;
    if (!rows_ok(dy, tokens) || !checkpoint_ok(x, tokens) || !fixed_ok(dw)) return ZB_ERR_ARG;
    if (tokens > 0 &&
        (!fixed_ok(scratch) || scratch_bytes < zb_op_backward_weight_checkpoint_scratch_bytes(tokens, in_features)))
        return ZB_ERR_WORKSPACE;
    ZB_TRY(device_ok());
    if (tokens == 0) return ZB_OK;
    cudaStream_t s = as_stream(stream);
    ZB_TRY(cuda_status(launch_unpack(x->codes, x->scales, scratch, tokens, in_features, s)));
    LinParams p{};
    p.m = out_features;
    p.n = in_features;
    return cuda_status(launch_linear<true, true, kLinAccumulate>(dy, scratch, dw, p, tokens, s));
}
