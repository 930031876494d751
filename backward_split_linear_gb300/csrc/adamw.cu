// AdamW over many tensors in one launch, with moments in 32 or 8 bits, and the
// global gradient norm that clips it.
//
// For every element, with g the gradient times *grad_scale:
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps).
// The kernels stream every tensor once and are bound by HBM: 30 bytes an
// element with float32 moments and master weights, 18 with 8-bit moments.
//
// 8-bit moments.  256 consecutive elements share a float32 scale per moment.
// A code's value is scale times an integer of the grid (8 + f) 2^(e - 1) (f for
// e = 0), e the code's upper bits and f its lower three: three significant
// bits over 2^18 (m: a sign and 7 bits) or 2^34 (v: 8 bits).  The scale is the
// block's largest value over the largest code's.  An exponential moving average
// moves by a fraction 1 - b of the difference per step, far less than a code's
// step for v (1 - b2 of 0.05 to 0.001 against 1/8): rounding to the nearest
// code would stand still, so the rounding can be stochastic, from a hash of
// (seed, step, tensor, element).  v rounds no nonzero value to zero: a
// vanished v would make the next update as large as m / eps.  m and v are
// formed with separately rounded products and sums, so that the codes are
// reproducible by any IEEE implementation of the formulas.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "chained.cuh"
#include "checks.h"
#include "device_common.cuh"

namespace zbk {

namespace {

constexpr int kAdamThreads = 256;
constexpr int kPerThread = 8;
constexpr int kChunk = kAdamThreads * kPerThread;  // elements a block takes at a time
constexpr int kStateBlock = 256;                   // elements per 8-bit scale: one warp's
constexpr float kMTop = 245760.f;                  // 15 * 2^14, the value of m's largest code
constexpr float kVTop = 16106127360.f;             // 15 * 2^30, the value of v's largest code

// The tensors of one launch, and the first chunk of each (first[n]: all chunks).  The
// table is a kernel parameter, copied at every launch, so short lists have a small one
// (12 tensors: a launch takes the host about 3 us less).
constexpr int kFewTensors = 16, kManyTensors = 64;
template <int N>
struct AdamTable {
    zb_adamw_tensor t[N];
    int first[N + 1];
    int n;
    int index0;  // number of t[0] in the caller's list (for the hash)
};
// Where adamw_unpack_kernel writes the moments of each tensor of a table.
template <int N>
struct AdamUnpack {
    float* m[N];
    float* v[N];
};

struct AdamArgs {
    float beta1, beta2, one_minus_beta1, one_minus_beta2, eps;
    float lr, bias1, rsqrt_bias2;          // bias1 = 1 - b1^t, rsqrt_bias2 = (1 - b2^t)^(-1/2)
    float log_beta1, log_beta2;            // for a step number on the device
    uint32_t seed, step;
    int stochastic;
    const float* grad_scale;
    const float* lr_dev;
    const int64_t* step_dev;
};

// The tensor that chunk c belongs to: the last one that starts at or before it.
template <int N>
__device__ __forceinline__ int find_tensor(const AdamTable<N>& tab, int c) {
    int lo = 0, hi = tab.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab.first[mid] <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Eight consecutive values from e on, zero past the end (kFull: there are eight).
template <bool kFull>
__device__ __forceinline__ void load8f(const float* p, int64_t e, int64_t n, float (&v)[8]) {
    if (kFull || e + 8 <= n) {
        const float4 a = *reinterpret_cast<const float4*>(p + e), b = *reinterpret_cast<const float4*>(p + e + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = e + k < n ? p[e + k] : 0.f;
    }
}
template <bool kFull>
__device__ __forceinline__ void store8f(float* p, int64_t e, int64_t n, const float (&v)[8]) {
    if (kFull || e + 8 <= n) {
        *reinterpret_cast<float4*>(p + e) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(p + e + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (e + k < n) p[e + k] = v[k];
    }
}
template <bool kFull>
__device__ __forceinline__ void load8h(const uint16_t* p, int64_t e, int64_t n, float (&v)[8]) {
    if (kFull || e + 8 <= n) {
        const uint4 q = *reinterpret_cast<const uint4*>(p + e);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = bf16_lo(w[k]);
            v[2 * k + 1] = bf16_hi(w[k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = e + k < n ? __uint_as_float(static_cast<uint32_t>(p[e + k]) << 16) : 0.f;
    }
}
template <bool kFull>
__device__ __forceinline__ void store8h(uint16_t* p, int64_t e, int64_t n, const uint32_t (&w)[4]) {
    if (kFull || e + 8 <= n) {
        *reinterpret_cast<uint4*>(p + e) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (e + k < n) p[e + k] = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
    }
}
template <bool kFull>
__device__ __forceinline__ uint2 load8b(const uint8_t* p, int64_t e, int64_t n) {
    if (kFull || e + 8 <= n) return *reinterpret_cast<const uint2*>(p + e);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (e + k < n) w[k >> 2] |= static_cast<uint32_t>(p[e + k]) << (8 * (k & 3));
    return make_uint2(w[0], w[1]);
}
template <bool kFull>
__device__ __forceinline__ void store8b(uint8_t* p, int64_t e, int64_t n, uint2 q) {
    if (kFull || e + 8 <= n) {
        *reinterpret_cast<uint2*>(p + e) = q;
    } else {
        const uint32_t w[2] = {q.x, q.y};
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (e + k < n) p[e + k] = static_cast<uint8_t>(w[k >> 2] >> (8 * (k & 3)));
    }
}

// A 32-bit hash of xorshifts and multiplications: constants and shifts are the ones that C. Wellons published in 2018
// as the result of a search for the least bias.
__device__ __forceinline__ uint32_t mix32(uint32_t x) {
    x = (x ^ (x >> 16)) * 0x7FEB352Du;
    x = (x ^ (x >> 15)) * 0x846CA68Bu;
    return x ^ (x >> 16);
}

// Byte k of w in bits 20 to 27.
__device__ __forceinline__ uint32_t code_field(uint32_t w, int k) { return k < 3 ? w << (20 - 8 * k) : w >> 4; }
// The grid's value of a code without its sign, given in bits 20 to 27.  The float with
// those bits under the exponent 128 is a quarter of (8 + f) 2^e, which is twice the
// value, or the value plus 8 for the codes below 8; the smaller of the two readings is
// the right one on both sides.
__device__ __forceinline__ float code_value(uint32_t field) {
    const float x = __uint_as_float(0x40000000u | field);
    return fminf(x + x, fmaf(4.f, x, -8.f));
}
// The code of a scaled value z >= 0, in bits 20 to 27: the inverse, rounded up when
// the remainder's 20 bits and `noise4` carry (16 bits above four; 0x80000: to the
// nearest).
__device__ __forceinline__ uint32_t code_bits(float z, uint32_t noise4) {
    return __float_as_uint(fmaxf(z + z, __fadd_rn(z, 8.f))) + noise4 - (1040u << 20);
}
__device__ __forceinline__ float decode_m(uint32_t w, int k, float scale) {
    const uint32_t sign = (k < 3 ? w << (24 - 8 * k) : w) & 0x80000000u;
    return __uint_as_float(__float_as_uint(__fmul_rn(code_value(code_field(w, k) & 0x07F00000u), scale)) | sign);
}
__device__ __forceinline__ float decode_v(uint32_t w, int k, float scale) {
    return __fmul_rn(code_value(code_field(w, k) & 0x0FF00000u), scale);
}
// Bits 20 to 27 of four words as four bytes.
__device__ __forceinline__ uint32_t pack_codes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a >> 20, b >> 20, 0x0040), __byte_perm(c >> 20, d >> 20, 0x0040), 0x5410);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ float sqrt_approx(float x) {
    float y;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What a launch's elements share.
struct AdamStep {
    float gs, decay, rate, rbias2;
    uint32_t key;
};

// Eight elements a thread, 256 a warp, from e on.  Whole warps run on (the 8-bit
// scales are reduced across a warp); elements past the end hold zeros and are not
// stored.  kFull: all of the warp's elements exist.
template <bool kState8, bool kFull>
__device__ __forceinline__ void adamw_elements(const zb_adamw_tensor& t, const AdamArgs& a, const AdamStep& st, int64_t e) {
    const int64_t n = t.count;
    float g[8], m[8], v[8], p[8];
    if (t.grad_dtype == ZB_F32)
        load8f<kFull>(static_cast<const float*>(t.grad), e, n, g);
    else
        load8h<kFull>(static_cast<const uint16_t*>(t.grad), e, n, g);
    if (t.master || t.param_dtype == ZB_F32)
        load8f<kFull>(t.master ? t.master : static_cast<const float*>(t.param), e, n, p);
    else
        load8h<kFull>(static_cast<const uint16_t*>(t.param), e, n, p);
    const int64_t block = e / kStateBlock;
    if constexpr (kState8) {
        const uint2 cm = load8b<kFull>(static_cast<const uint8_t*>(t.m), e, n),
                    cv = load8b<kFull>(static_cast<const uint8_t*>(t.v), e, n);
        const float sm = t.m_scale[block], sv = t.v_scale[block];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            m[k] = decode_m(k < 4 ? cm.x : cm.y, k & 3, sm);
            v[k] = decode_v(k < 4 ? cv.x : cv.y, k & 3, sv);
        }
    } else {
        load8f<kFull>(static_cast<const float*>(t.m), e, n, m);
        load8f<kFull>(static_cast<const float*>(t.v), e, n, v);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float gk = a.grad_scale ? __fmul_rn(g[k], st.gs) : g[k];
        m[k] = __fadd_rn(__fmul_rn(m[k], a.beta1), __fmul_rn(gk, a.one_minus_beta1));
        v[k] = __fadd_rn(__fmul_rn(v[k], a.beta2), __fmul_rn(__fmul_rn(gk, gk), a.one_minus_beta2));
        p[k] = p[k] * st.decay - st.rate * (m[k] * rcp_approx(fmaf(sqrt_approx(v[k]), st.rbias2, a.eps)));
    }
    uint32_t noise[8];
    if (a.stochastic) {
        // mix32(element ^ key): e is a multiple of 8, so the eight words differ in their
        // low bits alone and share the first shift; elements past 2^32 start another stream
        uint32_t x = static_cast<uint32_t>(e) ^ (st.key + static_cast<uint32_t>(static_cast<uint64_t>(e) >> 32) * 0x632BE5ABu);
        x ^= x >> 16;
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
            uint32_t r = (x ^ k) * 0x7FEB352Du;
            r = (r ^ (r >> 15)) * 0x846CA68Bu;
            noise[k] = r ^ (r >> 16);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) noise[k] = 0x80008000u;
    }
    if constexpr (kState8) {
        float mm = 0.f, mv = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (kFull || e + k < n) {
                mm = fmaxf(mm, fabsf(m[k]));
                mv = fmaxf(mv, v[k]);
            }
        mm = warp_max(mm);
        mv = warp_max(mv);
        // a value that is not finite takes the largest code: its scale, were it infinite,
        // would make NaN of the block's other values
        const float tiny = 1.17549435e-38f, huge = 3.402823466e38f;
        mm = fminf(mm, huge);
        mv = fminf(mv, huge);
        const float sm = fmaxf(__fmul_rn(mm, 1.f / kMTop), tiny), sv = fmaxf(__fmul_rn(mv, 1.f / kVTop), tiny);
        const float im = __fdiv_rn(1.f, sm), iv = __fdiv_rn(1.f, sv);
        uint32_t cm[8], cv[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            cm[k] = code_bits(fminf(__fmul_rn(fabsf(m[k]), im), kMTop), (noise[k] << 4) & 0xFFFF0u);
            // the sign above the code's seven bits (27 is m's bit 31 four places down)
            cm[k] = (cm[k] & 0x07FFFFFFu) | ((__float_as_uint(m[k]) >> 4) & 0x08000000u);
            const float z = fminf(__fmul_rn(v[k], iv), kVTop);
            cv[k] = code_bits(z, (noise[k] >> 12) & 0xFFFF0u);
            if (z > 0.f) cv[k] = max(cv[k], 1u << 20);
        }
        store8b<kFull>(static_cast<uint8_t*>(t.m), e, n,
                       make_uint2(pack_codes(cm[0], cm[1], cm[2], cm[3]), pack_codes(cm[4], cm[5], cm[6], cm[7])));
        store8b<kFull>(static_cast<uint8_t*>(t.v), e, n,
                       make_uint2(pack_codes(cv[0], cv[1], cv[2], cv[3]), pack_codes(cv[4], cv[5], cv[6], cv[7])));
        if ((threadIdx.x & 31) == 0) {
            t.m_scale[block] = sm;
            t.v_scale[block] = sv;
        }
    } else {
        store8f<kFull>(static_cast<float*>(t.m), e, n, m);
        store8f<kFull>(static_cast<float*>(t.v), e, n, v);
    }
    if (t.master) store8f<kFull>(t.master, e, n, p);
    if (t.param_dtype == ZB_F32) {
        store8f<kFull>(static_cast<float*>(t.param), e, n, p);
        return;
    }
    uint32_t w[4];
    if (a.stochastic && !t.master) {
        // without a master copy the parameter itself rounds stochastically: an
        // update below half a bf16 step would otherwise be lost every time
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t u[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float x = p[2 * k + i];
                const uint32_t b = __float_as_uint(x);
                u[i] = fabsf(x) <= 3.3895314e38f ? (b + ((noise[2 * k + i] * 0x9E3779B1u) >> 16)) >> 16 : pack_bf16x2(x, 0.f) & 0xFFFFu;
            }
            w[k] = u[0] | (u[1] << 16);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = pack_bf16x2(p[2 * k], p[2 * k + 1]);
    }
    store8h<kFull>(static_cast<uint16_t*>(t.param), e, n, w);
}

// Bound by HBM with float32 moments: 218 M elements in 912 us, 7.2 TB/s.  With 8-bit ones the
// codecs' instructions all but bind it (80 % of issue slots): five blocks an SM (48 registers) ran one 8B-shaped layer's step and its
// read-back in 1058 us, four in 1105, six in 1112 (at 48 registers a thread stores 24 bytes and loads 16 in
// its stack frame, which that includes); blocks that loop over four chunks, to share the setup, in 1225.
template <bool kState8, int N>
__global__ void __launch_bounds__(kAdamThreads, kState8 ? 5 : 4) adamw_kernel(const __grid_constant__ AdamTable<N> tab, const __grid_constant__ AdamArgs a) {
    wait_for_previous();
    AdamStep st;
    // A scale that is not finite (an overflowed or NaN gradient norm) skips the step.
    st.gs = 1.f;
    if (a.grad_scale) {
        st.gs = *a.grad_scale;
        if (!(fabsf(st.gs) <= 3.402823466e38f)) return;
    }
    const int chunk = static_cast<int>(blockIdx.x);
    const int ti = find_tensor(tab, chunk);
    const zb_adamw_tensor& t = tab.t[ti];
    const float lr = a.lr_dev ? *a.lr_dev : a.lr;
    float bias1 = a.bias1;
    st.rbias2 = a.rsqrt_bias2;
    uint32_t step = a.step;
    if (a.step_dev) {
        const int64_t s = *a.step_dev;
        step = static_cast<uint32_t>(s);
        bias1 = -expm1f(static_cast<float>(s) * a.log_beta1);
        st.rbias2 = rsqrtf(-expm1f(static_cast<float>(s) * a.log_beta2));
    }
    st.decay = 1.f - lr * t.weight_decay;
    st.rate = lr / bias1;
    st.key = mix32(mix32(a.seed ^ (step * 0x9E3779B1u)) + static_cast<uint32_t>(tab.index0 + ti) * 0x85EBCA77u);
    const int64_t e = static_cast<int64_t>(chunk - tab.first[ti]) * kChunk + threadIdx.x * kPerThread;
    const int64_t warp_e = e - (threadIdx.x & 31) * kPerThread;
    if (warp_e + kStateBlock <= t.count)
        adamw_elements<kState8, true>(t, a, st, e);
    else if (warp_e < t.count)
        adamw_elements<kState8, false>(t, a, st, e);
}

// The 8-bit moments as float32 values.
template <int N>
__global__ void __launch_bounds__(kAdamThreads) adamw_unpack_kernel(const __grid_constant__ AdamTable<N> tab,
                                                                    const __grid_constant__ AdamUnpack<N> out) {
    wait_for_previous();
    const int chunk = static_cast<int>(blockIdx.x);
    const int ti = find_tensor(tab, chunk);
    const zb_adamw_tensor& t = tab.t[ti];
    const int64_t n = t.count;
    const int64_t e = static_cast<int64_t>(chunk - tab.first[ti]) * kChunk + threadIdx.x * kPerThread;
    if (e >= n) return;
    const uint2 cm = load8b<false>(static_cast<const uint8_t*>(t.m), e, n), cv = load8b<false>(static_cast<const uint8_t*>(t.v), e, n);
    const float sm = t.m_scale[e / kStateBlock], sv = t.v_scale[e / kStateBlock];
    float m[8], v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        m[k] = decode_m(k < 4 ? cm.x : cm.y, k & 3, sm);
        v[k] = decode_v(k < 4 ? cv.x : cv.y, k & 3, sv);
    }
    store8f<false>(out.m[ti], e, n, m);
    store8f<false>(out.v[ti], e, n, v);
}

// Sums of squares.  The chunks of a launch go round-robin to a fixed number of
// blocks, whatever the device, and each block writes one float64: a fixed
// partition and order, so the norm is the same bits every time.  Squares are summed
// in float32, eight sums a thread: FP64 units are scarce, and positive terms'
// rounding errors average out (about 1e-7 of the norm measured).  Bound by HBM: 218 M
// float32 gradients in 122 us, 7.2 TB/s.
constexpr int kNormChunks = 4;       // chunks of a block in flight
constexpr int kNormBlocks = 1216;    // eight blocks on each of 152 SMs

// Sum of squares of thread `threadIdx.x`'s elements of chunks blockIdx.x + i gridDim.x;
// `top`: the largest of their sizes.
template <typename T, int N>
__device__ __forceinline__ T thread_squares(const AdamTable<N>& tab, int chunks, float& top) {
    T s[8] = {};
    top = 0.f;
    for (int64_t c0 = blockIdx.x; c0 < chunks; c0 += static_cast<int64_t>(kNormChunks) * gridDim.x) {
        float g[kNormChunks][8];
#pragma unroll
        for (int i = 0; i < kNormChunks; ++i) {
            const int64_t c = c0 + static_cast<int64_t>(i) * gridDim.x;
#pragma unroll
            for (int k = 0; k < 8; ++k) g[i][k] = 0.f;
            if (c < chunks) {
                const int ti = find_tensor(tab, static_cast<int>(c));
                const zb_adamw_tensor& t = tab.t[ti];
                const int64_t e = (c - tab.first[ti]) * kChunk + threadIdx.x * kPerThread;
                if (t.grad_dtype == ZB_F32)
                    load8f<false>(static_cast<const float*>(t.grad), e, t.count, g[i]);
                else
                    load8h<false>(static_cast<const uint16_t*>(t.grad), e, t.count, g[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kNormChunks; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                s[k] += static_cast<T>(g[i][k]) * static_cast<T>(g[i][k]);
                top = fmaxf(top, fabsf(g[i][k]));
            }
    }
    return ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
}

template <int N>
__global__ void __launch_bounds__(kAdamThreads) norm_partial_kernel(const __grid_constant__ AdamTable<N> tab, int chunks,
                                                                    double* part) {
    __shared__ double red[kAdamThreads / 32];
    wait_for_previous();
    float top;
    float sum = thread_squares<float>(tab, chunks, top);
    // squares that leave float32's range (or all but leave it) are summed again in
    // float64, by the whole warp
    const bool ok = sum <= 1e30f && (sum >= 1e-25f || top == 0.f);
    double total;
    if (__all_sync(0xffffffffu, ok)) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        total = sum;
    } else {
        total = thread_squares<double>(tab, chunks, top);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = total;
    __syncthreads();
    if (threadIdx.x < 8) {
        total = red[threadIdx.x];
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) total += __shfl_xor_sync(0xffu, total, o);
        if (threadIdx.x == 0) part[blockIdx.x] = total;
    }
}

// out[0] = the norm, out[1] = min(1, max_norm / (norm + 1e-6)).
__global__ void __launch_bounds__(256) norm_final_kernel(const double* part, int64_t n, float max_norm, float* out) {
    __shared__ double red[8];
    wait_for_previous();
    double sum = 0.0;
    for (int64_t i0 = threadIdx.x; i0 < n; i0 += 8 * 256) {
        double v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = i0 + k * 256 < n ? part[i0 + k * 256] : 0.0;
        sum += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x < 8) {
        sum = red[threadIdx.x];
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffu, sum, o);
        if (threadIdx.x == 0) {
            // float32's square root where the sum is in its range: float64's takes longer than all the rest
            const float norm = sum > 1e-30 && sum < 1e30 ? sqrtf(static_cast<float>(sum)) : static_cast<float>(sqrt(sum));
            out[0] = norm;
            // a NaN or infinite norm gives a NaN coefficient, which skips the step
            out[1] = fabsf(norm) <= 3.402823466e38f ? fminf(1.f, max_norm / (norm + 1e-6f)) : __int_as_float(0x7FC00000);
        }
    }
}

int64_t chunks_of(int64_t count, int64_t per) { return (count + per - 1) / per; }

// Calls fn(table, chunks, first tensor) for every group of tensors that fits a table;
// empty tensors take no chunk.
template <int N, typename Fn>
cudaError_t for_groups(const zb_adamw_tensor* ts, int n, int per, Fn&& fn) {
    for (int i0 = 0; i0 < n; i0 += N) {
        AdamTable<N> tab;
        tab.n = std::min(N, n - i0);
        tab.index0 = i0;
        int64_t c = 0;
        for (int i = 0; i < tab.n; ++i) {
            tab.t[i] = ts[i0 + i];
            tab.first[i] = static_cast<int>(c);
            c += chunks_of(ts[i0 + i].count, per);
            if (c > 0x7fffffff) return cudaErrorInvalidValue;
        }
        tab.first[tab.n] = static_cast<int>(c);
        if (c == 0) continue;
        const cudaError_t e = fn(tab, c, i0);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}
template <typename Fn>
cudaError_t for_tables(const zb_adamw_tensor* ts, int n, int per, Fn&& fn) {
    return n <= kFewTensors ? for_groups<kFewTensors>(ts, n, per, fn) : for_groups<kManyTensors>(ts, n, per, fn);
}

constexpr int64_t kMaxCount = int64_t(1) << 40;

zb_status tensors_ok(const zb_adamw_tensor* ts, int32_t n) {
    if (n < 0 || (n > 0 && !ts)) return ZB_ERR_ARG;
    int64_t total = 0;
    for (int i = 0; i < n; ++i) {
        if (ts[i].count < 0 || ts[i].count > kMaxCount) return ZB_ERR_SHAPE;
        total += ts[i].count;
        if (total > kMaxCount) return ZB_ERR_SHAPE;
        if ((ts[i].grad_dtype != ZB_BF16 && ts[i].grad_dtype != ZB_F32) ||
            (ts[i].param_dtype != ZB_BF16 && ts[i].param_dtype != ZB_F32))
            return ZB_ERR_ARG;
    }
    return ZB_OK;
}

zb_status moments_ok(const zb_adamw_tensor& t, bool state8) {
    if (t.count == 0) return ZB_OK;
    if (!fixed_ok(t.m) || !fixed_ok(t.v)) return ZB_ERR_ARG;
    if (state8 && (!fixed_ok(t.m_scale) || !fixed_ok(t.v_scale))) return ZB_ERR_ARG;
    return ZB_OK;
}

}  // namespace

}  // namespace zbk

using namespace zbk;

extern "C" zb_status zb_op_adamw_step(const zb_adamw_tensor* tensors, int32_t n, const zb_adamw_config* cfg, int64_t step,
                                      const float* grad_scale, const float* lr_device, const int64_t* step_device,
                                      void* stream) {
    if (!cfg) return ZB_ERR_ARG;
    ZB_TRY(tensors_ok(tensors, n));
    if (cfg->state_bits != 32 && cfg->state_bits != 8) return ZB_ERR_ARG;
    if (!(cfg->beta1 >= 0.0 && cfg->beta1 < 1.0) || !(cfg->beta2 >= 0.0 && cfg->beta2 < 1.0) || !(cfg->eps >= 1e-30) ||
        !std::isfinite(cfg->eps) || !std::isfinite(cfg->lr) || (!step_device && step < 1))
        return ZB_ERR_ARG;
    auto word_ok = [](const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; };
    if (!word_ok(grad_scale, 4) || !word_ok(lr_device, 4) || !word_ok(step_device, 8)) return ZB_ERR_ARG;
    const bool state8 = cfg->state_bits == 8;
    for (int i = 0; i < n; ++i) {
        const zb_adamw_tensor& t = tensors[i];
        if (!std::isfinite(t.weight_decay)) return ZB_ERR_ARG;
        if (t.count == 0) continue;
        if (!fixed_ok(t.param) || !fixed_ok(t.grad) || (t.master && !aligned16(t.master))) return ZB_ERR_ARG;
        if (t.master && t.param_dtype == ZB_F32) return ZB_ERR_ARG;  // a float32 parameter is its own master
        ZB_TRY(moments_ok(t, state8));
    }
    ZB_TRY(device_ok());
    AdamArgs a{};
    a.beta1 = static_cast<float>(cfg->beta1);
    a.beta2 = static_cast<float>(cfg->beta2);
    a.one_minus_beta1 = static_cast<float>(1.0 - cfg->beta1);
    a.one_minus_beta2 = static_cast<float>(1.0 - cfg->beta2);
    a.eps = static_cast<float>(cfg->eps);
    a.lr = static_cast<float>(cfg->lr);
    if (!step_device) {
        a.bias1 = static_cast<float>(1.0 - std::pow(cfg->beta1, static_cast<double>(step)));
        a.rsqrt_bias2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(cfg->beta2, static_cast<double>(step))));
        a.step = static_cast<uint32_t>(step);
    }
    a.log_beta1 = static_cast<float>(std::log(cfg->beta1));
    a.log_beta2 = static_cast<float>(std::log(cfg->beta2));
    a.seed = cfg->seed;
    a.stochastic = cfg->stochastic != 0;
    a.grad_scale = grad_scale;
    a.lr_dev = lr_device;
    a.step_dev = step_device;
    cudaStream_t s = as_stream(stream);
    return cuda_status(for_tables(tensors, n, kChunk, [&](const auto& tab, int64_t c, int) {
        if (state8)
            return launch_chained(adamw_kernel<true, std::extent<decltype(tab.t)>::value>, static_cast<unsigned>(c), kAdamThreads, 0, s, tab, a);
        return launch_chained(adamw_kernel<false, std::extent<decltype(tab.t)>::value>, static_cast<unsigned>(c), kAdamThreads, 0, s, tab, a);
    }));
}

extern "C" zb_status zb_op_adamw_unpack(const zb_adamw_tensor* tensors, int32_t n, float* const* m, float* const* v,
                                        void* stream) {
    ZB_TRY(tensors_ok(tensors, n));
    if (n > 0 && (!m || !v)) return ZB_ERR_ARG;
    for (int i = 0; i < n; ++i) {
        ZB_TRY(moments_ok(tensors[i], true));
        if (tensors[i].count > 0 && (!fixed_ok(m[i]) || !fixed_ok(v[i]))) return ZB_ERR_ARG;
    }
    ZB_TRY(device_ok());
    cudaStream_t s = as_stream(stream);
    return cuda_status(for_tables(tensors, n, kChunk, [&](const auto& tab, int64_t c, int i0) {
        AdamUnpack<std::extent<decltype(tab.t)>::value> out;
        for (int i = 0; i < tab.n; ++i) {
            out.m[i] = m[i0 + i];
            out.v[i] = v[i0 + i];
        }
        return launch_chained(adamw_unpack_kernel<std::extent<decltype(tab.t)>::value>, static_cast<unsigned>(c), kAdamThreads, 0, s, tab,
                              out);
    }));
}

extern "C" size_t zb_op_grad_norm_scratch_bytes(const zb_adamw_tensor* tensors, int32_t n) {
    if (tensors_ok(tensors, n) != ZB_OK) return 0;
    const int64_t launches = (n + kManyTensors - 1) / kManyTensors;
    return static_cast<size_t>(std::max<int64_t>(launches, 1)) * kNormBlocks * sizeof(double);
}

extern "C" zb_status zb_op_grad_norm(const zb_adamw_tensor* tensors, int32_t n, float max_norm, float* out, void* scratch,
                                     size_t scratch_bytes, void* stream) {
    ZB_TRY(tensors_ok(tensors, n));
    if (!(max_norm > 0.f) || !fixed_ok(out)) return ZB_ERR_ARG;
    for (int i = 0; i < n; ++i)
        if (tensors[i].count > 0 && !fixed_ok(tensors[i].grad)) return ZB_ERR_ARG;
    if (!scratch || !aligned16(scratch) || scratch_bytes < zb_op_grad_norm_scratch_bytes(tensors, n)) return ZB_ERR_WORKSPACE;
    ZB_TRY(device_ok());
    cudaStream_t s = as_stream(stream);
    double* part = static_cast<double*>(scratch);
    int64_t done = 0;
    const cudaError_t e = for_tables(tensors, n, kChunk, [&](const auto& tab, int64_t c, int) {
        const int64_t blocks = std::min<int64_t>(c, kNormBlocks);
        double* at = part + done;
        done += blocks;
        return launch_chained(norm_partial_kernel<std::extent<decltype(tab.t)>::value>, static_cast<unsigned>(blocks), kAdamThreads, 0, s,
                              tab, static_cast<int>(c), at);
    });
    if (e != cudaSuccess) return ZB_ERR_CUDA;
    return cuda_status(launch_chained(norm_final_kernel, 1, 256, 0, s, part, done, max_norm, out));
}
