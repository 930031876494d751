// The norms around a block with its gate and its residual scales, forward and split
// backward.  With y the block's output and x the residual stream that entered it:
//   F   u = PostNorm(y),  h = bf16(a x + b gate u),  n = PreNorm(h), the next block's input
//   B   dh = dres + PreNorm'(dn),  dx = a dh,  dy = PostNorm'(b gate dh),  dgate = b u dh
//   W   the norms' weights and biases, and a gate per channel
// Norm(v) = gamma (v - mean) rstd + beta; an RMS norm has mean 0 and no beta of its own.
//
// F and B take a row in one pass: its threads hold all of it in registers, so that every
// tensor is read and written once; the sums over the row go through shuffles, and shared
// memory where a row has more than one warp.  The data is bound by HBM, a row by its latency: loads,
// two sums, stores (6 us for 4096 columns), of which an SM has as many at a time as its registers
// hold.  So blocks bring the rows behind theirs into L2.  GB300, bytes at 6.8 TB/s in brackets: F with an
// 8-bit output 33.5 us for 4096 rows of 4096 columns (22.4) and 59 for 8192 columns (44.7); B
// 38.3 (29.7) and 71.5 (59.4).
#include <algorithm>
#include <cmath>

#include "chained.cuh"
#include "checkpoint.cuh"
#include "checks.h"
#include "device_common.cuh"

namespace zbk {

namespace {

constexpr int kNormMaxHidden = 32768;

struct NormParams {
    const uint16_t* x;   // F
    const uint16_t* y;
    const uint16_t* gate_token;
    const float* gate_channel;
    const float *post_gamma, *post_beta, *pre_gamma, *pre_beta;
    uint16_t* h;         // F: written, B: read
    uint16_t* n;
    uint8_t *codes, *scales;
    float4* stats;       // per row: post mean, post rstd, pre mean, pre rstd
    const uint16_t *dn, *dres;  // B
    uint16_t *dh, *dx, *dy, *dgate;
    float a, b, post_eps, pre_eps;
    int hidden, post, pre;
    int ahead;  // a row's block brings the row so far behind it into L2
};

// Eight values as four pairs, for the packed float32 instructions.
struct F8 {
    float2 p[4];
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ F8 widen(const uint4& q) {
    return F8{{make_float2(bf16_lo(q.x), bf16_hi(q.x)), make_float2(bf16_lo(q.y), bf16_hi(q.y)),
               make_float2(bf16_lo(q.z), bf16_hi(q.z)), make_float2(bf16_lo(q.w), bf16_hi(q.w))}};
}

__device__ __forceinline__ uint4 narrow(const F8& f) {
    return make_uint4(pack_bf16x2(f.p[0].x, f.p[0].y), pack_bf16x2(f.p[1].x, f.p[1].y), pack_bf16x2(f.p[2].x, f.p[2].y),
                      pack_bf16x2(f.p[3].x, f.p[3].y));
}

// Parameters.  They are constant from before a kernel that may run ahead of this one's start
// (release_next) to this one's end, so they may be read ahead of this kernel's stores, which
// took 10 us off the 70B-shaped backward (87 to 77, before rows came ahead into L2).
__device__ __forceinline__ F8 load_f8(const float* p) {
    float4 a, b;
    asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(a.x), "=f"(a.y), "=f"(a.z), "=f"(a.w) : "l"(p));
    asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(b.x), "=f"(b.y), "=f"(b.z), "=f"(b.w) : "l"(p + 4));
    return F8{{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)}};
}

// A row's data pass by L1, which keeps the parameters that every row reads.
__device__ __forceinline__ uint4 load_q(const uint16_t* p) {
    uint4 q;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "l"(p));
    return q;
}
// A row of a tensor into L2.
__device__ __forceinline__ void prefetch_row(const uint16_t* p, int64_t at, int hidden) {
    if (p) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p + at), "r"(2 * hidden) : "memory");
}

__device__ __forceinline__ void store_q(uint16_t* p, const uint4& q) { *reinterpret_cast<uint4*>(p) = q; }

__device__ __forceinline__ void affine(F8& v, float scale, float shift) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v.p[e] = __ffma2_rn(v.p[e], both(scale), both(shift));
}

// The normed value.  The difference first, which is exact where the mean is near: v rstd - mean rstd
// in one step would leave half a last place of mean rstd, 0.015 for a row of thousands.
__device__ __forceinline__ void centered(F8& v, float mean, float rstd) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v.p[e] = __fmul2_rn(__fadd2_rn(v.p[e], both(-mean)), both(rstd));
}

__device__ __forceinline__ void times(F8& v, const F8& g) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v.p[e] = __fmul2_rn(v.p[e], g.p[e]);
}

// v gamma + beta
__device__ __forceinline__ void weigh(F8& v, const float* gamma, const float* beta, int at) {
    const F8 g = load_f8(gamma + at);
    if (beta) {
        const F8 b = load_f8(beta + at);
#pragma unroll
        for (int e = 0; e < 4; ++e) v.p[e] = __ffma2_rn(v.p[e], g.p[e], b.p[e]);
    } else {
        times(v, g);
    }
}

// Sums of (s0, s1) over the threads of a row.  Each use of `round` has shared memory of its
// own, so that one barrier a sum is enough.
template <int kRow>
__device__ __forceinline__ float2 row_sum(float2 s, float2 (*red)[32], int round) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        s = __fadd2_rn(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, o), __shfl_xor_sync(0xffffffffu, s.y, o)));
    if constexpr (kRow > 32) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) red[round][warp] = s;
        __syncthreads();
        constexpr int kWarps = kRow / 32;
        s = red[round][lane & (kWarps - 1)];
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1)
            s = __fadd2_rn(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, o), __shfl_xor_sync(0xffffffffu, s.y, o)));
    }
    return s;
}

// Rows of a block, kRow threads each (one row where a row has more than a warp).
template <int kRow>
__host__ __device__ constexpr int norm_rows() {
    return kRow == 32 ? 4 : 1;
}

// Blocks that an SM takes at once with `regs` registers a thread.
template <int kRow>
__host__ __device__ constexpr int norm_blocks(int regs) {
    return 65536 / (kRow * norm_rows<kRow>() * regs) > 1 ? 65536 / (kRow * norm_rows<kRow>() * regs) : 1;
}

// Mean and 1 / sqrt(variance + eps) of a row whose thread holds kPer groups of 8 values
// (zeros past the row's end, unless kFull).  A layer norm's variance is of the differences from
// the mean: a second sum, which a mean far from zero cannot spoil.
template <int kRow, int kPer, bool kFull>
__device__ __forceinline__ float2 moments(const F8 (&v)[kPer], int tid, int chunks, int kind, float eps, float inv,
                                          float2 (*red)[32], int round) {
    float2 q = both(0.f);
    float mean = 0.f;
    if (kind == ZB_NORM_LAYER) {
        float2 s = both(0.f);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s = __fadd2_rn(s, v[i].p[e]);
        mean = row_sum<kRow>(make_float2(s.x + s.y, 0.f), red, round).x / static_cast<float>(8 * chunks);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (!kFull && tid + i * kRow >= chunks) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 d = __fadd2_rn(v[i].p[e], both(-mean));
                q = __ffma2_rn(d, d, q);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) q = __ffma2_rn(v[i].p[e], v[i].p[e], q);
    }
    const float var = row_sum<kRow>(make_float2(q.x + q.y, 0.f), red, round + 1).x * inv;
    return make_float2(mean, rsqrtf(var + eps));
}

template <int kRow, int kPer, bool kFull>
__global__ void __launch_bounds__(kRow * norm_rows<kRow>(), norm_blocks<kRow>(kRow == 512 ? 64 : 80))
    residual_norm_forward_kernel(const __grid_constant__ NormParams p, int tokens) {
    __shared__ float2 red[4][32];
    release_next();
    wait_for_previous();
    const int tid = kRow == 32 ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t row = kRow == 32 ? static_cast<int64_t>(blockIdx.x) * norm_rows<kRow>() + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= tokens) return;  // whole warps
    const int64_t base = row * p.hidden;
    const int chunks = p.hidden >> 3;
    const float inv = 1.f / static_cast<float>(p.hidden);
    auto inside = [&](int i) { return kFull || tid + i * kRow < chunks; };
    if (tid == 0 && row + p.ahead < tokens) {
        const int64_t at = (row + p.ahead) * p.hidden;
        prefetch_row(p.y, at, p.hidden);
        prefetch_row(p.x, at, p.hidden);
        prefetch_row(p.gate_token, at, p.hidden);
    }
    uint4 xq[kPer];
    F8 u[kPer];
    {
        uint4 yq[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            yq[i] = inside(i) ? load_q(p.y + base + 8 * (tid + i * kRow)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (inside(i)) xq[i] = load_q(p.x + base + 8 * (tid + i * kRow));
#pragma unroll
        for (int i = 0; i < kPer; ++i) u[i] = widen(yq[i]);
    }
    float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.post != ZB_NORM_NONE) {
        const float2 m = moments<kRow, kPer, kFull>(u, tid, chunks, p.post, p.post_eps, inv, red, 0);
        st.x = m.x;
        st.y = m.y;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (!inside(i)) continue;
        const int at = 8 * (tid + i * kRow);
        if (p.post != ZB_NORM_NONE) {
            centered(u[i], st.x, st.y);
            weigh(u[i], p.post_gamma, p.post_beta, at);
        }
        if (p.gate_channel)
            times(u[i], load_f8(p.gate_channel + at));
        else if (p.gate_token)
            times(u[i], widen(load_q(p.gate_token + base + at)));
        const F8 x = widen(xq[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) u[i].p[e] = __ffma2_rn(u[i].p[e], both(p.b), __fmul2_rn(x.p[e], both(p.a)));
        const uint4 hq = narrow(u[i]);
        store_q(p.h + base + at, hq);
        u[i] = widen(hq);  // n is the norm of the h that is stored
    }
    if (p.pre != ZB_NORM_NONE) {
        const float2 m = moments<kRow, kPer, kFull>(u, tid, chunks, p.pre, p.pre_eps, inv, red, 2);
        st.z = m.x;
        st.w = m.y;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = 8 * (tid + i * kRow);
            uint4 nq = make_uint4(0, 0, 0, 0);
            if (inside(i)) {
                centered(u[i], st.z, st.w);
                weigh(u[i], p.pre_gamma, p.pre_beta, at);
                nq = narrow(u[i]);
                if (p.n) store_q(p.n + base + at, nq);
            }
            if (p.codes) {  // four threads hold a block of 32 (a row has a multiple of 8 chunks)
                const uint32_t top2 = pack_top2(pack_top2(pack_top2(pack_top2(0u, nq.x), nq.y), nq.z), nq.w);
                uint32_t top = pack_top(top2);
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                if (inside(i)) {
                    const uint32_t scale = pack_scale(top);
                    const uint32_t f = pack_factor(scale);
                    *reinterpret_cast<uint2*>(p.codes + base + at) =
                        top < kPackLargest ? make_uint2(pack_codes(nq.x, nq.y, f), pack_codes(nq.z, nq.w, f))
                                           : make_uint2(pack_codes_slow(nq.x, nq.y, f, scale), pack_codes_slow(nq.z, nq.w, f, scale));
                    if ((tid & 3) == 0) p.scales[(base + at) >> 5] = static_cast<uint8_t>(scale);
                }
            }
        }
    }
    if (tid == 0) p.stats[row] = st;
}

// The input gradient of a norm of rows: d is the gradient of the normed values `hat`:
//   rstd (d - hat mean(d hat) - [layer] mean(d)).
template <int kRow, int kPer, bool kFull>
__global__ void __launch_bounds__(kRow * norm_rows<kRow>(), norm_blocks<kRow>(128))
    residual_norm_backward_kernel(const __grid_constant__ NormParams p, int tokens) {
    __shared__ float2 red[2][32];
    release_next();
    wait_for_previous();
    const int tid = kRow == 32 ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t row = kRow == 32 ? static_cast<int64_t>(blockIdx.x) * norm_rows<kRow>() + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= tokens) return;  // whole warps
    const int64_t base = row * p.hidden;
    const int chunks = p.hidden >> 3;
    const float inv = 1.f / static_cast<float>(p.hidden);
    const bool pre = p.pre != ZB_NORM_NONE, post = p.post != ZB_NORM_NONE;
    auto inside = [&](int i) { return kFull || tid + i * kRow < chunks; };
    if (tid == 0 && row + p.ahead < tokens) {
        const int64_t at = (row + p.ahead) * p.hidden;
        prefetch_row(pre ? p.dn : nullptr, at, p.hidden);
        prefetch_row(pre ? p.h : nullptr, at, p.hidden);
        prefetch_row(p.dres, at, p.hidden);
        prefetch_row(p.y, at, p.hidden);
        prefetch_row(p.gate_token, at, p.hidden);
    }
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 nq[kPer], hq[kPer], yq[kPer];
    F8 dh[kPer];
    const float4 st = p.stats[row];
#pragma unroll
    for (int i = 0; i < kPer; ++i) nq[i] = pre && inside(i) ? load_q(p.dn + base + 8 * (tid + i * kRow)) : zero;
#pragma unroll
    for (int i = 0; i < kPer; ++i) hq[i] = pre && inside(i) ? load_q(p.h + base + 8 * (tid + i * kRow)) : zero;
    {
        uint4 rq[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) rq[i] = p.dres && inside(i) ? load_q(p.dres + base + 8 * (tid + i * kRow)) : zero;
#pragma unroll
        for (int i = 0; i < kPer; ++i) yq[i] = p.y && inside(i) ? load_q(p.y + base + 8 * (tid + i * kRow)) : zero;
#pragma unroll
        for (int i = 0; i < kPer; ++i) dh[i] = widen(rq[i]);
    }
    if (pre) {
        float2 s0 = both(0.f), s1 = both(0.f);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (!inside(i)) continue;
            F8 d = widen(nq[i]), hat = widen(hq[i]);
            times(d, load_f8(p.pre_gamma + 8 * (tid + i * kRow)));
            centered(hat, st.z, st.w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s0 = __ffma2_rn(d.p[e], hat.p[e], s0);
                s1 = __fadd2_rn(s1, d.p[e]);
            }
        }
        const float2 s = row_sum<kRow>(make_float2(s0.x + s0.y, s1.x + s1.y), red, 0);
        const float m0 = -st.w * (s.x * inv), m1 = p.pre == ZB_NORM_LAYER ? -st.w * (s.y * inv) : 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (!inside(i)) continue;
            F8 d = widen(nq[i]), hat = widen(hq[i]);
            times(d, load_f8(p.pre_gamma + 8 * (tid + i * kRow)));
            centered(hat, st.z, st.w);
            affine(hat, m0, m1);
#pragma unroll
            for (int e = 0; e < 4; ++e) dh[i].p[e] = __fadd2_rn(__ffma2_rn(d.p[e], both(st.w), hat.p[e]), dh[i].p[e]);
        }
    }
    float2 s0 = both(0.f), s1 = both(0.f);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (!inside(i)) continue;
        const int at = 8 * (tid + i * kRow);
        store_q(p.dh + base + at, narrow(dh[i]));
        if (p.dx) {
            F8 dx = dh[i];
            affine(dx, p.a, 0.f);
            store_q(p.dx + base + at, narrow(dx));
        }
        // dh becomes the gradient of what the gate multiplies, then of the normed y
        affine(dh[i], p.b, 0.f);
        if (p.dgate) {
            F8 u = widen(yq[i]);
            if (post) {
                centered(u, st.x, st.y);
                weigh(u, p.post_gamma, p.post_beta, at);
            }
            times(u, dh[i]);
            store_q(p.dgate + base + at, narrow(u));
        }
        if (p.gate_channel)
            times(dh[i], load_f8(p.gate_channel + at));
        else if (p.gate_token)
            times(dh[i], widen(load_q(p.gate_token + base + at)));
        if (post) {
            times(dh[i], load_f8(p.post_gamma + at));
            F8 hat = widen(yq[i]);
            centered(hat, st.x, st.y);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s0 = __ffma2_rn(dh[i].p[e], hat.p[e], s0);
                s1 = __fadd2_rn(s1, dh[i].p[e]);
            }
        }
    }
    float m0 = 0.f, m1 = 0.f;
    if (post) {
        const float2 s = row_sum<kRow>(make_float2(s0.x + s0.y, s1.x + s1.y), red, 1);
        m0 = -st.y * (s.x * inv);
        m1 = p.post == ZB_NORM_LAYER ? -st.y * (s.y * inv) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (!inside(i)) continue;
        if (post) {
            F8 hat = widen(yq[i]);
            centered(hat, st.x, st.y);
            affine(hat, m0, m1);
#pragma unroll
            for (int e = 0; e < 4; ++e) dh[i].p[e] = __ffma2_rn(dh[i].p[e], both(st.y), hat.p[e]);
        }
        store_q(p.dy + base + 8 * (tid + i * kRow), narrow(dh[i]));
    }
}

// ---------------------------------------------------------------- weight gradients
//
// Two pairs of sums over the rows for every column: dn and dn hhat; gdh and gdh yhat, where
// gdh is dh (times the gate per token) and yhat the normed y (y itself without a post norm).
// A gate per channel is a factor of the sums, so dgate and the post norm's gradients come
// from the same two.  Where only a beta is asked for, its pair's h or y is not read (NULL) and
// the second sum not used.  Two passes in a fixed order: sums over parts of the rows
// ([parts][4][hidden]), then over the parts.

constexpr int kWThreads = 256;
constexpr int kWGroups = 8;
constexpr int kWUnroll = 2;
// Blocks of each pair, at most: 3 of 256 threads on each of 152 SMs, six for both pairs, all at
// once.  With a few more a second round starts: 8597 rows of 3776 columns in 60 us with 615 of 608 that
// fit, 45 with 450.  A gate per token takes the registers of four blocks an SM, so that both pairs' last blocks wait for a
// second round; that form is no further from its bytes all the same (4096 rows of 4096: 32.3 us of 24.7, 26.7 of 19.8 without; 8597
// of 3776: 55.7 of 47.9, 45.1 of 38.3).  The parts are the same whatever is formed, so that a gradient asked for alone has the
// same bits; one pair alone then fills half of the SMs' blocks (19 us for half the bytes).
constexpr int kWTargetBlocks = 456;
constexpr int kWMostParts = 152;     // few columns: 16384 rows of 256 in 19 us (608 parts: 29)

int norm_parts(int tokens, int hidden) {
    const int across = (hidden + 255) / 256;
    return std::max(1, std::min({kWTargetBlocks / across, kWMostParts, (tokens + kWGroups - 1) / kWGroups}));
}

// Block x + across (y + parts z): columns 256 x ..., the y-th part of the rows, pair first + z.
// Bound by HBM.  kMeans: a layer norm is among them (8B-shaped sums take 26.0 us without one, 27.1 with).
template <bool kTokenGate, bool kMeans>
__global__ void __launch_bounds__(kWThreads, kTokenGate ? 4 : 6)
    residual_norm_parts_kernel(const __grid_constant__ NormParams p, float* parts, int tokens, int first, int n_parts) {
    __shared__ float sums[2][kWGroups][256];
    release_next();
    wait_for_previous();
    const int across = (p.hidden + 255) / 256, bx = blockIdx.x % across;
    const int by = blockIdx.x / across % n_parts, bz = blockIdx.x / across / n_parts;
    const bool branch = first + bz == 1;
    const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
    const int col = bx * 256 + 8 * lane;
    const int per = (tokens + n_parts - 1) / n_parts;
    const int t0 = by * per, t1 = min(tokens, t0 + per);
    const uint16_t* d_of = branch ? p.dh : p.dn;
    const uint16_t* v_of = branch ? p.y : p.h;
    const uint16_t* gate = kTokenGate && branch ? p.gate_token : nullptr;
    const bool normed = v_of && (!branch || p.post != ZB_NORM_NONE);
    F8 s0{}, s1{};
    if (col < p.hidden) {
        for (int tb = t0 + group; tb < t1; tb += kWGroups * kWUnroll) {
            uint4 dq[kWUnroll], vq[kWUnroll], gq[kTokenGate ? kWUnroll : 1] = {};
            float2 st[kWUnroll];  // mean, rstd
#pragma unroll
            for (int i = 0; i < kWUnroll; ++i) {
                const int t = tb + i * kWGroups;
                dq[i] = vq[i] = make_uint4(0, 0, 0, 0);
                st[i] = make_float2(0.f, 1.f);
                if (t >= t1) continue;
                const int64_t at = static_cast<int64_t>(t) * p.hidden + col;
                dq[i] = load_q(d_of + at);
                if (v_of) vq[i] = load_q(v_of + at);
                if constexpr (kTokenGate)
                    if (gate) gq[i] = load_q(gate + at);
                if (normed) st[i] = reinterpret_cast<const float2*>(p.stats)[2 * static_cast<int64_t>(t) + (branch ? 0 : 1)];
            }
#pragma unroll
            for (int i = 0; i < kWUnroll; ++i) {
                const uint4& gi = gq[kTokenGate ? i : 0];
                const uint32_t dw[4] = {dq[i].x, dq[i].y, dq[i].z, dq[i].w}, vw[4] = {vq[i].x, vq[i].y, vq[i].z, vq[i].w};
                const uint32_t gw[4] = {gi.x, gi.y, gi.z, gi.w};
                // pair by pair: in steps of eight values, six blocks' registers do not hold them (layer norms 28.5 us, 27.1)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 d = make_float2(bf16_lo(dw[e]), bf16_hi(dw[e])), hat = make_float2(bf16_lo(vw[e]), bf16_hi(vw[e]));
                    if constexpr (kTokenGate)
                        if (gate) d = __fmul2_rn(d, make_float2(bf16_lo(gw[e]), bf16_hi(gw[e])));
                    if constexpr (kMeans) hat = __fadd2_rn(hat, both(-st[i].x));
                    hat = __fmul2_rn(hat, both(st[i].y));
                    s0.p[e] = __fadd2_rn(s0.p[e], d);
                    s1.p[e] = __ffma2_rn(d, hat, s1.p[e]);
                }
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        *reinterpret_cast<float2*>(&sums[0][group][8 * lane + 2 * e]) = s0.p[e];
        *reinterpret_cast<float2*>(&sums[1][group][8 * lane + 2 * e]) = s1.p[e];
    }
    __syncthreads();
    const int j = bx * 256 + threadIdx.x;
    if (j >= p.hidden) return;
    float* out = parts + (static_cast<int64_t>(by) * 4 + (branch ? 2 : 0)) * p.hidden + j;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float s = 0.f;
#pragma unroll
        for (int g = 0; g < kWGroups; ++g) s += sums[k][g][threadIdx.x];
        out[static_cast<int64_t>(k) * p.hidden] = s;
    }
}

struct NormGrads {
    float *post_gamma, *post_beta, *pre_gamma, *pre_beta, *gate;
};

// A block finishes 32 columns: warp (k, g) adds the parts g, g + 8, ... of sum k.
__global__ void __launch_bounds__(1024) residual_norm_sum_kernel(const __grid_constant__ NormParams p, const NormGrads out,
                                                                 const float* parts, int n_parts, bool pre,
                                                                 bool branch) {
    __shared__ float sums[4][8][32];
    release_next();
    wait_for_previous();
    const int c = threadIdx.x & 31, k0 = (threadIdx.x >> 5) & 3, g = threadIdx.x >> 7;
    const int j = blockIdx.x * 32 + c;
    if (k0 < 2 ? pre : branch) {
        float s = 0.f;
        for (int q0 = g; q0 < n_parts; q0 += 64) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = q0 + 8 * i < n_parts ? parts[(static_cast<int64_t>(q0 + 8 * i) * 4 + k0) * p.hidden + j] : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[i];
        }
        sums[k0][g][c] = s;
    }
    __syncthreads();
    if (threadIdx.x >= 32) return;
    float t[4] = {};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (k < 2 ? !pre : !branch) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) t[k] += sums[k][i][c];
    }
    if (out.pre_beta) out.pre_beta[j] += t[0];
    if (out.pre_gamma) out.pre_gamma[j] += t[1];
    const float gate = p.gate_channel ? p.gate_channel[j] : 1.f;
    if (out.post_beta) out.post_beta[j] += p.b * gate * t[2];
    if (out.post_gamma) out.post_gamma[j] += p.b * gate * t[3];
    if (out.gate) {
        const float u = p.post == ZB_NORM_NONE ? t[3] : p.post_gamma[j] * t[3] + (p.post_beta ? p.post_beta[j] * t[2] : 0.f);
        out.gate[j] += p.b * u;
    }
}

// ---------------------------------------------------------------- checks and launches

bool kind_ok(int32_t k) { return k >= ZB_NORM_NONE && k <= ZB_NORM_LAYER; }

// The options that all three calls read, checked.
zb_status norm_params(const zb_residual_norm* op, int32_t tokens, int32_t hidden, NormParams* p) {
    if (!op || !kind_ok(op->post_norm) || !kind_ok(op->pre_norm) || op->gate_kind < ZB_GATE_NONE ||
        op->gate_kind > ZB_GATE_TOKEN)
        return ZB_ERR_ARG;
    if (!tokens_ok(tokens) || !feature_ok(hidden) || hidden > kNormMaxHidden) return ZB_ERR_SHAPE;
    auto norm_ok = [](int32_t kind, const float* gamma, const float* beta, float eps) {
        if (kind == ZB_NORM_NONE) return !gamma && !beta;
        return fixed_ok(gamma) && eps >= 0.f && eps <= 1.f &&
               (kind == ZB_NORM_LAYER ? (!beta || aligned16(beta)) : !beta);
    };
    if (!norm_ok(op->post_norm, op->post_gamma, op->post_beta, op->post_eps) ||
        !norm_ok(op->pre_norm, op->pre_gamma, op->pre_beta, op->pre_eps))
        return ZB_ERR_ARG;
    if (op->gate_kind == ZB_GATE_NONE ? op->gate != nullptr
                                      : op->gate_kind == ZB_GATE_CHANNEL ? !fixed_ok(op->gate) : !rows_ok(op->gate, tokens))
        return ZB_ERR_ARG;
    if (!std::isfinite(op->residual_scale) || !std::isfinite(op->branch_scale)) return ZB_ERR_ARG;
    *p = NormParams{};
    p->post = op->post_norm;
    p->pre = op->pre_norm;
    p->post_gamma = op->post_gamma;
    p->post_beta = op->post_beta;
    p->pre_gamma = op->pre_gamma;
    p->pre_beta = op->pre_beta;
    if (op->gate_kind == ZB_GATE_CHANNEL) p->gate_channel = static_cast<const float*>(op->gate);
    if (op->gate_kind == ZB_GATE_TOKEN) p->gate_token = static_cast<const uint16_t*>(op->gate);
    p->a = op->residual_scale;
    p->b = op->branch_scale;
    p->post_eps = op->post_eps;
    p->pre_eps = op->pre_eps;
    p->hidden = hidden;
    return ZB_OK;
}

// Threads of a row: the fewest that hold it with four groups of 8 values each (three where a row of
// 512 threads is short: 1599 rows of 11712 columns in 44 us, 49 with four); kFull where it fills them all.
template <template <int, int, bool> class K>
cudaError_t launch_rows(NormParams& p, int regs, int tokens, cudaStream_t stream) {
    const int chunks = p.hidden / 8;
    const unsigned rows = static_cast<unsigned>(tokens), packed_rows = (rows + 3) / 4;
    auto go = [&](auto full, auto some, int most, unsigned grid, unsigned block) {
        // a third of the rows that are worked on at once: 8597 rows of 3776 columns in 55 us, 56 with all of them,
        // 60 with twice as many, 61 without; backward 71, 73, 79, 76
        const int blocks = std::max(1, 65536 / (static_cast<int>(block) * (block == 512 && regs < 128 ? 64 : regs)));
        p.ahead = std::max(1, sm_count() * blocks * (grid == rows ? 1 : 4) / 3);
        return launch_chained(chunks == most ? full : some, grid, block, 0, stream, p, tokens);
    };
    if (chunks <= 32) return go(K<32, 1, true>::get(), K<32, 1, false>::get(), 32, packed_rows, 128);
    if (chunks <= 64) return go(K<32, 2, true>::get(), K<32, 2, false>::get(), 64, packed_rows, 128);
    if (chunks <= 128) return go(K<32, 4, true>::get(), K<32, 4, false>::get(), 128, packed_rows, 128);
    if (chunks <= 256) return go(K<64, 4, true>::get(), K<64, 4, false>::get(), 256, rows, 64);
    if (chunks <= 512) return go(K<128, 4, true>::get(), K<128, 4, false>::get(), 512, rows, 128);
    if (chunks <= 1024) return go(K<256, 4, true>::get(), K<256, 4, false>::get(), 1024, rows, 256);
    if (chunks <= 1536) return go(K<512, 3, true>::get(), K<512, 3, false>::get(), 1536, rows, 512);
    if (chunks <= 2048) return go(K<512, 4, true>::get(), K<512, 4, false>::get(), 2048, rows, 512);
    return go(K<1024, 4, true>::get(), K<1024, 4, false>::get(), 4096, rows, 1024);
}

template <int kRow, int kPer, bool kFull>
struct ForwardKernel {
    static auto get() { return &residual_norm_forward_kernel<kRow, kPer, kFull>; }
};

template <int kRow, int kPer, bool kFull>
struct BackwardKernel {
    static auto get() { return &residual_norm_backward_kernel<kRow, kPer, kFull>; }
};

}  // namespace

}  // namespace zbk

extern "C" zb_status zb_op_residual_norm_forward(const zb_residual_norm* op, const void* x, const void* y, void* h, void* n,
                                                 const zb_checkpoint* n_packed, float* stats, int32_t tokens, int32_t hidden,
                                                 void* stream) {
    using namespace zbk;
    NormParams p;
    ZB_TRY(norm_params(op, tokens, hidden, &p));
    if (!rows_ok(x, tokens) || !rows_ok(y, tokens) || !rows_ok(h, tokens) || !rows_ok(stats, tokens)) return ZB_ERR_ARG;
    if (p.pre == ZB_NORM_NONE ? (n || n_packed) : (n ? !aligned16(n) : tokens > 0 && !n_packed)) return ZB_ERR_ARG;
    if (n_packed && (!rows_ok(n_packed->codes, tokens) || !rows_ok(n_packed->scales, tokens))) return ZB_ERR_ARG;
    ZB_TRY(device_ok());
    if (tokens == 0) return ZB_OK;
    p.x = static_cast<const uint16_t*>(x);
    p.y = static_cast<const uint16_t*>(y);
    p.h = static_cast<uint16_t*>(h);
    p.n = static_cast<uint16_t*>(n);
    if (n_packed) {
        p.codes = static_cast<uint8_t*>(n_packed->codes);
        p.scales = static_cast<uint8_t*>(n_packed->scales);
    }
    p.stats = reinterpret_cast<float4*>(stats);
    return cuda_status(launch_rows<ForwardKernel>(p, 80, tokens, as_stream(stream)));
}

extern "C" zb_status zb_op_residual_norm_backward_input(const zb_residual_norm* op, const void* dn, const void* dres,
                                                        const void* h, const void* y, const float* stats, void* dh, void* dx,
                                                        void* dy, void* dgate, int32_t tokens, int32_t hidden, void* stream) {
    using namespace zbk;
    NormParams p;
    ZB_TRY(norm_params(op, tokens, hidden, &p));
    const bool pre = p.pre != ZB_NORM_NONE, reads_y = p.post != ZB_NORM_NONE || dgate;
    if (!rows_ok(dh, tokens) || !rows_ok(dy, tokens) || !rows_ok(stats, tokens) || (dx && !aligned16(dx)) ||
        (dres && !aligned16(dres)) || (dgate && (!aligned16(dgate) || op->gate_kind != ZB_GATE_TOKEN)))
        return ZB_ERR_ARG;
    if (pre ? (!rows_ok(dn, tokens) || !rows_ok(h, tokens)) : (dn != nullptr || (tokens > 0 && !dres))) return ZB_ERR_ARG;
    if (reads_y && !rows_ok(y, tokens)) return ZB_ERR_ARG;
    ZB_TRY(device_ok());
    if (tokens == 0) return ZB_OK;
    p.dn = static_cast<const uint16_t*>(dn);
    p.dres = static_cast<const uint16_t*>(dres);
    p.h = static_cast<uint16_t*>(const_cast<void*>(h));
    p.y = reads_y ? static_cast<const uint16_t*>(y) : nullptr;
    p.stats = reinterpret_cast<float4*>(const_cast<float*>(stats));
    p.dh = static_cast<uint16_t*>(dh);
    p.dx = static_cast<uint16_t*>(dx);
    p.dy = static_cast<uint16_t*>(dy);
    p.dgate = static_cast<uint16_t*>(dgate);
    return cuda_status(launch_rows<BackwardKernel>(p, 128, tokens, as_stream(stream)));
}

extern "C" size_t zb_op_residual_norm_backward_weight_scratch_bytes(int32_t tokens, int32_t hidden) {
    if (!zbk::tokens_ok(tokens) || !zbk::feature_ok(hidden) || hidden > zbk::kNormMaxHidden) return 0;
    return static_cast<size_t>(zbk::norm_parts(tokens, hidden)) * 4 * static_cast<size_t>(hidden) * sizeof(float);
}

extern "C" zb_status zb_op_residual_norm_backward_weight(const zb_residual_norm* op, const void* dn, const void* h,
                                                         const void* dh, const void* y, const float* stats,
                                                         float* dpost_gamma, float* dpost_beta, float* dpre_gamma,
                                                         float* dpre_beta, float* dgate, int32_t tokens, int32_t hidden,
                                                         void* scratch, size_t scratch_bytes, void* stream) {
    using namespace zbk;
    NormParams p;
    ZB_TRY(norm_params(op, tokens, hidden, &p));
    // a gradient belongs to a parameter that the norms have
    if ((dpost_gamma && !p.post_gamma) || (dpost_beta && !p.post_beta) || (dpre_gamma && !p.pre_gamma) ||
        (dpre_beta && !p.pre_beta) || (dgate && !p.gate_channel))
        return ZB_ERR_ARG;
    for (const float* g : {dpost_gamma, dpost_beta, dpre_gamma, dpre_beta, dgate})
        if (g && !aligned16(g)) return ZB_ERR_ARG;
    const bool pre = dpre_gamma || dpre_beta, branch = dpost_gamma || dpost_beta || dgate;
    const bool reads_h = dpre_gamma, reads_y = dpost_gamma || dgate;
    if (!rows_ok(stats, tokens) || (pre && !rows_ok(dn, tokens)) || (reads_h && !rows_ok(h, tokens)) ||
        (branch && !rows_ok(dh, tokens)) || (reads_y && !rows_ok(y, tokens)))
        return ZB_ERR_ARG;
    if (tokens > 0 && (pre || branch) &&
        (!fixed_ok(scratch) || scratch_bytes < zb_op_residual_norm_backward_weight_scratch_bytes(tokens, hidden)))
        return ZB_ERR_WORKSPACE;
    ZB_TRY(device_ok());
    if (tokens == 0 || (!pre && !branch)) return ZB_OK;
    p.dn = static_cast<const uint16_t*>(dn);
    p.h = reads_h ? static_cast<uint16_t*>(const_cast<void*>(h)) : nullptr;
    p.dh = static_cast<uint16_t*>(const_cast<void*>(dh));
    p.y = reads_y ? static_cast<const uint16_t*>(y) : nullptr;
    p.stats = reinterpret_cast<float4*>(const_cast<float*>(stats));
    const int parts = norm_parts(tokens, hidden);
    cudaStream_t s = as_stream(stream);
    const unsigned grid = static_cast<unsigned>((hidden + 255) / 256 * parts * (pre && branch ? 2 : 1));
    const bool means = p.pre == ZB_NORM_LAYER || p.post == ZB_NORM_LAYER;
    auto kern = p.gate_token ? (means ? &residual_norm_parts_kernel<true, true> : &residual_norm_parts_kernel<true, false>)
                             : (means ? &residual_norm_parts_kernel<false, true> : &residual_norm_parts_kernel<false, false>);
    ZB_TRY(cuda_status(launch_chained(kern, grid, kWThreads, 0, s, p, static_cast<float*>(scratch), tokens, pre ? 0 : 1, parts)));
    const NormGrads out{dpost_gamma, dpost_beta, dpre_gamma, dpre_beta, dgate};
    return cuda_status(launch_chained(residual_norm_sum_kernel, static_cast<unsigned>(hidden / 32), 1024, 0, s, p, out,
                                      static_cast<const float*>(scratch), parts, pre, branch));
}
