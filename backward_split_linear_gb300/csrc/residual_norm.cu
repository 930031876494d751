// The norms around a block with its gate and its residual scales, forward and split
// backward.  With y the block's output and x the residual stream that entered it:
//   F   u = PostNorm(y),  h = bf16(a x + b gate u),  n = PreNorm(h), the next block's input
//   B   dh = dres + PreNorm'(dn),  dx = a dh,  dy = PostNorm'(b gate dh),  dgate = b u dh
//   W   the norms' weights and biases, and a gate per channel
// Norm(v) = gamma (v - mean) rstd + beta; an RMS norm has mean 0 and no beta of its own.
//
// F and B take a row in one pass: its threads hold all of it in registers, so that every
// tensor is read and written once; the sums over the row go through shuffles, and shared
// memory where a row has more than one warp.  Both are bound by HBM.
#include <algorithm>

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
};

struct F8 {
    float v[8];
};

__device__ __forceinline__ F8 widen(const uint4& q) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    F8 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        r.v[2 * e] = bf16_lo(w[e]);
        r.v[2 * e + 1] = bf16_hi(w[e]);
    }
    return r;
}

__device__ __forceinline__ uint4 narrow(const F8& f) {
    return make_uint4(pack_bf16x2(f.v[0], f.v[1]), pack_bf16x2(f.v[2], f.v[3]), pack_bf16x2(f.v[4], f.v[5]),
                      pack_bf16x2(f.v[6], f.v[7]));
}

__device__ __forceinline__ F8 load_f8(const float* p) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

__device__ __forceinline__ uint4 load_q(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

// Sums of (s0, s1) over the threads of a row.  Each use of `round` has shared memory of its
// own, so that one barrier a sum is enough.
template <int kRow>
__device__ __forceinline__ float2 row_sum(float s0, float s1, float2 (*red)[32], int round) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s0 += __shfl_xor_sync(0xffffffffu, s0, o);
        s1 += __shfl_xor_sync(0xffffffffu, s1, o);
    }
    if constexpr (kRow > 32) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) red[round][warp] = make_float2(s0, s1);
        __syncthreads();
        constexpr int kWarps = kRow / 32;
        const float2 part = lane < kWarps ? red[round][lane] : make_float2(0.f, 0.f);
        s0 = part.x;
        s1 = part.y;
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1) {
            s0 += __shfl_xor_sync(0xffffffffu, s0, o);
            s1 += __shfl_xor_sync(0xffffffffu, s1, o);
        }
        s0 = __shfl_sync(0xffffffffu, s0, 0);
        s1 = __shfl_sync(0xffffffffu, s1, 0);
    }
    return make_float2(s0, s1);
}

// Rows of a block, kRow threads each (one row where a row has more than a warp).
template <int kRow>
__host__ __device__ constexpr int norm_rows() {
    return kRow == 32 ? 4 : 1;
}

// Mean and 1 / sqrt(variance + eps) of a row whose thread holds kPer groups of 8 values.  The
// variance is of the differences from the mean: a second sum, which a mean far from zero
// cannot spoil.
template <int kRow, int kPer>
__device__ __forceinline__ float2 moments(const F8 (&v)[kPer], const bool (&in)[kPer], int kind, float eps, int hidden,
                                          float2 (*red)[32], int round) {
    const float inv = 1.f / static_cast<float>(hidden);
    float mean = 0.f;
    if (kind == ZB_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) s += in[i] ? v[i].v[e] : 0.f;
        mean = row_sum<kRow>(s, 0.f, red, round).x * inv;
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = v[i].v[e] - mean;
            q += in[i] ? d * d : 0.f;
        }
    const float var = row_sum<kRow>(q, 0.f, red, round + 1).x * inv;
    return make_float2(mean, rsqrtf(var + eps));
}

template <int kRow, int kPer>
__global__ void __launch_bounds__(kRow * norm_rows<kRow>()) residual_norm_forward_kernel(const __grid_constant__ NormParams p,
                                                                                         int tokens) {
    __shared__ float2 red[4][32];
    const int tid = kRow == 32 ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t row = kRow == 32 ? static_cast<int64_t>(blockIdx.x) * norm_rows<kRow>() + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= tokens) return;  // whole warps
    const int64_t base = row * p.hidden;
    const int chunks = p.hidden >> 3;
    bool in[kPer];
    uint4 xq[kPer], gq[kPer];
    F8 u[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int c = tid + i * kRow;
        in[i] = c < chunks;
        uint4 yq = make_uint4(0, 0, 0, 0);
        if (in[i]) {
            yq = load_q(p.y + base + 8 * c);
            xq[i] = load_q(p.x + base + 8 * c);
            if (p.gate_token) gq[i] = load_q(p.gate_token + base + 8 * c);
        }
        u[i] = widen(yq);
    }
    float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.post != ZB_NORM_NONE) {
        const float2 m = moments<kRow, kPer>(u, in, p.post, p.post_eps, p.hidden, red, 0);
        st.x = m.x;
        st.y = m.y;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int c = tid + i * kRow;
        if (!in[i]) continue;
        if (p.post != ZB_NORM_NONE) {
            const F8 g = load_f8(p.post_gamma + 8 * c);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[i].v[e] = (u[i].v[e] - st.x) * st.y * g.v[e];
            if (p.post_beta) {
                const F8 b = load_f8(p.post_beta + 8 * c);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[i].v[e] += b.v[e];
            }
        }
        if (p.gate_channel || p.gate_token) {
            const F8 g = p.gate_channel ? load_f8(p.gate_channel + 8 * c) : widen(gq[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[i].v[e] *= g.v[e];
        }
        const F8 x = widen(xq[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[i].v[e] = p.a * x.v[e] + p.b * u[i].v[e];
        const uint4 hq = narrow(u[i]);
        *reinterpret_cast<uint4*>(p.h + base + 8 * c) = hq;
        u[i] = widen(hq);  // n is the norm of the h that is stored
    }
    if (p.pre != ZB_NORM_NONE) {
        const float2 m = moments<kRow, kPer>(u, in, p.pre, p.pre_eps, p.hidden, red, 2);
        st.z = m.x;
        st.w = m.y;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = tid + i * kRow;
            uint4 nq = make_uint4(0, 0, 0, 0);
            if (in[i]) {
                const F8 g = load_f8(p.pre_gamma + 8 * c);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[i].v[e] = (u[i].v[e] - st.z) * st.w * g.v[e];
                if (p.pre_beta) {
                    const F8 b = load_f8(p.pre_beta + 8 * c);
#pragma unroll
                    for (int e = 0; e < 8; ++e) u[i].v[e] += b.v[e];
                }
                nq = narrow(u[i]);
                if (p.n) *reinterpret_cast<uint4*>(p.n + base + 8 * c) = nq;
            }
            if (p.codes) {  // four threads hold a block of 32 (a row has a multiple of 8 chunks)
                uint32_t top2 = pack_top2(pack_top2(pack_top2(pack_top2(0u, nq.x), nq.y), nq.z), nq.w);
                uint32_t top = max(top2 & 0xffffu, top2 >> 16);
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                if (in[i]) {
                    const uint32_t scale = pack_scale(top);
                    const float f = pack_factor(scale);
                    const bool fine = scale != kPackNotFinite;
                    reinterpret_cast<uint2*>(p.codes + base)[c] =
                        make_uint2(fine ? pack_codes(nq.x, nq.y, f) : 0u, fine ? pack_codes(nq.z, nq.w, f) : 0u);
                    if ((tid & 3) == 0) p.scales[(base >> 5) + (c >> 2)] = static_cast<uint8_t>(scale);
                }
            }
        }
    }
    if (tid == 0) p.stats[row] = st;
}

// The input gradient of a norm of rows: d is the gradient of the normed values `hat`:
//   rstd (d - hat mean(d hat) - [layer] mean(d)).
template <int kRow, int kPer>
__global__ void __launch_bounds__(kRow * norm_rows<kRow>()) residual_norm_backward_kernel(const __grid_constant__ NormParams p,
                                                                                          int tokens) {
    __shared__ float2 red[2][32];
    const int tid = kRow == 32 ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t row = kRow == 32 ? static_cast<int64_t>(blockIdx.x) * norm_rows<kRow>() + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= tokens) return;  // whole warps
    const int64_t base = row * p.hidden;
    const int chunks = p.hidden >> 3;
    const float inv = 1.f / static_cast<float>(p.hidden);
    const bool pre = p.pre != ZB_NORM_NONE, post = p.post != ZB_NORM_NONE;
    const float4 st = p.stats[row];
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 nq[kPer], hq[kPer], rq[kPer], yq[kPer], gq[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int c = tid + i * kRow;
        const bool in = c < chunks;
        nq[i] = in && pre ? load_q(p.dn + base + 8 * c) : zero;
        hq[i] = in && pre ? load_q(p.h + base + 8 * c) : zero;
        rq[i] = in && p.dres ? load_q(p.dres + base + 8 * c) : zero;
        yq[i] = in && p.y ? load_q(p.y + base + 8 * c) : zero;
        gq[i] = in && p.gate_token ? load_q(p.gate_token + base + 8 * c) : zero;
    }
    F8 dh[kPer];
    if (pre) {
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = tid + i * kRow;
            if (c < chunks) {
                const F8 d = widen(nq[i]), h = widen(hq[i]), g = load_f8(p.pre_gamma + 8 * c);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = d.v[e] * g.v[e];
                    s0 += v * ((h.v[e] - st.z) * st.w);
                    s1 += v;
                }
            }
        }
        const float2 s = row_sum<kRow>(s0, s1, red, 0);
        const float m0 = s.x * inv, m1 = p.pre == ZB_NORM_LAYER ? s.y * inv : 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = tid + i * kRow;
            dh[i] = widen(rq[i]);
            if (c < chunks) {
                const F8 d = widen(nq[i]), h = widen(hq[i]), g = load_f8(p.pre_gamma + 8 * c);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dh[i].v[e] += st.w * (d.v[e] * g.v[e] - (h.v[e] - st.z) * st.w * m0 - m1);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) dh[i] = widen(rq[i]);
    }
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int c = tid + i * kRow;
        if (c >= chunks) continue;
        *reinterpret_cast<uint4*>(p.dh + base + 8 * c) = narrow(dh[i]);
        if (p.dx) {
            F8 dx;
#pragma unroll
            for (int e = 0; e < 8; ++e) dx.v[e] = p.a * dh[i].v[e];
            *reinterpret_cast<uint4*>(p.dx + base + 8 * c) = narrow(dx);
        }
        // dh becomes du, the gradient of what the gate multiplies (times the norm's weight)
        const F8 y = widen(yq[i]);
        F8 g{{1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}};
        if (post) g = load_f8(p.post_gamma + 8 * c);
        if (p.dgate) {
            F8 dg, b{};
            if (p.post_beta) b = load_f8(p.post_beta + 8 * c);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float u = post ? (y.v[e] - st.x) * st.y * g.v[e] + b.v[e] : y.v[e];
                dg.v[e] = p.b * dh[i].v[e] * u;
            }
            *reinterpret_cast<uint4*>(p.dgate + base + 8 * c) = narrow(dg);
        }
        if (p.gate_channel || p.gate_token) {
            const F8 gate = p.gate_channel ? load_f8(p.gate_channel + 8 * c) : widen(gq[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) dh[i].v[e] *= gate.v[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dh[i].v[e] *= p.b * g.v[e];
            s0 += dh[i].v[e] * ((y.v[e] - st.x) * st.y);
            s1 += dh[i].v[e];
        }
    }
    float m0 = 0.f, m1 = 0.f, rstd = 1.f;
    if (post) {
        const float2 s = row_sum<kRow>(s0, s1, red, 1);
        m0 = s.x * inv;
        m1 = p.post == ZB_NORM_LAYER ? s.y * inv : 0.f;
        rstd = st.y;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int c = tid + i * kRow;
        if (c >= chunks) continue;
        if (post) {
            const F8 y = widen(yq[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) dh[i].v[e] = rstd * (dh[i].v[e] - (y.v[e] - st.x) * st.y * m0 - m1);
        }
        *reinterpret_cast<uint4*>(p.dy + base + 8 * c) = narrow(dh[i]);
    }
}

// ---------------------------------------------------------------- weight gradients
//
// Four sums over the rows for every column: dn, dn hhat, gdh, gdh yhat, where gdh is dh
// (times the gate per token) and yhat the normed y (y itself without a post norm).  A gate
// per channel is a factor of the sums, so dgate and the post norm's gradients come from the
// same two.  Two passes in a fixed order: parts of the rows ([parts][4][hidden]), then their sum.

constexpr int kWThreads = 256;
constexpr int kWGroups = 8;
constexpr int kWUnroll = 2;
constexpr int kWTargetBlocks = 608;  // 4 blocks of 256 threads on each of 152 SMs

int norm_parts(int tokens, int hidden) {
    const int across = (hidden + 255) / 256;
    return std::max(1, std::min((kWTargetBlocks + across - 1) / across, (tokens + kWGroups - 1) / kWGroups));
}

__global__ void __launch_bounds__(kWThreads) residual_norm_parts_kernel(const __grid_constant__ NormParams p,
                                                                        float* __restrict__ parts, int tokens, bool pre,
                                                                        bool branch) {
    __shared__ float sums[kWGroups][256];
    const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
    const int col = blockIdx.x * 256 + 8 * lane;
    const int per = (tokens + gridDim.y - 1) / gridDim.y;
    const int t0 = blockIdx.y * per, t1 = min(tokens, t0 + per);
    const bool post = p.post != ZB_NORM_NONE;
    float acc[4][8] = {};
    if (col < p.hidden) {
        for (int tb = t0 + group; tb < t1; tb += kWGroups * kWUnroll) {
            uint4 nq[kWUnroll], hq[kWUnroll], dq[kWUnroll], yq[kWUnroll], gq[kWUnroll];
            float4 st[kWUnroll];
#pragma unroll
            for (int i = 0; i < kWUnroll; ++i) {
                const int t = tb + i * kWGroups;
                if (t >= t1) continue;
                const int64_t at = static_cast<int64_t>(t) * p.hidden + col;
                st[i] = p.stats[t];
                if (pre) {
                    nq[i] = load_q(p.dn + at);
                    hq[i] = load_q(p.h + at);
                }
                if (branch) {
                    dq[i] = load_q(p.dh + at);
                    yq[i] = load_q(p.y + at);
                    if (p.gate_token) gq[i] = load_q(p.gate_token + at);
                }
            }
#pragma unroll
            for (int i = 0; i < kWUnroll; ++i) {
                if (tb + i * kWGroups >= t1) continue;
                if (pre) {
                    const F8 d = widen(nq[i]), h = widen(hq[i]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        acc[0][e] += d.v[e];
                        acc[1][e] += d.v[e] * ((h.v[e] - st[i].z) * st[i].w);
                    }
                }
                if (branch) {
                    F8 d = widen(dq[i]);
                    const F8 y = widen(yq[i]);
                    if (p.gate_token) {
                        const F8 g = widen(gq[i]);
#pragma unroll
                        for (int e = 0; e < 8; ++e) d.v[e] *= g.v[e];
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        acc[2][e] += d.v[e];
                        acc[3][e] += d.v[e] * (post ? (y.v[e] - st[i].x) * st[i].y : y.v[e]);
                    }
                }
            }
        }
    }
    const int j = blockIdx.x * 256 + threadIdx.x;
    float* out = parts + static_cast<int64_t>(blockIdx.y) * 4 * p.hidden;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (k < 2 ? !pre : !branch) continue;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[group][8 * lane + e] = acc[k][e];
        __syncthreads();
        if (j < p.hidden) {
            float s = 0.f;
#pragma unroll
            for (int g = 0; g < kWGroups; ++g) s += sums[g][threadIdx.x];
            out[static_cast<int64_t>(k) * p.hidden + j] = s;
        }
    }
}

struct NormGrads {
    float *post_gamma, *post_beta, *pre_gamma, *pre_beta, *gate;
};

__global__ void __launch_bounds__(256) residual_norm_sum_kernel(const __grid_constant__ NormParams p, const NormGrads out,
                                                                const float* __restrict__ parts, int n_parts, bool pre,
                                                                bool branch) {
    __shared__ float sums[4][8][32];
    const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int j = blockIdx.x * 32 + c;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (k < 2 ? !pre : !branch) continue;
        float s = 0.f;
        for (int q0 = g; q0 < n_parts; q0 += 64) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = q0 + 8 * i < n_parts ? parts[(static_cast<int64_t>(q0 + 8 * i) * 4 + k) * p.hidden + j] : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[i];
        }
        sums[k][g][c] = s;
    }
    __syncthreads();
    if (g != 0) return;
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
    auto finite = [](float v) { return v >= -3.4e38f && v <= 3.4e38f; };
    if (!finite(op->residual_scale) || !finite(op->branch_scale)) return ZB_ERR_ARG;
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

// Threads of a row: the fewest that hold it with four groups of 8 values each.
template <template <int, int> class K>
cudaError_t launch_rows(const NormParams& p, int tokens, cudaStream_t stream) {
    const int chunks = p.hidden / 8;
    const unsigned rows = static_cast<unsigned>(tokens), packed_rows = (rows + 3) / 4;
    if (chunks <= 32)
        K<32, 1>::get()<<<packed_rows, 128, 0, stream>>>(p, tokens);
    else if (chunks <= 64)
        K<32, 2>::get()<<<packed_rows, 128, 0, stream>>>(p, tokens);
    else if (chunks <= 128)
        K<32, 4>::get()<<<packed_rows, 128, 0, stream>>>(p, tokens);
    else if (chunks <= 256)
        K<64, 4>::get()<<<rows, 64, 0, stream>>>(p, tokens);
    else if (chunks <= 512)
        K<128, 4>::get()<<<rows, 128, 0, stream>>>(p, tokens);
    else if (chunks <= 1024)
        K<256, 4>::get()<<<rows, 256, 0, stream>>>(p, tokens);
    else if (chunks <= 2048)
        K<512, 4>::get()<<<rows, 512, 0, stream>>>(p, tokens);
    else
        K<1024, 4>::get()<<<rows, 1024, 0, stream>>>(p, tokens);
    return cudaGetLastError();
}

template <int kRow, int kPer>
struct ForwardKernel {
    static auto get() { return residual_norm_forward_kernel<kRow, kPer>; }
};

template <int kRow, int kPer>
struct BackwardKernel {
    static auto get() { return residual_norm_backward_kernel<kRow, kPer>; }
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
    return cuda_status(launch_rows<ForwardKernel>(p, tokens, as_stream(stream)));
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
    return cuda_status(launch_rows<BackwardKernel>(p, tokens, as_stream(stream)));
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
    if (!rows_ok(stats, tokens) || (pre && (!rows_ok(dn, tokens) || !rows_ok(h, tokens))) ||
        (branch && (!rows_ok(dh, tokens) || !rows_ok(y, tokens))))
        return ZB_ERR_ARG;
    if (tokens > 0 && (pre || branch) &&
        (!fixed_ok(scratch) || scratch_bytes < zb_op_residual_norm_backward_weight_scratch_bytes(tokens, hidden)))
        return ZB_ERR_WORKSPACE;
    ZB_TRY(device_ok());
    if (tokens == 0 || (!pre && !branch)) return ZB_OK;
    p.dn = static_cast<const uint16_t*>(dn);
    p.h = static_cast<uint16_t*>(const_cast<void*>(h));
    p.dh = static_cast<uint16_t*>(const_cast<void*>(dh));
    p.y = static_cast<const uint16_t*>(y);
    p.stats = reinterpret_cast<float4*>(const_cast<float*>(stats));
    const int parts = norm_parts(tokens, hidden);
    cudaStream_t s = as_stream(stream);
    const dim3 grid((hidden + 255) / 256, parts);
    residual_norm_parts_kernel<<<grid, kWThreads, 0, s>>>(p, static_cast<float*>(scratch), tokens, pre, branch);
    const NormGrads out{dpost_gamma, dpost_beta, dpre_gamma, dpre_beta, dgate};
    residual_norm_sum_kernel<<<hidden / 32, 256, 0, s>>>(p, out, static_cast<const float*>(scratch), parts, pre, branch);
    return cuda_status(cudaGetLastError());
}
