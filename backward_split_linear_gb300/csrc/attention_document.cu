// Softmax attention inside packed documents, on tcgen05 (sm_103a).
//
// Score of query i and key j of one document, h the head:
//   s = q_i . k_j / sqrt(d);  s = cap tanh(s / cap) with a cap;  s -= slope_h |i - j|.
// Key j is visible to query i when both are in the same document and j <= i or
// j is among the document's first `prefix` rows.
//
// A plan of intervals (attention_document.h) tells every tile of 128 rows which
// 128-row blocks it shares a visible pair with, and every row which columns:
// the work is that of the visible blocks, however the batch is packed.  The
// kernels are those of the causal core (attention.cu) with that in place of the
// diagonal, and differ where short documents ask for it: the forward is
// persistent, and the backward's two kernels are one launch.
//
//   document_fwd_kernel  two tiles a CTA (two heads of a group, or two
//                        consecutive query blocks of a head when the group is
//                        odd): S = Q K^T -> online softmax -> O += P V.
//   document_bwd_kernel  CTAs of two kinds: (kv head, key block) forms dK and dV
//                        over the group's heads and the query blocks that see
//                        the keys; the others take (head, query block) tiles
//                        from a counter and form dQ.
//
// Values that are not finite.  The tensor cores multiply every row of a tile
// with every other, and 0 times NaN is NaN: a hidden key's value, or a query of
// another document, would reach rows that do not see it.  Scores are selected,
// not multiplied, where they are hidden; padding's rows of an operand become zeros;
// and a result row that is not finite is formed again from its visible pairs
// alone, by the row-by-row code below.  In a batch of finite documents that
// code never runs.
#include "attention_common.cuh"
#include "attention_document.h"
#include "chained.cuh"
#include "checks.h"

namespace zbk {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------------ plan

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

// One block per 128 rows, one row per thread; a binary search finds the row's
// document.  Offsets are data: whatever they hold, every interval written lies
// inside [0, tokens].  Bound by a launch's latency: 2.8 us at 4096 tokens.
__global__ void __launch_bounds__(kDocBlock) document_plan_kernel(const int32_t* offsets, const int32_t* prefix, int n_docs,
                                                                  int tokens, int2* rows, int2* cols, int2* q_blocks,
                                                                  int2* k_blocks, int32_t* positions) {
    __shared__ int red[4][4];
    wait_for_previous();
    const int i = blockIdx.x * kDocBlock + threadIdx.x;
    int s = 0, e = 0, pre = 0, border = 0;
    if (i < tokens) {
        if (offsets) {
            int lo = 0, hi = n_docs;  // the last offset at or before row i
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (offsets[mid] <= i)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            border = clampi(offsets[lo], 0, tokens);  // where padding ends, or where it starts
            if (lo < n_docs) {
                s = border;
                e = clampi(offsets[lo + 1], 0, tokens);
                if (prefix) pre = prefix[lo];
            }
        } else {
            e = tokens;
            if (prefix) pre = prefix[0];
        }
        if (i < s || i >= e) s = e = 0;
    }
    const bool in = e > s;
    const int pend = in ? s + clampi(pre, 0, e - s) : 0;  // end of the prefix
    const int2 row = in ? make_int2(s, max(i + 1, pend)) : make_int2(border, border);
    const int2 col = in ? make_int2(i < pend ? s : i, e) : make_int2(border, border);
    rows[i] = row;
    cols[i] = col;
    if (positions && i < tokens) positions[i] = in ? i - s : 0;
    int v[4] = {in ? row.x : 0x7fffffff, in ? row.y : 0, in ? col.x : 0x7fffffff, in ? col.y : 0};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        v[0] = min(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
        v[1] = max(v[1], __shfl_xor_sync(0xffffffffu, v[1], o));
        v[2] = min(v[2], __shfl_xor_sync(0xffffffffu, v[2], o));
        v[3] = max(v[3], __shfl_xor_sync(0xffffffffu, v[3], o));
    }
    if ((threadIdx.x & 31) == 0)
        for (int k = 0; k < 4; ++k) red[k][threadIdx.x >> 5] = v[k];
    __syncthreads();
    if (threadIdx.x == 0) {
        const int q_lo = min(min(red[0][0], red[0][1]), min(red[0][2], red[0][3]));
        const int q_hi = max(max(red[1][0], red[1][1]), max(red[1][2], red[1][3]));
        const int k_lo = min(min(red[2][0], red[2][1]), min(red[2][2], red[2][3]));
        const int k_hi = max(max(red[3][0], red[3][1]), max(red[3][2], red[3][3]));
        q_blocks[blockIdx.x] = q_hi > 0 ? make_int2(q_lo / kDocBlock, (q_hi + kDocBlock - 1) / kDocBlock) : make_int2(0, 0);
        k_blocks[blockIdx.x] = k_hi > 0 ? make_int2(k_lo / kDocBlock, (k_hi + kDocBlock - 1) / kDocBlock) : make_int2(0, 0);
    }
}

// ------------------------------------------------------------------------ arguments

struct DocArgs {
    const uint16_t* qkv;
    const uint16_t* da;
    uint16_t* out;         // forward: a [T, n_heads d]; backward: dqkv
    const float* lse;      // [n_heads][ld_stat], backward
    float* lse_out;        // the same, forward
    const float* dvec;     // [n_heads][ld_stat]: rowsum(da * a)
    int* counter;          // backward: the next dQ tile
    DocPlan plan;
    const float* slopes;   // [n_heads] or null
    float cap, scale;
    float scale_log2;      // log2(e) / sqrt(d)
    float cap_log2;        // cap log2(e)
    float cap_limit;       // 3/4 cap sqrt(d): the polynomial's range
    float cap_poly[5];     // tanh(s / (cap sqrt(d))) / s as a polynomial in s^2
    float cap_exp;         // 2 log2(e) / (cap sqrt(d)): the exponent of e^(2 s / cap) per unit of q . k
    int tokens, n_heads, n_kv_heads, ld_stat, n_blocks;
    int* status;
    uint64_t wait_ns;      // the limit of every wait
};

// How scores are modified: not at all, by the distance, by the cap, or by both.
// Every kernel exists once for each: what a batch does not use would cost it
// instructions, and room in the instruction caches (the capped backward took 7 %
// longer with the distance's code beside it, never run).
enum DocMode : int { kDocPlain = 0, kDocBias = 1, kDocCap = 2, kDocCapBias = 3 };
__host__ __device__ constexpr bool mode_caps(int m) { return m >= kDocCap; }
__host__ __device__ constexpr bool mode_biases(int m) { return m == kDocBias || m == kDocCapBias; }

// ------------------------------------------------------------------------ row by row

template <int D>
__device__ __forceinline__ void load_row(const uint16_t* p, int lane, float (&v)[D / 32]) {
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(p + 64 * c + 2 * lane);
        v[2 * c] = bf16_lo(w);
        v[2 * c + 1] = bf16_hi(w);
    }
}
template <int D>
__device__ __forceinline__ void store_row(uint16_t* p, int lane, const float (&v)[D / 32], float f, int c0, int c1) {
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
        if (64 * c + 2 * lane >= c0 && 64 * c + 2 * lane < c1) *reinterpret_cast<uint32_t*>(p + 64 * c + 2 * lane) = pack_bf16x2(v[2 * c] * f, v[2 * c + 1] * f);
}
template <int N>
__device__ __forceinline__ float dot_rows(const float (&a)[N], const float (&b)[N]) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < N; ++c) s = fmaf(a[c], b[c], s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// Keys (or queries) whose rows are on their way together: one at a time, a row by row
// pass waits for memory.
constexpr int kAtOnce = 4;
constexpr uint64_t kRowPairNs = 1000;  // nanoseconds that a pair may take, for the waits' limits

// What a plan's row may walk, whatever the plan's memory holds.
__device__ __forceinline__ int2 inside(int2 see, int tokens) { return make_int2(max(see.x, 0), min(see.y, tokens)); }

// The score in base-2 units, and the cap's derivative.
__device__ __forceinline__ float score2(const DocArgs& p, float dot, float slope, int dist, float& slope_cap) {
    float s = dot * p.scale;
    slope_cap = 1.f;
    if (p.cap > 0.f) {
        const float t = tanhf(s / p.cap);
        slope_cap = 1.f - t * t;
        s = t * p.cap;
    }
    return (s - slope * static_cast<float>(dist)) * kLog2e;
}

// One query row and head by a whole warp: a and lse.
template <int D>
__device__ __forceinline__ void document_forward_row(const DocArgs& p, int i, int h, int lane) {
    const int64_t width = static_cast<int64_t>(p.n_heads + 2 * p.n_kv_heads) * D;
    const int g = h / (p.n_heads / p.n_kv_heads);
    const uint16_t* k = p.qkv + (p.n_heads + g) * D;
    const uint16_t* v = p.qkv + (p.n_heads + p.n_kv_heads + g) * D;
    const float slope = p.slopes ? p.slopes[h] : 0.f;
    float q[D / 32], acc[D / 32] = {};
    load_row<D>(p.qkv + i * width + h * D, lane, q);
    const int2 see = inside(p.plan.rows[i], p.tokens);
    float m = -INFINITY, l = 0.f;
    for (int j0 = see.x; j0 < see.y && l == l; j0 += kAtOnce) {  // once l is NaN, so is everything
        float x[kAtOnce][D / 32], y[kAtOnce][D / 32], dot[kAtOnce], unused;
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int64_t j = min(j0 + u, see.y - 1);
            load_row<D>(k + j * width, lane, x[u]);
            load_row<D>(v + j * width, lane, y[u]);
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) dot[u] = dot_rows(q, x[u]);
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            if (j0 + u >= see.y) break;
            const float s = score2(p, dot[u], slope, abs(i - j0 - u), unused);
            // a score of -infinity has no weight; ahead of every finite one, s - top would be NaN
            const float top = fmaxf(m, s), f = m == -INFINITY ? 0.f : exp2f(m - top), e = s == -INFINITY ? 0.f : exp2f(s - top);
            m = top;
            l = l * f + e;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) acc[c] = acc[c] * f + e * y[u][c];
        }
    }
    store_row<D>(p.out + (static_cast<int64_t>(i) * p.n_heads + h) * D, lane, acc, 1.f / l, 0, D);
    if (lane == 0) p.lse_out[static_cast<int64_t>(h) * p.ld_stat + i] = m + log2f(l);
}

// Columns [c0, c1) of dq of one query row and head.
template <int D>
__device__ __noinline__ void document_dq_row(const DocArgs& p, int i, int h, int lane, int c0, int c1) {
    const int64_t width = static_cast<int64_t>(p.n_heads + 2 * p.n_kv_heads) * D;
    const int g = h / (p.n_heads / p.n_kv_heads);
    const uint16_t* k = p.qkv + (p.n_heads + g) * D;
    const uint16_t* v = p.qkv + (p.n_heads + p.n_kv_heads + g) * D;
    const float slope = p.slopes ? p.slopes[h] : 0.f;
    float q[D / 32], dy[D / 32], acc[D / 32] = {};
    load_row<D>(p.qkv + i * width + h * D, lane, q);
    load_row<D>(p.da + (static_cast<int64_t>(i) * p.n_heads + h) * D, lane, dy);
    const float lse = p.lse[static_cast<int64_t>(h) * p.ld_stat + i], dsum = p.dvec[static_cast<int64_t>(h) * p.ld_stat + i];
    const int2 see = inside(p.plan.rows[i], p.tokens);
    float ds = 0.f;
    for (int j0 = see.x; j0 < see.y && ds == ds; j0 += kAtOnce) {  // a NaN ds makes every sum NaN
        float x[kAtOnce][D / 32], dot[kAtOnce], dp[kAtOnce], f;
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            float y[D / 32];
            const int64_t j = min(j0 + u, see.y - 1);
            load_row<D>(k + j * width, lane, x[u]);
            load_row<D>(v + j * width, lane, y);
            dot[u] = dot_rows(q, x[u]);
            dp[u] = dot_rows(dy, y);
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            if (j0 + u >= see.y) break;
            const float e = exp2f(score2(p, dot[u], slope, abs(i - j0 - u), f) - lse);
            ds = e * (dp[u] - dsum) * f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) acc[c] += ds * x[u][c];
            if (ds != ds) break;
        }
    }
    store_row<D>(p.out + i * width + h * D, lane, acc, p.scale, c0, c1);
}

// dk (or dv, with `value`) of one key row and kv head.
template <int D>
__device__ __noinline__ void document_dkv_row(const DocArgs& p, int j, int g, int lane, bool value) {
    const int64_t width = static_cast<int64_t>(p.n_heads + 2 * p.n_kv_heads) * D;
    const int group = p.n_heads / p.n_kv_heads;
    const int64_t kcol = (p.n_heads + g) * D, vcol = (p.n_heads + p.n_kv_heads + g) * D;
    float k[D / 32], v[D / 32], acc[D / 32] = {};
    load_row<D>(p.qkv + j * width + kcol, lane, k);
    load_row<D>(p.qkv + j * width + vcol, lane, v);
    const int2 see = inside(p.plan.cols[j], p.tokens);
    float w = 0.f;
    for (int h = g * group; h < (g + 1) * group && w == w; ++h) {
        const float slope = p.slopes ? p.slopes[h] : 0.f;
        const float* lse = p.lse + static_cast<int64_t>(h) * p.ld_stat;
        const float* dsum = p.dvec + static_cast<int64_t>(h) * p.ld_stat;
        for (int i0 = see.x; i0 < see.y && w == w; i0 += kAtOnce) {  // a NaN weight makes every sum NaN
            float x[kAtOnce][D / 32], y[kAtOnce][D / 32], dot[kAtOnce], dp[kAtOnce], f;
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int64_t i = min(i0 + u, see.y - 1);
                load_row<D>(p.qkv + i * width + h * D, lane, x[u]);
                load_row<D>(p.da + (i * p.n_heads + h) * D, lane, y[u]);
                dot[u] = dot_rows(k, x[u]);
                dp[u] = dot_rows(v, y[u]);
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int i = i0 + u;
                if (i >= see.y) break;
                const float e = exp2f(score2(p, dot[u], slope, abs(i - j), f) - lse[i]);
                w = value ? e : e * (dp[u] - dsum[i]) * f;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) acc[c] += w * (value ? y[u][c] : x[u][c]);
                if (w != w) break;
            }
        }
    }
    store_row<D>(p.out + j * width + (value ? vcol : kcol), lane, acc, value ? 1.f : p.scale, 0, D);
}

// ------------------------------------------------------------------------ scores on the tensor-core path

// The largest of three, one instruction (NaN operands give way, as in fmaxf).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Two float32 operations in one instruction.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split_pair(uint64_t r, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// s <- tanh(x), x = s / (cap sqrt(d)), for N columns of a row.  Where all of a
// warp's |x| are at most 3/4 (scores below 3/4 of the cap, the usual case), an odd
// polynomial of degree 9 on the FMA pipe, relative error below 6e-7: x P(x^2), P a
// weighted least-squares fit of tanh(x) / x reweighted to equal ripple, with the
// factor between s and x in its coefficients.  Else 1 - 2 / (1 + e^(2x)): two more
// special-function operations an element beside the softmax's one, and off by
// 2^-22 of the cap, which there is not far above the largest score.
template <int N>
__device__ __forceinline__ void cap_tanh(const DocArgs& p, float* s) {
    float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < N; c += 2) top[(c >> 1) & 3] = max3(top[(c >> 1) & 3], fabsf(s[c]), fabsf(s[c + 1]));
    if (__all_sync(0xffffffffu, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) <= p.cap_limit)) {
        uint64_t k[5];
#pragma unroll
        for (int e = 0; e < 5; ++e) k[e] = pair_of(p.cap_poly[e], p.cap_poly[e]);
#pragma unroll
        for (int c = 0; c < N; c += 2) {
            const uint64_t x = pair_of(s[c], s[c + 1]), u = mul_pair(x, x);
            uint64_t r = fma_pair(k[4], u, k[3]);
            r = fma_pair(r, u, k[2]);
            r = fma_pair(r, u, k[1]);
            r = fma_pair(r, u, k[0]);
            split_pair(mul_pair(x, r), s[c], s[c + 1]);
        }
    } else {
#pragma unroll
        for (int c = 0; c < N; ++c) s[c] = 1.f - __fdividef(2.f, 1.f + ex2(s[c] * p.cap_exp));
    }
}

// s <- mul s - slope |c - at| + add for N columns c of a row, and its power of two.
// Where the warp's columns all lie on one side of their rows' distance 0 the distance
// is linear: one multiply-add of the column number, without an absolute value.
// (kSides: with that form as well; under a cap its code would only crowd the rest out
// of the instruction caches.)  Column numbers come as eight's start and the place in
// it: a constant pair (c, c + 1) for every two columns takes two moves each.
template <bool kExp, int N, bool kSides>
__device__ __forceinline__ void bias_scores(float* s, float mul, float slope, float at, float add) {
    const uint64_t mul2 = pair_of(mul, mul);
    const bool before = kSides && __all_sync(0xffffffffu, at >= static_cast<float>(N - 1));
    if (before || (kSides && __all_sync(0xffffffffu, at <= 0.f))) {
        const float step = before ? slope : -slope;
        const float base = fmaf(-step, at, add);
        uint64_t part[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) part[e] = pair_of(step * (2 * e), step * (2 * e + 1));
#pragma unroll
        for (int c = 0; c < N; c += 2) {
            const float rest = fmaf(static_cast<float>(c & ~7), step, base);
            split_pair(fma_pair(pair_of(s[c], s[c + 1]), mul2, add_pair(part[(c >> 1) & 3], pair_of(rest, rest))), s[c], s[c + 1]);
            if (kExp) s[c] = ex2(s[c]), s[c + 1] = ex2(s[c + 1]);
        }
        return;
    }
    const uint64_t step2 = pair_of(-slope, -slope), add2 = pair_of(add, add);
    uint64_t part[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) part[e] = pair_of(2.f * e, 2.f * e + 1.f);
#pragma unroll
    for (int c = 0; c < N; c += 2) {
        const float c8 = static_cast<float>(c & ~7) - at;
        float a, b;
        split_pair(add_pair(part[(c >> 1) & 3], pair_of(c8, c8)), a, b);
        const uint64_t rest = fma_pair(step2, pair_of(fabsf(a), fabsf(b)), add2);
        split_pair(fma_pair(pair_of(s[c], s[c + 1]), mul2, rest), s[c], s[c + 1]);
        if (kExp) s[c] = ex2(s[c]), s[c + 1] = ex2(s[c + 1]);
    }
}

// s <- 2^(mul s + add).
template <int N>
__device__ __forceinline__ void exp_scores(float* s, float mul, float add) {
    const uint64_t mul2 = pair_of(mul, mul), add2 = pair_of(add, add);
#pragma unroll
    for (int c = 0; c < N; c += 2) {
        float a, b;
        split_pair(fma_pair(pair_of(s[c], s[c + 1]), mul2, add2), a, b);
        s[c] = ex2(a);
        s[c + 1] = ex2(b);
    }
}
// s <- s (v + add), and s <- s (1 - t^2).
template <int N>
__device__ __forceinline__ void times_sum(float* s, const uint32_t* v, float add) {
    const uint64_t add2 = pair_of(add, add);
#pragma unroll
    for (int c = 0; c < N; c += 2)
        split_pair(mul_pair(pair_of(s[c], s[c + 1]), add_pair(pair_of(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), add2)),
                   s[c], s[c + 1]);
}
template <int N>
__device__ __forceinline__ void times_cap_slope(float* s, const float* t) {
    const uint64_t one2 = pair_of(1.f, 1.f), minus2 = pair_of(-1.f, -1.f);
#pragma unroll
    for (int c = 0; c < N; c += 2) {
        const uint64_t x = pair_of(t[c], t[c + 1]);
        split_pair(mul_pair(pair_of(s[c], s[c + 1]), fma_pair(mul_pair(x, minus2), x, one2)), s[c], s[c + 1]);
    }
}

// Bit c: column c of 32 lies in [lo, hi).
__device__ __forceinline__ uint32_t columns_in(int lo, int hi) {
    const uint32_t below_hi = hi >= 32 ? 0xffffffffu : hi <= 0 ? 0u : (1u << hi) - 1u;
    const uint32_t below_lo = lo >= 32 ? 0xffffffffu : lo <= 0 ? 0u : (1u << lo) - 1u;
    return below_hi & ~below_lo;
}

// `hidden` outside the columns [lo, hi) of a row: a select per element on a bit of
// one word per 32 columns, for both ends at once.  A warp whose rows all see the 32
// columns skips them.
template <int N>
__device__ __forceinline__ void hide_columns(float* s, int lo, int hi, float hidden) {
    if (__all_sync(0xffffffffu, lo <= 0 && hi >= N)) return;
#pragma unroll
    for (int b = 0; b < N; b += 32) {
        const uint32_t in = columns_in(lo - b, hi - b);
        if (__all_sync(0xffffffffu, in == 0xffffffffu)) continue;
#pragma unroll
        for (int c = 0; c < 32; ++c) s[b + c] = (in & (1u << c)) ? s[b + c] : hidden;
    }
}

// The blocks that a tile of the plan walks, whatever the plan's memory holds.
__device__ __forceinline__ int2 block_range(const int2* blocks, int b, int n_blocks) {
    if (b >= n_blocks) return make_int2(0, 0);
    const int2 r = blocks[b];
    const int first = min(max(r.x, 0), n_blocks);
    return make_int2(first, min(max(r.y, first), n_blocks));
}

// Padding: rows before the first document and behind the last, which see nothing and
// which nothing sees.  They hold anything, NaN as well as what a fresh allocation left,
// and a product over a tile would carry that into all its rows.  So the warp that issues
// the products makes their rows of such an operand zeros in shared memory first.  (Formed
// again pair by pair, as for what a document itself holds, the backward of a document of
// 4000 rows behind which 96 rows were NaN took 182 ms, 32 heads of 128; with zeros 0.3.
// By the row warps, the test alone cost batches without padding 1 to 2 %; here at most 1.)
//
// The rows that are not padding, [x, y): empty intervals of the first and the last row
// say where it ends and starts.
__device__ __forceinline__ int2 document_rows(const DocArgs& p) {
    const int2 a = p.plan.rows[0], b = p.plan.rows[p.tokens - 1];
    return make_int2(a.y <= a.x ? a.x : 0, b.y <= b.x ? b.x : 0x7fffffff);
}
__device__ __forceinline__ bool has_padding(int r0, int2 live) { return r0 < live.x || r0 + kRows > live.y; }
// By the warp that issues the products, while it would wait for the row warps: zeros in the
// padding rows of a tile of D columns whose first row is the tensor's r0 (boxes of 128
// 128-byte rows; the swizzle permutes within a row), or of two tiles `other` bytes apart.
template <int D>
__device__ __forceinline__ void zero_padding(uint32_t tile, int r0, int2 live, int lane, uint32_t other = 0) {
    constexpr int kLanes = D / 8;  // 16 bytes a lane
    // rows before `head` and from `tail` on, inside the tile whatever the plan's memory holds
    const int head = min(live.x - r0, kRows), tail = max(live.y - r0, 0);
    const uint32_t at = tile + static_cast<uint32_t>((lane % kLanes >> 3) * 16384 + (lane & 7) * 16);
    const int first = head > 0 ? 0 : tail, end = tail < kRows ? kRows : head;
#pragma unroll 1
    for (int i = first + lane / kLanes; i < end; i += 32 / kLanes)
        if (i < head || i >= tail) {
            st_shared_v4(at + static_cast<uint32_t>(i * 128), make_uint4(0u, 0u, 0u, 0u));
            if (other) st_shared_v4(at + static_cast<uint32_t>(i * 128) + other, make_uint4(0u, 0u, 0u, 0u));
        }
    fence_proxy_async_smem();  // the products read through the other proxy
    __syncwarp();
}

__device__ __forceinline__ bool finite32(const float (&v)[32]) {
    float m[4] = {0.f, 0.f, 0.f, 0.f};  // 0 v is NaN for a v that is not finite
#pragma unroll
    for (int e = 0; e < 32; ++e) m[e & 3] = fmaf(v[e], 0.f, m[e & 3]);
    return (m[0] + m[1]) + (m[2] + m[3]) == 0.f;
}

// Results leave through shared memory and TMA: a warp packs 32 rows of 64 columns
// into 4 KiB (128-byte rows, 128-byte swizzle; 64-byte rows have theirs) and one
// thread stores the box, rows behind the tensor clipped.  Stored from registers, each lane to its own row, a
// tile's results held its warps for about 5000 cycles, three passes over its keys;
// the copy runs beside the next tile's work.
constexpr uint32_t kStageBytes = 4096;
template <int kRowBytes = 128>
__device__ __forceinline__ void stage32(uint32_t stage, int lane, int half, const float (&v)[32], float f, bool zero) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint4 w = make_uint4(pack_bf16x2(v[8 * k] * f, v[8 * k + 1] * f), pack_bf16x2(v[8 * k + 2] * f, v[8 * k + 3] * f),
                             pack_bf16x2(v[8 * k + 4] * f, v[8 * k + 5] * f), pack_bf16x2(v[8 * k + 6] * f, v[8 * k + 7] * f));
        if (zero) w = make_uint4(0u, 0u, 0u, 0u);
        const uint32_t at = static_cast<uint32_t>(lane * kRowBytes + (4 * half + k) * 16);
        st_shared_v4(stage + (at ^ (((at >> 7) & (kRowBytes / 16 - 1)) << 4)), w);
    }
}
__device__ __forceinline__ void store_stage(const CUtensorMap* map, uint32_t stage, int lane, int col, int row) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        tma_store_2d(map, stage, col, row);
        bulk_commit_group();
    }
}
// The stage may be written again: its last store has read it.
__device__ __forceinline__ void stage_free(int lane) {
    if (lane == 0) bulk_wait_group_read<0>();
    __syncwarp();
}
// This warp's stores have been written, before some of their rows are written again.
__device__ __forceinline__ void stores_done(int lane) {
    if (lane == 0) bulk_wait_group_all();
    __syncwarp();
}

__device__ __forceinline__ void load_tmem32(uint32_t t, float (&v)[32]) {
    uint32_t r[32];
    tmem_load_32(t, r);
    tmem_wait_load();
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
}

// ------------------------------------------------------------------------ forward

// Every warp of a warpgroup takes part.  A claim waits until the releases of the
// other warpgroups of the block have made room.
template <int N>
__device__ __forceinline__ void registers_release() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_claim() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Cancels the launch of the next CTA of the grid that has not started and
// writes its place to `slot` (16 bytes), completing on `bar`: the CTA takes that
// one's work.  Tiles go to whichever CTA is free, with no counter in memory that
// two calls or two graphs could share.
__device__ __forceinline__ void next_cta_request(uint32_t slot, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(slot),
                 "r"(bar)
                 : "memory");
}
// The answer: the CTA's number, or -1 when none is left (after which no request
// may follow).
__device__ __forceinline__ int next_cta_answer(uint32_t slot) {
    uint32_t got, x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
        : "=r"(got), "=r"(x)
        : "r"(slot)
        : "memory");
    return got ? static_cast<int>(x) : -1;
}

// The two tiles of forward tile t: the same kv group and one K / V stream.
struct FwdTile {
    int h[2], q0[2];
    int g, first, nk;
};

__host__ __device__ inline int fwd_tiles(const DocArgs& p) {
    return (p.n_heads / p.n_kv_heads) % 2 == 0 ? p.n_blocks * (p.n_heads / 2) : (p.n_blocks + 1) / 2 * p.n_heads;
}

// Where tile t lies: heads, query rows, kv head.
__device__ __forceinline__ FwdTile fwd_place(const DocArgs& p, int t) {
    FwdTile f{};
    const int group = p.n_heads / p.n_kv_heads;
    if (group % 2 == 0) {
        const int pairs = p.n_heads / 2;
        const int qb = p.n_blocks - 1 - t / pairs;  // in one long document, the longest rows first
        f.h[0] = 2 * (t % pairs);
        f.h[1] = f.h[0] + 1;
        f.q0[0] = f.q0[1] = qb * kRows;
    } else {
        const int b = (p.n_blocks + 1) / 2 - 1 - t / p.n_heads;
        f.h[0] = f.h[1] = t % p.n_heads;
        f.q0[0] = 2 * b * kRows;
        f.q0[1] = f.q0[0] + kRows;
    }
    f.g = f.h[0] / group;
    return f;
}

// The same with its key blocks: those that a row of either tile sees.
__device__ __forceinline__ FwdTile fwd_tile(const DocArgs& p, int t) {
    FwdTile f = fwd_place(p, t);
    const int2 x = block_range(p.plan.q_blocks, f.q0[0] / kRows, p.n_blocks), y = block_range(p.plan.q_blocks, f.q0[1] / kRows, p.n_blocks);
    const bool ex = x.x == x.y, ey = y.x == y.y;
    f.first = ex ? y.x : ey ? x.x : min(x.x, y.x);
    f.nk = (ex ? y.y : ey ? x.y : max(x.y, y.y)) - f.first;
    return f;
}

template <int D>
struct DocFwdSmem {
    static constexpr int kStages = D == 64 ? 4 : 2;
    static constexpr uint32_t kTile = D * 256;
    static constexpr uint32_t kQ = 0;           // Q of tile A, then Q of tile B
    static constexpr uint32_t kKV = 2 * kTile;  // stage s: K at kKV + 2 s kTile, V after it
    static constexpr uint32_t kStage = kKV + 2 * kStages * kTile;  // results, 4 KiB a row warp
    static constexpr uint32_t kAnswer = kStage + 8 * kStageBytes;   // 16 bytes
    static constexpr uint32_t kBars = kAnswer + 16;
    // Q full / empty, the K / V ring, S, P and PV of both tiles (two of each in turn), tile slots full / empty,
    // answer, drain
    static constexpr int kNumBars = 2 + 2 * kStages + 12 + 4 + 2;
    static constexpr uint32_t kTmemSlot = (kBars + 8 * kNumBars + 15) / 16 * 16;
    static constexpr uint32_t kTileSlot = kTmemSlot + 16;  // two slots of a tile's place, first key block and steps
    static constexpr uint32_t kRowSlot = kTileSlot + 2 * 16;  // and of its rows' intervals
    static constexpr size_t kUsed = kRowSlot + 2 * 1024;
    static constexpr size_t kBytes = kUsed > kMinSmem ? kUsed : kMinSmem;
};

// The two-head forward of the causal core over the steps of many tiles: the
// K / V ring, the score buffers and the barriers' phases run on from one tile to
// the next, and the next tile's Q loads as soon as the last scores of the
// current one are formed, while its softmax, last product and stores run.  A
// tile that sees nothing (padding) has no steps.
//
// Key blocks are taken from the last to the first: a row meets its own key, and with
// a distance bias its largest scores, in its first block, and its accumulator is
// seldom rescaled (from first to last, a tile of a steep slope rescaled at every
// step, 700 cycles of 2800).
//
// Three warpgroups: warp 0 loads, warp 1 issues products (warps 2 and 3 only hold
// their place), warps 4-7 and 8-11 are the softmax rows of tiles A and B.  The
// first hands registers to the other two.
//
// Bound by the softmax rows: a step of two tiles takes 2700 to 2900 cycles where
// its products take 2048 (heads of 128; 4900 with a cap, 1500 of them for tanh, 900
// for the exponential, 1400 until the next scores), and 4000 cycles lie between two
// tiles (last product, normalising, stores, first scores).  32 heads of 128 on 8,
// 4096 tokens: 9 documents in 40 us (2.2 M pairs in visible blocks, 900 TFLOP/s of
// theirs), 2 with a cap in 95; 16 heads of 64, one document of 16384 with a bias in
// 532 (1034 TFLOP/s of its visible pairs).  Slower, each against its time then (9
// documents; bias): sixteen row warps of half the columns (45 -> 50 us; 805 -> 826),
// a quarter of the exponentials as polynomials on the FMA pipe (45 -> 46; 645 -> 714:
// the exponential unit, now 44 % busy, does not bind), scores loaded in four parts beside the work on
// them (45 -> 49; 604 -> 722), four more warps that store the results while the rows
// go on (41 -> 43; 601 -> 630), at heads of 128 steps of 64 keys with two score
// buffers a tile (40 -> 42; a bias over 8192 rows 198 -> 232).
constexpr int kDocFwdThreads = 384;
constexpr int kDocFwdRegs = 168, kDocFwdFew = 56, kDocFwdMany = 224;
static_assert(kDocFwdFew + 2 * kDocFwdMany <= 3 * kDocFwdRegs, "registers of the launch");

template <int D, int M>
__global__ void __launch_bounds__(kDocFwdThreads, 1)
    document_fwd_kernel(const __grid_constant__ CUtensorMap map_qkv, const __grid_constant__ CUtensorMap map_a,
                        const __grid_constant__ DocArgs p) {
    using L = DocFwdSmem<D>;
    constexpr int NS = L::kStages;
    constexpr uint32_t kTile = L::kTile;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = smem_addr(smem_raw);
    if (base & 1023u) {  // the tiles' 128-byte swizzle needs a 1 KiB-aligned start
        if (threadIdx.x == 0) atomicCAS(p.status, 0, kSiteAttn);
        return;
    }
    const uint32_t s_q = base + L::kQ, s_kv = base + L::kKV, s_answer = base + L::kAnswer;
    const uint32_t bars = base + L::kBars;
    const uint32_t q_full = bars, q_empty = bars + 8u;
    auto kv_full = [&](uint32_t s) { return bars + 8u * (2 + s); };
    auto kv_empty = [&](uint32_t s) { return bars + 8u * (2 + NS + s); };
    constexpr int kB = 2 + 2 * NS;
    // Step g of tile x.  Two barriers in turn: a third score buffer lets a tile's scores
    // run one step ahead of its softmax, so one warp of it can be a step ahead of
    // another, and its arrival must not count for the step before.
    auto s_full = [&](int x, uint32_t g) { return bars + 8u * (kB + 2 * x + (g & 1u)); };
    auto p_full = [&](int x, uint32_t g) { return bars + 8u * (kB + 4 + 2 * x + (g & 1u)); };
    auto pv_done = [&](int x, uint32_t g) { return bars + 8u * (kB + 8 + 2 * x + (g & 1u)); };
    auto tile_full = [&](uint32_t s) { return bars + 8u * (kB + 12 + s); };
    auto tile_empty = [&](uint32_t s) { return bars + 8u * (kB + 14 + s); };
    const uint32_t answer_full = bars + 8u * (kB + 16), drain = bars + 8u * (kB + 17);
    const uint32_t tmem_slot = base + L::kTmemSlot;
    volatile uint32_t* tmem_slot_ptr = reinterpret_cast<volatile uint32_t*>(smem_raw + L::kTmemSlot);
    const int4* tile_slot = reinterpret_cast<const int4*>(smem_raw + L::kTileSlot);
    const int2* row_slot = reinterpret_cast<const int2*>(smem_raw + L::kRowSlot);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int s = 0; s < NS; ++s) {
            mbar_init(kv_full(s), 1);
            mbar_init(kv_empty(s), 1);
        }
        for (int x = 0; x < 2; ++x) {
            for (uint32_t g = 0; g < 2; ++g) {
                mbar_init(s_full(x, g), 1);
                mbar_init(p_full(x, g), 4);
                mbar_init(pv_done(x, g), 1);
            }
            mbar_init(tile_full(x), 1);
            mbar_init(tile_empty(x), 9);  // the MMA warp and the eight row warps
        }
        mbar_init(answer_full, 1);
        mbar_init(drain, 1);
        mbar_fence_init();
        tma_prefetch_map(&map_qkv);
    }
    if (warp == 1) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    wait_for_previous();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot_ptr;
    // Tensor memory, heads of 128: S_A 0-127, S_B 128-255, O_A 256-383, O_B 384-511.
    // Heads of 64 leave room for a third score buffer: the tiles' score blocks A0, B0,
    // A1, B1, .. take buffers 0-127, 128-255, 256-383 in turn, O_A is 384-447, O_B
    // 448-511.  P is packed into the first 64 columns of its scores' buffer.
    auto t_s = [&](int x, uint32_t g) {
        return tmem_base + 128u * (D == 64 ? (2u * g + static_cast<uint32_t>(x)) % 3u : static_cast<uint32_t>(x));
    };
    auto t_o = [&](int x) { return tmem_base + (D == 64 ? 384u + 64u * x : 256u + 128u * x); };
    // Tile B is the next head, or (odd groups) the next query block.
    const bool two_heads = (p.n_heads / p.n_kv_heads) % 2 == 0;
    // A consumer warp's view of tile slot n & 1: the first query row of tile A (-1: no
    // tile left), its head, the first key block and the steps; `see`: the intervals of
    // its row of tile A.  Then the warp releases the slot.
    auto take_tile = [&](uint32_t n, int row, int4& tile, int2& see) {
        if (!warp_wait(tile_full(n & 1u), (n >> 1) & 1u, p.status, p.wait_ns)) return false;
        tile = tile_slot[n & 1u];
        see = row_slot[(n & 1u) * kRows + row];
        __syncwarp();
        if (lane == 0) mbar_arrive(tile_empty(n & 1u));
        return tile.x >= 0;
    };

    if (warp < 4) {
        registers_release<kDocFwdFew>();
        if (warp == 0) {
            if (lane == 0) {
                uint32_t nq = 0, nkv = 0, nt = 0;  // Q loads, K / V steps and tile slots issued
                int t = static_cast<int>(blockIdx.x);
                for (uint32_t n = 0;; ++n) {
                    if (!mbar_wait_fast(tile_empty(n & 1u), ((n >> 1) & 1u) ^ 1u, p.status, kSiteAttn, p.wait_ns)) break;
                    const FwdTile f = t >= 0 ? fwd_tile(p, t) : FwdTile{};
                    *reinterpret_cast<int4*>(smem_raw + L::kTileSlot + 16 * (n & 1u)) = t < 0 ? make_int4(-1, 0, 0, 0) : make_int4(f.q0[0], f.h[0], f.first, f.nk);
                    ++nt;
                    if (t < 0) {
                        mbar_arrive(tile_full(n & 1u));
                        break;
                    }
                    // the intervals of tile A's rows land on the same barrier (tile B's own rows,
                    // in odd groups, are read where they are needed)
                    mbar_arrive_expect_tx(tile_full(n & 1u), 1024);
                    bulk_load_1d(base + L::kRowSlot + 1024u * (n & 1u), p.plan.rows + f.q0[0], 1024, tile_full(n & 1u));
                    if (f.nk > 0) {
                        // Q once the previous tile's scores are formed
                        if (!mbar_wait_fast(q_empty, (nq & 1u) ^ 1u, p.status, kSiteAttn, p.wait_ns)) break;
                        mbar_arrive_expect_tx(q_full, 2 * kTile);
                        load_tile<D>(s_q, &map_qkv, q_full, f.h[0] * D, f.q0[0]);
                        load_tile<D>(s_q + kTile, &map_qkv, q_full, f.h[1] * D, f.q0[1]);
                        ++nq;
                    }
                    const int kcol = (p.n_heads + f.g) * D, vcol = (p.n_heads + p.n_kv_heads + f.g) * D;
                    bool ok = true;
                    for (int j = 0; j < f.nk; ++j) {
                        const uint32_t st = nkv % NS;
                        if (!mbar_wait_fast(kv_empty(st), ((nkv / NS) & 1u) ^ 1u, p.status, kSiteAttn, p.wait_ns)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(kv_full(st), 2 * kTile);
                        const int k0 = (f.first + f.nk - 1 - j) * kRows;
                        load_tile<D>(s_kv + 2 * st * kTile, &map_qkv, kv_full(st), kcol, k0);
                        load_tile<D>(s_kv + (2 * st + 1) * kTile, &map_qkv, kv_full(st), vcol, k0);
                        ++nkv;
                    }
                    if (!ok) break;
                    // the next tile's number after this tile's last load, a ring's depth before its end
                    mbar_arrive_expect_tx(answer_full, 16);
                    next_cta_request(s_answer, answer_full);
                    if (!mbar_wait_fast(answer_full, n & 1u, p.status, kSiteAttn, p.wait_ns)) break;
                    t = next_cta_answer(s_answer);
                    fence_proxy_async_smem();  // the answer is read before another one is written over it
                    if (t >= 0) {
                        const FwdTile nx = fwd_tile(p, t);
                        prefetch_tile<D>(&map_qkv, nx.h[0] * D, nx.q0[0]);
                        if (nx.q0[1] < p.tokens) prefetch_tile<D>(&map_qkv, nx.h[1] * D, nx.q0[1]);
                    }
                }
                // no copy may land after the CTA has gone
                if (nq > 0) mbar_wait_fast(q_full, (nq - 1) & 1u, p.status, kSiteDrain, p.wait_ns);
                for (int s = 0; s < NS; ++s) {
                    const uint32_t u = ring_uses(nkv, NS, s);
                    if (u > 0) mbar_wait_fast(kv_full(s), (u - 1) & 1u, p.status, kSiteDrain, p.wait_ns);
                }
                for (int s = 0; s < 2; ++s) {
                    const uint32_t u = ring_uses(nt, 2, s);
                    if (u > 0) mbar_wait_fast(tile_full(s), (u - 1) & 1u, p.status, kSiteDrain, p.wait_ns);
                }
            }
        } else if (warp == 1) {
            // the whole warp runs the issue loop; its elected lane carries each instruction
            const uint32_t leader = elect_one_sync();
            constexpr uint32_t idesc_s = mma_idesc_bf16(128, 128, false, false);
            constexpr uint32_t idesc_o = mma_idesc_bf16(128, D, false, true);
            auto issue_s = [&](int x, uint32_t g) {
                const uint64_t a_desc = kdesc_base(s_q + static_cast<uint32_t>(x) * kTile),
                               b_desc = kdesc_base(s_kv + 2 * (g % NS) * kTile);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    umma_bf16_elected(leader, t_s(x, g), kdesc_at(a_desc, kk), kdesc_at(b_desc, kk), idesc_s, kk > 0);
                umma_commit_elected(leader, s_full(x, g));
            };
            auto issue_pv = [&](int x, uint32_t g, bool first) {
                if (!warp_wait(p_full(x, g), (g >> 1) & 1u, p.status, p.wait_ns)) return false;
                tc_fence_after();
                const uint64_t v_desc = mndesc_base(s_kv + (2 * (g % NS) + 1) * kTile);
#pragma unroll
                for (int kk = 0; kk < kRows / 16; ++kk)
                    umma_bf16_ts_elected(leader, t_o(x), t_s(x, g) + 8 * kk, mndesc_at(v_desc, kk), idesc_o,
                                         (!first || kk > 0) ? 1u : 0u);
                umma_commit_elected(leader, pv_done(x, g));
                return true;
            };
            auto kv_ready = [&](uint32_t g) {
                if (!warp_wait(kv_full(g % NS), (g / NS) & 1u, p.status, p.wait_ns)) return false;
                tc_fence_after();
                return true;
            };
            const int2 live = document_rows(p);
            uint32_t g = 0, nq = 0;  // steps and tiles with steps so far
            bool ok = true;
            for (uint32_t n = 0; ok; ++n) {
                int4 tile;
                int2 unused;
                if (!take_tile(n, 0, tile, unused)) break;
                const int nk = tile.w;
                if (nk == 0) continue;
                if (!warp_wait(q_full, nq & 1u, p.status, p.wait_ns) || !kv_ready(g)) break;
                ++nq;
                issue_s(0, g);
                issue_s(1, g);
                if (nk == 1) umma_commit_elected(leader, q_empty);
                // Heads of 128: PV_A[j], S_A[j+1], PV_B[j], S_B[j+1]; S_X[j+1] overwrites
                // P_X[j].  Heads of 64: S_A[j+1], PV_A[j], S_B[j+1], PV_B[j]; S_A[j+1]
                // overwrites P_B[j-1], S_B[j+1] P_A[j]: a tile's next scores are there when
                // its softmax has finished the last ones.
                for (int j = 0; j < nk; ++j, ++g) {
                    const bool more = j + 1 < nk;
                    const int k0 = (tile.z + nk - 1 - j) * kRows;
                    ok = false;
                    if (D == 64 && more) {
                        if (!kv_ready(g + 1)) break;
                        issue_s(0, g + 1);
                    }
                    if (has_padding(k0, live)) zero_padding<D>(s_kv + (2 * (g % NS) + 1) * kTile, k0, live, lane);  // V[g]
                    if (!issue_pv(0, g, j == 0)) break;
                    if (D == 128 && more) {
                        if (!kv_ready(g + 1)) break;
                        issue_s(0, g + 1);
                    }
                    if (D == 64 && more) issue_s(1, g + 1);
                    if (!issue_pv(1, g, j == 0)) break;
                    umma_commit_elected(leader, kv_empty(g % NS));
                    if (D == 128 && more) issue_s(1, g + 1);
                    // Q is free for the next tile once its last scores are formed
                    if (j + 2 == nk) umma_commit_elected(leader, q_empty);
                    ok = true;
                }
            }
            umma_commit_elected(leader, drain);
            mbar_wait_fast(drain, 0, p.status, kSiteDrain, p.wait_ns);
        }
    } else {
        registers_claim<kDocFwdMany>();
        // ---------------- softmax rows: warps 4-7 tile A, warps 8-11 tile B
        const int x = (warp - 4) >> 2;
        const int qw = warp & 3;
        const int row = qw * 32 + lane;
        const uint32_t t_row = static_cast<uint32_t>(qw * 32) << 16;
        const uint32_t to = t_o(x);
        uint32_t g = 0;  // steps so far
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            int4 tile;
            int2 see;
            if (!take_tile(n, row, tile, see)) break;
            const int first = tile.z, nk = tile.w;
            const int h = two_heads ? tile.y + x : tile.y;
            const int q = (two_heads ? tile.x : tile.x + x * kRows) + row;
            const bool valid = q < p.tokens;
            if (!two_heads && x && valid) see = p.plan.rows[q];
            if (!valid) see = make_int2(0, 0);
            const bool empty = see.y <= see.x;
            const float slope2 = mode_biases(M) ? p.slopes[h] * kLog2e : 0.f;
            // -1e30, not -infinity: a row that has seen no key yet keeps finite differences
            float m = -1e30f, l = 0.f;
            for (int j = 0; j < nk; ++j, ++g) {
                if (!warp_wait(s_full(x, g), (g >> 1) & 1u, p.status, p.wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t ts = t_s(x, g);
                float s[128];
                {
                    uint32_t r[128];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        tmem_load_32(ts + t_row + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(r + 32 * c));
                    tmem_wait_load();
#pragma unroll
                    for (int e = 0; e < 128; ++e) s[e] = __uint_as_float(r[e]);
                }
                const int k0 = (first + nk - 1 - j) * kRows;  // the diagonal first
                // unmodified (and capped, undistanced) scores are scaled below and in the exponent's FMA
                float sc = 1.f;
                if constexpr (M == kDocPlain) sc = p.scale_log2;
                if constexpr (mode_caps(M)) {
#pragma unroll
                    for (int c = 0; c < 128; c += 32) cap_tanh<32>(p, s + c);
                    sc = p.cap_log2;
                }
                // Distances: in a block whose keys all lie on one side of the warp's rows
                // (all but the diagonal's) a score is mul s + step c + base.  Its step
                // (c mod 8) is added here and the rest, which eight columns share, to their
                // maximum and in the exponent: 64 constant pairs (c, c + 1) would cost two
                // moves each.
                float step = 0.f, off = 0.f;
                if constexpr (mode_biases(M)) {
                    const float mul = M == kDocBias ? p.scale_log2 : p.cap_log2, at = static_cast<float>(q - k0);
                    const bool before = __all_sync(0xffffffffu, at >= 127.f);
                    if (before || __all_sync(0xffffffffu, at <= 0.f)) {
                        step = before ? slope2 : -slope2;
                        off = -step * at;
                        const uint64_t mul2 = pair_of(mul, mul);
                        uint64_t rest[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) rest[e] = pair_of(step * (2 * e), step * (2 * e + 1));
#pragma unroll
                        for (int c = 0; c < 128; c += 2)
                            split_pair(fma_pair(pair_of(s[c], s[c + 1]), mul2, rest[(c >> 1) & 3]), s[c], s[c + 1]);
                    } else {
                        bias_scores<false, 128, false>(s, mul, slope2, at, 0.f);
                    }
                    sc = 1.f;
                }
                hide_columns<128>(s, see.x - k0, see.y - k0, -INFINITY);
                // eight running maxima and sums, not one chain of 128 dependent operations
                float mx8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) mx8[e] = -INFINITY;
                if constexpr (mode_biases(M)) {
#pragma unroll
                    for (int c = 0; c < 128; c += 8) {
                        const float m8 = max3(max3(max3(s[c], s[c + 1], s[c + 2]), s[c + 3], s[c + 4]), s[c + 5], fmaxf(s[c + 6], s[c + 7]));
                        mx8[(c >> 3) & 7] = fmaxf(mx8[(c >> 3) & 7], m8 + fmaf(static_cast<float>(c), step, off));
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 128; c += 2) mx8[(c >> 1) & 7] = max3(mx8[(c >> 1) & 7], s[c], s[c + 1]);
                }
                float mx = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                 fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
                mx *= sc;
                // A row's maximum rose far above its reference: the warp rescales O and l of
                // all its rows to their new maxima (warp-wide tensor-memory loads and
                // stores; rescaling to any larger reference is exact), after PV_X[j-1].  Rows
                // that have seen no key yet hold zeros and take their first maximum freely.
                if (__any_sync(0xffffffffu, mx > m + 8.f)) {
                    const float m_new = fmaxf(m, mx);
                    if (__any_sync(0xffffffffu, mx > m + 8.f && l > 0.f)) {
                        if (!warp_wait(pv_done(x, g - 1), ((g - 1) >> 1) & 1u, p.status, p.wait_ns)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const float alpha = ex2(m - m_new);
                        l *= alpha;
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t r[32];
                            tmem_load_32(to + t_row + 32 * c, r);
                            tmem_wait_load();
#pragma unroll
                            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
                            tmem_store_32(to + t_row + 32 * c, r);
                        }
                        m = m_new;
                    } else if (!(l > 0.f)) {
                        m = m_new;
                    }
                }
                const uint64_t sc2 = pair_of(sc, sc), m2 = pair_of(-m, -m);
                uint64_t sum[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float a, b;
                        if constexpr (mode_biases(M)) {
                            const int c8 = (32 * c + 2 * e) & ~7;
                            const float add = fmaf(static_cast<float>(c8), step, off - m);
                            split_pair(add_pair(pair_of(s[32 * c + 2 * e], s[32 * c + 2 * e + 1]), pair_of(add, add)), a, b);
                        } else {
                            split_pair(fma_pair(pair_of(s[32 * c + 2 * e], s[32 * c + 2 * e + 1]), sc2, m2), a, b);
                        }
                        a = ex2(a);
                        b = ex2(b);
                        sum[e & 3] = add_pair(sum[e & 3], pair_of(a, b));
                        w[e] = pack_bf16x2(a, b);  // P to bf16: the tensor cores' operand; l sums it unrounded
                    }
                    tmem_store_16(ts + t_row + 16 * c, w);
                }
                float la, lb;
                split_pair(add_pair(add_pair(sum[0], sum[1]), add_pair(sum[2], sum[3])), la, lb);
                l += la + lb;
                tmem_wait_store();
                tc_fence_before();
                warp_arrive(p_full(x, g), lane);
            }
            if (!ok) break;
            bool again = false;  // not finite: formed again below
            float inv = 0.f;
            if (nk > 0) {
                if (!warp_wait(pv_done(x, g - 1), ((g - 1) >> 1) & 1u, p.status, p.wait_ns)) break;
                tc_fence_after();
                inv = 1.f / l;
                again = !(fabsf(inv) <= 3e38f);
            }
            const uint32_t stage = base + L::kStage + kStageBytes * static_cast<uint32_t>(warp - 4);
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                float o[2][32] = {};
                if (nk > 0) {
                    load_tmem32(to + t_row + 64 * c, o[0]);
                    load_tmem32(to + t_row + 64 * c + 32, o[1]);
                    again |= !finite32(o[0]) || !finite32(o[1]);
                }
                stage_free(lane);
                stage32(stage, lane, 0, o[0], inv, empty);
                stage32(stage, lane, 1, o[1], inv, empty);
                if (q - lane < p.tokens) store_stage(&map_a, stage, lane, h * D + 64 * c, q - lane);
            }
            tc_fence_before();
            if (valid) p.lse_out[static_cast<int64_t>(h) * p.ld_stat + q] = empty ? -INFINITY : m + lg2(l);
            uint32_t redo = __ballot_sync(0xffffffffu, again && valid && !empty);
            if (redo) stores_done(lane);
            while (redo) {
                const int src = __ffs(redo) - 1;
                redo &= redo - 1;
                document_forward_row<D>(p, q - lane + src, h, lane);
            }
        }
        stage_free(lane);  // shared memory outlives the stores that read it
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

// ------------------------------------------------------------------------ backward: dq

// The causal core's dQ tiles and pipeline (attention.cu): S and dP by warp 1, dQ
// by warp 10, two groups of row warps with 64 key columns each.  Bound, as dK / dV
// below, by the row warps and the chain from one product to the next.
template <int D>
struct DocDqSmem {
    // One V stage where the results' 32 KiB leave no room for two: V[g + 1] lands while
    // the row warps still turn dP[g] into dS[g].
    static constexpr int kKStages = 3, kVStages = D == 64 ? 2 : 1;
    static constexpr uint32_t kTile = D * 256;
    static constexpr uint32_t kQ = 0, kDO = kTile, kK = 2 * kTile;
    static constexpr uint32_t kV = kK + kKStages * kTile;
    static constexpr uint32_t kStage = kV + kVStages * kTile;  // results, 4 KiB a row warp
    static constexpr uint32_t kBars = kStage + 8 * kStageBytes;
    // q full / empty, the K ring (full, empty), the V ring (full, empty), S (2), dP,
    // dS (2), done, drain, the two tile slots (full, empty), dQ issued (2), dP issued (2)
    static constexpr int kNumBars = 2 + 2 * kKStages + 2 * kVStages + 2 + 5 + 4 + 4;
    static constexpr uint32_t kTmemSlot = kBars + 8 * kNumBars;
    static constexpr uint32_t kTileSlot = kTmemSlot + 8;  // the tile number held by each slot (two ints)
    static constexpr size_t kUsed = kTileSlot + 8;
};

struct DqTile {
    int h, q0, kb0, nk;
};
__device__ __forceinline__ DqTile dq_tile(const DocArgs& p, int t) {
    DqTile d;
    const int qb = p.n_blocks - 1 - t / p.n_heads;
    d.h = t % p.n_heads;
    d.q0 = qb * kRows;
    const int2 r = block_range(p.plan.q_blocks, qb, p.n_blocks);
    d.kb0 = r.x;
    d.nk = r.y - r.x;
    return d;
}

template <int D, int M>
__device__ __forceinline__ void document_dq(const CUtensorMap& map_qkv, const CUtensorMap& map_do, const CUtensorMap& map_dq,
                                            const DocArgs& p, uint8_t* smem_raw) {
    using L = DocDqSmem<D>;
    constexpr int NK = L::kKStages, NV = L::kVStages;
    constexpr uint32_t kTile = L::kTile;
    const uint32_t base = smem_addr(smem_raw);
    const uint32_t s_q = base + L::kQ, s_do = base + L::kDO, s_k = base + L::kK, s_v = base + L::kV,
                   s_stage = base + L::kStage;
    const uint32_t bars = base + L::kBars;
    const uint32_t q_full = bars, q_empty = bars + 8u;
    auto k_full = [&](uint32_t s) { return bars + 8u * (2 + s); };
    auto k_empty = [&](uint32_t s) { return bars + 8u * (2 + NK + s); };
    auto v_full = [&](uint32_t s) { return bars + 8u * (2 + 2 * NK + s); };
    auto v_empty = [&](uint32_t s) { return bars + 8u * (2 + 2 * NK + NV + s); };
    constexpr int kB = 2 + 2 * NK + 2 * NV;
    auto s_full = [&](uint32_t b) { return bars + 8u * (kB + b); };
    const uint32_t dp_full = bars + 8u * (kB + 2), done = bars + 8u * (kB + 3), drain = bars + 8u * (kB + 4);
    auto ds_full = [&](uint32_t g) { return bars + 8u * (kB + 5 + (g & 1u)); };
    auto tile_full = [&](uint32_t s) { return bars + 8u * (kB + 7 + s); };
    auto tile_empty = [&](uint32_t s) { return bars + 8u * (kB + 9 + s); };
    auto dq_issued = [&](uint32_t g) { return bars + 8u * (kB + 11 + (g & 1u)); };
    auto dp_issued = [&](uint32_t g) { return bars + 8u * (kB + 13 + (g & 1u)); };
    const uint32_t tmem_slot = base + L::kTmemSlot;
    volatile uint32_t* tmem_slot_ptr = reinterpret_cast<volatile uint32_t*>(smem_raw + L::kTmemSlot);
    volatile int* tile_slot = reinterpret_cast<volatile int*>(smem_raw + L::kTileSlot);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_tiles = p.n_blocks * p.n_heads;
    const int group = p.n_heads / p.n_kv_heads;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int s = 0; s < NK; ++s) {
            mbar_init(k_full(s), 1);
            mbar_init(k_empty(s), 1);
        }
        for (int s = 0; s < NV; ++s) {
            mbar_init(v_full(s), 1);
            mbar_init(v_empty(s), 1);
        }
        mbar_init(s_full(0), 1);
        mbar_init(s_full(1), 1);
        mbar_init(dp_full, 1);
        mbar_init(done, 1);
        mbar_init(drain, 2);  // both MMA warps
        for (int s = 0; s < 2; ++s) {
            mbar_init(ds_full(s), 8);
            mbar_init(tile_full(s), 1);
            mbar_init(tile_empty(s), 10);  // the two MMA warps and the eight row warps
            mbar_init(dq_issued(s), 1);
            mbar_init(dp_issued(s), 1);
        }
        mbar_fence_init();
        tma_prefetch_map(&map_qkv);
        tma_prefetch_map(&map_do);
    }
    if (warp == 1) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    wait_for_previous();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot_ptr;
    // columns: S buffers 0-127 and 128-255 (dS packed into columns 0-31 and
    // 64-95 of a buffer once read), dP 256-383, dQ 384..
    const uint32_t t_dp = tmem_base + 256, t_dq = tmem_base + 384;
    auto t_s = [&](uint32_t g) { return tmem_base + 128u * (g & 1u); };
    auto take_tile = [&](uint32_t n, int& t) {
        if (!warp_wait(tile_full(n & 1u), (n >> 1) & 1u, p.status, p.wait_ns)) return false;
        t = tile_slot[n & 1u];
        __syncwarp();
        if (lane == 0) mbar_arrive(tile_empty(n & 1u));
        return true;
    };

    if (warp == 0) {
        if (lane == 0) {
            auto fetch = [&](uint32_t n) {
                if (!mbar_wait_fast(tile_empty(n & 1u), ((n >> 1) & 1u) ^ 1u, p.status, kSiteAttn, p.wait_ns)) return -2;
                int t = atomicAdd(p.counter, 1);
                if (t >= n_tiles) t = -1;
                tile_slot[n & 1u] = t;
                mbar_arrive(tile_full(n & 1u));
                return t;
            };
            uint32_t nq = 0, nkf = 0, nvf = 0;  // Q / dO, K and V loads issued
            int t = fetch(0);
            for (uint32_t n = 0; t >= 0; ++n) {
                const DqTile tl = dq_tile(p, t);
                if (tl.nk > 0) {
                    // Q and dO once the previous tile's S and dP products are done
                    if (!mbar_wait_fast(q_empty, (nq & 1u) ^ 1u, p.status, kSiteAttn, p.wait_ns)) break;
                    mbar_arrive_expect_tx(q_full, 2 * kTile);
                    load_tile<D>(s_q, &map_qkv, q_full, tl.h * D, tl.q0);
                    load_tile<D>(s_do, &map_do, q_full, tl.h * D, tl.q0);
                    ++nq;
                }
                const int g = tl.h / group;
                const int kcol = (p.n_heads + g) * D, vcol = (p.n_heads + p.n_kv_heads + g) * D;
                int t_next = tl.nk > 0 ? -2 : fetch(n + 1);
                for (int j = 0; j < tl.nk; ++j) {
                    const uint32_t u = nkf;
                    if (!mbar_wait_fast(k_empty(u % NK), ((u / NK) & 1u) ^ 1u, p.status, kSiteAttn, p.wait_ns)) break;
                    mbar_arrive_expect_tx(k_full(u % NK), kTile);
                    load_tile<D>(s_k + (u % NK) * kTile, &map_qkv, k_full(u % NK), kcol, (tl.kb0 + j) * kRows);
                    ++nkf;
                    if (!mbar_wait_fast(v_empty(u % NV), ((u / NV) & 1u) ^ 1u, p.status, kSiteAttn, p.wait_ns)) break;
                    mbar_arrive_expect_tx(v_full(u % NV), kTile);
                    load_tile<D>(s_v + (u % NV) * kTile, &map_qkv, v_full(u % NV), vcol, (tl.kb0 + j) * kRows);
                    ++nvf;
                    // the next tile's number at this tile's last load, and its Q and dO into L2
                    if (j == tl.nk - 1) {
                        t_next = fetch(n + 1);
                        if (t_next >= 0) {
                            const DqTile nx = dq_tile(p, t_next);
                            prefetch_tile<D>(&map_qkv, nx.h * D, nx.q0);
                            prefetch_tile<D>(&map_do, nx.h * D, nx.q0);
                        }
                    }
                }
                t = t_next;  // -2 after a failed wait ends the loop
            }
            // no copy may land after the CTA has gone
            if (nq > 0) mbar_wait_fast(q_full, (nq - 1) & 1u, p.status, kSiteDrain, p.wait_ns);
            for (int s = 0; s < NK; ++s) {
                const uint32_t u = ring_uses(nkf, NK, s);
                if (u > 0) mbar_wait_fast(k_full(s), (u - 1) & 1u, p.status, kSiteDrain, p.wait_ns);
            }
            for (int s = 0; s < NV; ++s) {
                const uint32_t u = ring_uses(nvf, NV, s);
                if (u > 0) mbar_wait_fast(v_full(s), (u - 1) & 1u, p.status, kSiteDrain, p.wait_ns);
            }
        }
    } else if (warp == 1) {
        // ---------------- S and dP products
        const uint32_t leader = elect_one_sync();
        constexpr uint32_t idesc_s = mma_idesc_bf16(128, 128, false, false);
        const uint64_t q_desc = kdesc_base(s_q), do_desc = kdesc_base(s_do);
        auto issue_s = [&](uint32_t g) {
            const uint32_t st = g % NK;
            if (!warp_wait(k_full(st), (g / NK) & 1u, p.status, p.wait_ns)) return false;
            tc_fence_after();
            const uint64_t k_desc = kdesc_base(s_k + st * kTile);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                umma_bf16_elected(leader, t_s(g), kdesc_at(q_desc, kk), kdesc_at(k_desc, kk), idesc_s, kk > 0);
            umma_commit_elected(leader, s_full(g & 1u));
            return true;
        };
        auto issue_dp = [&](uint32_t g) {
            const uint32_t st = g % NV;
            if (!warp_wait(v_full(st), (g / NV) & 1u, p.status, p.wait_ns)) return false;
            tc_fence_after();
            const uint64_t v_desc = kdesc_base(s_v + st * kTile);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                umma_bf16_elected(leader, t_dp, kdesc_at(do_desc, kk), kdesc_at(v_desc, kk), idesc_s, kk > 0);
            umma_commit_elected(leader, dp_full);
            umma_commit_elected(leader, v_empty(st));
            return true;
        };
        // S[g] overwrites the S buffer of step g - 2 once the dQ warp has issued
        // dQ[g - 2], which reads dS[g - 2] from it; dP[g] overwrites dP[g - 1]
        // once the row warps are done with it.
        auto may_issue_s = [&](uint32_t g) {
            if (g < 2) return true;
            if (!warp_wait(dq_issued(g - 2), ((g - 2) >> 1) & 1u, p.status, p.wait_ns)) return false;
            tc_fence_after();
            return true;
        };
        auto may_issue_dp = [&](uint32_t g) {
            if (g < 1) return true;
            if (!warp_wait(ds_full(g - 1), ((g - 1) >> 1) & 1u, p.status, p.wait_ns)) return false;
            tc_fence_after();
            return true;
        };
        uint32_t g = 0, nq = 0;  // steps and tiles with steps so far
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            int t;
            if (!take_tile(n, t) || t < 0) break;
            const int nk = dq_tile(p, t).nk;
            if (nk == 0) continue;
            if (!warp_wait(q_full, nq & 1u, p.status, p.wait_ns)) break;
            ++nq;
            tc_fence_after();
            // the MMA order per step is S[g+1], dP[g+1] (here) beside dQ[g] (the dQ warp)
            for (int j = 0; j < nk; ++j, ++g) {
                if (!may_issue_s(g) || !issue_s(g) || !may_issue_dp(g) || !issue_dp(g)) {
                    ok = false;
                    break;
                }
                tc_fence_before();
                if (leader) mbar_arrive(dp_issued(g));
                // Q and dO are free for the next tile once its last S and dP are done
                if (j + 1 == nk) umma_commit_elected(leader, q_empty);
            }
        }
        umma_commit_elected(leader, drain);
        mbar_wait_fast(drain, 0, p.status, kSiteDrain, p.wait_ns);
    } else if (warp == kDqWarp) {
        // ---------------- dQ products
        const uint32_t leader = elect_one_sync();
        constexpr uint32_t idesc_q = mma_idesc_bf16(128, D, false, true);
        const int2 live = document_rows(p);
        uint32_t g = 0;
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            int t;
            if (!take_tile(n, t) || t < 0) break;
            const DqTile tl = dq_tile(p, t);
            const int nk = tl.nk;
            if (nk == 0) continue;
            for (int j = 0; j < nk; ++j, ++g) {
                const int k0 = (tl.kb0 + j) * kRows;
                if (has_padding(k0, live)) {  // K[g], once S[g] has read it
                    if (!warp_wait(s_full(g & 1u), (g >> 1) & 1u, p.status, p.wait_ns)) {
                        ok = false;
                        break;
                    }
                    zero_padding<D>(s_k + (g % NK) * kTile, k0, live, lane);
                }
                if (!warp_wait(ds_full(g), (g >> 1) & 1u, p.status, p.wait_ns) ||
                    (j + 1 < nk && !warp_wait(dp_issued(g + 1), ((g + 1) >> 1) & 1u, p.status, p.wait_ns))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t k_mn = mndesc_base(s_k + (g % NK) * kTile);
#pragma unroll
                for (int kk = 0; kk < kRows / 16; ++kk)
                    umma_bf16_ts_elected(leader, t_dq, t_s(g) + packed_col(kk), mndesc_at(k_mn, kk), idesc_q,
                                         (j > 0 || kk > 0) ? 1u : 0u);
                umma_commit_elected(leader, k_empty(g % NK));
                tc_fence_before();
                if (leader) mbar_arrive(dq_issued(g));
            }
            if (ok) umma_commit_elected(leader, done);
        }
        umma_commit_elected(leader, drain);
        mbar_wait_fast(drain, 0, p.status, kSiteDrain, p.wait_ns);
    } else {
        // ---------------- row warps: group gi takes key columns 64 gi .. 64 gi + 63 of every step
        const int gi = (warp - 2) >> 2;
        const int qw = warp & 3;
        const int row = qw * 32 + lane;
        const uint32_t t_row = (static_cast<uint32_t>(qw * 32) << 16) + 64u * gi;
        uint32_t g = 0, nd = 0;  // steps and tiles with steps so far
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            int t;
            if (!take_tile(n, t) || t < 0) break;
            const DqTile tl = dq_tile(p, t);
            const int q = tl.q0 + row;
            const bool valid = q < p.tokens;
            const int2 see = valid ? p.plan.rows[q] : make_int2(0, 0);
            const bool empty = see.y <= see.x;
            const float lse = empty ? 0.f : p.lse[static_cast<int64_t>(tl.h) * p.ld_stat + q];
            const float dv = empty ? 0.f : p.dvec[static_cast<int64_t>(tl.h) * p.ld_stat + q];
            const float slope2 = mode_biases(M) ? p.slopes[tl.h] * kLog2e : 0.f;
            for (int j = 0; j < tl.nk; ++j, ++g) {
                const int c0 = (tl.kb0 + j) * kRows + 64 * gi;
                if (!warp_wait(s_full(g & 1u), (g >> 1) & 1u, p.status, p.wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                float pr[64];  // P, times the cap's derivative
                {
                    uint32_t rs[64];
                    tmem_load_32(t_s(g) + t_row, *reinterpret_cast<uint32_t(*)[32]>(rs));
                    tmem_load_32(t_s(g) + t_row + 32, *reinterpret_cast<uint32_t(*)[32]>(rs + 32));
                    tmem_wait_load();
#pragma unroll
                    for (int i = 0; i < 64; ++i) pr[i] = __uint_as_float(rs[i]);
                }
                const float x = static_cast<float>(q - c0);
                if constexpr (M == kDocPlain) {
                    exp_scores<64>(pr, p.scale_log2, -lse);
                } else if constexpr (M == kDocBias) {
                    bias_scores<true, 64, true>(pr, p.scale_log2, slope2, x, -lse);
                } else {
                    float th[64];
                    cap_tanh<32>(p, pr);
                    cap_tanh<32>(p, pr + 32);
#pragma unroll
                    for (int i = 0; i < 64; ++i) th[i] = pr[i];
                    if constexpr (mode_biases(M))
                        bias_scores<true, 64, false>(pr, p.cap_log2, slope2, x, -lse);
                    else
                        exp_scores<64>(pr, p.cap_log2, -lse);
                    times_cap_slope<64>(pr, th);
                }
                if (!warp_wait(dp_full, g & 1u, p.status, p.wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t rp[64];
                tmem_load_32(t_dp + t_row, *reinterpret_cast<uint32_t(*)[32]>(rp));
                tmem_load_32(t_dp + t_row + 32, *reinterpret_cast<uint32_t(*)[32]>(rp + 32));
                tmem_wait_load();
                times_sum<64>(pr, rp, -dv);
                // hidden pairs last: their P or dP may be anything
                hide_columns<64>(pr, see.x - c0, see.y - c0, 0.f);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(pr[32 * c + 2 * e], pr[32 * c + 2 * e + 1]);
                    // packed columns 16 c .. 16 c + 15 of the group's S columns, all read above
                    tmem_store_16(t_s(g) + t_row + 16 * c, w);
                }
                tmem_wait_store();
                tc_fence_before();
                warp_arrive(ds_full(g), lane);
            }
            if (!ok) break;
            // group gi stores dQ columns [D/2 gi, D/2 (gi + 1)); the tile's next
            // dQ product waits for this group's next dS arrival, after these loads
            constexpr int kChunks = D / 64;  // 32-column chunks of this group's half
            const uint32_t stage = s_stage + kStageBytes * static_cast<uint32_t>(warp - 2);
            bool again = false;
            float r[kChunks][32] = {};
            if (tl.nk > 0) {
                if (!warp_wait(done, nd & 1u, p.status, p.wait_ns)) break;
                ++nd;
                tc_fence_after();
                const uint32_t t_q = t_dq + (static_cast<uint32_t>(qw * 32) << 16) + 32u * (gi * kChunks);
#pragma unroll
                for (int c = 0; c < kChunks; ++c) load_tmem32(t_q + 32 * c, r[c]);
                tc_fence_before();
#pragma unroll
                for (int c = 0; c < kChunks; ++c) again |= !finite32(r[c]);
            }
            stage_free(lane);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) stage32<D>(stage, lane, c, r[c], p.scale, empty);
            if (q - lane < p.tokens) store_stage(&map_dq, stage, lane, tl.h * D + gi * (D / 2), q - lane);
            uint32_t redo = __ballot_sync(0xffffffffu, again && valid && !empty);
            if (redo) stores_done(lane);
            while (redo) {
                const int src = __ffs(redo) - 1;
                redo &= redo - 1;
                document_dq_row<D>(p, q - lane + src, tl.h, lane, gi * (D / 2), (gi + 1) * (D / 2));
            }
        }
        stage_free(lane);  // shared memory outlives the stores that read it
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

// ------------------------------------------------------------------------ backward: dk, dv

// The causal core's dK / dV pipeline (attention.cu).  lse enters the score
// product as an extra K step where scores are linear in q . k; a cap applies to
// the product alone, so there the row warps read lse themselves (broadcast reads
// that the L1 serves).  A plain step takes 2900 cycles where its products take 2176:
// S^T, P^T, dV and the next S^T follow one another.
template <int D>
struct DocDkvSmem {
    static constexpr int kQStages = 2, kDoStages = 2, kStatStages = 2, kAugStages = 2;
    static constexpr uint32_t kTile = D * 256;
    static constexpr uint32_t kAugTile = 128 * 16 * 2;  // 128 rows x one K step of 16 bf16, no swizzle
    static constexpr uint32_t kK = 0, kV = kTile, kQ = 2 * kTile;
    static constexpr uint32_t kDO = kQ + kQStages * kTile;
    static constexpr uint32_t kOnes = kDO + kDoStages * kTile;  // two constant A operands: lse, D selectors
    static constexpr uint32_t kAug = kOnes + 2 * kAugTile;      // stage s: the B operand of step s
    static constexpr uint32_t kStat = kAug + kAugStages * kAugTile;  // stage s: lse (512 bytes) then D (512 bytes)
    static constexpr uint32_t kBars = kStat + 1024 * kStatStages;
    static constexpr int kNumBars = 1 + 2 * (kQStages + kStatStages) + kAugStages + 8;
    static constexpr size_t kUsed = kBars + 8 * kNumBars + 16;
};

template <int D>
constexpr size_t doc_bwd_smem() {
    return std::max({DocDqSmem<D>::kUsed, DocDkvSmem<D>::kUsed, kMinSmem});
}

template <int D, int M>
__device__ __forceinline__ void document_dkv(const CUtensorMap& map_qkv, const CUtensorMap& map_do, const CUtensorMap& map_out,
                                             const DocArgs& p, uint8_t* smem_raw) {
    using L = DocDkvSmem<D>;
    constexpr int NQ = L::kQStages, ND = L::kDoStages, NT = L::kStatStages, NA = L::kAugStages;
    constexpr uint32_t kTile = L::kTile;
    constexpr int kThreads = kAttnDqThreads, kStats = kDqWarp;  // warp 10: statistics
    const uint32_t base = smem_addr(smem_raw);
    const uint32_t s_k = base + L::kK, s_v = base + L::kV, s_q = base + L::kQ, s_do = base + L::kDO,
                   s_ones = base + L::kOnes, s_aug = base + L::kAug, s_stat = base + L::kStat;
    const uint32_t bars = base + L::kBars;
    const uint32_t kv_full = bars;
    auto q_full = [&](int s) { return bars + 8u * (1 + s); };
    // q_empty(s) releases Q, dO (same ring position, ND == NQ) and nothing else
    auto q_empty = [&](int s) { return bars + 8u * (1 + NQ + s); };
    auto st_full = [&](int s) { return bars + 8u * (1 + 2 * NQ + s); };
    auto st_empty = [&](int s) { return bars + 8u * (1 + 2 * NQ + NT + s); };
    auto aug_empty = [&](int s) { return bars + 8u * (1 + 2 * NQ + 2 * NT + s); };
    constexpr int kB = 1 + 2 * (NQ + NT) + NA;
    static_assert(NQ == ND, "Q and dO share their ring position and release");
    // p_full(c) / ds_full(c): chunk c (32 query columns of each group) of P^T / dS^T is packed
    auto p_full = [&](int c) { return bars + 8u * (kB + 2 + c); };
    auto ds_full = [&](int c) { return bars + 8u * (kB + 4 + c); };
    const uint32_t s_full = bars + 8u * kB, dp_full = bars + 8u * (kB + 1), done = bars + 8u * (kB + 6),
                   drain = bars + 8u * (kB + 7);
    const uint32_t tmem_slot = bars + 8u * L::kNumBars;
    volatile uint32_t* tmem_slot_ptr = reinterpret_cast<volatile uint32_t*>(smem_raw + (tmem_slot - base));

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = p.n_heads / p.n_kv_heads;
    const int kb = static_cast<int>(blockIdx.x) / p.n_kv_heads;  // in one long document, the most work first
    const int g = static_cast<int>(blockIdx.x) % p.n_kv_heads;
    const int k0 = kb * kRows;
    const int kcol = (p.n_heads + g) * D, vcol = (p.n_heads + p.n_kv_heads + g) * D;

    // The constant A operands of the statistics step (ones in bf16 columns 0-2
    // for lse, 8-10 for D) and zeros in the B operands' unused columns; the
    // statistics warp rewrites only columns 0-2 and 8-10 of a B operand.
    {
        uint4* z = reinterpret_cast<uint4*>(smem_raw + L::kOnes);
        constexpr int n16 = (2 + NA) * L::kAugTile / 16;
        for (int e = threadIdx.x; e < n16; e += kThreads) {
            const int tile = e / (L::kAugTile / 16);
            const int kc = (e >> 3) & 1;  // 16-byte rows: 8 rows per chunk, chunks alternate every 128 bytes
            const bool ones = tile < 2 && kc == tile;
            z[e] = ones ? make_uint4(0x3F803F80u, 0x3F80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
    }
    if (threadIdx.x == 0) {
        mbar_init(kv_full, 1);
        for (int s = 0; s < NQ; ++s) {
            mbar_init(q_full(s), 2);  // the Q and dO tiles' TMA and the statistics warp's B operand
            mbar_init(q_empty(s), 1);
        }
        for (int s = 0; s < NT; ++s) {
            mbar_init(st_full(s), 1);
            mbar_init(st_empty(s), 1);
        }
        for (int s = 0; s < NA; ++s) mbar_init(aug_empty(s), 1);
        mbar_init(s_full, 1);
        mbar_init(dp_full, 1);
        for (int c = 0; c < 2; ++c) {
            mbar_init(p_full(c), 8);
            mbar_init(ds_full(c), 8);
        }
        mbar_init(done, 1);
        mbar_init(drain, 1);
        mbar_fence_init();
        tma_prefetch_map(&map_qkv);
        tma_prefetch_map(&map_do);
    }
    if (warp == 1) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    wait_for_previous();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot_ptr;
    const int2 range = block_range(p.plan.k_blocks, kb, p.n_blocks);
    const int n_steps = group * (range.y - range.x);  // (query block, head of the group) pairs
    // columns: S^T 0-127 (P^T packed into 0-31 and 64-95 once read), dP^T
    // 128-255 (dS^T likewise), dV 256.., dK 256 + D..
    const uint32_t t_s = tmem_base, t_dp = tmem_base + 128, t_dv = tmem_base + 256, t_dk = tmem_base + 256 + D;

    if (n_steps == 0) {  // keys that nothing sees
        const int64_t width = static_cast<int64_t>(p.n_heads + 2 * p.n_kv_heads) * D;
        for (int e = threadIdx.x; e < kRows * D / 4; e += kThreads) {
            const int r = e / (D / 4), c = e % (D / 4);  // 16-byte pieces: D / 8 of dk, then D / 8 of dv
            if (k0 + r < p.tokens)
                *reinterpret_cast<uint4*>(p.out + (k0 + r) * width + (c < D / 8 ? kcol + 8 * c : vcol + 8 * (c - D / 8))) =
                    make_uint4(0u, 0u, 0u, 0u);
        }
    } else if (warp == 0) {
        if (lane == 0) {
            mbar_arrive_expect_tx(kv_full, 2 * kTile);
            load_tile<D>(s_k, &map_qkv, kv_full, kcol, k0);
            load_tile<D>(s_v, &map_qkv, kv_full, vcol, k0);
            uint32_t nq = 0, nt = 0;
            for (int i = 0; i < n_steps; ++i) {
                const int h = g * group + i % group;
                const int r0 = (range.x + i / group) * kRows;
                if (!mbar_wait_fast(st_empty(i % NT), ((i / NT) & 1) ^ 1u, p.status, kSiteAttn, p.wait_ns)) break;
                const uint32_t stat = s_stat + 1024u * (i % NT);
                mbar_arrive_expect_tx(st_full(i % NT), 1024);
                bulk_load_1d(stat, p.lse + static_cast<int64_t>(h) * p.ld_stat + r0, 512, st_full(i % NT));
                bulk_load_1d(stat + 512, p.dvec + static_cast<int64_t>(h) * p.ld_stat + r0, 512, st_full(i % NT));
                ++nt;
                // Q[i] and dO[i] land on one barrier (with the statistics operand); one
                // release covers both stages (dK[i - 2], after dV[i - 2], read the last of them)
                if (!mbar_wait_fast(q_empty(i % NQ), ((i / NQ) & 1) ^ 1u, p.status, kSiteAttn, p.wait_ns)) break;
                mbar_arrive_expect_tx(q_full(i % NQ), 2 * kTile);
                load_tile<D>(s_q + (i % NQ) * kTile, &map_qkv, q_full(i % NQ), h * D, r0);
                load_tile<D>(s_do + (i % ND) * kTile, &map_do, q_full(i % NQ), h * D, r0);
                ++nq;
            }
            mbar_wait_fast(kv_full, 0, p.status, kSiteDrain, p.wait_ns);
            for (int s = 0; s < NQ; ++s) {
                const uint32_t u = ring_uses(nq, NQ, s);
                if (u > 0) mbar_wait_fast(q_full(s), (u - 1) & 1, p.status, kSiteDrain, p.wait_ns);
            }
            for (int s = 0; s < NT; ++s) {
                const uint32_t u = ring_uses(nt, NT, s);
                if (u > 0) mbar_wait_fast(st_full(s), (u - 1) & 1, p.status, kSiteDrain, p.wait_ns);
            }
        }
    } else if (warp == 1) {
        // the whole warp runs the issue loop; its elected lane carries each instruction
        const uint32_t leader = elect_one_sync();
        constexpr uint32_t idesc_s = mma_idesc_bf16(128, 128, false, false);
        constexpr uint32_t idesc_g = mma_idesc_bf16(128, D, false, true);
        const uint64_t k_desc = kdesc_base(s_k), v_desc = kdesc_base(s_v);
        const uint64_t ones_lse = aug_desc(s_ones), ones_d = aug_desc(s_ones + L::kAugTile);
        auto issue_s = [&](int i) {
            const int st = i % NQ;
            // Q tile i and statistics operand i % NA (NA = NQ) complete one phase together
            if (!warp_wait(q_full(st), (i / NQ) & 1, p.status, p.wait_ns)) return false;
            tc_fence_after();
            const uint64_t q_desc = kdesc_base(s_q + st * kTile);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                umma_bf16_elected(leader, t_s, kdesc_at(k_desc, kk), kdesc_at(q_desc, kk), idesc_s, kk > 0);
            if constexpr (!mode_caps(M))
                umma_bf16_elected(leader, t_s, ones_lse, aug_desc(s_aug + (i % NA) * L::kAugTile), idesc_s, 1u);
            umma_commit_elected(leader, s_full);
            return true;
        };
        auto issue_dp = [&](int i) {  // after issue_s(i), which waited for dO[i] and the statistics too
            const int st = i % ND;
            const uint64_t do_desc = kdesc_base(s_do + st * kTile);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                umma_bf16_elected(leader, t_dp, kdesc_at(v_desc, kk), kdesc_at(do_desc, kk), idesc_s, kk > 0);
            umma_bf16_elected(leader, t_dp, ones_d, aug_desc(s_aug + (i % NA) * L::kAugTile), idesc_s, 1u);
            umma_commit_elected(leader, dp_full);
            umma_commit_elected(leader, aug_empty(i % NA));
            return true;
        };
        bool ok = warp_wait(kv_full, 0, p.status, p.wait_ns) && issue_s(0) && issue_dp(0);
        // K steps of dV / dK in the order their P^T / dS^T chunks are packed:
        // chunk c of group g holds the K steps 4 g + 2 c and 4 g + 2 c + 1
        constexpr int kOrder[8] = {0, 1, 4, 5, 2, 3, 6, 7};
        // steps before pad_end and from pad_start on have padding among their queries
        const int2 live = document_rows(p);
        const int pad_end = has_padding(range.x * kRows, live) ? group : 0;
        const int pad_start = n_steps - (has_padding((range.y - 1) * kRows, live) ? group : 0);
        for (int i = 0; ok && i < n_steps; ++i) {
            if (i < pad_end || i >= pad_start) {  // Q[i] and dO[i], once S[i] and dP[i] have read them
                if (!warp_wait(s_full, i & 1, p.status, p.wait_ns) || !warp_wait(dp_full, i & 1, p.status, p.wait_ns)) break;
                zero_padding<D>(s_q + (i % NQ) * kTile, (range.x + i / group) * kRows, live, lane, s_do - s_q);
            }
            const uint64_t do_mn = mndesc_base(s_do + (i % ND) * kTile);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (!warp_wait(p_full(c), i & 1, p.status, p.wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int kk = kOrder[4 * c + e];
                    umma_bf16_ts_elected(leader, t_dv, t_s + packed_col(kk), mndesc_at(do_mn, kk), idesc_g,
                                         (i > 0 || kk > 0) ? 1u : 0u);
                }
            }
            if (!ok) break;
            // S^T[i+1] overwrites the S^T buffer after dV[i] has read P^T[i] from it
            if (i + 1 < n_steps && !issue_s(i + 1)) break;
            const uint64_t q_mn = mndesc_base(s_q + (i % NQ) * kTile);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (!warp_wait(ds_full(c), i & 1, p.status, p.wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int kk = kOrder[4 * c + e];
                    umma_bf16_ts_elected(leader, t_dk, t_dp + packed_col(kk), mndesc_at(q_mn, kk), idesc_g,
                                         (i > 0 || kk > 0) ? 1u : 0u);
                }
            }
            if (!ok) break;
            // Q[i] and dO[i]: dK[i] is the last product that reads either
            umma_commit_elected(leader, q_empty(i % NQ));
            if (i + 1 < n_steps && !issue_dp(i + 1)) break;
        }
        umma_commit_elected(leader, done);
        umma_commit_elected(leader, drain);
        mbar_wait_fast(drain, 0, p.status, kSiteDrain, p.wait_ns);
    } else if (warp == kStats) {
        // ---------------- statistics warp: step i's lse and D into B operand i % NA
        const float inv_c = 1.f / p.scale_log2;
        for (int i = 0; i < n_steps; ++i) {
            if (!warp_wait(st_full(i % NT), (i / NT) & 1, p.status, p.wait_ns) ||
                !warp_wait(aug_empty(i % NA), ((i / NA) & 1) ^ 1u, p.status, p.wait_ns))
                break;
            const float* stat = reinterpret_cast<const float*>(smem_raw + L::kStat + 1024u * (i % NT));
            uint8_t* aug = smem_raw + L::kAug + (i % NA) * L::kAugTile;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int r = lane + 32 * u;
                // statistics of rows that see nothing, or behind the last row, reach
                // hidden columns only, whatever they hold
                if constexpr (!mode_caps(M))
                    *reinterpret_cast<uint2*>(aug + aug_offset(r, 0)) = split3_bf16(-stat[r] * inv_c);
                *reinterpret_cast<uint2*>(aug + aug_offset(r, 1)) = split3_bf16(-stat[128 + r]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(q_full(i % NQ));
                mbar_arrive(st_empty(i % NT));
            }
        }
    } else {
        // ---------------- two groups of four warps, one key row per thread in each:
        // group gi takes query columns 64 gi .. 64 gi + 63 of every step
        const int gi = (warp - 2) >> 2;
        const int qw = warp & 3;
        const int row = qw * 32 + lane;
        const int k = k0 + row;
        const bool valid = k < p.tokens;
        const int2 see = valid ? p.plan.cols[k] : make_int2(0, 0);
        const bool empty = see.y <= see.x;
        const uint32_t t_row = (static_cast<uint32_t>(qw * 32) << 16) + 64u * gi;
        bool ok = true;
        for (int i = 0; i < n_steps; ++i) {
            const int qc0 = (range.x + i / group) * kRows + 64 * gi;  // query of this group's first column
            const int h = g * group + i % group;
            const float slope2 = mode_biases(M) ? p.slopes[h] * kLog2e : 0.f;
            const float x = static_cast<float>(k - qc0);  // the column at distance 0
            const int lo = see.x - qc0, hi = see.y - qc0;  // this key's queries
            if (!warp_wait(s_full, i & 1, p.status, p.wait_ns)) {
                ok = false;
                break;
            }
            tc_fence_after();
            float pr[64];  // P; after the first pass, times the cap's derivative
            {
                uint32_t rs[64];
                tmem_load_32(t_s + t_row, *reinterpret_cast<uint32_t(*)[32]>(rs));
                tmem_load_32(t_s + t_row + 32, *reinterpret_cast<uint32_t(*)[32]>(rs + 32));
                tmem_wait_load();
#pragma unroll
                for (int j = 0; j < 64; ++j) pr[j] = __uint_as_float(rs[j]);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float th[32];
                if constexpr (M == kDocPlain) {
                    exp_scores<32>(pr + 32 * c, p.scale_log2, 0.f);
                } else if constexpr (M == kDocBias) {
                    bias_scores<true, 32, true>(pr + 32 * c, p.scale_log2, slope2, x - 32 * c, 0.f);
                } else {
                    const float4* lse4 = reinterpret_cast<const float4*>(p.lse + static_cast<int64_t>(h) * p.ld_stat + qc0 + 32 * c);
                    cap_tanh<32>(p, pr + 32 * c);
#pragma unroll
                    for (int j = 0; j < 32; ++j) th[j] = pr[32 * c + j];
                    if constexpr (mode_biases(M)) bias_scores<false, 32, false>(pr + 32 * c, p.cap_log2, slope2, x - 32 * c, 0.f);
                    const float cap2 = mode_biases(M) ? 1.f : p.cap_log2;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float4 v = lse4[e];
                        float* s = pr + 32 * c + 4 * e;
                        split_pair(fma_pair(pair_of(s[0], s[1]), pair_of(cap2, cap2), pair_of(-v.x, -v.y)), s[0], s[1]);
                        split_pair(fma_pair(pair_of(s[2], s[3]), pair_of(cap2, cap2), pair_of(-v.z, -v.w)), s[2], s[3]);
#pragma unroll
                        for (int u = 0; u < 4; ++u) s[u] = ex2(s[u]);
                    }
                }
                hide_columns<32>(pr + 32 * c, lo - 32 * c, hi - 32 * c, 0.f);
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(pr[32 * c + 2 * e], pr[32 * c + 2 * e + 1]);
                // packed columns 16 c .. 16 c + 15 of the group's columns, all read above
                tmem_store_16(t_s + t_row + 16 * c, w);
                if constexpr (mode_caps(M)) times_cap_slope<32>(pr + 32 * c, th);
                tmem_wait_store();
                tc_fence_before();
                warp_arrive(p_full(c), lane);
            }
            if (!warp_wait(dp_full, i & 1, p.status, p.wait_ns)) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t rp[64];
            tmem_load_32(t_dp + t_row, *reinterpret_cast<uint32_t(*)[32]>(rp));
            tmem_load_32(t_dp + t_row + 32, *reinterpret_cast<uint32_t(*)[32]>(rp + 32));
            tmem_wait_load();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float* ds = pr + 32 * c;
                times_sum<32>(ds, rp + 32 * c, 0.f);
                hide_columns<32>(ds, lo - 32 * c, hi - 32 * c, 0.f);  // a hidden column's dP may be anything
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(ds[2 * e], ds[2 * e + 1]);
                tmem_store_16(t_dp + t_row + 16 * c, w);
                tmem_wait_store();
                tc_fence_before();
                warp_arrive(ds_full(c), lane);
            }
        }
        // group 0 stores dK, group 1 dV
        if (ok && warp_wait(done, 0, p.status, p.wait_ns)) {
            tc_fence_after();
            const uint32_t t_acc = (gi == 0 ? t_dk : t_dv) + (static_cast<uint32_t>(qw * 32) << 16);
            const float sc = gi == 0 ? p.scale : 1.f;
            // every product has been formed: the Q stages serve the results, D / 64 boxes a warp
            const uint32_t stage = s_q + kStageBytes * static_cast<uint32_t>((warp - 2) * (D / 64));
            bool again = false;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                float r[2][32];
                load_tmem32(t_acc + 64 * c, r[0]);
                load_tmem32(t_acc + 64 * c + 32, r[1]);
                again |= !finite32(r[0]) || !finite32(r[1]);
                stage32(stage + c * kStageBytes, lane, 0, r[0], sc, empty);
                stage32(stage + c * kStageBytes, lane, 1, r[1], sc, empty);
                if (k - lane < p.tokens) store_stage(&map_out, stage + c * kStageBytes, lane, (gi == 0 ? kcol : vcol) + 64 * c, k - lane);
            }
            uint32_t redo = __ballot_sync(0xffffffffu, again && valid && !empty);
            if (redo) stores_done(lane);
            while (redo) {
                const int src = __ffs(redo) - 1;
                redo &= redo - 1;
                document_dkv_row<D>(p, k - lane + src, g, lane, gi == 1);
            }
            stage_free(lane);  // shared memory outlives the stores that read it
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

// One launch for both halves of the backward: the first n_blocks * n_kv_heads
// CTAs form dK and dV, the rest, one per SM at most, take dQ tiles as SMs come
// free.  (The causal core runs them on two streams, which costs a small call a
// fork and a join, and makes one stream and counter the whole device's.)
// 32 heads of 128 on 8, 4096 tokens: 9 documents in 98 us (tensor pipe 58 % busy), 4
// with prefixes and a cap in 243.  Sixteen row warps of half the columns took 123 and
// 262 with the row sums, against 118 and 269 then: kept at eight for the plain form.
template <int D, int M>
__global__ void __launch_bounds__(kAttnDqThreads, 1)
    document_bwd_kernel(const __grid_constant__ CUtensorMap map_qkv, const __grid_constant__ CUtensorMap map_do,
                        const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_dq,
                        const __grid_constant__ DocArgs p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    if (smem_addr(smem_raw) & 1023u) {  // the tiles' 128-byte swizzle needs a 1 KiB-aligned start
        if (threadIdx.x == 0) atomicCAS(p.status, 0, kSiteAttn);
        return;
    }
    if (static_cast<int>(blockIdx.x) < p.n_blocks * p.n_kv_heads)
        document_dkv<D, M>(map_qkv, map_do, map_out, p, smem_raw);
    else
        document_dq<D, M>(map_qkv, map_do, map_dq, p, smem_raw);
}

DocArgs doc_args(const DocShape& s, const void* qkv, const void* plan, const float* slopes, float cap) {
    DocArgs p{};
    p.qkv = static_cast<const uint16_t*>(qkv);
    p.plan = doc_plan(plan, s.tokens);
    p.slopes = slopes;
    p.cap = cap;
    p.scale = 1.f / sqrtf(static_cast<float>(s.head_dim));
    p.scale_log2 = kLog2e * p.scale;
    p.cap_log2 = cap * kLog2e;
    const float cap_rate = cap > 0.f ? p.scale / cap : 0.f;
    p.cap_limit = cap > 0.f ? 0.75f / cap_rate : 0.f;
    p.cap_exp = 2.f * kLog2e * cap_rate;
    const double tanh_poly[5] = {0.999999434947, -0.333282515696, 0.132589833556, -0.0500563036011, 0.0129296314219};
    double power = cap_rate;  // cap_rate^(2 k + 1)
    for (int k = 0; k < 5; ++k, power *= static_cast<double>(cap_rate) * cap_rate)
        p.cap_poly[k] = static_cast<float>(tanh_poly[k] * power);
    p.tokens = s.tokens;
    p.n_heads = s.n_heads;
    p.n_kv_heads = s.n_kv_heads;
    p.ld_stat = s.ld_stat;
    p.n_blocks = static_cast<int>(doc_blocks(s.tokens));
    p.status = status_word();
    // a warp may be forming 32 rows over, one by one, while others wait for it
    p.wait_ns = kWaitLimitNs + static_cast<uint64_t>(s.tokens) * 32u * kRowPairNs;
    return p;
}

DocMode mode_of(const DocArgs& p) {
    return p.cap > 0.f ? (p.slopes ? kDocCapBias : kDocCap) : (p.slopes ? kDocBias : kDocPlain);
}

// A kernel whose warpgroups trade registers must have been launched with as many as
// they claim in all, or the last claim would wait for ever.
template <typename K>
cudaError_t prepare_kernel(K kern, size_t smem, int regs) {
    cudaFuncAttributes attr;
    const cudaError_t e = cudaFuncGetAttributes(&attr, kern);
    if (e != cudaSuccess) return e;
    return attr.numRegs >= regs ? set_smem(kern, smem) : cudaErrorInvalidConfiguration;
}

template <int D, int M>
cudaError_t forward(const DocArgs& p, cudaStream_t stream) {
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    std::call_once(once, [] { err = prepare_kernel(document_fwd_kernel<D, M>, DocFwdSmem<D>::kBytes, kDocFwdRegs); });
    if (err != cudaSuccess) return err;
    const int width = (p.n_heads + 2 * p.n_kv_heads) * D;
    CUtensorMap map, out;
    if (!attn_map(&map, p.qkv, p.tokens, width, width) || !attn_map(&out, p.out, p.tokens, p.n_heads * D, p.n_heads * D, 32))
        return cudaErrorInvalidValue;
    const int64_t tiles = static_cast<int64_t>(fwd_tiles(p));
    return launch_chained(document_fwd_kernel<D, M>, static_cast<unsigned>(tiles), kDocFwdThreads, DocFwdSmem<D>::kBytes, stream, map,
                          out, p);
}

template <int D, int M>
cudaError_t backward(const DocArgs& p, const uint16_t* a, float* dvec, bool d_ready, cudaStream_t stream) {
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    std::call_once(once, [] { err = set_smem(document_bwd_kernel<D, M>, doc_bwd_smem<D>()); });
    if (err != cudaSuccess) return err;
    const int width = (p.n_heads + 2 * p.n_kv_heads) * D;
    CUtensorMap mq, md, mo, mdq;  // dq leaves in boxes of half a head
    if (!attn_map(&mq, p.qkv, p.tokens, width, width) || !attn_map(&md, p.da, p.tokens, p.n_heads * D, p.n_heads * D) ||
        !attn_map(&mo, p.out, p.tokens, width, width, 32) || !attn_map(&mdq, p.out, p.tokens, width, width, 32, D / 2))
        return cudaErrorInvalidValue;
    if (d_ready) {
        const cudaError_t e = cudaMemsetAsync(p.counter, 0, sizeof(int), stream);
        if (e != cudaSuccess) return e;
    } else {
        const int64_t warps = (static_cast<int64_t>(p.tokens) * p.n_heads + 7) / 8;  // 8 rows per warp
        const cudaError_t e = launch_chained(attn_causal_rowsum_kernel<D>, static_cast<unsigned>((warps + 7) / 8), 256, 0, stream, p.da, a,
                                             dvec, p.tokens, p.n_heads, p.ld_stat, p.counter);
        if (e != cudaSuccess) return e;
    }
    const int64_t dkv = static_cast<int64_t>(p.n_blocks) * p.n_kv_heads;
    const int64_t dq = std::min<int64_t>(static_cast<int64_t>(p.n_blocks) * p.n_heads, sm_count());
    return launch_chained(document_bwd_kernel<D, M>, static_cast<unsigned>(dkv + dq), kAttnDqThreads, doc_bwd_smem<D>(), stream, mq, md,
                          mo, mdq, p);
}

template <int D>
cudaError_t forward_mode(const DocArgs& p, cudaStream_t stream) {
    switch (mode_of(p)) {
        case kDocPlain: return forward<D, kDocPlain>(p, stream);
        case kDocBias: return forward<D, kDocBias>(p, stream);
        case kDocCap: return forward<D, kDocCap>(p, stream);
        default: return forward<D, kDocCapBias>(p, stream);
    }
}

template <int D>
cudaError_t backward_mode(const DocArgs& p, const uint16_t* a, float* dvec, bool d_ready, cudaStream_t stream) {
    switch (mode_of(p)) {
        case kDocPlain: return backward<D, kDocPlain>(p, a, dvec, d_ready, stream);
        case kDocBias: return backward<D, kDocBias>(p, a, dvec, d_ready, stream);
        case kDocCap: return backward<D, kDocCap>(p, a, dvec, d_ready, stream);
        default: return backward<D, kDocCapBias>(p, a, dvec, d_ready, stream);
    }
}

}  // namespace

cudaError_t launch_document_plan(const int32_t* offsets, const int32_t* prefix, int n_docs, int tokens, void* plan,
                                 int32_t* positions, cudaStream_t stream) {
    if (tokens <= 0) return cudaSuccess;
    const DocPlan p = doc_plan(plan, tokens);
    return launch_chained(document_plan_kernel, static_cast<unsigned>(doc_blocks(tokens)), kDocBlock, 0, stream, offsets, prefix, n_docs,
                          tokens, const_cast<int2*>(p.rows), const_cast<int2*>(p.cols), const_cast<int2*>(p.q_blocks),
                          const_cast<int2*>(p.k_blocks), positions);
}

cudaError_t launch_document_forward(const DocShape& s, const void* qkv, void* a, float* lse, const void* plan,
                                    const float* slopes, float cap, cudaStream_t stream) {
    if (s.tokens <= 0) return cudaSuccess;
    DocArgs p = doc_args(s, qkv, plan, slopes, cap);
    if (!p.status) return cudaErrorInvalidDevice;
    p.out = static_cast<uint16_t*>(a);
    p.lse_out = lse;
    return s.head_dim == 128 ? forward_mode<128>(p, stream) : forward_mode<64>(p, stream);
}

cudaError_t launch_document_backward(const DocShape& s, const void* qkv, const void* a, const void* da, const float* lse,
                                     void* dqkv, const void* plan, const float* slopes, float cap, void* scratch,
                                     cudaStream_t stream, bool d_ready) {
    if (s.tokens <= 0) return cudaSuccess;
    DocArgs p = doc_args(s, qkv, plan, slopes, cap);
    if (!p.status) return cudaErrorInvalidDevice;
    float* dvec = static_cast<float*>(scratch);
    p.da = static_cast<const uint16_t*>(da);
    p.out = static_cast<uint16_t*>(dqkv);
    p.lse = lse;
    p.dvec = dvec;
    p.counter = reinterpret_cast<int*>(dvec + static_cast<int64_t>(s.n_heads) * s.ld_stat);
    const uint16_t* av = static_cast<const uint16_t*>(a);
    return s.head_dim == 128 ? backward_mode<128>(p, av, dvec, d_ready, stream)
                             : backward_mode<64>(p, av, dvec, d_ready, stream);
}

namespace {

bool word_ok(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

zb_status document_ok(int32_t tokens, int32_t nh, int32_t nkv, int32_t hd, const void* plan, const float* slopes, float cap) {
    if (!tokens_ok(tokens) || !heads_ok(nh, nkv, hd) || (hd != 64 && hd != 128)) return ZB_ERR_SHAPE;
    if (!rows_ok(plan, tokens) || !word_ok(slopes) || !cap_ok(cap)) return ZB_ERR_ARG;
    return ZB_OK;
}

DocShape shape_of(int32_t tokens, int32_t nh, int32_t nkv, int32_t hd) { return {tokens, nh, nkv, hd, stat_stride(tokens)}; }

}  // namespace

}  // namespace zbk

using namespace zbk;

extern "C" size_t zb_op_attention_document_plan_bytes(int32_t tokens) { return tokens_ok(tokens) ? doc_plan_bytes(tokens) : 0; }

extern "C" zb_status zb_op_attention_document_plan(const int32_t* doc_offsets, const int32_t* prefix_len, int32_t n_docs,
                                                   int32_t tokens, void* plan, size_t plan_bytes, int32_t* positions,
                                                   void* stream) {
    if (!tokens_ok(tokens)) return ZB_ERR_SHAPE;
    if (n_docs < 1 || n_docs > kMaxDocuments || (!doc_offsets && n_docs != 1) || !word_ok(doc_offsets) || !word_ok(prefix_len) || !word_ok(positions))
        return ZB_ERR_ARG;
    if (tokens > 0 && (!plan || !aligned16(plan) || plan_bytes < doc_plan_bytes(tokens))) return ZB_ERR_WORKSPACE;
    ZB_TRY(device_ok());
    return cuda_status(launch_document_plan(doc_offsets, prefix_len, n_docs, tokens, plan, positions, as_stream(stream)));
}

extern "C" size_t zb_op_attention_document_scratch_bytes(int32_t tokens, int32_t n_heads) {
    return tokens_ok(tokens) && n_heads > 0 && n_heads <= kMaxFeature ? document_scratch_bytes(n_heads, stat_stride(tokens)) : 0;
}

extern "C" zb_status zb_op_attention_document_forward(const void* qkv, void* a, float* lse, const void* plan,
                                                      const float* slopes, float cap, int32_t tokens, int32_t n_heads,
                                                      int32_t n_kv_heads, int32_t head_dim, void* stream) {
    ZB_TRY(document_ok(tokens, n_heads, n_kv_heads, head_dim, plan, slopes, cap));
    if (!rows_ok(qkv, tokens) || !rows_ok(a, tokens) || !rows_ok(lse, tokens)) return ZB_ERR_ARG;
    ZB_TRY(device_ok());
    return cuda_status(launch_document_forward(shape_of(tokens, n_heads, n_kv_heads, head_dim), qkv, a, lse, plan, slopes, cap,
                                               as_stream(stream)));
}

extern "C" zb_status zb_op_attention_document_backward(const void* qkv, const void* a, const void* da, const float* lse,
                                                       void* dqkv, const void* plan, const float* slopes, float cap,
                                                       int32_t tokens, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                                       void* scratch, size_t scratch_bytes, void* stream) {
    ZB_TRY(document_ok(tokens, n_heads, n_kv_heads, head_dim, plan, slopes, cap));
    const void* rows[] = {qkv, a, da, lse, dqkv};
    for (const void* p : rows)
        if (!rows_ok(p, tokens)) return ZB_ERR_ARG;
    const DocShape s = shape_of(tokens, n_heads, n_kv_heads, head_dim);
    if (tokens > 0 && (!scratch || !aligned16(scratch) || scratch_bytes < document_scratch_bytes(n_heads, s.ld_stat)))
        return ZB_ERR_WORKSPACE;
    ZB_TRY(device_ok());
    return cuda_status(launch_document_backward(s, qkv, a, da, lse, dqkv, plan, slopes, cap, scratch, as_stream(stream)));
}
