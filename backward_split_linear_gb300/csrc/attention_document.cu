// Softmax attention inside packed documents: the plan of a batch, and the
// kernels row by row.
//
// Score of query i and key j of one document, h the head:
//   s = q_i . k_j / sqrt(d);  s = cap tanh(s / cap) with a cap;  s -= slope_h |i - j|.
// Key j is visible to query i when both are in the same document and j <= i or
// j is among the document's first `prefix` rows.
#include "checks.h"
#include "attention_document.h"

namespace zbk {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------------ plan

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

// One block per 128 rows, one row per thread.  Offsets are data: whatever they
// hold, every interval written lies inside [0, tokens].
__global__ void __launch_bounds__(kDocBlock) document_plan_kernel(const int32_t* offsets, const int32_t* prefix, int n_docs,
                                                                  int tokens, int2* rows, int2* cols, int2* q_blocks,
                                                                  int2* k_blocks, int32_t* positions) {
    __shared__ int red[4][4];
    const int i = blockIdx.x * kDocBlock + threadIdx.x;
    int s = 0, e = 0, pre = 0;
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
            if (lo < n_docs) {
                s = clampi(offsets[lo], 0, tokens);
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
    const int2 row = in ? make_int2(s, max(i + 1, pend)) : make_int2(0, 0);
    const int2 col = in ? make_int2(i < pend ? s : i, e) : make_int2(0, 0);
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

// ------------------------------------------------------------------------ row by row

struct DocArgs {
    const uint16_t* qkv;
    const uint16_t* a;
    const uint16_t* da;
    uint16_t* out;
    const float* lse;
    float* lse_out;
    const float* dvec;
    DocPlan plan;
    const float* slopes;
    float cap, scale;
    int tokens, n_heads, n_kv_heads, ld_stat;
};

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
__device__ __forceinline__ void store_row(uint16_t* p, int lane, const float (&v)[D / 32], float f) {
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
        *reinterpret_cast<uint32_t*>(p + 64 * c + 2 * lane) = pack_bf16x2(v[2 * c] * f, v[2 * c + 1] * f);
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

// One warp per query row and head.
template <int D>
__global__ void __launch_bounds__(128) document_forward_rows(const DocArgs p) {
    const int lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int i = static_cast<int>(w / p.n_heads), h = static_cast<int>(w % p.n_heads);
    if (i >= p.tokens) return;
    const int64_t width = static_cast<int64_t>(p.n_heads + 2 * p.n_kv_heads) * D;
    const int g = h / (p.n_heads / p.n_kv_heads);
    const uint16_t* k = p.qkv + (p.n_heads + g) * D;
    const uint16_t* v = p.qkv + (p.n_heads + p.n_kv_heads + g) * D;
    const float slope = p.slopes ? p.slopes[h] : 0.f;
    float q[D / 32], acc[D / 32] = {};
    load_row<D>(p.qkv + i * width + h * D, lane, q);
    const int2 see = p.plan.rows[i];
    float m = -INFINITY, l = 0.f;
    for (int j = see.x; j < see.y; ++j) {
        float x[D / 32], unused;
        load_row<D>(k + j * width, lane, x);
        const float s = score2(p, dot_rows(q, x), slope, abs(i - j), unused);
        const float top = fmaxf(m, s), f = m == -INFINITY ? 0.f : exp2f(m - top), e = exp2f(s - top);
        m = top;
        l = l * f + e;
        load_row<D>(v + j * width, lane, x);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) acc[c] = acc[c] * f + e * x[c];
    }
    store_row<D>(p.out + (static_cast<int64_t>(i) * p.n_heads + h) * D, lane, acc, see.y > see.x ? 1.f / l : 0.f);
    if (lane == 0) p.lse_out[static_cast<int64_t>(h) * p.ld_stat + i] = see.y > see.x ? m + log2f(l) : -INFINITY;
}

// D = rowsum(da * a) of one row and head per warp.
template <int D>
__global__ void __launch_bounds__(128) document_rowsum(const DocArgs p, float* dvec) {
    const int lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (w >= static_cast<int64_t>(p.tokens) * p.n_heads) return;
    float x[D / 32], y[D / 32];
    load_row<D>(p.da + w * D, lane, x);
    load_row<D>(p.a + w * D, lane, y);
    const float s = dot_rows(x, y);
    if (lane == 0) dvec[(w % p.n_heads) * p.ld_stat + w / p.n_heads] = s;
}

// dq: one warp per query row and head.
template <int D>
__global__ void __launch_bounds__(128) document_dq_rows(const DocArgs p) {
    const int lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int i = static_cast<int>(w / p.n_heads), h = static_cast<int>(w % p.n_heads);
    if (i >= p.tokens) return;
    const int64_t width = static_cast<int64_t>(p.n_heads + 2 * p.n_kv_heads) * D;
    const int g = h / (p.n_heads / p.n_kv_heads);
    const uint16_t* k = p.qkv + (p.n_heads + g) * D;
    const uint16_t* v = p.qkv + (p.n_heads + p.n_kv_heads + g) * D;
    const float slope = p.slopes ? p.slopes[h] : 0.f;
    float q[D / 32], dy[D / 32], acc[D / 32] = {};
    load_row<D>(p.qkv + i * width + h * D, lane, q);
    load_row<D>(p.da + (static_cast<int64_t>(i) * p.n_heads + h) * D, lane, dy);
    const float lse = p.lse[static_cast<int64_t>(h) * p.ld_stat + i], dsum = p.dvec[static_cast<int64_t>(h) * p.ld_stat + i];
    const int2 see = p.plan.rows[i];
    for (int j = see.x; j < see.y; ++j) {
        float x[D / 32], y[D / 32], f;
        load_row<D>(k + j * width, lane, x);
        load_row<D>(v + j * width, lane, y);
        const float e = exp2f(score2(p, dot_rows(q, x), slope, abs(i - j), f) - lse);
        const float ds = e * (dot_rows(dy, y) - dsum) * f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) acc[c] += ds * x[c];
    }
    store_row<D>(p.out + i * width + h * D, lane, acc, p.scale);
}

// dk and dv: one warp per key row and kv head.
template <int D>
__global__ void __launch_bounds__(128) document_dkv_rows(const DocArgs p) {
    const int lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int j = static_cast<int>(w / p.n_kv_heads), g = static_cast<int>(w % p.n_kv_heads);
    if (j >= p.tokens) return;
    const int64_t width = static_cast<int64_t>(p.n_heads + 2 * p.n_kv_heads) * D;
    const int group = p.n_heads / p.n_kv_heads;
    const int64_t kcol = (p.n_heads + g) * D, vcol = (p.n_heads + p.n_kv_heads + g) * D;
    float k[D / 32], v[D / 32], dk[D / 32] = {}, dv[D / 32] = {};
    load_row<D>(p.qkv + j * width + kcol, lane, k);
    load_row<D>(p.qkv + j * width + vcol, lane, v);
    const int2 see = p.plan.cols[j];
    for (int h = g * group; h < (g + 1) * group; ++h) {
        const float slope = p.slopes ? p.slopes[h] : 0.f;
        for (int i = see.x; i < see.y; ++i) {
            float x[D / 32], y[D / 32], f;
            load_row<D>(p.qkv + i * width + h * D, lane, x);
            load_row<D>(p.da + (static_cast<int64_t>(i) * p.n_heads + h) * D, lane, y);
            const float lse = p.lse[static_cast<int64_t>(h) * p.ld_stat + i], dsum = p.dvec[static_cast<int64_t>(h) * p.ld_stat + i];
            const float e = exp2f(score2(p, dot_rows(k, x), slope, abs(i - j), f) - lse);
            const float ds = e * (dot_rows(v, y) - dsum) * f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                dv[c] += e * y[c];
                dk[c] += ds * x[c];
            }
        }
    }
    store_row<D>(p.out + j * width + kcol, lane, dk, p.scale);
    store_row<D>(p.out + j * width + vcol, lane, dv, 1.f);
}

unsigned warps4(int64_t n) { return static_cast<unsigned>((n + 3) / 4); }

DocArgs doc_args(const DocShape& s, const void* qkv, const void* plan, const float* slopes, float cap) {
    DocArgs p{};
    p.qkv = static_cast<const uint16_t*>(qkv);
    p.plan = doc_plan(plan, s.tokens);
    p.slopes = slopes;
    p.cap = cap;
    p.scale = 1.f / sqrtf(static_cast<float>(s.head_dim));
    p.tokens = s.tokens;
    p.n_heads = s.n_heads;
    p.n_kv_heads = s.n_kv_heads;
    p.ld_stat = s.ld_stat;
    return p;
}

template <int D>
cudaError_t forward(const DocArgs& p, cudaStream_t stream) {
    document_forward_rows<D><<<warps4(static_cast<int64_t>(p.tokens) * p.n_heads), 128, 0, stream>>>(p);
    return cudaGetLastError();
}

template <int D>
cudaError_t backward(DocArgs p, float* dvec, bool d_ready, cudaStream_t stream) {
    const unsigned rows = warps4(static_cast<int64_t>(p.tokens) * p.n_heads);
    p.dvec = dvec;
    if (!d_ready) document_rowsum<D><<<rows, 128, 0, stream>>>(p, dvec);
    document_dkv_rows<D><<<warps4(static_cast<int64_t>(p.tokens) * p.n_kv_heads), 128, 0, stream>>>(p);
    document_dq_rows<D><<<rows, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_document_plan(const int32_t* offsets, const int32_t* prefix, int n_docs, int tokens, void* plan,
                                 int32_t* positions, cudaStream_t stream) {
    if (tokens <= 0) return cudaSuccess;
    const DocPlan p = doc_plan(plan, tokens);
    document_plan_kernel<<<static_cast<unsigned>(doc_blocks(tokens)), kDocBlock, 0, stream>>>(
        offsets, prefix, n_docs, tokens, const_cast<int2*>(p.rows), const_cast<int2*>(p.cols), const_cast<int2*>(p.q_blocks),
        const_cast<int2*>(p.k_blocks), positions);
    return cudaGetLastError();
}

cudaError_t launch_document_forward(const DocShape& s, const void* qkv, void* a, float* lse, const void* plan,
                                    const float* slopes, float cap, cudaStream_t stream) {
    if (s.tokens <= 0) return cudaSuccess;
    DocArgs p = doc_args(s, qkv, plan, slopes, cap);
    p.out = static_cast<uint16_t*>(a);
    p.lse_out = lse;
    return s.head_dim == 128 ? forward<128>(p, stream) : forward<64>(p, stream);
}

cudaError_t launch_document_backward(const DocShape& s, const void* qkv, const void* a, const void* da, const float* lse,
                                     void* dqkv, const void* plan, const float* slopes, float cap, void* scratch,
                                     cudaStream_t stream, bool d_ready) {
    if (s.tokens <= 0) return cudaSuccess;
    DocArgs p = doc_args(s, qkv, plan, slopes, cap);
    p.a = static_cast<const uint16_t*>(a);
    p.da = static_cast<const uint16_t*>(da);
    p.out = static_cast<uint16_t*>(dqkv);
    p.lse = lse;
    float* dvec = static_cast<float*>(scratch);
    return s.head_dim == 128 ? backward<128>(p, dvec, d_ready, stream) : backward<64>(p, dvec, d_ready, stream);
}

namespace {

bool word_ok(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

zb_status document_ok(int32_t tokens, int32_t nh, int32_t nkv, int32_t hd, const void* plan, const float* slopes, float cap) {
    if (!tokens_ok(tokens) || !heads_ok(nh, nkv, hd) || (hd != 64 && hd != 128)) return ZB_ERR_SHAPE;
    if (!rows_ok(plan, tokens) || !word_ok(slopes) || !(cap >= 0.f && cap <= 1e30f)) return ZB_ERR_ARG;
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
    if (n_docs < 1 || (!doc_offsets && n_docs != 1) || !word_ok(doc_offsets) || !word_ok(prefix_len) || !word_ok(positions))
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
