// What the document attention kernels share: the plan of a packed batch, the
// scores' modifications, and the row-by-row forms.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace zbk {

// The visibility of a packed batch of T rows, as intervals.  Row i sees the keys
// [rows[i].x, rows[i].y); key j is seen by the queries [cols[j].x, cols[j].y).
// Both are intervals: a document is one, and a prefix key is seen by all of it.
// Per 128-row block: the key blocks [q_blocks.x, q_blocks.y) that any of its
// rows sees, the query blocks [k_blocks.x, k_blocks.y) that see any of its keys.
// Every array covers whole blocks; rows behind T are empty.  So are padding's, as (x, x)
// with x where the documents start (rows before them) or end.
struct DocPlan {
    const int2* rows;
    const int2* cols;
    const int2* q_blocks;
    const int2* k_blocks;
};

constexpr int kDocBlock = 128;
constexpr int kMaxDocuments = 1 << 28;  // the search for a row's document adds two of their numbers

__host__ __device__ inline int64_t doc_blocks(int64_t tokens) { return (tokens + kDocBlock - 1) / kDocBlock; }
inline size_t doc_plan_bytes(int64_t tokens) { return static_cast<size_t>(doc_blocks(tokens)) * (2 * kDocBlock + 2) * sizeof(int2); }
inline DocPlan doc_plan(const void* plan, int64_t tokens) {
    const int64_t nb = doc_blocks(tokens);
    DocPlan p;
    p.rows = static_cast<const int2*>(plan);
    p.cols = p.rows + nb * kDocBlock;
    p.q_blocks = p.cols + nb * kDocBlock;
    p.k_blocks = p.q_blocks + nb;
    return p;
}

// The caps that the kernels take: none, or a size at which its polynomial's
// coefficients, odd powers of 1 / (cap sqrt(d)) up to the ninth, are normal float32
// numbers: at 512 and d = 128 the last is 1.8e-36, at 1e-3 and d = 64 it is 1e17.
inline bool cap_ok(float cap) { return cap == 0.f || (cap >= 1e-3f && cap <= 512.f); }

struct DocShape {
    int tokens, n_heads, n_kv_heads, head_dim, ld_stat;
};

cudaError_t launch_document_plan(const int32_t* offsets, const int32_t* prefix, int n_docs, int tokens, void* plan,
                                 int32_t* positions, cudaStream_t stream);
cudaError_t launch_document_forward(const DocShape& s, const void* qkv, void* a, float* lse, const void* plan,
                                    const float* slopes, float cap, cudaStream_t stream);
// scratch: D = rowsum(da * a), [n_heads][ld_stat], then one tile counter.  With
// d_ready the caller has written D (but not the counter).
cudaError_t launch_document_backward(const DocShape& s, const void* qkv, const void* a, const void* da, const float* lse,
                                     void* dqkv, const void* plan, const float* slopes, float cap, void* scratch,
                                     cudaStream_t stream, bool d_ready = false);
inline size_t document_scratch_bytes(int n_heads, int ld_stat) { return (static_cast<size_t>(n_heads) * ld_stat + 64) * sizeof(float); }

}  // namespace zbk
