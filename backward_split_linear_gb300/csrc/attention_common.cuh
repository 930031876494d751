// What the attention kernels share: operand descriptors, waits, the packing of
// P and dS, the statistics operand, the row kernel that forms D and the tensor
// maps.  Everything is local to the translation unit that includes it.
#pragma once

#include <cudaTypedefs.h>

#include <mutex>

#include "chained.cuh"
#include "device_common.cuh"

namespace zbk {

namespace {

constexpr int kAttnThreads = 192;
// The backward kernels run two groups of four row warps (warps 2-5 and 6-9),
// each on every other sub-block.
constexpr int kAttnBwdThreads = 320;
// The dQ kernel adds a warp that issues the dQ products (warp 10).
constexpr int kAttnDqThreads = kAttnBwdThreads + 32;
constexpr int kDqWarp = kAttnBwdThreads / 32;
constexpr int kRows = 128;             // query and key block
// Every attention CTA allocates all 512 tensor-memory columns; asking for at
// least this much shared memory keeps two CTAs off one SM (the second would
// wait in its allocation until the first ends).
constexpr size_t kMinSmem = 120 * 1024;

// K-major operand from a tile whose rows are the M (or N) index and whose
// columns are the contraction: step kk covers columns 16 kk .. 16 kk + 15.
// The descriptor of step kk is the tile's descriptor plus the step's byte
// offset / 16 in its start-address field, so callers build the base once.
__device__ __forceinline__ uint64_t kdesc_base(uint32_t tile) { return smem_desc_sw128(tile, 16, 1024); }
__device__ __forceinline__ uint64_t kdesc_at(uint64_t base, int kk) {
    return base + static_cast<uint64_t>(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
}

// MN-major operand from the same kind of tile: the contraction runs over its
// 128 rows (step kk = rows 16 kk .. +15), the MN index over its columns.
__device__ __forceinline__ uint64_t mndesc_base(uint32_t tile) { return smem_desc_sw128(tile, 16384, 1024); }
__device__ __forceinline__ uint64_t mndesc_at(uint64_t base, int kk) {
    return base + static_cast<uint64_t>((kk * 2048) >> 4);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// v where `visible`, else +0.0: a bit mask, not a branch.  A select written as a
// short-circuit condition per element compiled to a branch per element, and
// branch resolution then dominated the elementwise passes.
__device__ __forceinline__ float keep_if(float v, bool visible) {
    return __uint_as_float(__float_as_uint(v) & (0u - static_cast<uint32_t>(visible)));
}

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A wait taken by every lane of a warp, with one verdict for the warp (the
// tensor-memory loads that follow are warp-wide).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int* status, uint64_t limit_ns = kWaitLimitNs) {
    const bool ok = mbar_wait_fast(bar, parity, status, kSiteAttn, limit_ns);
    return __all_sync(0xffffffffu, ok);
}

// One arrival for the whole warp, after every lane's prior work: each lane has
// waited for its tensor-memory stores and fenced them before this call.  One
// arrival per warp instead of one per thread keeps 256 shared-memory atomics
// on one barrier off the path between the row warps and the MMA thread.
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// Loads one 128-row tile (d / 64 boxes) of columns col .. col + d - 1 at row r0.
template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar, int col, int r0) {
#pragma unroll
    for (int b = 0; b < D / 64; ++b) tma_load_2d(dst + b * 16384u, map, bar, col + 64 * b, r0);
}
// The same boxes into L2 only.
template <int D>
__device__ __forceinline__ void prefetch_tile(const CUtensorMap* map, int col, int r0) {
#pragma unroll
    for (int b = 0; b < D / 64; ++b) tma_prefetch_l2_2d(map, col + 64 * b, r0);
}

// Tensor-memory column of the packed bf16 operand of K step kk (16 rows of the
// contraction) when the two groups of row warps each pack their 64 columns of
// a 128-column buffer into its first 32: group kk / 4 at 64 (kk / 4), then 8
// columns per K step.
__device__ __forceinline__ uint32_t packed_col(int kk) { return static_cast<uint32_t>(64 * (kk >> 2) + 8 * (kk & 3)); }

// Byte offset of row r, K chunk kc (8 bf16) of a no-swizzle K-major operand of
// one K step: 8-row groups 256 bytes apart (the stride-dimension offset), the
// two 8-column chunks of a row group 128 bytes apart (the leading-dimension
// offset), rows of a chunk 16 bytes apart.
__device__ __forceinline__ uint32_t aug_offset(int r, int kc) {
    return static_cast<uint32_t>((r >> 3) * 256 + kc * 128 + (r & 7) * 16);
}
__device__ __forceinline__ uint64_t aug_desc(uint32_t tile) {
    return static_cast<uint64_t>((tile & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 16) |
           (static_cast<uint64_t>(256 >> 4) << 32) | (1ull << 46);  // swizzle mode 0: none
}

// v as hi + mid + lo, each bf16 (round to nearest), as the low 48 bits of a
// 64-bit word (bf16 columns 0, 1, 2; column 3 zero).
__device__ __forceinline__ uint2 split3_bf16(float v) {
    const __nv_bfloat16 hi = __float2bfloat16_rn(v);
    const float r1 = v - __bfloat162float(hi);
    const __nv_bfloat16 mid = __float2bfloat16_rn(r1);
    const __nv_bfloat16 lo = __float2bfloat16_rn(r1 - __bfloat162float(mid));
    return make_uint2(static_cast<uint32_t>(__bfloat16_as_ushort(hi)) | (static_cast<uint32_t>(__bfloat16_as_ushort(mid)) << 16),
                      static_cast<uint32_t>(__bfloat16_as_ushort(lo)));
}

// ------------------------------------------------------------------------ D = rowsum(dO * O)

// dvec[h][t] = sum_c da[t, h d + c] * a[t, h d + c].  Row r = t n_heads + h of
// da and a starts at element r d (rows are contiguous); d / 8 lanes read one
// row in 16-byte pieces (pointers and d keep them 16-byte aligned), so every
// load instruction covers 512 contiguous bytes of each tensor, and a warp
// takes 8 consecutive rows.  All of a warp's loads are issued before the first
// sum: with a reduction between one pair of rows and the next, the kernel ran
// at about 0.6 of the HBM bandwidth.
template <int D>
__global__ void attn_causal_rowsum_kernel(const uint16_t* __restrict__ da, const uint16_t* __restrict__ a, float* dvec,
                                          int tokens, int n_heads, int ld_stat, int* counter = nullptr) {
    // the tile counter of the kernel that follows on the stream, if it has one
    wait_for_previous();
    if (counter && blockIdx.x == 0 && threadIdx.x == 0) *counter = 0;
    constexpr int kLanesPerRow = D / 8;
    constexpr int kRowsPerPass = 32 / kLanesPerRow;
    constexpr int kRowsPerWarp = 8;
    constexpr int kPasses = kRowsPerWarp / kRowsPerPass;
    const int64_t warp_id = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31, sub = lane / kLanesPerRow, pl = lane % kLanesPerRow;
    const int64_t n_rows = static_cast<int64_t>(tokens) * n_heads;
    uint4 u[kPasses], v[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int64_t r = warp_id * kRowsPerWarp + i * kRowsPerPass + sub;
        u[i] = make_uint4(0u, 0u, 0u, 0u);
        v[i] = u[i];
        if (r < n_rows) {
            u[i] = *reinterpret_cast<const uint4*>(da + r * D + 8 * pl);
            v[i] = *reinterpret_cast<const uint4*>(a + r * D + 8 * pl);
        }
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        float acc = bf16_lo(u[i].x) * bf16_lo(v[i].x) + bf16_hi(u[i].x) * bf16_hi(v[i].x) +
                    bf16_lo(u[i].y) * bf16_lo(v[i].y) + bf16_hi(u[i].y) * bf16_hi(v[i].y) +
                    bf16_lo(u[i].z) * bf16_lo(v[i].z) + bf16_hi(u[i].z) * bf16_hi(v[i].z) +
                    bf16_lo(u[i].w) * bf16_lo(v[i].w) + bf16_hi(u[i].w) * bf16_hi(v[i].w);
#pragma unroll
        for (int o = kLanesPerRow / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);  // within a row's lanes
        const int64_t r = warp_id * kRowsPerWarp + i * kRowsPerPass + sub;
        if (pl == 0 && r < n_rows) {
            const int t = static_cast<int>(r / n_heads), h = static_cast<int>(r % n_heads);
            dvec[static_cast<int64_t>(h) * ld_stat + t] = acc;
        }
    }
}

// ------------------------------------------------------------------------ host side

PFN_cuTensorMapEncodeTiled_v12000 attn_encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// [rows, cols] bf16, row stride ld elements; boxes of 64 columns x 128 rows, 128B swizzle
// (or box_rows rows, and box_cols = 32 columns with 64B swizzle).
bool attn_map(CUtensorMap* map, const void* ptr, int64_t rows, int64_t cols, int64_t ld, uint32_t box_rows = 128,
              uint32_t box_cols = 64) {
    auto fn = attn_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, box_cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename K>
cudaError_t set_smem(K kern, size_t bytes) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

}  // namespace

}  // namespace zbk
