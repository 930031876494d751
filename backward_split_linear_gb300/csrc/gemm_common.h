// What the tcgen05 GEMM kernels share on the host: tensor maps and the tile order.
#pragma once

#include <cstdint>
#include <cuda.h>

namespace zbk {

// Row-major matrix of `rows` x `cols` with row stride `ld` elements (bf16, float32 or bytes), in
// boxes of box_cols x box_rows; zero fill out of range on loads, no writes there on stores.
bool gemm_encode_map(CUtensorMap* map, const void* ptr, int64_t rows, int64_t cols, int64_t ld, uint32_t box_cols,
                     uint32_t box_rows, CUtensorMapSwizzle swizzle, CUtensorMapDataType dtype);

// Tiles per group of the grouped tile order of a launch whose waves hold `grid` tiles;
// *group_m: groups of tile rows (else of tile columns).
int gemm_raster(int tiles_m, int tiles_n, int bm, int bn, int k, int grid, bool* group_m);

}  // namespace zbk
