// Host-side launchers of the training operators beside the stage's own steps
// (internal to libzb): rotary positions.  As in launch.h, every launcher
// enqueues on `stream`; arguments are checked in the C-ABI layer.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace zbk {

// Rows of n_heads heads of head_dim bf16 elements, ld elements apart; y may be
// x.  sign is +1 (forward) or -1 (backward).
cudaError_t launch_rotary(const void* x, int64_t ld_x, void* y, int64_t ld_y, const int32_t* positions,
                          const uint64_t* turns, float magnitude, int tokens, int n_heads, int head_dim, int rotary_dim,
                          bool half, float sign, cudaStream_t stream);

}  // namespace zbk
