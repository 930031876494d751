// Launches whose blocks start while the last blocks of the stream's previous kernel
// end, so that a short kernel's setup hides behind the one before it.
#pragma once

#include <cuda_runtime.h>
#include <utility>

namespace zbk {

// Returns once the kernels before this one on its stream have ended and their writes
// are visible.  Every block of a kernel launched by `launch_chained` calls it before
// its first access to global memory (the status word aside, which is only ever set), on
// every path: a later kernel takes this one's end for the end of those before it.
// Elsewhere it returns at once.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream, A&&... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace zbk
