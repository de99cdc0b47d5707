// Launches of one call that follow one another: a kernel's blocks take the SMs that the launch before leaves, and set
// themselves up, while that launch's last blocks still run.  A stream otherwise starts a kernel about 2.5 us after the
// last block of the one before (a graph: about 1 us).
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace sdv2 {

// What the launch before wrote may be read, and what it reads written, behind this.  Every launch of a chain waits in
// every block that has something to wait for and in one at least, so that the chain's end is the end of all of it.
__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The launch that follows may start once all blocks have come here (or are done).
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A&&... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace sdv2
