// Launches that follow one another in a stream, those of one call and of two: a kernel's blocks take the SMs that the
// launch before leaves, and set themselves up, while that launch's last blocks still run or its end is on the way.  A
// stream otherwise starts a kernel about 2.5 us after the last block of the one before (a graph: about 1 us).  Every
// kernel of these operators is launched so and waits before it touches memory (inside cross attention's backward pass:
// memory that the call's own launches write); calls in a row measured, unchained and
// chained, in a stream: cross attention 480p 23.4 and 21.3 us, 720p 60.1 and 57.6, layer norm of 4680 x 5120 35.1 and
// 32.4.  A launch that lets the next one start before its own blocks are done (launch_dependents) is faster inside the
// backward passes, in 4-bit quantisation of rows, in the 4-bit products and in the rotations, where comments say so, and no
// faster or slower elsewhere (cross attention of the ragged batch: 42.8 us without, 46.0 with).
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace sdv2 {

// What the launch before wrote may be read, and what it reads written, behind this.  Every launch of a chain waits in
// every block that has something to wait for and in one at least, so that the chain's end is the end of all of it.
__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The launch that follows may start once all blocks have come here (or are done).
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

inline cudaLaunchAttribute chained_attribute()
{
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    return attr;
}

template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A&&... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr = chained_attribute();
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace sdv2
