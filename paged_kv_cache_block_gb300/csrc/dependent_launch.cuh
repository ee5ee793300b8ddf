// Launches as programmatic dependents of the kernel before in the stream: the launch is prepared, and the
// CTAs set themselves up, while that kernel still runs.  Such a kernel calls previous_kernel_done() in
// every thread before it reads or writes anything that an earlier kernel may have written or read; it
// returns when all of that kernel has completed.  After anything but a kernel it is a plain launch.
// Nor does it load through the read-only path (__ldg, ld.global.nc), which takes the data for unchanged from
// the kernel's launch on, when the kernel before may still be writing it.
#pragma once

#include <cuda_runtime.h>

namespace pkv {

__device__ __forceinline__ void previous_kernel_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel may be launched once every CTA has come here (or ended).
__device__ __forceinline__ void let_next_kernel_launch() { asm volatile("griddepcontrol.launch_dependents;"); }

template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                             const Args &...args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace pkv
