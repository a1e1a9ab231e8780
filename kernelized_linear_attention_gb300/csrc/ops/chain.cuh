// Kernels of one call that are launched before the one ahead of them has ended (programmatic dependent launch), so that
// nothing waits for a launch: 40009 x 8 x 64 packed 129 us, 136 without; 1025 x 3 x 37 x 53 22 and 27.  The first one is
// launched like any other; every later one has chain_wait() as its first step, in all of its threads, before anything is
// read, written or allocated (tensor memory that a waiting block held could be what a block of the kernel ahead still
// needs), so that the end of the last kernel is the end of all.  (Product passes of the gradients that wait for one
// another at their ends only, side by side, were slower by a twenty-fifth for 8 x 4096 x 8 x 64.)
#pragma once

#include <cuda_runtime.h>

namespace la {

__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel's blocks start as soon as all of this one's have.
__device__ __forceinline__ void chain_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

struct Chain {
    cudaStream_t stream;
    bool after = false;          // the call's last launch was a kernel of the chain
};

template <typename... Params, typename... Args>
cudaError_t launch_in(Chain& chain, void (*kernel)(Params...), dim3 grid, dim3 threads, size_t smem, Args&&... args) {
    if (!chain.after) {
        chain.after = true;
        kernel<<<grid, threads, smem, chain.stream>>>(Params(args)...);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cfg.gridDim = grid;
    cfg.blockDim = threads;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = chain.stream;
    return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

}  // namespace la
