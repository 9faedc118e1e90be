// dependent.cuh -- launches of one call whose starts overlap the end of the kernel before (programmatic
// dependent launch): the launch latency and a kernel's set-up then cost nothing.
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"

namespace prism {

// A kernel lets the next one of the call start once it has itself seen its predecessor complete, so whatever a
// kernel reads before dependent_wait() is older than the call.  Every block of every kernel of a chain executes
// it: a kernel's end then implies the end of all before.
__device__ __forceinline__ void dependent_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launches `kern` so that its start may overlap the end of the call's previous kernel (`dependent`).
template <typename... P, typename... A>
cudaError_t dependent_launch(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, bool dependent, const A &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = dependent ? 1 : 0;
    launch_probe_mark(s);
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, args...);
    if (err != cudaSuccess) cudaGetLastError();  // reported here, not by the caller's next check
    return err;
}

}  // namespace prism
