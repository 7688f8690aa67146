// pdl.cuh -- launches that start while the previous kernel of the stream still runs.
//
// A kernel launched by launch_after() may have its CTAs placed, and run up to pdl_wait(),
// before the kernel ahead of it has finished; pdl_wait() returns when that kernel has
// completed and its writes are visible, so a kernel that touches no global memory before it
// (kernel parameters aside) behaves as if launched normally.  pdl_trigger() lets the next
// launch do the same: it takes effect when every CTA of this grid has called it or ended.
#pragma once

#include <cuda_runtime.h>

namespace mxk {

__device__ __forceinline__ void pdl_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void pdl_trigger() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem,
                         cudaStream_t s, unsigned cluster, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mxk
