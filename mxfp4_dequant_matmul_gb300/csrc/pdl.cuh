// pdl.cuh -- launches that start while the previous kernel of the stream still runs.
//
// A kernel launched by launch_after() may have its CTAs placed, and run up to pdl_wait(),
// before the kernel ahead of it has finished; pdl_wait() returns when that kernel has
// completed and its writes are visible, so a kernel that touches no global memory before it
// (kernel parameters aside) behaves as if launched normally.  pdl_trigger() lets the next
// launch do the same: it takes effect when every CTA of this grid has called it or ended.
//
// Such a kernel reads global memory by ld_dep(), plain loads that pdl_wait() orders behind
// the kernel ahead.  Not by ld.global.nc (__ldg, or what the compiler may make of a const
// __restrict__ pointer): that form is defined only for memory that nobody writes while the
// kernel lives, and here it lives, waiting, while the kernel ahead writes what it will read.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace mxk {

__device__ __forceinline__ void pdl_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void pdl_trigger() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Loads of what a kernel ahead may have written, after pdl_wait().
__device__ __forceinline__ uint16_t ld_dep(const uint16_t* p) {
    uint16_t v;
    asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ld_dep(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ int32_t ld_dep(const int32_t* p) {
    return static_cast<int32_t>(ld_dep(reinterpret_cast<const uint32_t*>(p)));
}
__device__ __forceinline__ float ld_dep(const float* p) {
    return __uint_as_float(ld_dep(reinterpret_cast<const uint32_t*>(p)));
}
__device__ __forceinline__ uint2 ld_dep(const uint2* p) {
    uint2 v;
    asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint4 ld_dep(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ float4 ld_dep(const float4* p) {
    const uint4 v = ld_dep(reinterpret_cast<const uint4*>(p));
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                       __uint_as_float(v.w));
}
// Data that is read once does not stay in L1.
__device__ __forceinline__ uint4 ld_dep_stream(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ void ld_dep_stream32(const void* p, uint32_t (&v)[8]) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                   "=r"(v[6]), "=r"(v[7])
                 : "l"(p));
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
