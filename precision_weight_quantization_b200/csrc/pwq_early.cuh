// pwq_early.cuh -- programmatic dependent launch: kernels that are set up while
// the kernel ahead of them on the stream still runs (the products and the
// norms), and the loads that such kernels use.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace pwq {

// Launches `kernel` so that it may start while the kernel before it on the
// stream still runs (programmatic dependent launch); the kernel itself calls
// wait_for_earlier_kernels() before it touches global memory, so stream order
// is kept.  cluster > 1: thread-block clusters of that many CTAs.
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream,
                         unsigned cluster, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// The device side.  Every kernel launched that way calls both: kernels behind
// it on the stream may then be set up on SMs that it leaves, and none reads or
// writes memory before the kernels ahead of it have ended.
__device__ __forceinline__ void let_later_kernels_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_earlier_kernels() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Loads of such kernels.  griddepcontrol.wait makes the earlier kernels' writes
// visible to ordinary loads; the non-coherent path (ld.global.nc, __ldg) is
// defined only for memory that nothing writes during the kernel's lifetime,
// which here begins before those writes (and an in-place output is written by
// the kernel itself).  _once: not kept in L1.
__device__ __forceinline__ uint4 ld_v4(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ float ld_f32(const float* p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

}  // namespace pwq
