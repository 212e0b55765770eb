// pdl.cuh -- programmatic dependent launch: a kernel whose blocks may start,
// and set themselves up, while the one before it on the stream still runs.
// Nothing is read or written before griddep_wait(), which returns once every
// earlier kernel has completed and its writes are visible; every block calls
// it.  griddep_launch_dependents() lets the next such kernel start.
// What such a kernel reads may have been written by a kernel that still ran
// when it started.  Its loads are therefore plain ones (ld_plain(),
// ld_stream_v4(), bulk and TMA copies), never __ldg, ld.global.nc or a
// `const __restrict__` parameter: the read-only path is defined only for
// memory that nothing writes while the kernel runs, and the compiler need not
// keep such a load behind griddep_wait().
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace swiglu {

__device__ __forceinline__ void griddep_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void griddep_launch_dependents() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Loads that stay behind griddep_wait(): volatile, as it is.

__device__ __forceinline__ uint4 ld_plain(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ float4 ld_plain(const float4 *p) {
    float4 v;
    asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ld_plain(const uint2 *p) {
    uint2 v;
    asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ float ld_plain(const float *p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

// (B200: 2.3 us of the host per launch, against 2.7 of a plain one.)
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, dim3 block, uint32_t smem, cudaStream_t stream,
                             const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace swiglu
