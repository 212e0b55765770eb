// api_util.cuh -- host-side checks shared by the C entry points.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.cuh"
#include "swiglu.h"

namespace swiglu {

constexpr int64_t kMaxDim = (1LL << 31) - 1;  // TMA coordinates are 32-bit

// Current device's properties; returns a status code.
int current_device(DeviceInfo &out);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool overlaps(const void *a, int64_t abytes, const void *b, int64_t bbytes) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + static_cast<uintptr_t>(bbytes) && b0 < a0 + static_cast<uintptr_t>(abytes);
}

inline int elem_size(int dtype) { return dtype == SWIGLU_BF16 ? 2 : 4; }

inline int from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return SWIGLU_OK;
    (void)cudaGetLastError();
    return SWIGLU_ERR_CUDA;
}

}  // namespace swiglu
