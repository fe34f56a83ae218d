// Storage types of the sequence-layer kernels: loads to and rounding from
// float32, and adjacent elements in one access.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace pn {

using bf16 = __bf16;
using f16 = _Float16;

template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
    T v[N];
};

// The workgroup's number in a launch of grid_of(); below 2^32.
__device__ __forceinline__ uint32_t block_id() { return blockIdx.y * gridDim.x + blockIdx.x; }

// Round to nearest even; NaN stays NaN.
template <typename T>
__device__ __forceinline__ T from_f32(float x) { return static_cast<T>(x); }
template <typename T>
__device__ __forceinline__ float to_f32(T x) { return static_cast<float>(x); }

}  // namespace pn
