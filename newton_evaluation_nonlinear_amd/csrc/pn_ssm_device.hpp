// Functions of the state-space kernels.
#pragma once

#include "pn_seq_device.hpp"

namespace pn {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Keeps a value's computation where it stands: before a select, not in a branch made of it.
__device__ __forceinline__ float pinned(float v) {
    asm("" : "+v"(v));
    return v;
}

// v if on, otherwise 0, by a select and not a branch around what v takes.
__device__ __forceinline__ float kept(bool on, float v) {
    v = pinned(v);
    return on ? v : 0.0f;
}

// log(1 + e^v) = max(v, 0) + log(1 + t), t = e^-|v|; log(1 + t) as log(w) +
// (t - (w - 1)) / w, w = 1 + t as rounded, which leaves 2^-48 of its rounding.
__device__ __forceinline__ float softplus(float v, float* slope) {
    const float t = __builtin_amdgcn_exp2f(-fabsf(v) * kLog2e), w = 1.0f + t, r = __builtin_amdgcn_rcpf(w);
    *slope = (v >= 0.0f ? 1.0f : t) * r;
    return fmaxf(v, 0.0f) + fmaf(__builtin_amdgcn_logf(w), kLn2, (t - (w - 1.0f)) * r);
}
// e^-v past float32 is infinite and its reciprocal 0: v logistic(v) is -0 for v far below 0.
__device__ __forceinline__ float logistic(float v) { return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kLog2e)); }

}  // namespace
}  // namespace pn
