// vn_act.cuh -- the activations of the linear layer and their derivatives, in fp32.
#pragma once

#include <cuda_runtime.h>

#include "vn.h"

namespace vn {

template <int kAct>
__device__ __forceinline__ float activate(float z) {
  if constexpr (kAct == VN_ACT_TANH) return tanhf(z);
  if constexpr (kAct == VN_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
  if constexpr (kAct == VN_ACT_GELU) return z * normcdff(z);
  if constexpr (kAct == VN_ACT_SILU) return z / (1.f + expf(-z));
  return z;
}

template <int kAct>
__device__ __forceinline__ float slope(float z) {
  if constexpr (kAct == VN_ACT_TANH) {
    const float t = tanhf(z);
    return fmaf(-t, t, 1.f);
  }
  if constexpr (kAct == VN_ACT_RELU) return z > 0.f ? 1.f : (z != z ? z : 0.f);
  if constexpr (kAct == VN_ACT_GELU)
    return fmaf(z * 0.3989422804014327f, expf(-0.5f * z * z), normcdff(z));
  if constexpr (kAct == VN_ACT_SILU) {
    const float t = 1.f / (1.f + expf(-z));
    return t * fmaf(z, 1.f - t, 1.f);
  }
  return 1.f;
}

// The same with the activation chosen at run time (uniform over the launch).
__device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    case VN_ACT_TANH: return activate<VN_ACT_TANH>(z);
    case VN_ACT_RELU: return activate<VN_ACT_RELU>(z);
    case VN_ACT_GELU: return activate<VN_ACT_GELU>(z);
    case VN_ACT_SILU: return activate<VN_ACT_SILU>(z);
    default: return z;
  }
}
__device__ __forceinline__ float slope(int act, float z) {
  switch (act) {
    case VN_ACT_TANH: return slope<VN_ACT_TANH>(z);
    case VN_ACT_RELU: return slope<VN_ACT_RELU>(z);
    case VN_ACT_GELU: return slope<VN_ACT_GELU>(z);
    case VN_ACT_SILU: return slope<VN_ACT_SILU>(z);
    default: return 1.f;
  }
}

}  // namespace vn
