// vn_act.cuh -- the activations of the linear layer and their derivatives.
//
// Two forms of each: with CUDA's full-precision functions, for results in fp32, and one good to
// 2^-14 (1 + |z|) and better, for results that are rounded to bf16 (2^-8): a quotient and an
// exponential on the special-function unit and a few multiply-adds, a third of the
// instructions, so that an epilogue over a whole tile stays shorter than the tile's products.
#pragma once

#include <cuda_runtime.h>

#include "vn.h"

namespace vn {

__device__ __forceinline__ float quick_reciprocal(float x) { return __fdividef(1.f, x); }

// tanh: 1 - 2 / (1 + e^2z), and its Taylor series where that difference would cancel
// (to z^9 62/2835: below 1e-6 of the value at 1/4).
__device__ __forceinline__ float quick_tanh(float z) {
  const float s = z * z;
  const float series = z * fmaf(s, fmaf(s, fmaf(s, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
  const float quotient = 1.f - 2.f * quick_reciprocal(1.f + __expf(2.f * z));
  return fabsf(z) < 0.25f ? series : quotient;
}
// The normal distribution function and e^(-z^2/2): Abramowitz and Stegun 7.1.26,
// erfc(x) = (a1 t + .. + a5 t^5) e^(-x^2), t = 1 / (1 + p x), off by at most 1.5e-7.
__device__ __forceinline__ float quick_cdf(float z, float* e) {
  const float x = fabsf(z) * 0.70710678118654752f;
  const float t = quick_reciprocal(fmaf(0.3275911f, x, 1.f));
  const float poly =
      t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f), 0.254829592f);
  *e = __expf(-0.5f * z * z);
  const float tail = 0.5f * poly * *e;
  return z >= 0.f ? 1.f - tail : tail;
}

template <int kAct, bool kQuick>
__device__ __forceinline__ float activate(float z) {
  if constexpr (kAct == VN_ACT_TANH) return kQuick ? quick_tanh(z) : tanhf(z);
  if constexpr (kAct == VN_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
  if constexpr (kAct == VN_ACT_GELU) {
    float e;
    return z * (kQuick ? quick_cdf(z, &e) : normcdff(z));
  }
  if constexpr (kAct == VN_ACT_SILU) return kQuick ? z * quick_reciprocal(1.f + __expf(-z)) : z / (1.f + expf(-z));
  return z;
}

template <int kAct, bool kQuick>
__device__ __forceinline__ float slope(float z) {
  if constexpr (kAct == VN_ACT_TANH) {
    const float t = kQuick ? quick_tanh(z) : tanhf(z);
    return fmaf(-t, t, 1.f);
  }
  if constexpr (kAct == VN_ACT_RELU) return z > 0.f ? 1.f : (z != z ? z : 0.f);
  if constexpr (kAct == VN_ACT_GELU) {
    if constexpr (kQuick) {
      float e;
      const float c = quick_cdf(z, &e);
      return fmaf(z * 0.3989422804014327f, e, c);
    }
    return fmaf(z * 0.3989422804014327f, expf(-0.5f * z * z), normcdff(z));
  }
  if constexpr (kAct == VN_ACT_SILU) {
    const float t = kQuick ? quick_reciprocal(1.f + __expf(-z)) : 1.f / (1.f + expf(-z));
    return t * fmaf(z, 1.f - t, 1.f);
  }
  return 1.f;
}

// v[i] = act(v[i]); the activation is the same for the whole launch.
template <bool kQuick, int N>
__device__ __forceinline__ void activate_all(int act, float (&v)[N]) {
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = f(v[i]);
  };
  switch (act) {
    case VN_ACT_TANH: each([](float z) { return activate<VN_ACT_TANH, kQuick>(z); }); break;
    case VN_ACT_RELU: each([](float z) { return activate<VN_ACT_RELU, kQuick>(z); }); break;
    case VN_ACT_GELU: each([](float z) { return activate<VN_ACT_GELU, kQuick>(z); }); break;
    case VN_ACT_SILU: each([](float z) { return activate<VN_ACT_SILU, kQuick>(z); }); break;
    default: break;
  }
}
// v[i] *= act'(z[i]).
template <bool kQuick, int N>
__device__ __forceinline__ void slope_all(int act, const float (&z)[N], float (&v)[N]) {
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= f(z[i]);
  };
  switch (act) {
    case VN_ACT_TANH: each([](float x) { return slope<VN_ACT_TANH, kQuick>(x); }); break;
    case VN_ACT_RELU: each([](float x) { return slope<VN_ACT_RELU, kQuick>(x); }); break;
    case VN_ACT_GELU: each([](float x) { return slope<VN_ACT_GELU, kQuick>(x); }); break;
    case VN_ACT_SILU: each([](float x) { return slope<VN_ACT_SILU, kQuick>(x); }); break;
    default: break;
  }
}

}  // namespace vn
