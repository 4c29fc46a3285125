// vn_act.cuh -- the activations of the linear layer and their derivatives.
//
// Two forms of each: with CUDA's full-precision functions, and a quick one good to 2^-20 (1 + |z|) or
// better, with a quotient and an exponential on the special-function unit and a few multiply-adds: a
// third of the instructions, so that an epilogue over a whole tile stays shorter than the tile's
// products. The quick one serves every bf16 result (rounded to 2^-8), and fp32 ones where the
// products' own rounding is of that size: those gathered on the tensor cores and the gradients. There the
// full-precision functions cost, with GELU, 1024 x 256 to 256 7.7 us for 7.2, its gradients 19.3 for 13.7, and
// the gradients of 8192 x 1024 to 1024 233 for 199 (SiLU 7.6 for 7.1, 16.9 for 13.4 and 207 for 199).
#pragma once

#include <cuda_runtime.h>

#include "vn.h"
#include "vn_pair.cuh"

namespace vn {

// 1 / x and 2^x as single instructions of the special-function unit (to 1 and 2 units of the last place;
// subnormal operands and results are 0): the CUDA functions' care for subnormals took as many
// instructions again.
__device__ __forceinline__ float quick_reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float quick_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2E = 1.4426950408889634f;

// tanh: 1 - 2 / (1 + e^2z), and its Taylor series where that difference would cancel
// (to z^9 62/2835: below 1e-6 of the value at 1/4).
__device__ __forceinline__ float quick_tanh(float z) {
  const float s = z * z;
  const float series = z * fmaf(s, fmaf(s, fmaf(s, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
  const float quotient = fmaf(-2.f, quick_reciprocal(1.f + quick_exp2(2.f * kLog2E * z)), 1.f);
  return fabsf(z) < 0.25f ? series : quotient;
}
// The normal distribution function and e^(-z^2/2): Abramowitz and Stegun 7.1.26,
// erfc(x) = (a1 t + .. + a5 t^5) e^(-x^2), t = 1 / (1 + p x), off by at most 1.5e-7.
// The constants have 1/sqrt(2) and the half of erfc folded in.
__device__ __forceinline__ float quick_cdf(float z, float* e) {
  const float t = quick_reciprocal(fmaf(0.3275911f * 0.70710678118654752f, fabsf(z), 1.f));
  const float poly = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 0.5307027145f, -0.7265760135f), 0.7107068705f), -0.142248368f),
                              0.127414796f);
  *e = quick_exp2(z * (-0.5f * kLog2E * z));
  const float tail = poly * *e;
  return z >= 0.f ? 1.f - tail : tail;
}

// Two of z times quick_cdf(z), with two-lane multiply-adds.
__device__ __forceinline__ void quick_gelu(float* z0, float* z1) {
  auto both = [](float x) { return f2(x, x); };
  const F2 z = f2(*z0, *z1);
  float a, b;
  split(fma2(both(0.3275911f * 0.70710678118654752f), f2(fabsf(*z0), fabsf(*z1)), both(1.f)), &a, &b);
  const F2 t = f2(quick_reciprocal(a), quick_reciprocal(b));
  F2 poly = fma2(t, both(0.5307027145f), both(-0.7265760135f));
  poly = fma2(t, poly, both(0.7107068705f));
  poly = fma2(t, poly, both(-0.142248368f));
  poly = mul2(t, fma2(t, poly, both(0.127414796f)));
  split(mul2(z, mul2(z, both(-0.5f * kLog2E))), &a, &b);
  split(mul2(poly, f2(quick_exp2(a), quick_exp2(b))), &a, &b);
  *z0 *= *z0 >= 0.f ? 1.f - a : a;
  *z1 *= *z1 >= 0.f ? 1.f - b : b;
}

template <int kAct, bool kQuick>
__device__ __forceinline__ float activate(float z) {
  if constexpr (kAct == VN_ACT_TANH) return kQuick ? quick_tanh(z) : tanhf(z);
  if constexpr (kAct == VN_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
  if constexpr (kAct == VN_ACT_GELU) {
    float e;
    return z * (kQuick ? quick_cdf(z, &e) : normcdff(z));
  }
  if constexpr (kAct == VN_ACT_SILU) return kQuick ? z * quick_reciprocal(1.f + quick_exp2(-kLog2E * z)) : z / (1.f + expf(-z));
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
    const float t = kQuick ? quick_reciprocal(1.f + quick_exp2(-kLog2E * z)) : 1.f / (1.f + expf(-z));
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
    case VN_ACT_GELU:
      if constexpr (kQuick && N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2) quick_gelu(&v[i], &v[i + 1]);
      } else {
        each([](float z) { return activate<VN_ACT_GELU, kQuick>(z); });
      }
      break;
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
