// vn_pair.cuh -- fp32 arithmetic two lanes at a time.
#pragma once

#include <cuda_runtime.h>

namespace vn {

// Two fp32 values in one register pair, and the two-lane instructions on them: one does the work of two
// where issue slots are what a kernel runs out of. The compiler may contract a product and a sum of
// them to a multiply-add, .rn or not: where every rounding counts, sums are taken as single
// instructions.
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void split(F2 v, float* a, float* b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(v));
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float sum_of(F2 v) {
  float a, b;
  split(v, &a, &b);
  return a + b;
}
}  // namespace vn
