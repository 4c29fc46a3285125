// vn_split.cuh -- an fp32 value as the sum of three bf16 values.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace vn {

// The three bf16 terms of a finite fp32 value, exactly: its top 8 significant bits, the next 8,
// the last 8. The terms of an infinity or a NaN hold a NaN.
__device__ __forceinline__ void split3(float v, uint32_t (&t)[3]) {
  const uint32_t u = __float_as_uint(v);
  const float r1 = v - __uint_as_float(u & 0xFFFF0000u);
  const uint32_t u1 = __float_as_uint(r1);
  const float r2 = r1 - __uint_as_float(u1 & 0xFFFF0000u);
  t[0] = u;
  t[1] = u1;
  t[2] = __float_as_uint(r2);
}
// Terms of two values (each in its word's upper half), the first one's in the lower half.
__device__ __forceinline__ uint32_t join_terms(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }

}  // namespace vn
