// vn_dense_rows.cu -- the centre network's linear layer on few rows (acting on one observation,
// or on a handful): y[r, j] = act(sum_k x[r, k] W[j, k] + b[j]) + residual[r, j], up to 8 rows.
//
// Every weight is used once per row, so the bound is reading W once. A warp owns two rows of
// W (features), or a slice of their k where features are few (up to 8 warps then share two
// features and add their sums through shared memory); its lanes walk along k with 16-byte loads of W,
// eight in flight a lane, and x comes from the caches. fp32 sums, in a fixed order.
// 4096 x 4096 bf16 on one row: 6.2 us, 5.4 TB/s; the tensor-core kernels take 11.3, on one row as on 16.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "vn_act.cuh"
#include "vn_dense.h"
#include "vn_internal.h"
#include "vn_launch.cuh"

namespace vn {
namespace {

constexpr int kWarps = 8;
constexpr int kFeatures = 2;  // of a warp

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// V consecutive elements: 16 bytes, or one.
template <typename T, int V>
struct Group {
  uint4 raw;
  __device__ __forceinline__ void load_stream(const T* p) { raw = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void load(const T* p) { raw = fetch(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { raw = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&v)[V]) const {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[2 * q] = __uint_as_float(w[q] << 16);
        v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = __uint_as_float(w[q]);
    }
  }
};
template <typename T>
struct Group<T, 1> {
  T e;
  __device__ __forceinline__ void load_stream(const T* p) { e = __ldcs(p); }
  __device__ __forceinline__ void load(const T* p) { e = fetch(p); }
  __device__ __forceinline__ void zero() { e = narrow<T>(0.f); }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = value(e); }
};

// kRows: rows rounded up to 1, 2, 4 or 8. slices: warps that share a pair of features.
template <typename T, int V, int kRows>
__global__ void __launch_bounds__(kWarps * 32) rows_kernel(const DenseArgs a, int slices) {
  let_next();
  constexpr int kDepth = kRows <= 2 ? 4 : 2;  // steps of k whose loads are in flight at once
  __shared__ float s[kWarps][kFeatures * kRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slice = warp % slices;
  const int64_t j0 = (static_cast<int64_t>(blockIdx.x) * (kWarps / slices) + warp / slices) * kFeatures;
  const T* x = static_cast<const T*>(a.x);
  const T* w = static_cast<const T*>(a.w);
  if constexpr (V == 8) {
    // While the kernel before this one ends, the warp's first weights are asked for into L2, which is
    // where any write to them is seen too: a hint that reads nothing. A lane takes one of a step's four
    // lines, for eight steps at a time. Calls one after the other, one row of 4096 to 4096 6.3 us for
    // 8.0, eight rows 20.0 for 21.5; all of longer rows, or fp32's, cost more than they gave (one
    // row of 4096 to 4096 13.4 us for 11.7).
    const int64_t end = a.in < 4096 ? a.in : 4096;
    for (int64_t k = ((slice + (lane >> 2) * static_cast<int64_t>(slices)) * 32 + (lane & 3) * 8) * V; k < end;
         k += static_cast<int64_t>(slices) * 256 * V) {
#pragma unroll
      for (int f = 0; f < kFeatures; ++f)
        if (j0 + f < a.out) prefetch(w + (j0 + f) * a.in + k);
    }
  }
  after_previous();
  const int rows = static_cast<int>(a.rows);
  float sum[kFeatures][kRows] = {};
  if (j0 < a.out) {
    const T* w0 = w + j0 * a.in;
    const T* w1 = j0 + 1 < a.out ? w0 + a.in : w0;  // the last feature of an odd number reads itself twice
    const int64_t step = static_cast<int64_t>(slices) * 32 * V;
    for (int64_t k = (static_cast<int64_t>(slice) * 32 + lane) * V; k < a.in; k += kDepth * step) {
      Group<T, V> wg[kFeatures][kDepth];
#pragma unroll
      for (int u = 0; u < kDepth; ++u) {
        const int64_t at = k + u * step;
        if (at < a.in) {
          wg[0][u].load_stream(w0 + at);
          wg[1][u].load_stream(w1 + at);
        } else {
          wg[0][u].zero();
          wg[1][u].zero();
        }
      }
#pragma unroll
      for (int u = 0; u < kDepth; ++u) {
        const int64_t at = k + u * step;
        if (at < a.in) {
          float v0[V], v1[V];
          wg[0][u].get(v0);
          wg[1][u].get(v1);
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            if (r < rows) {
              Group<T, V> xg;
              float xv[V];
              xg.load(x + r * a.in + at);
              xg.get(xv);
#pragma unroll
              for (int q = 0; q < V; ++q) {
                sum[0][r] = fmaf(xv[q], v0[q], sum[0][r]);
                sum[1][r] = fmaf(xv[q], v1[q], sum[1][r]);
              }
            }
          }
        }
      }
    }
  }
#pragma unroll
  for (int f = 0; f < kFeatures; ++f)
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum[f][r] += __shfl_xor_sync(0xFFFFFFFFu, sum[f][r], o);
      if (lane == 0) s[warp][f * kRows + r] = sum[f][r];
    }
  __syncthreads();
  // Output (feature f, row r) of a pair: one lane of its first warp.
  if (slice != 0 || lane >= kFeatures * kRows) return;
  const int f = lane / kRows, r = lane % kRows;
  const int64_t j = j0 + f;
  if (j >= a.out || r >= rows) return;
  float z[1] = {0.f};
  for (int k = 0; k < slices; ++k) z[0] += s[warp + k][lane];
  if (a.b != nullptr)
    z[0] += a.b_dt == VN_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.b)[j]) : static_cast<const float*>(a.b)[j];
  const int64_t at = r * a.out + j;
  if (a.preact != nullptr) static_cast<T*>(a.preact)[at] = narrow<T>(z[0]);
  activate_all<false>(a.act, z);
  if (a.residual != nullptr) z[0] += value(static_cast<const T*>(a.residual)[at]);
  static_cast<T*>(a.y)[at] = narrow<T>(z[0]);
}

template <typename T, int V, int kRows>
cudaError_t run(const DenseArgs& a, int slices, cudaStream_t stream) {
  const int64_t per = kWarps / slices * kFeatures;
  const int64_t grid = (a.out + per - 1) / per;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  return launch_overlapped(rows_kernel<T, V, kRows>, dim3(static_cast<unsigned>(grid)), kWarps * 32, 0, 0, stream, a,
                           slices);
}

template <typename T, int V>
cudaError_t run_rows(const DenseArgs& a, cudaStream_t stream) {
  DeviceInfo dev;
  const cudaError_t err = device_info(&dev);
  if (err != cudaSuccess) return err;
  // Slices until 16 warps an SM are at work, while a slice still has a full step for its lanes.
  int slices = 1;
  const int64_t pairs = (a.out + kFeatures - 1) / kFeatures;
  while (slices < kWarps && pairs * slices < 16 * dev.sm_count && a.in > slices * 32 * V) slices *= 2;
  if (a.rows <= 1) return run<T, V, 1>(a, slices, stream);
  if (a.rows <= 2) return run<T, V, 2>(a, slices, stream);
  if (a.rows <= 4) return run<T, V, 4>(a, slices, stream);
  return run<T, V, 8>(a, slices, stream);
}

template <typename T>
cudaError_t run_typed(const DenseArgs& a, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  const bool vec = a.in % V == 0 && (reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.w)) % 16 == 0;
  return vec ? run_rows<T, V>(a, stream) : run_rows<T, 1>(a, stream);
}

}  // namespace

cudaError_t launch_rows_forward(const DenseArgs& a, cudaStream_t stream) {
  return a.dt == VN_BF16 ? run_typed<__nv_bfloat16>(a, stream) : run_typed<float>(a, stream);
}

}  // namespace vn
