// vn_dense.cu -- the centre network's linear layer and its gradients.
//
//   z = x W^T + b, y = act(z) + residual
//   d = g act'(z), dx = d W, dw = d^T x, db = sum_rows d
//
// Every product is brought to one form, D[q, p] = sum_k A(p, k) B(q, k), with p the
// contiguous dimension of the result:
//   forward  p = out, q = row, k = in    A = W (k contiguous)   B = x (k contiguous)
//   dx       p = in,  q = row, k = out   A = W (p contiguous)   B = d (k contiguous)
//   dw       p = in,  q = out, k = row   A = x (p contiguous)   B = d (q contiguous)
// so one kernel with two stride pairs serves all three.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "vn_act.cuh"
#include "vn_internal.h"

namespace vn {
namespace {

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

constexpr int kTile = 64, kStep = 16, kThreads = 256;

struct Product {
  const void* a;
  const void* b;
  int64_t ap, ak, bq, bk;  // element strides
  int64_t np, nq, nk;
  const void* bias;        // [np] or NULL
  int bias_bf16, act;
  const void* residual;    // [nq, np] or NULL
  void* out;               // [nq, np]
  void* preact;            // [nq, np] or NULL
  int64_t p_tiles;
};

// 64 x 64 outputs a CTA, 4 x 4 a thread; 16 of k at a time through shared memory.
template <typename T>
__global__ void __launch_bounds__(kThreads) product_kernel(const Product d) {
  __shared__ float sa[kStep][kTile + 4], sb[kStep][kTile + 4];
  const int64_t p0 = static_cast<int64_t>(blockIdx.x % d.p_tiles) * kTile;
  const int64_t q0 = static_cast<int64_t>(blockIdx.x / d.p_tiles) * kTile;
  const int tp = threadIdx.x % 16, tq = threadIdx.x / 16;
  const T* a = static_cast<const T*>(d.a);
  const T* b = static_cast<const T*>(d.b);
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < d.nk; k0 += kStep) {
#pragma unroll
    for (int r = 0; r < kTile * kStep / kThreads; ++r) {
      const int e = r * kThreads + threadIdx.x;
      {
        const int k = d.ak == 1 ? e % kStep : e / kTile, p = d.ak == 1 ? e / kStep : e % kTile;
        sa[k][p] = (k0 + k < d.nk && p0 + p < d.np) ? value(a[(p0 + p) * d.ap + (k0 + k) * d.ak]) : 0.f;
      }
      {
        const int k = d.bk == 1 ? e % kStep : e / kTile, q = d.bk == 1 ? e / kStep : e % kTile;
        sb[k][q] = (k0 + k < d.nk && q0 + q < d.nq) ? value(b[(q0 + q) * d.bq + (k0 + k) * d.bk]) : 0.f;
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
      float av[4], bv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        av[i] = sa[k][tp * 4 + i];
        bv[i] = sb[k][tq * 4 + i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(bv[i], av[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t q = q0 + tq * 4 + i, p = p0 + tp * 4 + j;
      if (q < d.nq && p < d.np) {
        float z = acc[i][j];
        if (d.bias != nullptr)
          z += d.bias_bf16 ? value(static_cast<const __nv_bfloat16*>(d.bias)[p]) : static_cast<const float*>(d.bias)[p];
        if (d.preact != nullptr) static_cast<T*>(d.preact)[q * d.np + p] = narrow<T>(z);
        z = activate(d.act, z);
        if (d.residual != nullptr) z += value(static_cast<const T*>(d.residual)[q * d.np + p]);
        static_cast<T*>(d.out)[q * d.np + p] = narrow<T>(z);
      }
    }
}

// d = g act'(z) (rounded to T), and column sums of the unrounded d over every
// gridDim.y-th group of 8 rows.
template <typename T>
__global__ void __launch_bounds__(256)
delta_kernel(const T* __restrict__ g, const T* __restrict__ z, int act, int64_t rows, int64_t n,
             T* __restrict__ d, float* __restrict__ part) {
  __shared__ float s[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float sum = 0.f;
  if (c < n) {
    for (int64_t r = static_cast<int64_t>(blockIdx.y) * 8 + warp; r < rows; r += static_cast<int64_t>(gridDim.y) * 8) {
      float v = value(g[r * n + c]);
      if (act != VN_ACT_NONE) v *= slope(act, value(z[r * n + c]));
      if (d != nullptr) d[r * n + c] = narrow<T>(v);
      sum += v;
    }
  }
  s[warp][lane] = sum;
  __syncthreads();
  if (part != nullptr && warp == 0 && c < n) {
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += s[k][lane];
    part[static_cast<int64_t>(blockIdx.y) * n + c] = sum;
  }
}

template <typename T>
cudaError_t run_product(Product d, cudaStream_t stream) {
  if (d.np == 0 || d.nq == 0) return cudaSuccess;
  d.p_tiles = (d.np + kTile - 1) / kTile;
  const int64_t q_tiles = (d.nq + kTile - 1) / kTile;
  if (d.p_tiles > 0x7FFFFFFFll / q_tiles) return cudaErrorInvalidConfiguration;
  product_kernel<T><<<static_cast<unsigned>(d.p_tiles * q_tiles), kThreads, 0, stream>>>(d);
  return cudaGetLastError();
}

cudaError_t product(const Product& d, vn_dtype dt, cudaStream_t stream) {
  return dt == VN_BF16 ? run_product<__nv_bfloat16>(d, stream) : run_product<float>(d, stream);
}

constexpr int64_t kAlign = 256;
int64_t rounded(int64_t bytes) { return (bytes + kAlign - 1) / kAlign * kAlign; }

// Row groups that the column sums are split over.
int64_t delta_parts(int64_t rows) { return std::max<int64_t>(1, std::min<int64_t>(64, (rows + 63) / 64)); }

}  // namespace

int64_t dense_workspace(int64_t rows, int64_t in, int64_t out, vn_dtype dt, bool aligned) {
  (void)rows; (void)in; (void)out; (void)dt; (void)aligned;
  return 0;
}

int64_t dense_backward_workspace(int64_t rows, int64_t in, int64_t out, vn_dtype dt, vn_act act, bool aligned) {
  (void)in; (void)aligned;
  const int64_t size = dt == VN_BF16 ? 2 : 4;
  return (act != VN_ACT_NONE ? rounded(rows * out * size) : 0) + rounded(delta_parts(rows) * out * 4);
}

cudaError_t launch_dense(const DenseArgs& a, cudaStream_t stream) {
  Product d = {};
  d.a = a.w; d.ap = a.in; d.ak = 1;
  d.b = a.x; d.bq = a.in; d.bk = 1;
  d.np = a.out; d.nq = a.rows; d.nk = a.in;
  d.bias = a.b; d.bias_bf16 = a.b_dt == VN_BF16; d.act = a.act;
  d.residual = a.residual; d.out = a.y; d.preact = a.preact;
  return product(d, a.dt, stream);
}

cudaError_t launch_dense_backward(const DenseGradArgs& a, cudaStream_t stream) {
  const int64_t size = a.dt == VN_BF16 ? 2 : 4;
  uint8_t* work = static_cast<uint8_t*>(a.workspace);
  void* delta = nullptr;
  if (a.act != VN_ACT_NONE) {
    delta = work;
    work += rounded(a.rows * a.out * size);
  }
  float* part = a.grad_b != nullptr ? reinterpret_cast<float*>(work) : nullptr;
  const bool products = a.grad_x != nullptr || a.grad_w != nullptr;
  if (!products) delta = nullptr;
  cudaError_t err = cudaSuccess;
  const int64_t parts = a.rows > 0 ? delta_parts(a.rows) : 0;
  if (a.rows > 0 && a.out > 0 && (delta != nullptr || part != nullptr)) {
    const int64_t tiles = (a.out + 31) / 32;
    if (tiles > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(parts));
    if (a.dt == VN_BF16)
      delta_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(
          static_cast<const __nv_bfloat16*>(a.grad), static_cast<const __nv_bfloat16*>(a.preact), a.act, a.rows,
          a.out, static_cast<__nv_bfloat16*>(delta), part);
    else
      delta_kernel<float><<<grid, 256, 0, stream>>>(static_cast<const float*>(a.grad),
                                                    static_cast<const float*>(a.preact), a.act, a.rows, a.out,
                                                    static_cast<float*>(delta), part);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
  }
  if (a.grad_b != nullptr && a.out > 0 &&
      (err = launch_column_sum(part, parts, a.out, a.out, a.grad_b, nullptr, a.gb_dt, stream)) != cudaSuccess)
    return err;
  Product d = {};
  d.b = delta != nullptr ? delta : a.grad;
  if (a.grad_x != nullptr) {
    d.a = a.w; d.ap = 1; d.ak = a.in;
    d.bq = a.out; d.bk = 1;
    d.np = a.in; d.nq = a.rows; d.nk = a.out;
    d.out = a.grad_x;
    if ((err = product(d, a.dt, stream)) != cudaSuccess) return err;
  }
  if (a.grad_w != nullptr) {
    d.a = a.x; d.ap = 1; d.ak = a.in;
    d.bq = 1; d.bk = a.out;
    d.np = a.in; d.nq = a.out; d.nk = a.rows;
    d.out = a.grad_w;
    if ((err = product(d, a.dt, stream)) != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace vn
