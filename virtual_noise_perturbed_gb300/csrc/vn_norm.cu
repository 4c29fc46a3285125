// vn_norm.cu -- layer norm and its gradients.
//
//   mean = sum x / n, rstd = (sum (x - mean)^2 / n + eps)^-1/2, y = (x - mean) rstd w + b
//   h = (x - mean) rstd, t = g w:  dx = rstd (t - mean(t) - h mean(t h)),
//   dw = sum_rows g h, db = sum_rows g
//
// Forward: a row lives in the registers of T threads (8 to 512 by its length),
// so it is read from memory once although the variance is taken from the centred
// values (a second pass over registers, not the cancelling sum of squares).
//
// Backward: the two row means come from one reduction of two numbers. The sums over rows
// stay in registers: a group of T threads walks over rows of its own (every G-th), each
// thread on the same columns in each, and its column sums leave once at the end, as one
// partial row per CTA; a second small kernel adds the partial rows in order. No atomics, so
// the sums do not depend on the order in which CTAs run.
//
// Rows beyond what registers hold take the looping kernels at the end of this file.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "vn_internal.h"
#include "vn_launch.cuh"
#include "vn_pair.cuh"

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

// V consecutive elements, as they are in memory: 16 bytes (V > 1) or one element.
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T e[V];
};
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p) {
  Pack<T, V> r;
  if constexpr (V > 1) {
    static_assert(sizeof(T) * V == 16, "16-byte packs");
    *reinterpret_cast<uint4*>(&r) = __ldcs(reinterpret_cast<const uint4*>(p));
  } else {
    r.e[0] = p[0];
  }
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void store_pack(T* p, const float (&v)[V]) {
  if constexpr (V > 1) {
    Pack<T, V> r;
#pragma unroll
    for (int q = 0; q < V; ++q) r.e[q] = narrow<T>(v[q]);
    __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(&r));
  } else {
    p[0] = narrow<T>(v[0]);
  }
}
// V consecutive parameters (fp32 or bf16, 16-byte aligned at multiples of V when V > 1).
template <int V>
__device__ __forceinline__ void load_param(const void* w, int bf16, int64_t i, float absent, float (&v)[V]) {
  if (w == nullptr) {
#pragma unroll
    for (int q = 0; q < V; ++q) v[q] = absent;
  } else if (bf16) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(w) + i;
    if constexpr (V == 8) {
      const uint4 a = fetch(reinterpret_cast<const uint4*>(p));
      const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[2 * q] = __uint_as_float(u[q] << 16);
        v[2 * q + 1] = __uint_as_float(u[q] & 0xFFFF0000u);
      }
    } else if constexpr (V == 4) {
      const uint2 a = fetch(reinterpret_cast<const uint2*>(p));
      v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xFFFF0000u);
      v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xFFFF0000u);
    } else {
      v[0] = __bfloat162float(p[0]);
    }
  } else {
    const float* p = static_cast<const float*>(w) + i;
    if constexpr (V > 1) {
#pragma unroll
      for (int q = 0; q < V; q += 4) {
        const float4 a = fetch(reinterpret_cast<const float4*>(p + q));
        v[q] = a.x; v[q + 1] = a.y; v[q + 2] = a.z; v[q + 3] = a.w;
      }
    } else {
      v[0] = fetch(p);
    }
  }
}

// Sums over the T threads of a row (a part of a warp, a warp, or the whole CTA), the same in every thread.
// `scratch`: 64 floats for one sum, 128 for two, halves of which calls use in turn.
template <int T>
__device__ __forceinline__ float row_sum(float v, float* scratch, int& turn) {
#pragma unroll
  for (int o = (T < 32 ? T : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if constexpr (T > 32) {
    constexpr int kW = T / 32;
    float* s = scratch + (turn++ & 1) * 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) s[warp] = v;
    __syncthreads();
    v = s[lane % kW];
#pragma unroll
    for (int o = kW / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  }
  return v;
}
// Two sums: the first step leaves each half of a warp with one of them.
template <int T>
__device__ __forceinline__ void row_sum2(float& v0, float& v1, float* scratch, int& turn) {
  const int lane = threadIdx.x & 31;
  const bool upper = lane >= 16;
  float v = (upper ? v1 : v0) + __shfl_xor_sync(0xFFFFFFFFu, upper ? v0 : v1, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if constexpr (T > 32) {
    constexpr int kW = T / 32;
    static_assert(kW <= 16, "a half-warp takes a sum's partial sums");
    float* s = scratch + (turn++ & 1) * 64 + (upper ? 32 : 0);
    if ((lane & 15) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = s[lane % kW];
#pragma unroll
    for (int o = kW / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  }
  v0 = __shfl_sync(0xFFFFFFFFu, v, 0);
  v1 = __shfl_sync(0xFFFFFFFFu, v, 16);
}

// A 16-byte pack as pairs of fp32: 4 of bf16, 2 of fp32.
template <typename X>
constexpr int kPairs = 8 / sizeof(X);
template <typename X>
__device__ __forceinline__ void pairs_of(const uint4& p, F2 (&v)[kPairs<X>]) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
  if constexpr (sizeof(X) == 2) {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = f2(__uint_as_float(w[q] << 16), __uint_as_float(w[q] & 0xFFFF0000u));
  } else {
#pragma unroll
    for (int q = 0; q < 2; ++q) v[q] = f2(__uint_as_float(w[2 * q]), __uint_as_float(w[2 * q + 1]));
  }
}
template <typename X>
__device__ __forceinline__ void store_pairs(X* p, const F2 (&v)[kPairs<X>]) {
  float o[16 / sizeof(X)];
#pragma unroll
  for (int q = 0; q < kPairs<X>; ++q) split(v[q], &o[2 * q], &o[2 * q + 1]);
  store_pack<X, 16 / sizeof(X)>(p, o);
}
// The first `left` of V consecutive parameters, 0 beyond.
template <int V>
__device__ __forceinline__ void load_params(const void* w, int bf16, int64_t i, int left, float absent, float (&v)[V]) {
  if (left >= V) {
    load_param<V>(w, bf16, i, absent, v);
    return;
  }
#pragma unroll
  for (int q = 0; q < V; ++q) {
    float one[1] = {0.f};
    if (q < left) load_param<1>(w, bf16, i + q, absent, one);
    v[q] = one[0];
  }
}
// V consecutive parameters as pairs.
template <int V>
__device__ __forceinline__ void load_pairs(const void* w, int bf16, int64_t i, int left, float absent, F2 (&v)[V / 2]) {
  float u[V];
  load_params<V>(w, bf16, i, left, absent, u);
#pragma unroll
  for (int q = 0; q < V / 2; ++q) v[q] = f2(u[2 * q], u[2 * q + 1]);
}
// Rows that start anywhere. Their elements are taken in packs of 16 bytes all the same: a pack comes from
// the two aligned words that hold it, and leaves as one aligned word with the end of the pack
// before it, which the lane below has. Single elements are moved at the ends of a row and of a
// warp, and where an aligned word would pass the tensor's ends.
//
// 16 bytes from element e of a and b on.
template <typename X>
__device__ __forceinline__ uint4 pick(const uint4& a, const uint4& b, int e) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  constexpr int kOne = sizeof(X) == 2 ? 2 : 1, kTwo = 2 * kOne;
  uint32_t x[6], y[5];
#pragma unroll
  for (int i = 0; i < 6; ++i) x[i] = e & kTwo ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) y[i] = e & kOne ? x[i + 1] : x[i];
  if constexpr (sizeof(X) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __funnelshift_r(y[i], y[i + 1], (e & 1) * 16);
  }
  return make_uint4(y[0], y[1], y[2], y[3]);
}
template <typename X>
__device__ __forceinline__ int misplaced(const X* p) {  // elements since the last 16-byte boundary
  return static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(X));
}
template <typename X>
__device__ __forceinline__ int misplaced(const void* tensor, int64_t row, int n) {  // of row `row`
  return (misplaced(static_cast<const X*>(tensor)) + static_cast<uint32_t>(row) * static_cast<uint32_t>(n)) & (16 / sizeof(X) - 1);
}
// The first `left` elements of a pack, 0 beyond.
template <typename X>
__device__ __forceinline__ uint4 keep(const uint4& v, int left) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(X) == 2) w[i] = left >= 2 * i + 2 ? w[i] : left > 2 * i ? w[i] & 0xFFFFu : 0u;
    else w[i] = left > i ? w[i] : 0u;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename X>
__device__ __forceinline__ uint4 gather_pack(const X* p, int left) {
  uint32_t w[4] = {};
  if constexpr (sizeof(X) == 2) {
    const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < left) w[q / 2] |= static_cast<uint32_t>(fetch(h + q)) << (q % 2 * 16);
  } else {
    const uint32_t* h = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < left) w[q] = fetch(h + q);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Whether the aligned words of a row's `packs` packs, whose first element is `at`, lie within the tensor.
template <typename X>
__device__ __forceinline__ bool within(int64_t at, int packs, int64_t elements) {
  constexpr int V = 16 / sizeof(X);
  return at >= V && at + static_cast<int64_t>(packs + 1) * V <= elements;
}
// One pack of outputs, the row's elements from i on, by all lanes of the warp. `before`: the group's pack
// ahead of its first lane's; `first` and `last`: this lane's pack is the group's first or last of the row,
// whose neighbour is not at hand. m: misplaced(row).
template <typename X, int kGroup>
__device__ __forceinline__ void store_any(X* row, int m, int i, int n, bool first, bool last, const uint4& before, const uint4& o) {
  constexpr int V = 16 / sizeof(X);
  const int lane = threadIdx.x & (kGroup - 1);
  const bool top = lane == kGroup - 1;
  const int from = (lane + kGroup - 1) & (kGroup - 1);
  uint4 below;
  below.x = __shfl_sync(0xFFFFFFFFu, top ? before.x : o.x, from, kGroup);
  below.y = __shfl_sync(0xFFFFFFFFu, top ? before.y : o.y, from, kGroup);
  below.z = __shfl_sync(0xFFFFFFFFu, top ? before.z : o.z, from, kGroup);
  below.w = __shfl_sync(0xFFFFFFFFu, top ? before.w : o.w, from, kGroup);
  const int left = n - i;
  if (left <= 0) return;
  const bool whole = left >= V - m && (m == 0 || !first);  // this lane's aligned word
  const bool above = left - V >= V - m && !last;           // the next one, by the lane above
  if (whole) __stcs(reinterpret_cast<uint4*>(row + i - m), m == 0 ? o : pick<X>(below, o, V - m));
  if (!whole || (m > 0 && !above)) {
    const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int q = 0; q < V; ++q) {
      if (q >= left || (q < V - m ? whole : above)) continue;
      if constexpr (sizeof(X) == 2) reinterpret_cast<unsigned short*>(row + i)[q] = static_cast<unsigned short>(w[q / 2] >> (q % 2 * 16));
      else reinterpret_cast<uint32_t*>(row + i)[q] = w[q];
    }
  }
}
template <typename X>
__device__ __forceinline__ uint4 pack_of(const F2 (&v)[kPairs<X>]) {
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < kPairs<X>; ++q) {
    float a, b;
    split(v[q], &a, &b);
    if constexpr (sizeof(X) == 2) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      w[q] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      w[2 * q] = __float_as_uint(a);
      w[2 * q + 1] = __float_as_uint(b);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest `pending` groups of copies are complete.
__device__ __forceinline__ void wait_copies(int pending) {
  if (pending == 4) asm volatile("cp.async.wait_group 4;" ::: "memory");
  else if (pending == 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (pending == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else asm volatile("cp.async.wait_group 1;" ::: "memory");
}

struct NormArgsK {
  const void* x;
  const void* w;
  const void* b;
  void* y;
  float* mean;
  float* rstd;
  int64_t rows, n;
  float eps, inv_n;
  int w_bf16;
};

constexpr int cta_threads(int t) { return t < 64 ? 128 : t; }

// Rows of 16-byte packs, NV of them a thread; kAny: that start anywhere and end within a pack.
template <typename X, int T, int NV, bool kAny>
__global__ void __launch_bounds__(cta_threads(T)) norm_pairs_kernel(const NormArgsK a) {
  let_next();
  after_previous();
  constexpr int kRows = cta_threads(T) / T, V = 16 / sizeof(X), P = kPairs<X>;
  __shared__ float scratch[T > 32 ? 64 : 1];
  int turn = 0;
  const int t = threadIdx.x % T;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / T;
  if (T == 32 && row >= a.rows) return;
  const bool live = row < a.rows;  // below a warp a row, its lanes stay together
  if (!live) row = a.rows - 1;
  const int n = live ? static_cast<int>(a.n) : 0;
  const X* in = static_cast<const X*>(a.x) + row * a.n;
  uint4 raw[NV];
  // The thread's packs: every T-th, or in a warp's groups one after the other, so that all
  // neighbours but a warp's first and last are at hand.
  constexpr int kGroup = T < 32 ? T : 32;
  auto at = [&](int j) { return (kAny && T > 32 ? ((t >> 5) * NV + j) * 32 + (t & 31) : j * T + t) * V; };
  if constexpr (kAny) {
    const int m = misplaced<X>(a.x, row, static_cast<int>(a.n));
    bool inside = within<X>(row * a.n, static_cast<int>((a.n + V - 1) / V), a.rows * a.n);
    if (T < 32) inside = __all_sync(0xFFFFFFFFu, inside);  // a warp's rows go one way
    if (inside) {
      const uint4 none = make_uint4(0u, 0u, 0u, 0u);
      const bool top = (t & (kGroup - 1)) == kGroup - 1;
      uint4 beyond = none;  // the word after the thread's last group's
#pragma unroll
      for (int j = 0; j < NV; ++j) raw[j] = at(j) < n + m ? fetch(reinterpret_cast<const uint4*>(in - m + at(j))) : none;
      if (top && at(NV - 1) + V < n + m) beyond = fetch(reinterpret_cast<const uint4*>(in - m + at(NV - 1) + V));
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        // The next word: the lane above's, or the next group's first.
        const uint4 next = j + 1 < NV ? raw[j + 1] : beyond;
        const bool low = (t & (kGroup - 1)) == 0;
        uint4 high;
        const int from = (t + 1) & (kGroup - 1);
        high.x = __shfl_sync(0xFFFFFFFFu, low && j + 1 < NV ? next.x : raw[j].x, from, kGroup);
        high.y = __shfl_sync(0xFFFFFFFFu, low && j + 1 < NV ? next.y : raw[j].y, from, kGroup);
        high.z = __shfl_sync(0xFFFFFFFFu, low && j + 1 < NV ? next.z : raw[j].z, from, kGroup);
        high.w = __shfl_sync(0xFFFFFFFFu, low && j + 1 < NV ? next.w : raw[j].w, from, kGroup);
        if (j + 1 == NV && top) high = beyond;
        raw[j] = pick<X>(raw[j], high, m);
        const int left = n - at(j);
        if (left < V) raw[j] = keep<X>(raw[j], left);
      }
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) raw[j] = gather_pack(in + at(j), n - at(j));
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = at(j);
      if (i < n) raw[j] = __ldcs(reinterpret_cast<const uint4*>(in + i));
    }
  }
  // The row stays as it was loaded and is unpacked in each pass: bf16 in half the registers
  // that its fp32 values would take, for more rows at work (84 us against 116 us, 32768 x 4096).
  F2 s = f2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (at(j) < n) {
      F2 x[P];
      pairs_of<X>(raw[j], x);
#pragma unroll
      for (int q = 0; q < P; ++q) s = add2(s, x[q]);
    }
  const float mean = row_sum<T>(sum_of(s), scratch, turn) * a.inv_n;
  const F2 minus = f2(-mean, -mean);
  s = f2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (at(j) < n) {
      F2 x[P];
      pairs_of<X>(raw[j], x);
      const int left = n - at(j);
#pragma unroll
      for (int q = 0; q < P; ++q) {
        x[q] = add2(x[q], minus);
        if (kAny && left < V) {
          float u, v;
          split(x[q], &u, &v);
          x[q] = f2(2 * q < left ? u : 0.f, 2 * q + 1 < left ? v : 0.f);
        }
        s = fma2(x[q], x[q], s);
      }
    }
  const float rstd = 1.f / sqrtf(row_sum<T>(sum_of(s), scratch, turn) * a.inv_n + a.eps);
  const F2 r2 = f2(rstd, rstd);
  X* y = static_cast<X*>(a.y) + row * a.n;
  uint4 before = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = at(j);
    uint4 o = make_uint4(0u, 0u, 0u, 0u);
    if (i < n) {
      F2 x[P], w[P], b[P];
      const int left = kAny ? n - i : V;
      load_pairs<V>(a.w, a.w_bf16, i, left, 1.f, w);
      load_pairs<V>(a.b, a.w_bf16, i, left, 0.f, b);
      pairs_of<X>(raw[j], x);
#pragma unroll
      for (int q = 0; q < P; ++q) x[q] = fma2(mul2(add2(x[q], minus), r2), w[q], b[q]);
      if constexpr (kAny) o = pack_of<X>(x);
      else store_pairs<X>(y + i, x);
    }
    if constexpr (kAny) {
      const int lane = t & (kGroup - 1);
      store_any<X, kGroup>(y, misplaced(y), i, n, j == 0 && lane == 0, j == NV - 1 && lane == kGroup - 1, before, o);
      before = o;
    }
  }
  if (t == 0 && live) {
    if (a.mean != nullptr) a.mean[row] = mean;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
}

// Parameters that do not start on 16 bytes: single elements, NV of them a thread.
template <typename X, int T, int V, int NV>
__global__ void __launch_bounds__(cta_threads(T)) norm_kernel(const NormArgsK a) {
  let_next();
  after_previous();
  constexpr int kRows = cta_threads(T) / T;
  __shared__ float scratch[T > 32 ? 64 : 1];
  int turn = 0;
  const int t = threadIdx.x % T;
  const int n = static_cast<int>(a.n);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / T;
  if (T == 32 && row >= a.rows) return;
  const X* x = static_cast<const X*>(a.x) + row * a.n;
  Pack<X, V> v[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = (j * T + t) * V;
    if (i < n) v[j] = load_pack<X, V>(x + i);
  }
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if ((j * T + t) * V < n)
#pragma unroll
      for (int q = 0; q < V; ++q) s += value(v[j].e[q]);
  const float mean = row_sum<T>(s, scratch, turn) * a.inv_n;
  s = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if ((j * T + t) * V < n)
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const float c = value(v[j].e[q]) - mean;
        s = fmaf(c, c, s);
      }
  const float rstd = 1.f / sqrtf(row_sum<T>(s, scratch, turn) * a.inv_n + a.eps);
  X* y = static_cast<X*>(a.y) + row * a.n;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = (j * T + t) * V;
    if (i < n) {
      float w[V], b[V], o[V];
      load_param<V>(a.w, a.w_bf16, i, 1.f, w);
      load_param<V>(a.b, a.w_bf16, i, 0.f, b);
#pragma unroll
      for (int q = 0; q < V; ++q) o[q] = fmaf((value(v[j].e[q]) - mean) * rstd, w[q], b[q]);
      store_pack<X, V>(y + i, o);
    }
  }
  if (t == 0) {
    if (a.mean != nullptr) a.mean[row] = mean;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
}

// Rows longer than the registers hold: three passes over the row (the second and third
// mostly from L2).
template <typename X>
__global__ void __launch_bounds__(512) norm_long_kernel(const NormArgsK a) {
  let_next();
  after_previous();
  __shared__ float scratch[64];
  int turn = 0;
  const int64_t row = blockIdx.x;
  const X* x = static_cast<const X*>(a.x) + row * a.n;
  X* y = static_cast<X*>(a.y) + row * a.n;
  float s = 0.f;
  for (int64_t i = threadIdx.x; i < a.n; i += 512) s += value(x[i]);
  const float mean = row_sum<512>(s, scratch, turn) * a.inv_n;
  s = 0.f;
  for (int64_t i = threadIdx.x; i < a.n; i += 512) {
    const float c = value(x[i]) - mean;
    s = fmaf(c, c, s);
  }
  const float rstd = 1.f / sqrtf(row_sum<512>(s, scratch, turn) * a.inv_n + a.eps);
  for (int64_t i = threadIdx.x; i < a.n; i += 512) {
    float w[1], b[1];
    load_param<1>(a.w, a.w_bf16, i, 1.f, w);
    load_param<1>(a.b, a.w_bf16, i, 0.f, b);
    y[i] = narrow<X>(fmaf((value(x[i]) - mean) * rstd, w[0], b[0]));
  }
  if (threadIdx.x == 0) {
    if (a.mean != nullptr) a.mean[row] = mean;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
}

// ---------------------------------------------------------------- gradients
struct NormGradK {
  const void* g;
  const void* x;
  const float* mean;
  const float* rstd;
  const void* w;
  void* dx;
  float* part;  // [CTAs][2][n] column sums, or NULL
  int64_t rows, n;
  float inv_n;
  int w_bf16;
};

// Threads of a CTA: 16 warps where a warp has a row, for few partial sums. Up to four elements a thread leave
// registers for two such CTAs an SM (60000 x 63 bf16: 12.8 us for 25.3).
constexpr int grad_threads(int t) { return t < 64 ? 512 : t; }

template <typename X, int T, int V, int NV>
__global__ void __launch_bounds__(grad_threads(T), T < 64 && V * NV <= 4 ? 2 : 1) norm_grad_kernel(const NormGradK a) {
  let_next();
  after_previous();
  constexpr int kRows = grad_threads(T) / T;
  __shared__ float scratch[T > 32 ? 128 : 1];
  extern __shared__ float columns[];  // T == 32: kRows x 2 x n column sums to be added
  int turn = 0;
  const int t = threadIdx.x % T;
  const int group = threadIdx.x / T;
  const int n = static_cast<int>(a.n);
  float w[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = (j * T + t) * V;
#pragma unroll
    for (int q = 0; q < V; ++q) w[j][q] = dw[j][q] = db[j][q] = 0.f;
    if (i < n) load_param<V>(a.w, a.w_bf16, i, 1.f, w[j]);
  }
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + group;
  // The next row's loads are issued before this row's arithmetic.
  Pack<X, V> gn[NV], xn[NV];
  float mean_n = 0.f, rstd_n = 0.f;
  auto fetch = [&](int64_t r) {
    const X* g = static_cast<const X*>(a.g) + r * a.n;
    const X* x = static_cast<const X*>(a.x) + r * a.n;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = (j * T + t) * V;
      if (i < n) {
        gn[j] = load_pack<X, V>(g + i);
        xn[j] = load_pack<X, V>(x + i);
      }
    }
    mean_n = a.mean[r];
    rstd_n = a.rstd[r];
  };
  if (row < a.rows) fetch(row);
  for (; row < a.rows; row += stride) {
    Pack<X, V> gv[NV], xv[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      gv[j] = gn[j];
      xv[j] = xn[j];
    }
    const float mean = mean_n, rstd = rstd_n;
    if (row + stride < a.rows) fetch(row + stride);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if ((j * T + t) * V < n)
#pragma unroll
        for (int q = 0; q < V; ++q) {
          const float d = value(gv[j].e[q]), h = (value(xv[j].e[q]) - mean) * rstd;
          const float u = d * w[j][q];
          s[0] += u;
          s[1] = fmaf(u, h, s[1]);
          dw[j][q] = fmaf(d, h, dw[j][q]);
          db[j][q] += d;
        }
    row_sum2<T>(s[0], s[1], scratch, turn);
    const float m1 = s[0] * a.inv_n, m2 = s[1] * a.inv_n;
    X* dx = static_cast<X*>(a.dx) + row * a.n;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = (j * T + t) * V;
      if (i < n) {
        float o[V];
#pragma unroll
        for (int q = 0; q < V; ++q) {
          const float h = (value(xv[j].e[q]) - mean) * rstd;
          o[q] = rstd * (fmaf(value(gv[j].e[q]), w[j][q], -m1) - h * m2);
        }
        store_pack<X, V>(dx + i, o);
      }
    }
  }
  if (a.part == nullptr) return;
  float* out = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.n;
  if constexpr (T == 32) {  // the CTA's warps hold sums of the same columns
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const int i = (j * T + t) * V + q;
        if (i < n) {
          columns[(group * 2) * n + i] = dw[j][q];
          columns[(group * 2 + 1) * n + i] = db[j][q];
        }
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * n; i += grad_threads(T)) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < kRows; ++k) s += columns[k * 2 * n + i];
      out[i] = s;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const int i = (j * T + t) * V + q;
        if (i < n) {
          out[i] = dw[j][q];
          out[a.n + i] = db[j][q];
        }
      }
  }
}

// The same for longer rows of 16-byte packs, which come through a ring of rows in shared memory: with
// straight loads of one row ahead 32 KB an SM were on their way, 4 TB/s; and on pairs: 35
// instructions an element were the next bound (193 us on 32768 x 4096 bf16).
template <typename X, int T, int NV>
__global__ void __launch_bounds__(T) norm_grad_ring_kernel(const NormGradK a, const int depth) {
  let_next();
  after_previous();
  constexpr int V = 16 / sizeof(X), P = kPairs<X>;
  extern __shared__ uint4 ring[];  // [depth][2][NV][T]
  __shared__ float scratch[128];
  const int t = threadIdx.x;
  const int n = static_cast<int>(a.n);
  // The number of the thread's pack j: a warp's NV groups of 32 follow one another, so that it reads and
  // writes in few places (32768 x 4096 fp32: 235 us, with every T-th pack 273).
  auto at = [&](int j) { return ((t >> 5) * NV + j) * 32 + (t & 31); };
  F2 w[NV][P], dw[NV][P], db[NV][P];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = at(j) * V;
    float u[V] = {};
    if (i < n) load_param<V>(a.w, a.w_bf16, i, 1.f, u);
#pragma unroll
    for (int q = 0; q < P; ++q) {
      w[j][q] = f2(u[2 * q], u[2 * q + 1]);
      dw[j][q] = db[j][q] = f2(0.f, 0.f);
    }
  }
  const int64_t stride = gridDim.x;
  auto fetch = [&](int64_t row, int slot) {  // one group of copies, empty beyond the last row
    if (row < a.rows) {
      const X* g = static_cast<const X*>(a.g) + row * a.n;
      const X* x = static_cast<const X*>(a.x) + row * a.n;
      const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(ring + slot * (2 * NV * T)));
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i = at(j) * V;
        if (i < n) {
          copy16(to + at(j) * 16, g + at(j) * V);
          copy16(to + (NV * T + at(j)) * 16, x + at(j) * V);
        }
      }
    }
    commit_copies();
  };
  // Row k's sums and row k - 1's outputs share an iteration, with one barrier at its end: the
  // reduction's latency is covered by the other row's arithmetic (in sequence, a row of 4096
  // took a CTA 1.7 us, 0.9 of it waiting). Row k - 1 is read a second time from the ring.
  const int64_t first = blockIdx.x;
  const int64_t count = first < a.rows ? (a.rows - first + stride - 1) / stride : 0;
  for (int d = 0; d < depth - 1; ++d) fetch(first + d * stride, d);
  float mean = 0.f, rstd = 0.f, mean_n = 0.f, rstd_n = 0.f;  // row k's, and row k + 1's
  if (count > 0) {
    mean_n = a.mean[first];
    rstd_n = a.rstd[first];
  }
  const int warp = t >> 5, lane = t & 31;
  int slot = 0;
  F2 r2, shift;  // row k - 1's, then row k's
  for (int64_t k = 0; k <= count; ++k) {
    const F2 r2_old = r2, shift_old = shift;
    const int old = slot == 0 ? depth - 1 : slot - 1;
    if (k < count) {
      mean = mean_n;
      rstd = rstd_n;
      if (k + 1 < count) {
        mean_n = a.mean[first + (k + 1) * stride];
        rstd_n = a.rstd[first + (k + 1) * stride];
      }
      // h = (x - mean) rstd; in bf16, whose x is coarser than the rounding of mean rstd, as
      // one multiply-add.
      r2 = f2(rstd, rstd);
      shift = sizeof(X) == 2 ? f2(-mean * rstd, -mean * rstd) : f2(-mean, -mean);
      wait_copies(depth - 2);
      const uint4* const from = ring + slot * (2 * NV * T);
      F2 s1 = f2(0.f, 0.f), s2 = f2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (at(j) * V < n) {
          F2 g[P], h[P];
          pairs_of<X>(from[at(j)], g);
          pairs_of<X>(from[NV * T + at(j)], h);
#pragma unroll
          for (int q = 0; q < P; ++q) {
            h[q] = sizeof(X) == 2 ? fma2(h[q], r2, shift) : mul2(add2(h[q], shift), r2);
            db[j][q] = add2(db[j][q], g[q]);
            const F2 gh = mul2(g[q], h[q]);
            dw[j][q] = add2(dw[j][q], gh);
            s1 = fma2(g[q], w[j][q], s1);
            s2 = fma2(gh, w[j][q], s2);
          }
        }
      // The warp's two sums, one in each half of its lanes, to its place.
      const float v0 = sum_of(s1), v1 = sum_of(s2);
      float v = (lane >= 16 ? v1 : v0) + __shfl_xor_sync(0xFFFFFFFFu, lane >= 16 ? v0 : v1, 16);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      if ((lane & 15) == 0) scratch[(k & 1) * 64 + (lane >> 4) * 32 + warp] = v;
    }
    if (k > 0) {
      constexpr int kW = T / 32;
      float v = scratch[((k - 1) & 1) * 64 + (lane >> 4) * 32 + lane % kW];
#pragma unroll
      for (int o = kW / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      const float m1 = -__shfl_sync(0xFFFFFFFFu, v, 0) * a.inv_n, m2 = -__shfl_sync(0xFFFFFFFFu, v, 16) * a.inv_n;
      // rstd (g w - m1 - h m2)
      const F2 c1 = f2(m1, m1), c2 = f2(m2, m2);
      const uint4* const from = ring + old * (2 * NV * T);
      X* dx = static_cast<X*>(a.dx) + (first + (k - 1) * stride) * a.n;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int i = at(j) * V;
        if (i < n) {
          F2 g[P], h[P], o[P];
          pairs_of<X>(from[at(j)], g);
          pairs_of<X>(from[NV * T + at(j)], h);
#pragma unroll
          for (int q = 0; q < P; ++q) {
            h[q] = sizeof(X) == 2 ? fma2(h[q], r2_old, shift_old) : mul2(add2(h[q], shift_old), r2_old);
            o[q] = mul2(fma2(h[q], c2, fma2(g[q], w[j][q], c1)), r2_old);
          }
          store_pairs<X>(dx + i, o);
        }
      }
    }
    // Row k - 1's place is free: the row `depth` after it.
    if (k < count) {
      fetch(first + (k + depth - 1) * stride, old);
      slot = slot + 1 == depth ? 0 : slot + 1;
    }
    __syncthreads();
  }
  if (a.part == nullptr) return;
  float* out = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.n;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = at(j) * V;
    if (i < n) {
#pragma unroll
      for (int q = 0; q < P; q += 2) {
        float4 u, v;
        split(dw[j][q], &u.x, &u.y);
        split(dw[j][q + 1], &u.z, &u.w);
        split(db[j][q], &v.x, &v.y);
        split(db[j][q + 1], &v.z, &v.w);
        *reinterpret_cast<float4*>(out + i + 2 * q) = u;
        *reinterpret_cast<float4*>(out + a.n + i + 2 * q) = v;
      }
    }
  }
}

// Long rows, beyond 8192 elements: grad_x in two passes over the row, of single elements (16384 x 8200 bf16 541 us
// with the column sums, 568 in fp32, where 16384 x 8192 on the ring takes 151 and 206) ...
template <typename X>
__global__ void __launch_bounds__(512) norm_grad_long_kernel(const NormGradK a) {
  let_next();
  after_previous();
  __shared__ float scratch[128];
  int turn = 0;
  const int64_t row = blockIdx.x;
  const X* g = static_cast<const X*>(a.g) + row * a.n;
  const X* x = static_cast<const X*>(a.x) + row * a.n;
  X* dx = static_cast<X*>(a.dx) + row * a.n;
  const float mean = a.mean[row], rstd = a.rstd[row];
  float s[2] = {0.f, 0.f};
  for (int64_t i = threadIdx.x; i < a.n; i += 512) {
    float w[1];
    load_param<1>(a.w, a.w_bf16, i, 1.f, w);
    const float u = value(g[i]) * w[0];
    s[0] += u;
    s[1] = fmaf(u, (value(x[i]) - mean) * rstd, s[1]);
  }
  row_sum2<512>(s[0], s[1], scratch, turn);
  const float m1 = s[0] * a.inv_n, m2 = s[1] * a.inv_n;
  for (int64_t i = threadIdx.x; i < a.n; i += 512) {
    float w[1];
    load_param<1>(a.w, a.w_bf16, i, 1.f, w);
    const float h = (value(x[i]) - mean) * rstd;
    dx[i] = narrow<X>(rstd * (fmaf(value(g[i]), w[0], -m1) - h * m2));
  }
}
// ... and the column sums from a pass of their own: CTA (c, p) adds its 256 columns over
// every gridDim.y-th row.
template <typename X>
__global__ void __launch_bounds__(256) norm_columns_kernel(const NormGradK a) {
  let_next();
  after_previous();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= a.n) return;
  float dw = 0.f, db = 0.f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float d = value(static_cast<const X*>(a.g)[row * a.n + i]);
    const float h = (value(static_cast<const X*>(a.x)[row * a.n + i]) - a.mean[row]) * a.rstd[row];
    dw = fmaf(d, h, dw);
    db += d;
  }
  float* out = a.part + static_cast<int64_t>(blockIdx.y) * 2 * a.n;
  out[i] = dw;
  out[a.n + i] = db;
}

// out[c] = sum over parts, in order, of part[p][c], c < n; a second output takes columns
// n .. 2n-1. 32 columns a CTA; warp k adds every kSumWarps-th part from k, 20 loads at a time, then the
// warps' sums.
constexpr int kSumLoads = 20;
template <int kSumWarps>
__global__ void __launch_bounds__(kSumWarps * 32)
column_sum_kernel(const float* part, int64_t parts, int64_t width, int64_t n, void* o1, void* o2,
                  int bf16) {
  let_next();
  after_previous();
  __shared__ float s[kSumWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float v = 0.f;
  if (c < width) {
    for (int64_t p = warp; p < parts; p += kSumWarps * kSumLoads) {
      const float* from = part + p * width + c;
      float u[kSumLoads];
#pragma unroll
      for (int k = 0; k < kSumLoads; ++k) {
        u[k] = p + k * kSumWarps < parts ? fetch(from) : 0.f;
        from += kSumWarps * width;
      }
#pragma unroll
      for (int k = 0; k < kSumLoads; ++k) v += u[k];
    }
  }
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < width) {
    v = 0.f;
#pragma unroll
    for (int k = 0; k < kSumWarps; ++k) v += s[k][lane];
    void* o = c < n ? o1 : o2;
    const int64_t i = c < n ? c : c - n;
    if (o != nullptr) {
      if (bf16) static_cast<__nv_bfloat16*>(o)[i] = __float2bfloat16_rn(v);
      else static_cast<float*>(o)[i] = v;
    }
  }
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <typename X, int T, int V, int NV, bool kAny>
cudaError_t run_norm(const NormArgsK& a, cudaStream_t stream) {
  constexpr int kRows = cta_threads(T) / T;
  const int64_t ctas = (a.rows + kRows - 1) / kRows;
  if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(ctas));
  if constexpr (V > 1) return launch_overlapped(norm_pairs_kernel<X, T, NV, kAny>, grid, cta_threads(T), 0, 0, stream, a);
  else return launch_overlapped(norm_kernel<X, T, V, NV>, grid, cta_threads(T), 0, 0, stream, a);
}

// The threads of a row by its number of packs: as few as 8 packs a thread allow, so that many rows
// are at work on an SM and few barriers join them (32768 x 4096 bf16: 81 us with 64 threads a
// row, 84 with 128, 102 with 256; 16384 x 8192: 81 with 128, 88 with 256); eight lanes for short rows
// (60000 x 63 bf16: 9.7 us, 17.0 with a warp a row).
template <typename X, int V, bool kAny>
cudaError_t norm_by_length(const NormArgsK& a, cudaStream_t stream) {
  const int64_t packs = (a.n + V - 1) / V;
  if constexpr (V > 1) {
    if (packs <= 8) return run_norm<X, 8, V, 1, kAny>(a, stream);
    if (packs <= 16) return run_norm<X, 8, V, 2, kAny>(a, stream);
    if (packs <= 32) return run_norm<X, 8, V, 4, kAny>(a, stream);
  } else {
    if (packs <= 32) return run_norm<X, 32, V, 1, kAny>(a, stream);
  }
  if (packs <= 64) return run_norm<X, 32, V, 2, kAny>(a, stream);
  if (packs <= 128) return run_norm<X, 32, V, 4, kAny>(a, stream);
  if (packs <= 256) return run_norm<X, 32, V, 8, kAny>(a, stream);
  if (packs <= 512) return run_norm<X, 64, V, 8, kAny>(a, stream);
  if (packs <= 1024) return run_norm<X, 128, V, 8, kAny>(a, stream);
  if (packs <= 2048) return run_norm<X, 256, V, 8, kAny>(a, stream);
  if (packs <= 4096) return run_norm<X, 512, V, 8, kAny>(a, stream);
  if (a.rows > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  return launch_overlapped(norm_long_kernel<X>, dim3(static_cast<unsigned>(a.rows)), 512, 0, 0, stream, a);
}

template <typename X>
cudaError_t norm_typed(const NormArgsK& a, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(X);
  if (!aligned16(a.w) || !aligned16(a.b)) return norm_by_length<X, 1, false>(a, stream);
  if (a.n % V == 0 && aligned16(a.x) && aligned16(a.y)) return norm_by_length<X, V, false>(a, stream);
  // Rows that start anywhere. In packs their loads are fewer, but each is shifted into place, and how many of a
  // thread's packs a length fills matters; single elements run out of registers at 4096 and read a longer row
  // three times. 40 M elements, packs and single elements, us: fp32 127 69 82, 129 153 81, 255 87 48, 257
  // 114 158, 511 69 81, 513 106 82, 4097 127 79, 8191 80 74, 12289 79 78, 16383 69 82; bf16 127 73 81, 129 94 81,
  // 255 57 43, 257 117 158, 511 70 81, 513 91 81, 4097 86 75, 6001 66 80, 8191 55 62, 8193 86 58, 12289 70 57,
  // 16383 60 64.
  const int64_t n = a.n;
  const bool packs = n <= 128 || (n > 256 && n <= 512) || n > 14000 || (sizeof(X) == 2 && n > 5000 && n <= 8192);
  return packs ? norm_by_length<X, V, true>(a, stream) : norm_by_length<X, 1, false>(a, stream);
}

// Partial rows of the column sums: at most this many CTAs walk the rows.
constexpr int64_t kMaxParts = 152 * 4;

template <typename X, int T, int V, int NV>
cudaError_t run_norm_grad(const NormGradK& a, int64_t parts, cudaStream_t stream) {
  const size_t smem = T == 32 ? sizeof(float) * 2 * (grad_threads(T) / T) * a.n : 0;
  static SmemRecord record;
  const cudaError_t err = ensure_dynamic_smem(reinterpret_cast<const void*>(norm_grad_kernel<X, T, V, NV>), smem, record);
  if (err != cudaSuccess) return err;
  return launch_overlapped(norm_grad_kernel<X, T, V, NV>, dim3(static_cast<unsigned>(parts)), grad_threads(T), 0, smem,
                           stream, a);
}

template <typename X, int T, int NV>
cudaError_t run_norm_grad_ring(const NormGradK& a, int64_t parts, cudaStream_t stream) {
  // Two rows at work and up to four on their way, in an SM's 192 KB for 512 threads.
  constexpr size_t kRow = 2 * NV * T * sizeof(uint4), kRoom = 384 * T;
  constexpr int kDepth = kRow * 6 <= kRoom ? 6 : kRow * 5 <= kRoom ? 5 : kRow * 4 <= kRoom ? 4 : 3;
  constexpr size_t kSmem = kRow * kDepth;
  static SmemRecord record;
  const cudaError_t err =
      ensure_dynamic_smem(reinterpret_cast<const void*>(norm_grad_ring_kernel<X, T, NV>), kSmem, record);
  if (err != cudaSuccess) return err;
  return launch_overlapped(norm_grad_ring_kernel<X, T, NV>, dim3(static_cast<unsigned>(parts)), T, 0, kSmem, stream, a,
                           kDepth);
}

template <typename X, int V>
cudaError_t norm_grad_by_length(const NormGradK& a, int64_t* parts, cudaStream_t stream) {
  // Elements of a thread: each takes three fp32 registers (weight and both sums) besides the rows
  // at work. 16 with 16-byte loads; 8 with single ones, for more loads in flight an SM.
  constexpr int kNv = V > 1 ? 16 / V : 8;
  auto ctas = [&](int t, int64_t an_sm) {  // as many as are resident at once
    const int64_t rows = grad_threads(t) / t;
    return std::max<int64_t>(1, std::min<int64_t>(152 * an_sm, (a.rows + rows - 1) / rows));
  };
  const int64_t per = kNv * V;
  if (a.n <= 32 * per) {
    if constexpr (V == 1) {
      if (a.n <= 64) { *parts = ctas(32, 2); return run_norm_grad<X, 32, V, 2>(a, *parts, stream); }
    }
    if (a.n <= 32 * per / 2) {
      *parts = ctas(32, per <= 8 ? 2 : 1);
      return run_norm_grad<X, 32, V, kNv / 2>(a, *parts, stream);
    }
    *parts = ctas(32, 1);
    return run_norm_grad<X, 32, V, kNv>(a, *parts, stream);
  }
  if constexpr (V > 1) {
    if (a.n <= 64 * per) { *parts = ctas(128, 4); return run_norm_grad_ring<X, 128, kNv / 2>(a, *parts, stream); }
    if (a.n <= 128 * per) { *parts = ctas(128, 4); return run_norm_grad_ring<X, 128, kNv>(a, *parts, stream); }
    if (a.n <= 256 * per) { *parts = ctas(256, 2); return run_norm_grad_ring<X, 256, kNv>(a, *parts, stream); }
    if (a.n <= 512 * per) { *parts = ctas(512, 1); return run_norm_grad_ring<X, 512, kNv>(a, *parts, stream); }
  } else {
    if (a.n <= 128 * per) { *parts = ctas(128, 4); return run_norm_grad<X, 128, V, kNv>(a, *parts, stream); }
    if (a.n <= 256 * per) { *parts = ctas(256, 2); return run_norm_grad<X, 256, V, kNv>(a, *parts, stream); }
    if (a.n <= 512 * per) { *parts = ctas(512, 1); return run_norm_grad<X, 512, V, kNv>(a, *parts, stream); }
    if (a.n <= 512 * 16) { *parts = ctas(512, 1); return run_norm_grad<X, 512, V, 16>(a, *parts, stream); }
  }
  if (a.rows > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  cudaError_t err = launch_overlapped(norm_grad_long_kernel<X>, dim3(static_cast<unsigned>(a.rows)), 512, 0, 0, stream, a);
  if (err != cudaSuccess || a.part == nullptr) return err;
  const int64_t tiles = (a.n + 255) / 256;
  *parts = std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(a.rows, kMaxParts), 4 * 152 / tiles));
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(*parts));
  return launch_overlapped(norm_columns_kernel<X>, grid, 256, 0, 0, stream, a);
}

template <typename X>
cudaError_t norm_grad_typed(const NormGradK& a, int64_t* parts, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(X);
  const bool vec = a.n % V == 0 && aligned16(a.g) && aligned16(a.x) && aligned16(a.dx) && aligned16(a.w);
  return vec ? norm_grad_by_length<X, V>(a, parts, stream) : norm_grad_by_length<X, 1>(a, parts, stream);
}

}  // namespace

cudaError_t launch_layer_norm(const NormArgs& a, cudaStream_t stream) {
  NormArgsK k;
  k.x = a.x; k.w = a.w; k.b = a.b; k.y = a.y; k.mean = a.mean; k.rstd = a.rstd;
  k.rows = a.rows; k.n = a.n; k.eps = a.eps;
  k.inv_n = static_cast<float>(1.0 / static_cast<double>(a.n));
  k.w_bf16 = a.w_dt == VN_BF16;
  return a.dt == VN_BF16 ? norm_typed<__nv_bfloat16>(k, stream) : norm_typed<float>(k, stream);
}

int64_t layer_norm_parts(int64_t rows) { return std::max<int64_t>(1, std::min(rows, kMaxParts)); }

cudaError_t launch_column_sum(const float* part, int64_t parts, int64_t width, int64_t n, void* o1, void* o2,
                                 vn_dtype dt, cudaStream_t stream) {
  const int64_t grid = (width + 31) / 32;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  // 32 warps take all of 608 parts in one round of loads (layer norm's gradients of 4096 x 640 bf16: 12.3 us
  // for 16.5 with 16); with more CTAs than the SMs begin at once, 16 are faster (8192 x 1536: 19.8 for 26.5).
  auto* const fn = grid <= 76 ? column_sum_kernel<32> : column_sum_kernel<16>;
  return launch_overlapped(fn, dim3(static_cast<unsigned>(grid)), grid <= 76 ? 1024 : 512, 0, 0, stream, part, parts,
                           width, n, o1, o2, dt == VN_BF16);
}

cudaError_t launch_layer_norm_backward(const NormGradArgs& a, cudaStream_t stream) {
  NormGradK k;
  k.g = a.grad; k.x = a.x; k.mean = a.mean; k.rstd = a.rstd; k.w = a.w; k.dx = a.grad_x;
  k.part = (a.grad_w != nullptr || a.grad_b != nullptr) ? a.part : nullptr;
  k.rows = a.rows; k.n = a.n;
  k.inv_n = static_cast<float>(1.0 / static_cast<double>(a.n));
  k.w_bf16 = a.w_dt == VN_BF16;
  int64_t parts = 0;
  if (a.rows > 0) {
    const cudaError_t err = a.dt == VN_BF16 ? norm_grad_typed<__nv_bfloat16>(k, &parts, stream)
                                            : norm_grad_typed<float>(k, &parts, stream);
    if (err != cudaSuccess) return err;
  }
  if (k.part == nullptr) return cudaSuccess;
  return launch_column_sum(k.part, parts, 2 * a.n, a.n, a.grad_w, a.grad_b, a.w_dt, stream);
}

}  // namespace vn
