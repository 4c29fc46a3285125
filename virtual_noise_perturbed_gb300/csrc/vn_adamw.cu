// vn_adamw.cu -- the AdamW step over many tensors in one launch, with moments in 32
// bits or in 8, and the reading-out of 8-bit moments.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Every element is read and written once, so the bound is memory: p, m and v both ways
// and g once. A warp owns a block of 256 consecutive elements of one tensor (also the
// block that shares a scale), a lane two groups of four: loads of 16 bytes in fp32, 8 in
// bf16 and 4 in e4m3, all of them issued before the first use. The tensors' addresses
// travel in the kernel's parameters, so a step needs no table in device memory and no copy;
// a CTA finds its tensor by bisecting the table's first chunks.
//
// 8-bit moments: m as e4m3 codes in units of max|m| / 448 of its block, v as the same of
// sqrt(v) -- e4m3's 2^-9..448 then spans 36 binary orders of v -- and a positive root
// never becomes code 0: as a denominator it would turn the next step into m / eps.
// The maxima are integer maxima of the magnitudes' bits, so that a NaN or infinity wins
// and reaches its block's scale. Every operation on the way to a code is a single rounding
// (no contraction), which makes the stored codes a function of the formulas alone.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "vn_internal.h"

namespace vn {
namespace {

constexpr int kBlock = 256;                // elements of a warp's block, and of a scale
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = kWarps * kBlock;    // elements of a CTA
constexpr float kTop = 448.f;              // largest finite e4m3 value
constexpr float kTiny = 1e-30f;            // blocks below this are stored as zeros

struct Entry {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  int64_t n;
  int64_t first;  // first chunk of this tensor within the launch
  float keep;     // 1 - lr * weight_decay
  int vec;        // every array takes a group of four elements in one access
};

template <int kCap>
struct Table {
  int count;
  float b1, c1, b2, c2;     // beta and 1 - beta
  float inv_root, eps;      // 1 / sqrt(1 - beta2^t), eps
  float size;               // lr / (1 - beta1^t)
  float sign;               // -1 to ascend
  Entry e[kCap];
};

template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&v)[4]);
template <>
__device__ __forceinline__ void load4<float>(const float* p, float (&v)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
template <>
__device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 a = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xFFFF0000u);
  v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xFFFF0000u);
}
__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float decode(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}
__device__ __forceinline__ void decode4(uint32_t c, float (&v)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c >> (16 * h)), __NV_E4M3);
    const float2 f = __half22float2(__half2(r));
    v[2 * h] = f.x;
    v[2 * h + 1] = f.y;
  }
}
__device__ __forceinline__ uint32_t encode4(const float (&v)[4]) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// The scale of a block whose largest magnitude has these bits, and the factor that takes
// values to its units.
__device__ __forceinline__ float block_scale(uint32_t top_bits, float* inv) {
  const float top = __uint_as_float(top_bits);
  const float scale = top < kTiny ? 0.f : __fmul_rn(top, 1.f / kTop);
  *inv = scale == 0.f ? 0.f : __fdiv_rn(1.f, scale);
  return scale;
}

// Two groups of four elements: lane l of a warp owns elements 4l..4l+3 and
// 128+4l..128+4l+3 of its block (kVec), or 32 j + l, j < 8 (any alignment, and the last
// block of a tensor).
template <typename P, typename G, bool k8, bool kVec, int kCap>
__device__ __forceinline__ void step_block(const Table<kCap>& t, const Entry& e, int64_t block, int lane) {
  const int64_t base = block * kBlock;
  P* p = static_cast<P*>(e.p) + base;
  const G* gp = static_cast<const G*>(e.g) + base;
  const int left = static_cast<int>(min(static_cast<int64_t>(kBlock), e.n - base));
  auto at = [&](int h, int q) { return kVec ? h * 128 + lane * 4 + q : (h * 4 + q) * 32 + lane; };
  float pv[2][4], gv[2][4], mv[2][4], vv[2][4];
  uint32_t mc[2], vc[2];
  float ms = 0.f, vs = 0.f;
  if constexpr (k8) {
    ms = e.ms[block];
    vs = e.vs[block];
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (kVec) {
      load4<P>(p + at(h, 0), pv[h]);
      load4<G>(gp + at(h, 0), gv[h]);
      if constexpr (k8) {
        mc[h] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(e.m) + base + at(h, 0));
        vc[h] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(e.v) + base + at(h, 0));
      } else {
        load4<float>(static_cast<const float*>(e.m) + base + at(h, 0), mv[h]);
        load4<float>(static_cast<const float*>(e.v) + base + at(h, 0), vv[h]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bool in = at(h, q) < left;
        pv[h][q] = in ? value(p[at(h, q)]) : 0.f;
        gv[h][q] = in ? value(gp[at(h, q)]) : 0.f;
        if constexpr (k8) {
          mv[h][q] = in ? decode(static_cast<const uint8_t*>(e.m)[base + at(h, q)]) : 0.f;
          vv[h][q] = in ? decode(static_cast<const uint8_t*>(e.v)[base + at(h, q)]) : 0.f;
        } else {
          mv[h][q] = in ? static_cast<const float*>(e.m)[base + at(h, q)] : 0.f;
          vv[h][q] = in ? static_cast<const float*>(e.v)[base + at(h, q)] : 0.f;
        }
      }
    }
  }
  uint32_t mtop = 0, rtop = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (k8 && kVec) {
      decode4(mc[h], mv[h]);
      decode4(vc[h], vv[h]);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (k8) {
        mv[h][q] = __fmul_rn(mv[h][q], ms);
        vv[h][q] = __fmul_rn(vv[h][q], vs);
        vv[h][q] = __fmul_rn(vv[h][q], vv[h][q]);
      }
      const float g = gv[h][q] * t.sign;
      const float m = __fadd_rn(__fmul_rn(mv[h][q], t.b1), __fmul_rn(g, t.c1));
      const float v = __fadd_rn(__fmul_rn(vv[h][q], t.b2), __fmul_rn(__fmul_rn(g, g), t.c2));
      const float root = __fsqrt_rn(v);
      const float move = __fmul_rn(__fdividef(m, fmaf(root, t.inv_root, t.eps)), t.size);
      pv[h][q] = fmaf(pv[h][q], e.keep, -move);
      mv[h][q] = m;
      vv[h][q] = k8 ? root : v;
      if constexpr (k8) {
        mtop = max(mtop, __float_as_uint(m) & 0x7FFFFFFFu);
        rtop = max(rtop, __float_as_uint(root) & 0x7FFFFFFFu);
      }
    }
  }
  if constexpr (k8) {
    mtop = __reduce_max_sync(0xFFFFFFFFu, mtop);
    rtop = __reduce_max_sync(0xFFFFFFFFu, rtop);
    float minv, rinv;
    ms = block_scale(mtop, &minv);
    vs = block_scale(rtop, &rinv);
    if (lane == 0) {
      e.ms[block] = ms;
      e.vs[block] = vs;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mq[4], rq[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        mq[q] = __fmul_rn(mv[h][q], minv);  // a block stored as zeros has factor 0
        rq[q] = __fmul_rn(vv[h][q], rinv);
        // A positive root takes code 1, 2^-9, at least (a NaN stays one).
        const float least = max_nan(rq[q], 0x1p-9f);
        rq[q] = vv[h][q] > 0.f && vs > 0.f ? least : rq[q];
      }
      const uint32_t mo = encode4(mq);
      const uint32_t ro = encode4(rq);
      uint8_t* mp = static_cast<uint8_t*>(e.m) + base;
      uint8_t* vp = static_cast<uint8_t*>(e.v) + base;
      if constexpr (kVec) {
        *reinterpret_cast<uint32_t*>(mp + at(h, 0)) = mo;
        *reinterpret_cast<uint32_t*>(vp + at(h, 0)) = ro;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (at(h, q) < left) {
            mp[at(h, q)] = static_cast<uint8_t>(mo >> (8 * q));
            vp[at(h, q)] = static_cast<uint8_t>(ro >> (8 * q));
          }
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float* mp = static_cast<float*>(e.m) + base;
    float* vp = static_cast<float*>(e.v) + base;
    if constexpr (kVec) {
      store4(p + at(h, 0), pv[h]);
      if constexpr (!k8) {
        store4(mp + at(h, 0), mv[h]);
        store4(vp + at(h, 0), vv[h]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (at(h, q) < left) {
          store1(p + at(h, q), pv[h][q]);
          if constexpr (!k8) {
            mp[at(h, q)] = mv[h][q];
            vp[at(h, q)] = vv[h][q];
          }
        }
    }
  }
}

template <typename P, typename G, bool k8, int kCap>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Table<kCap> t) {
  const int64_t chunk = blockIdx.x;
  int lo = 0, hi = t.count;  // the last entry whose first chunk is not beyond this one
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.e[mid].first <= chunk) lo = mid; else hi = mid;
  }
  const Entry& e = t.e[lo];
  const int64_t block = (chunk - e.first) * kWarps + (threadIdx.x >> 5);
  if (block * kBlock >= e.n) return;
  const int lane = threadIdx.x & 31;
  if (e.vec && (block + 1) * kBlock <= e.n)
    step_block<P, G, k8, true>(t, e, block, lane);
  else
    step_block<P, G, k8, false>(t, e, block, lane);
}

__global__ void __launch_bounds__(kThreads)
moments_kernel(const uint8_t* __restrict__ mc, const uint8_t* __restrict__ vc, const float* __restrict__ ms,
               const float* __restrict__ vs, int64_t n, float* __restrict__ m, float* __restrict__ v, int vec) {
  const int64_t block = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t base = block * kBlock;
  if (base >= n) return;
  const int lane = threadIdx.x & 31;
  const float a = ms[block], r = vs[block];
  if (vec && base + kBlock <= n) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t i = base + h * 128 + lane * 4;
      float mv[4], vv[4];
      decode4(*reinterpret_cast<const uint32_t*>(mc + i), mv);
      decode4(*reinterpret_cast<const uint32_t*>(vc + i), vv);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        mv[q] = __fmul_rn(mv[q], a);
        vv[q] = __fmul_rn(vv[q], r);
        vv[q] = __fmul_rn(vv[q], vv[q]);
      }
      store4(m + i, mv);
      store4(v + i, vv);
    }
  } else {
    for (int64_t i = base + lane; i < min(n, base + kBlock); i += 32) {
      m[i] = __fmul_rn(decode(mc[i]), a);
      const float q = __fmul_rn(decode(vc[i]), r);
      v[i] = __fmul_rn(q, q);
    }
  }
}

template <typename P, typename G, bool k8, int kCap>
cudaError_t launch_table(const AdamwArgs& a, int64_t from, int64_t count, cudaStream_t stream) {
  Table<kCap> t;
  t.count = 0;
  t.b1 = static_cast<float>(a.beta1); t.c1 = static_cast<float>(1.0 - a.beta1);
  t.b2 = static_cast<float>(a.beta2); t.c2 = static_cast<float>(1.0 - a.beta2);
  const double s = static_cast<double>(a.step);
  t.inv_root = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(a.beta2, s)));
  t.eps = static_cast<float>(a.eps);
  t.size = static_cast<float>(a.lr / (1.0 - std::pow(a.beta1, s)));
  t.sign = a.maximize ? -1.f : 1.f;
  int64_t chunks = 0;
  auto fits = [](const void* q, size_t bytes) { return reinterpret_cast<uintptr_t>(q) % bytes == 0; };
  for (int64_t i = from; i < from + count; ++i) {
    const vn_adamw_tensor& x = a.tensors[i];
    if (x.n == 0) continue;
    Entry& e = t.e[t.count++];
    e.p = x.param; e.g = x.grad; e.m = x.exp_avg; e.v = x.exp_avg_sq;
    e.ms = x.exp_avg_scale; e.vs = x.exp_avg_sq_scale;
    e.n = x.n;
    e.first = chunks;
    e.keep = static_cast<float>(1.0 - a.lr * x.weight_decay);
    const size_t state = k8 ? 4 : 16;
    e.vec = fits(x.param, 4 * sizeof(P)) && fits(x.grad, 4 * sizeof(G)) && fits(x.exp_avg, state) &&
            fits(x.exp_avg_sq, state);
    chunks += (x.n + kChunk - 1) / kChunk;
  }
  if (chunks == 0) return cudaSuccess;
  if (chunks > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  adamw_kernel<P, G, k8, kCap><<<static_cast<unsigned>(chunks), kThreads, 0, stream>>>(t);
  return cudaGetLastError();
}

// Tensors per launch: the table's 64 bytes a tensor must fit the 32,764 bytes of a kernel's
// parameters. The small table serves calls of a few tensors (their parameters are copied
// at every launch).
constexpr int kSmall = 16, kLarge = 448;
static_assert(sizeof(Table<kLarge>) <= 32764, "kernel parameters");

template <typename P, typename G, bool k8>
cudaError_t launch_typed(const AdamwArgs& a, cudaStream_t stream) {
  for (int64_t from = 0; from < a.count; from += kLarge) {
    const int64_t count = std::min<int64_t>(kLarge, a.count - from);
    const cudaError_t err = count <= kSmall ? launch_table<P, G, k8, kSmall>(a, from, count, stream)
                                            : launch_table<P, G, k8, kLarge>(a, from, count, stream);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

template <typename P, typename G>
cudaError_t launch_bits(const AdamwArgs& a, cudaStream_t stream) {
  return a.state_bits == 8 ? launch_typed<P, G, true>(a, stream) : launch_typed<P, G, false>(a, stream);
}

}  // namespace

cudaError_t launch_adamw(const AdamwArgs& a, cudaStream_t stream) {
  if (a.param_dt == VN_BF16)
    return a.grad_dt == VN_BF16 ? launch_bits<__nv_bfloat16, __nv_bfloat16>(a, stream)
                                : launch_bits<__nv_bfloat16, float>(a, stream);
  return a.grad_dt == VN_BF16 ? launch_bits<float, __nv_bfloat16>(a, stream)
                              : launch_bits<float, float>(a, stream);
}

cudaError_t launch_adamw_moments(const void* mc, const void* vc, const float* ms, const float* vs, int64_t n,
                                 float* m, float* v, cudaStream_t stream) {
  const int64_t grid = (n + kChunk - 1) / kChunk;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  auto fits = [](const void* q, size_t bytes) { return reinterpret_cast<uintptr_t>(q) % bytes == 0; };
  const int vec = fits(mc, 4) && fits(vc, 4) && fits(m, 16) && fits(v, 16);
  moments_kernel<<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(
      static_cast<const uint8_t*>(mc), static_cast<const uint8_t*>(vc), ms, vs, n, m, v, vec);
  return cudaGetLastError();
}

}  // namespace vn
