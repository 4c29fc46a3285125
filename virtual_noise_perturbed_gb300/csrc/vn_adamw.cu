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
#include "vn_launch.cuh"
#include "vn_pair.cuh"

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
  float b1, c1, b2, c2;     // beta and 1 - beta; c1 negative to ascend
  float inv_root, eps;      // 1 / sqrt(1 - beta2^t), eps
  float size;               // -lr / (1 - beta1^t)
  Entry e[kCap];
};

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

// Four elements as they are in memory.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float4 v;
  __device__ __forceinline__ void get(F2 (&o)[2]) const { o[0] = f2(v.x, v.y); o[1] = f2(v.z, v.w); }
};
template <>
struct Raw<__nv_bfloat16> {
  uint2 v;
  __device__ __forceinline__ void get(F2 (&o)[2]) const {
    o[0] = f2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u));
    o[1] = f2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
  }
};
struct Codes {
  uint32_t v;
  __device__ __forceinline__ void get(F2 (&o)[2]) const {
    float f[4];
    decode4(v, f);
    o[0] = f2(f[0], f[1]);
    o[1] = f2(f[2], f[3]);
  }
};
// Elements 32 apart, the first from p; those at or beyond `left` are zeros.
__device__ __forceinline__ void gather(const float* p, int at, int left, Raw<float>* r) {
  float v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = at + q * 32 < left ? p[at + q * 32] : 0.f;
  r->v = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void gather(const __nv_bfloat16* p, int at, int left, Raw<__nv_bfloat16>* r) {
  uint32_t v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    v[q] = at + q * 32 < left ? static_cast<uint32_t>(__bfloat16_as_ushort(p[at + q * 32])) : 0u;
  r->v = make_uint2(v[0] | (v[1] << 16), v[2] | (v[3] << 16));
}
__device__ __forceinline__ void gather(const uint8_t* p, int at, int left, Codes* r) {
  uint32_t v = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) v |= at + q * 32 < left ? static_cast<uint32_t>(p[at + q * 32]) << (8 * q) : 0u;
  r->v = v;
}
template <bool k8>
struct Moment {
  using Element = float;
  using Four = Raw<float>;
};
template <>
struct Moment<true> {
  using Element = uint8_t;
  using Four = Codes;
};

// A warp's block: lane l owns two groups of four elements, 4l..4l+3 and 128+4l..128+4l+3
// (kVec), or the elements l, l + 32, .. (any alignment, and the last block of a tensor). The
// operands stay as they were loaded until their group's turn, in few registers: what is in
// flight per SM is what bounds this kernel.
template <typename P, typename G, bool k8, bool kVec, int kCap>
__device__ __forceinline__ void step_block(const Table<kCap>& t, const Entry& e, int64_t block, int lane) {
  using M = typename Moment<k8>::Element;
  using Four = typename Moment<k8>::Four;
  const int64_t base = block * kBlock;
  P* p = static_cast<P*>(e.p) + base;
  const G* gp = static_cast<const G*>(e.g) + base;
  M* mp = static_cast<M*>(e.m) + base;
  M* vp = static_cast<M*>(e.v) + base;
  const int left = static_cast<int>(min(static_cast<int64_t>(kBlock), e.n - base));
  Raw<P> rp[2];
  Raw<G> rg[2];
  Four rm[2], rv[2];
  float ms = 0.f, vs = 0.f;
  if constexpr (k8) {
    ms = e.ms[block];
    vs = e.vs[block];
  }
  auto at = [&](int h) { return kVec ? h * 128 + lane * 4 : h * 128 + lane; };
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (kVec) {
      rp[h] = *reinterpret_cast<const Raw<P>*>(p + at(h));
      rg[h] = *reinterpret_cast<const Raw<G>*>(gp + at(h));
      rm[h] = *reinterpret_cast<const Four*>(mp + at(h));
      rv[h] = *reinterpret_cast<const Four*>(vp + at(h));
    } else {
      gather(p, at(h), left, &rp[h]);
      gather(gp, at(h), left, &rg[h]);
      gather(mp, at(h), left, &rm[h]);
      gather(vp, at(h), left, &rv[h]);
    }
  }
  float m[2][4], r[2][4];  // the new moments; of 8-bit ones the root of the second
  float mtop = 0.f, rtop = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    F2 pv[2], gv[2], mv[2], vv[2];
    rp[h].get(pv);
    rg[h].get(gv);
    rm[h].get(mv);
    rv[h].get(vv);
    float np[4];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if constexpr (k8) {
        mv[q] = mul2(mv[q], f2(ms, ms));
        vv[q] = mul2(vv[q], f2(vs, vs));
        vv[q] = mul2(vv[q], vv[q]);
      }
      // The sums as single instructions: two-lane ones the compiler contracts with the products.
      float v0, v1, d0, d1, a0, a1;
      split(mul2(mv[q], f2(t.b1, t.b1)), &v0, &v1);
      split(mul2(gv[q], f2(t.c1, t.c1)), &a0, &a1);
      m[h][2 * q] = __fadd_rn(v0, a0);
      m[h][2 * q + 1] = __fadd_rn(v1, a1);
      split(mul2(vv[q], f2(t.b2, t.b2)), &v0, &v1);
      split(mul2(mul2(gv[q], gv[q]), f2(t.c2, t.c2)), &a0, &a1);
      v0 = __fadd_rn(v0, a0);
      v1 = __fadd_rn(v1, a1);
      const float r0 = __fsqrt_rn(v0), r1 = __fsqrt_rn(v1);
      split(fma2(f2(r0, r1), f2(t.inv_root, t.inv_root), f2(t.eps, t.eps)), &d0, &d1);
      const F2 move = mul2(f2(__fdividef(m[h][2 * q], d0), __fdividef(m[h][2 * q + 1], d1)), f2(t.size, t.size));
      split(fma2(pv[q], f2(e.keep, e.keep), move), &np[2 * q], &np[2 * q + 1]);
      r[h][2 * q] = k8 ? r0 : v0;
      r[h][2 * q + 1] = k8 ? r1 : v1;
      if constexpr (k8) {
        mtop = max_nan(mtop, max_nan(fabsf(m[h][2 * q]), fabsf(m[h][2 * q + 1])));
        rtop = max_nan(rtop, max_nan(r0, r1));
      }
    }
    if constexpr (kVec) {
      store4(p + at(h), np);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (at(h) + q * 32 < left) store1(p + at(h) + q * 32, np[q]);
    }
    if constexpr (!k8) {
      if constexpr (kVec) {
        store4(mp + at(h), m[h]);
        store4(vp + at(h), r[h]);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (at(h) + q * 32 < left) {
            mp[at(h) + q * 32] = m[h][q];
            vp[at(h) + q * 32] = r[h][q];
          }
      }
    }
  }
  if constexpr (k8) {
    // A NaN's bits, without its sign, are above every number's.
    const uint32_t mbits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(mtop) & 0x7FFFFFFFu);
    const uint32_t rbits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(rtop) & 0x7FFFFFFFu);
    float minv, rinv;
    ms = block_scale(mbits, &minv);
    vs = block_scale(rbits, &rinv);
    if (lane == 0) {
      e.ms[block] = ms;
      e.vs[block] = vs;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mq[4], rq[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        mq[q] = __fmul_rn(m[h][q], minv);  // a block stored as zeros has factor 0
        rq[q] = __fmul_rn(r[h][q], rinv);
        // A positive root takes code 1, 2^-9, at least (a NaN stays one).
        const float least = max_nan(rq[q], 0x1p-9f);
        rq[q] = r[h][q] > 0.f && vs > 0.f ? least : rq[q];
      }
      const uint32_t mo = encode4(mq), ro = encode4(rq);
      if constexpr (kVec) {
        *reinterpret_cast<uint32_t*>(mp + at(h)) = mo;
        *reinterpret_cast<uint32_t*>(vp + at(h)) = ro;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (at(h) + q * 32 < left) {
            mp[at(h) + q * 32] = static_cast<uint8_t>(mo >> (8 * q));
            vp[at(h) + q * 32] = static_cast<uint8_t>(ro >> (8 * q));
          }
      }
    }
  }
}

// Five CTAs an SM: 105 us on 54.5 M parameters with 8 bits, 114 us with the four that 56
// registers leave, 111 us with six.
template <typename P, typename G, bool k8, int kCap>
__global__ void __launch_bounds__(kThreads, 5) adamw_kernel(const __grid_constant__ Table<kCap> t) {
  let_next();
  after_previous();
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
moments_kernel(const uint8_t* mc, const uint8_t* vc, const float* ms,
               const float* vs, int64_t n, float* m, float* v, int vec) {
  let_next();
  after_previous();
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
  t.b1 = static_cast<float>(a.beta1); t.c1 = static_cast<float>(a.maximize ? a.beta1 - 1.0 : 1.0 - a.beta1);
  t.b2 = static_cast<float>(a.beta2); t.c2 = static_cast<float>(1.0 - a.beta2);
  const double s = static_cast<double>(a.step);
  t.inv_root = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(a.beta2, s)));
  t.eps = static_cast<float>(a.eps);
  t.size = static_cast<float>(-a.lr / (1.0 - std::pow(a.beta1, s)));
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
  const dim3 grid(static_cast<unsigned>(chunks));
  return launch_overlapped(adamw_kernel<P, G, k8, kCap>, grid, kThreads, 0, 0, stream, t);
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
  return launch_overlapped(moments_kernel, dim3(static_cast<unsigned>(grid)), kThreads, 0, 0, stream,
                           static_cast<const uint8_t*>(mc), static_cast<const uint8_t*>(vc), ms, vs, n, m, v, vec);
}

}  // namespace vn
