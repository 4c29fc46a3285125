// vn_clip.cu -- the norm of a gradient over many tensors, and the gradient scaled to a bound of it:
//
//   norm = sqrt(sum over all tensors of g^2),   factor = norm <= bound ? 1 : bound / norm,   out = g factor
//
// The norm reads every element once and the scaling reads and writes it, so the bound is memory (the
// second reading comes from L2 where the gradient fits there). Sums: squares and their sums in pairs of fp32 of which the second
// carries what the first rounds off, its own roundings below 2^-37; the warps' and the CTAs' in 64 bits, in a fixed order:
// results do not depend on the order of CTAs, and the norm is the exact one rounded once but where that falls within 2^-36
// of a border. Eight squares whose sum leaves what fp32 holds to full precision are taken in 64 bits, so the norm is
// right over the whole range of the types (fp64 has 1/64 of fp32's rate here: no other element sees it).
// The norm of 805 MB fp32 takes 117 us, 6.9 TB/s; 109 MB of bf16 20 us and, scaled to other buffers, 47 (three launches: squares,
// their join, scaling); a policy's 0.3 MB 4.5 of the GPU in one launch, and 6.3 with the call on the host.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "vn_internal.h"
#include "vn_launch.cuh"
#include "vn_pair.cuh"

namespace cg = cooperative_groups;

namespace vn {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 8;                      // elements that are squared and summed in fp32
constexpr int kLoads = 4;                      // 16-byte loads of a thread in flight
template <typename T>
constexpr int kChunkOf = kThreads * kLoads * 16 / static_cast<int>(sizeof(T));  // elements of a CTA's turn
constexpr int kPerSm = 6;                      // CTAs an SM that sum squares: 805 MB of fp32 127 us with 4, 117 with 6, 135 with 8
constexpr int kCluster = 16;                   // CTAs of the kernel for few chunks
// Up to here (1 MB) that kernel: clipping 8, 32 and 64 chunks takes 3.3, 3.8 and 5.0 us of the device for 4.6, 5.1 and 5.6
// of the three launches, which cost 9 us of the host for 4 to 6; with 128 chunks 6.4 for 6.6.
constexpr int64_t kFewChunks = 64;
constexpr int kSmall = 16, kLarge = 896;       // tensors of a launch

struct Piece {
  const void* g;
  void* out;
  int64_t n;
  int64_t first;  // first chunk of this tensor within the launch
};
template <int kCap>
struct Table {
  int count;
  int64_t chunks;
  Piece e[kCap];
};
static_assert(sizeof(Table<kLarge>) + 64 <= 32764, "kernel parameters");

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// A sum of squares: fp32 in two lanes, what its additions round off, and what fp32 cannot hold. `hi` starts from `base`, a power of
// two above the squares to come. Then, with t = RN(hi + x^2) below 2 hi, t - hi has no rounding, and x^2 - (t - hi), a multiply-add good to
// 2^-24 of itself, is what t rounds off: four instructions for two elements. Where t is not below 2 hi, the base is raised.
struct Sum {
  F2 hi = 0, lo = 0;
  float base = 0.f;  // in each lane of hi
  double wide = 0.0;
  __device__ __forceinline__ void add(const float (&x)[kGroup]) {
    const F2 minus = f2(-1.f, -1.f);
#pragma unroll 1
    for (int turn = 0;; ++turn) {
      F2 t = hi, rest = 0;
#pragma unroll
      for (int q = 0; q < kGroup; q += 2) {
        const F2 v = f2(x[q], x[q + 1]), next = fma2(v, v, t), r = fma2(v, v, fma2(next, minus, t));
        rest = q == 0 ? r : add2(rest, r);
        t = next;
      }
      float a, b, c, d;
      split(t, &a, &b);
      split(hi, &c, &d);
      if (a < 2.f * c && b < 2.f * d && fmaxf(a, b) < kMost) {
        hi = t;
        lo = add2(lo, rest);
        return;
      }
      if (turn == 1 || !raise(x)) break;
    }
    wide += squares(x[0], x[1], x[2], x[3]) + squares(x[4], x[5], x[6], x[7]);
  }
  // A warp adds 64 lanes up. (A thread's squares that are below 2^100 by eights do not get there; ones that grow from eight to eight may.)
  static constexpr float kMost = 0x1p118f;
  // A base of four to eight times these squares' sum. Below 2^-76 the squares that fp32 cannot hold would count (they are below
  // 2^-149, however many); from 2^100 on `hi` could pass its largest value; a NaN is neither.
  __device__ __forceinline__ bool raise(const float (&x)[kGroup]) {
    F2 s = mul2(f2(x[0], x[1]), f2(x[0], x[1]));
#pragma unroll
    for (int q = 2; q < kGroup; q += 2) s = fma2(f2(x[q], x[q + 1]), f2(x[q], x[q + 1]), s);
    const float v = sum_of(s);
    if (!(v >= 0x1p-76f && v < 0x1p100f)) return false;
    const float up = __uint_as_float((__float_as_uint(v) & 0x7F800000u) + (3u << 23));
    if (up <= base) return false;  // it was kMost
    float a, b, c, d;
    split(hi, &a, &b);
    split(lo, &c, &d);
    c += plus(a, up) + plus(a, -base);
    d += plus(b, up) + plus(b, -base);
    hi = f2(a, b);
    lo = f2(c, d);
    base = up;
    return true;
  }
  // What `lo` has gathered, to `hi`: its own roundings stay below 2^-37 of the sum.
  __device__ __forceinline__ void settle() {
    const F2 minus = f2(-1.f, -1.f), t = add2(hi, lo);
    lo = add2(lo, fma2(t, minus, hi));
    hi = t;
  }
  // Out of line and by value: the sums of every other element stay in registers.
  static __device__ __noinline__ double squares(float a, float b, float c, float d) {
    if (a == 0.f && b == 0.f && c == 0.f && d == 0.f) return 0.0;
    const double x = a, y = b, z = c, w = d;
    return x * x + y * y + z * z + w * w;
  }
  // The sum over a warp, in lane 0: pairs of fp32 (below 2^124) whose additions are as exact, and 64 bits where a lane has them.
  __device__ __forceinline__ double warp_total() const {
    float h, l, o, c, d;
    split(hi, &h, &o);
    split(lo, &c, &d);
    l = (plus(h, -base) + plus(o, -base)) + (c + d);
    l += plus(h, o);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) {
      const float more = l + __shfl_xor_sync(0xFFFFFFFFu, l, i);
      l = plus(h, __shfl_xor_sync(0xFFFFFFFFu, h, i)) + more;
    }
    double w = 0.0;
    if (__any_sync(0xFFFFFFFFu, wide != 0.0)) {
      w = wide;
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) w += __shfl_xor_sync(0xFFFFFFFFu, w, i);
    }
    return static_cast<double>(h) + (static_cast<double>(l) + w);
  }
  // a += b, and what that rounds off.
  static __device__ __forceinline__ float plus(float& a, float b) {
    const float t = __fadd_rn(a, b), n = __fsub_rn(t, a);
    const float rest = __fadd_rn(__fsub_rn(a, __fsub_rn(t, n)), __fsub_rn(b, n));
    a = t;
    return rest;
  }
};

// The sum over a CTA's warps of what their lanes 0 have, in thread 0. (64 bits are 16 cycles an instruction and warp, so few take part:
// with every thread adding them up, and lanes in 64 bits too, the norm of 4 M elements in fp32 took 8.5 us for 6.8.)
__device__ __forceinline__ double cta_sum(double v) {
  __shared__ double s[kThreads / 32];
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = threadIdx.x < kThreads / 32 ? s[threadIdx.x] : 0.0;
#pragma unroll
    for (int o = kThreads / 64; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  }
  return v;
}

// What a launch reads per thread and 16 bytes.
template <typename T>
__device__ __forceinline__ void unpack(const uint4& raw, float* x) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      x[2 * q] = __uint_as_float(w[q] << 16);
      x[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = __uint_as_float(w[q]);
  }
}

template <int kCap>
__device__ __forceinline__ const Piece& piece_of(const Table<kCap>& t, int64_t chunk) {
  int lo = 0, hi = t.count;  // the last piece whose first chunk is not beyond this one
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.e[mid].first <= chunk) lo = mid; else hi = mid;
  }
  return t.e[lo];
}

// A chunk's elements one at a time, 256 apart: any alignment, and the last chunk of a tensor.
template <typename T, typename F>
__device__ __forceinline__ void each_single(const T* g, int64_t left, F f) {
  constexpr int kChunk = kChunkOf<T>;
  const int end = static_cast<int>(min(static_cast<int64_t>(kChunk), left));
  for (int i = threadIdx.x; i < end; i += kThreads * kGroup) {
    float x[kGroup];
#pragma unroll
    for (int q = 0; q < kGroup; ++q) x[q] = i + q * kThreads < end ? value(fetch(g + i + q * kThreads)) : 0.f;
    f(i, end, x);
  }
}

// The squares of one chunk.
template <typename T, int kCap>
__device__ __forceinline__ void square_chunk(const Table<kCap>& t, int64_t chunk, Sum& sum) {
  constexpr int kChunk = kChunkOf<T>;
  const Piece& e = piece_of(t, chunk);
  const int64_t base = (chunk - e.first) * kChunk;
  const T* g = static_cast<const T*>(e.g) + base;
  if (base + kChunk <= e.n && reinterpret_cast<uintptr_t>(g) % 16 == 0) {
    uint4 raw[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) raw[u] = fetch(reinterpret_cast<const uint4*>(g) + u * kThreads + threadIdx.x);
    constexpr int kPer = 16 / sizeof(T);
#pragma unroll
    for (int u = 0; u < kLoads; u += kGroup / kPer) {
      float x[kGroup];
#pragma unroll
      for (int k = 0; k < kGroup / kPer; ++k) unpack<T>(raw[u + k], x + k * kPer);
      sum.add(x);
    }
  } else {
    each_single(g, e.n - base, [&](int, int, const float(&x)[kGroup]) { sum.add(x); });
  }
  sum.settle();
}

// out = g f over one chunk.
template <typename T, int kCap>
__device__ __forceinline__ void scale_chunk(const Table<kCap>& t, int64_t chunk, float f) {
  constexpr int kChunk = kChunkOf<T>;
  const Piece& e = piece_of(t, chunk);
  if (f == 1.f && e.out == e.g) return;
  const int64_t base = (chunk - e.first) * kChunk;
  const T* g = static_cast<const T*>(e.g) + base;
  T* o = static_cast<T*>(e.out) + base;
  if (base + kChunk <= e.n && (reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(o)) % 16 == 0) {
    uint4 raw[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) raw[u] = fetch(reinterpret_cast<const uint4*>(g) + u * kThreads + threadIdx.x);
    constexpr int kPer = 16 / sizeof(T);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      float x[kPer];
      unpack<T>(raw[u], x);
      uint32_t w[4];
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(__fmul_rn(x[2 * q], f), __fmul_rn(x[2 * q + 1], f));
          w[q] = *reinterpret_cast<const uint32_t*>(&b);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = __float_as_uint(__fmul_rn(x[q], f));
      }
      __stcs(reinterpret_cast<uint4*>(o) + u * kThreads + threadIdx.x, make_uint4(w[0], w[1], w[2], w[3]));
    }
  } else {
    each_single(g, e.n - base, [&](int i, int end, const float(&x)[kGroup]) {
#pragma unroll
      for (int q = 0; q < kGroup; ++q)
        if (i + q * kThreads < end) put(o + i + q * kThreads, __fmul_rn(x[q], f));
    });
  }
}

__device__ __forceinline__ float factor_of(double norm, double bound) {
  return norm <= bound ? 1.f : static_cast<float>(bound / norm);
}

template <typename T, int kCap>
__global__ void __launch_bounds__(kThreads) square_kernel(const __grid_constant__ Table<kCap> t, double* parts) {
  let_next();
  after_previous();
  Sum sum;
  for (int64_t chunk = blockIdx.x; chunk < t.chunks; chunk += gridDim.x) square_chunk<T>(t, chunk, sum);
  const double total = cta_sum(sum.warp_total());
  if (threadIdx.x == 0) parts[blockIdx.x] = total;
}

// The parts of all launches to the norm and the factor: one CTA.
__global__ void __launch_bounds__(kThreads) join_kernel(const double* parts, int64_t count, double bound, float* norm, float* factor) {
  let_next();
  after_previous();
  double v = 0.0;
  for (int64_t i = threadIdx.x; i < count; i += kThreads) v += fetch(parts + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  v = cta_sum(v);
  if (threadIdx.x != 0) return;
  const double n = sqrt(v);
  *norm = static_cast<float>(n);
  *factor = factor_of(n, bound);
}

// A CTA a chunk, from the last one to the first: what the norm's launch read last is still in L2.
template <typename T, int kCap>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Table<kCap> t, const float* factor) {
  let_next();
  after_previous();
  scale_chunk<T>(t, t.chunks - 1 - blockIdx.x, fetch(factor));
}

// Few chunks: all of it in one cluster of CTAs, which add their sums over distributed shared memory.
template <typename T, int kCap>
__global__ void __launch_bounds__(kThreads)
few_kernel(const __grid_constant__ Table<kCap> t, double bound, float* norm, float* factor, int scale) {
  __shared__ double mine;
  __shared__ float shared_factor;
  cg::cluster_group cluster = cg::this_cluster();
  let_next();
  after_previous();
  Sum sum;
  for (int64_t chunk = blockIdx.x; chunk < t.chunks; chunk += kCluster) square_chunk<T>(t, chunk, sum);
  const double total = cta_sum(sum.warp_total());
  if (threadIdx.x == 0) mine = total;
  cluster.sync();
  double parts = 0.0;
  if (threadIdx.x < 32) {
    parts = threadIdx.x < kCluster ? *cluster.map_shared_rank(&mine, threadIdx.x) : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) parts += __shfl_xor_sync(0xFFFFFFFFu, parts, o);
  }
  if (threadIdx.x == 0) {
    const double n = sqrt(parts);
    shared_factor = factor_of(n, bound);
    if (blockIdx.x == 0) {
      *norm = static_cast<float>(n);
      *factor = shared_factor;
    }
  }
  cluster.sync();  // no CTA ends while another may read its sum
  if (!scale) return;
  const float f = shared_factor;
  for (int64_t chunk = blockIdx.x; chunk < t.chunks; chunk += kCluster) scale_chunk<T>(t, chunk, f);
}

template <typename T, int kCap>
void fill(const ClipArgs& a, int64_t from, int64_t count, Table<kCap>* t) {
  t->count = 0;
  t->chunks = 0;
  for (int64_t i = from; i < from + count; ++i) {
    const vn_gradient& x = a.tensors[i];
    if (x.n == 0) continue;
    Piece& e = t->e[t->count++];
    e.g = x.grad;
    e.out = x.out;
    e.n = x.n;
    e.first = t->chunks;
    t->chunks += (x.n + kChunkOf<T> - 1) / kChunkOf<T>;
  }
}

// Calls f with the table of every launch's tensors.
template <typename T, typename F>
cudaError_t each_table(const ClipArgs& a, F f) {
  for (int64_t from = 0; from < a.count; from += kLarge) {
    const int64_t count = std::min<int64_t>(kLarge, a.count - from);
    cudaError_t err;
    if (count <= kSmall) {
      Table<kSmall> t;
      fill<T>(a, from, count, &t);
      err = f(t);
    } else {
      Table<kLarge> t;
      fill<T>(a, from, count, &t);
      err = f(t);
    }
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

template <typename T, int kCap>
cudaError_t launch_square(const Table<kCap>& t, int64_t grid, double* parts, cudaStream_t stream) {
  return launch_overlapped(square_kernel<T, kCap>, dim3(static_cast<unsigned>(grid)), kThreads, 0, 0, stream, t, parts);
}
template <typename T, int kCap>
cudaError_t launch_scale(const Table<kCap>& t, const float* factor, cudaStream_t stream) {
  return launch_overlapped(scale_kernel<T, kCap>, dim3(static_cast<unsigned>(t.chunks)), kThreads, 0, 0, stream, t, factor);
}
template <typename T, int kCap>
cudaError_t launch_few(const Table<kCap>& t, const ClipArgs& a, float* factor, cudaStream_t stream) {
  static SmemRecord wide;
  const cudaError_t err = allow_wide_clusters(reinterpret_cast<const void*>(few_kernel<T, kCap>), wide);
  if (err != cudaSuccess) return err;
  return launch_overlapped(few_kernel<T, kCap>, dim3(kCluster), kThreads, kCluster, 0, stream, t, a.bound, a.norm, factor,
                           a.scale ? 1 : 0);
}

template <typename T>
cudaError_t run(const ClipArgs& a, cudaStream_t stream) {
  DeviceInfo dev;
  cudaError_t err = device_info(&dev);
  if (err != cudaSuccess) return err;
  const int64_t most = std::min<int64_t>(static_cast<int64_t>(dev.sm_count) * kPerSm, kClipParts);
  float* const factor = static_cast<float*>(a.workspace);
  double* const parts = static_cast<double*>(a.workspace) + 1;  // the factor's place comes first
  int64_t done = 0;
  bool few = false;
  err = each_table<T>(a, [&](const auto& t) {
    if (t.chunks > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    few = a.count <= kLarge && t.chunks <= kFewChunks;
    if (few) return launch_few<T>(t, a, factor, stream);
    const int64_t grid = std::min(t.chunks, most);
    if (grid == 0) return cudaSuccess;
    double* const to = parts + done;
    done += grid;
    return launch_square<T>(t, grid, to, stream);
  });
  if (err != cudaSuccess || few) return err;
  err = launch_overlapped(join_kernel, dim3(1), kThreads, 0, 0, stream, static_cast<const double*>(parts), done, a.bound, a.norm,
                          factor);
  if (err != cudaSuccess || !a.scale) return err;
  return each_table<T>(a, [&](const auto& t) { return t.chunks == 0 ? cudaSuccess : launch_scale<T>(t, factor, stream); });
}

}  // namespace

int64_t clip_workspace(int64_t count) { return 8 * (1 + (count + kLarge - 1) / kLarge * kClipParts); }

cudaError_t launch_clip(const ClipArgs& a, cudaStream_t stream) {
  return a.dt == VN_BF16 ? run<__nv_bfloat16>(a, stream) : run<float>(a, stream);
}

}  // namespace vn
