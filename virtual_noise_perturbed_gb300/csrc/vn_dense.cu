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
// so every kernel serves all three. Which one a call goes to is reckoned from its sizes (below): few
// rows, operands gathered by threads, or tiles by TMA, whose operands are converted first where TMA
// cannot take them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "vn_act.cuh"
#include "vn_dense.h"
#include "vn_internal.h"
#include "vn_launch.cuh"
#include "vn_split.cuh"

namespace vn {
namespace {

template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Eight values to row-major memory. kPlanes 1: in T, 16-byte stores where they fit; 3: bf16
// planes, `plane` elements apart, the whole group written (pitch is a multiple of 8).
template <typename T, int kPlanes>
__device__ __forceinline__ void store8(void* dst, int64_t at, int64_t plane, const float (&v)[8], int count, bool vec) {
  if constexpr (kPlanes == 3) {
    uint32_t w[3][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t a[3], b[3];
      split3(v[2 * q], a);
      split3(v[2 * q + 1], b);
#pragma unroll
      for (int k = 0; k < 3; ++k) w[k][q] = join_terms(a[k], b[k]);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(dst) + k * plane + at) =
          make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
  } else {
    T* d = static_cast<T*>(dst) + at;
    if (vec) {
      if constexpr (sizeof(T) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * q], v[2 * q + 1]);
          w[q] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        *reinterpret_cast<float4*>(d) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(d + 4) = make_float4(v[4], v[5], v[6], v[7]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < count) d[q] = narrow<T>(v[q]);
    }
  }
}
// Eight elements of a row as they are in memory (zeros beyond `count`); vec: 16-byte loads,
// count >= 8 or none.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int count, bool vec) {
    a = make_uint4(0u, 0u, 0u, 0u);
    if (vec) {
      if (count > 0) a = __ldcs(reinterpret_cast<const uint4*>(p));
    } else {
      uint32_t h[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) h[q] = q < count ? static_cast<uint32_t>(__bfloat16_as_ushort(p[q])) : 0u;
      a = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = __uint_as_float(w[q] << 16);
      v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
    }
  }
};
template <>
struct Eight<float> {
  float v8[8];
  __device__ __forceinline__ void load(const float* p, int count, bool vec) {
#pragma unroll
    for (int q = 0; q < 8; ++q) v8[q] = 0.f;
    if (vec) {
      if (count > 0) {
        const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
        v8[0] = a.x; v8[1] = a.y; v8[2] = a.z; v8[3] = a.w;
        v8[4] = b.x; v8[5] = b.y; v8[6] = b.z; v8[7] = b.w;
      }
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < count) v8[q] = p[q];
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = v8[q];
  }
};

// A matrix as the tensor cores take it: rows padded to `pitch`, fp32 split into planes.
template <typename T>
__global__ void __launch_bounds__(256)
convert_kernel(const T* src, int64_t rows, int64_t cols, void* dst, int64_t pitch,
               int64_t plane, int vec) {
  let_next();
  after_previous();
  const int64_t groups = pitch / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= rows * groups) return;
  const int64_t r = i / groups, c = (i - r * groups) * 8;
  Eight<T> e;
  float v[8];
  e.load(src + r * cols + c, static_cast<int>(min(static_cast<int64_t>(8), cols - c)), vec != 0);
  e.get(v);
  if constexpr (sizeof(T) == 2) store8<T, 1>(dst, r * pitch + c, 0, v, 8, true);
  else store8<T, 3>(dst, r * pitch + c, plane, v, 8, true);
}

// d = g act'(z), stored as the products take it, and column sums of the unrounded d: a
// CTA's 8 warps walk over every 8 gridDim.y-th row of 256 columns.
struct Delta {
  const void* g;
  const void* z;
  void* d;      // NULL: only the sums
  float* part;  // NULL: only d
  int64_t rows, n, pitch, plane;
  int act;
  int vec_in, vec_out;
};
template <typename T, int kPlanes>
__global__ void __launch_bounds__(256) delta_kernel(const Delta a) {
  let_next();
  after_previous();
  __shared__ float s[8][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + lane * 8;
  const int count = static_cast<int>(min(static_cast<int64_t>(8), a.n - c));
  const T* g = static_cast<const T*>(a.g);
  const T* z = static_cast<const T*>(a.z);
  float sum[8] = {};
  if (count > 0) {
    // A few rows at a time, their loads before the first use.
    constexpr int kAhead = sizeof(T) == 2 ? 4 : 2;
    const int64_t step = static_cast<int64_t>(gridDim.y) * 8;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.y) * 8 + warp; r0 < a.rows; r0 += kAhead * step) {
      Eight<T> eg[kAhead], ez[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t r = r0 + i * step;
        const int have = r < a.rows ? count : 0;
        eg[i].load(g + r * a.n + c, have, a.vec_in != 0);
        if (a.act != VN_ACT_NONE) ez[i].load(z + r * a.n + c, have, a.vec_in != 0);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t r = r0 + i * step;
        float v[8];
        eg[i].get(v);
        if (a.act != VN_ACT_NONE) {
          float u[8];
          ez[i].get(u);
          slope_all<true>(a.act, u, v);
        }
        if (a.d != nullptr && r < a.rows) store8<T, kPlanes>(a.d, r * a.pitch + c, a.plane, v, count, a.vec_out != 0);
#pragma unroll
        for (int q = 0; q < 8; ++q) sum[q] += v[q];
      }
    }
  }
  if (a.part == nullptr) return;
#pragma unroll
  for (int q = 0; q < 8; ++q) s[warp][q * 32 + lane] = sum[q];
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) t += s[k][threadIdx.x];
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 256 + (threadIdx.x & 31) * 8 + (threadIdx.x >> 5);
  if (col < a.n) a.part[static_cast<int64_t>(blockIdx.y) * a.n + col] = t;
}

constexpr int64_t kAlign = 256;
int64_t rounded(int64_t bytes) { return (bytes + kAlign - 1) / kAlign * kAlign; }
int64_t pitch_of(int64_t cols) { return (cols + 7) / 8 * 8; }

// Bytes of a matrix as the tensor cores take it.
int64_t operand_bytes(int64_t rows, int64_t cols, vn_dtype dt) {
  return rounded(rows * pitch_of(cols) * (dt == VN_BF16 ? 2 : 6));
}
// Whether a matrix can be taken as it is.
bool as_is(vn_dtype dt, int64_t cols, bool aligned) { return dt == VN_BF16 && cols % 8 == 0 && aligned; }

// ---------------------------------------------------------------- which kernel
// The times below are what calls one after the other took on a GB300, over sizes from 64 to 8192: a few
// microseconds a launch, more of them the larger its tile, and a CTA's (or pair's) time per 64 of k.
// They are reckoned here, from sizes alone, so that a call and its workspace agree without a device.
enum class Route {
  kRows = 0,    // few rows, at most 8: vn_dense_rows.cu
  kGather = 2,  // one launch, operands gathered by threads: vn_dense_gather.cu
  kTiles = 3,   // operands by TMA, in bf16 (converted where they are not): vn_dense_tc.cu
};
// More rows than 32-bit coordinates reach are taken in slices.
constexpr int64_t kSlice = int64_t{1} << 30;
double tiles_of(int64_t n, int64_t tile) { return static_cast<double>((n + tile - 1) / tile); }
// CTAs that the GPU holds at once in clusters of 2^log_cluster, `per_sm` to an SM: fewer than 152 SMs
// have room for, as clusters stay within a part of the GPU.
double resident(int log_cluster, int per_sm) {
  static const double kOne[5] = {152, 152, 144, 120, 112}, kTwo[5] = {304, 304, 296, 288, 224};
  return per_sm == 1 ? kOne[log_cluster] : kTwo[log_cluster];
}

// A product on tiles. iters: chunks of 64 k, six times as many of fp32's planes.
TilePlan tile_plan(int64_t np, int64_t nq, int64_t nk, vn_dtype dt, bool b_mn) {
  TilePlan best;
  if (np == 0 || nq == 0) {
    best.us = 0;
    return best;
  }
  const double iters = tiles_of(nk, 64) * (dt == VN_BF16 ? 1 : 6);
  // Pairs: rounds of tiles over 76 pairs. Up to 128 columns the four MMAs of 64 k take as long as each
  // other's latency; with every SM at work, operands come slower. 256 x 4096 to 4096 in bf16: one
  // round of 64 columns 14.8 us, of 128 15.5, of 256 24.7; 4096 cubed: 4 rounds of 224 columns 76, 4 of
  // 256 81, 7 of 128 95.
  for (int bn = 256; bn >= 32; bn -= 16) {
    const double rounds = std::ceil(tiles_of(np, 256) * tiles_of(nq, bn) / 76);
    const double stage = rounds > 1 ? 0.135 + 0.00059 * bn : std::max(0.15, 0.00104 * bn);
    const double us = 4.0 + rounds * iters * stage + (rounds - 1) * 0.8 + 0.0165 * bn;
    if (us < best.us) best = TilePlan{us, true, bn, 0};
  }
  // Single CTAs, two an SM, which then share its loads.
  for (int bn : {16, 64, 128}) {
    if (b_mn && bn == 16) continue;
    const double stage = bn == 128 ? 0.29 : bn == 64 ? 0.25 : 0.22;
    for (int l = 0; l < 4 && (1 << l) <= iters; ++l) {  // each CTA has a share of k
      const double ctas = tiles_of(np, 128) * tiles_of(nq, bn) * (1 << l);
      const double rounds = std::ceil(ctas / resident(l, 2));
      const double us = (bn == 128 ? 5.3 : bn == 64 ? 2.6 : 1.9) + (l > 0 ? 0.4 + 1.4 * l : 0.0) +
                        rounds * (std::ceil(iters / (1 << l)) * stage * (ctas > 152 ? 1.6 : 1.0) + 2.0);
      if (us < best.us) best = TilePlan{us, false, bn, l};
    }
  }
  return best;
}

// Products (one, or a layer's two gradients) gathered in one launch: the time of the longest CTA, or of
// all of them over those that run at once.
struct Shape {
  int64_t np, nq, nk;
};
GatherPlan gather_plan(const Shape (&shapes)[2], vn_dtype dt, bool backward, bool vectors) {
  GatherPlan best;
  const bool bf16 = dt == VN_BF16;
  for (int bn : {16, 64, 128}) {
    if (backward && bn == 16) continue;
    // Not built: what would hold too many registers, and forward products in bf16 of more columns, which a
    // sweep over sizes never chose (tiles by TMA are faster where rows start on 16 bytes).
    if (bf16 && bn > (backward ? (vectors ? 128 : 64) : (vectors ? 16 : 64))) continue;
    const double stage = (vectors ? 1.0 : !bf16 ? 1.7 : bn > 16 ? 2.4 : 2.0) *  // rows that start anywhere
                         (backward    ? (bn == 128 ? (bf16 ? 2.2 : 3.1) : (bf16 ? 1.2 : 1.7))
                          : bn == 128 ? (bf16 ? 0.9 : 1.4)
                          : bn == 64  ? (bf16 ? 0.65 : 1.2)
                                      : (bf16 ? 0.75 : 0.95));
    const double launch = backward ? (bf16 || bn == 128 ? 5.3 : 6.7) : bn == 128 ? 8.5 : bn == 64 ? 6.0 : 3.5;
    for (int l0 = 0; l0 < 4; ++l0)
      // Clusters of 16, where the sums over rows are long.
      for (int l1 = 0; l1 < (!backward ? 1 : shapes[1].nk >= 4096 ? 5 : 4); ++l1) {
        const int l[2] = {l0, l1};
        double work = 0, longest = 0, ctas = 0, chunks = 0;
        for (int i = 0; i < 2; ++i) {
          const Shape& s = shapes[i];
          if (s.np == 0 || s.nq == 0) continue;
          const double n = tiles_of(s.np, 128) * tiles_of(s.nq, bn) * (1 << l[i]);
          chunks = std::max(chunks, std::ceil(tiles_of(s.nk, 64) / (1 << l[i])));
          const double t = std::ceil(tiles_of(s.nk, 64) / (1 << l[i])) * stage + launch + (l[i] > 3 ? 2.5 : l[i] > 0 ? 1.5 : 0.0) +
                           (backward && bn == 128 ? 2.0 * l[i] : 0.0);
          ctas += n;
          work += n * t;
          longest = std::max(longest, t);
        }
        const int per_sm = bf16 ? 2 : 1;
        const double room = resident(std::max(l0, l1), per_sm);
        // Two CTAs of an SM share its threads' time.
        double crowd = per_sm == 2 && ctas > resident(std::max(l0, l1), 1) ? 1.7 : 1.0;
        if (backward && ctas > 0) crowd = 1 + (crowd - 1) * work / (ctas * longest);  // short ones leave soon
        if (!backward) crowd = (longest + (crowd - 1) * 0.4 * chunks * stage) / std::max(longest, 1e-9);
        const double us = crowd * (ctas <= room ? longest : std::max(longest, work / room) + 0.5 * longest);
        if (us < best.us) {
          best.us = us;
          best.bn = bn;
          best.log_split[0] = l0;
          best.log_split[1] = l1;
        }
      }
  }
  return best;
}
// Converting a matrix for the tensor cores.
double convert_us(int64_t rows, int64_t cols, vn_dtype dt, bool as_it_is) {
  if (as_it_is) return 0;
  return 3.2 + static_cast<double>(rows) * static_cast<double>(cols) * (dt == VN_BF16 ? 4 : 10) / 4e6;
}

struct ForwardPlan {
  Route route;
  GatherPlan gather;
  TilePlan tiles;
};
ForwardPlan reckon_forward(int64_t rows, int64_t in, int64_t out, vn_dtype dt, bool aligned) {
  ForwardPlan p;
  p.route = Route::kRows;
  // fp32 keeps its products unsplit up to 8 rows; in bf16 the tensor cores take over where they are faster
  // (4096 to 4096: one row 6.2 us, eight 20.0 and on tiles 11.3; 4095 to 4095: one row 23.6, eight 49.1 and
  // gathered 18.6).
  if (rows <= 8 && (dt == VN_F32 || in == 0 || in > kDenseMost || out > kDenseMost)) return p;
  const double few = rows > 8 ? 1e30
                              : 3.2 + static_cast<double>(in) * static_cast<double>(out) / 16.8e6 *
                                          (aligned && in % 8 == 0 ? 1.2 + 2.0 * static_cast<double>(rows)
                                                                  : 16.0 + 4.5 * static_cast<double>(rows));
  const Shape shapes[2] = {{out, rows, in}, {0, 0, 0}};
  const int64_t vec = dt == VN_BF16 ? 8 : 4;
  p.gather = gather_plan(shapes, dt, false, aligned && in % vec == 0);
  p.route = Route::kGather;
  if (in == 0) return p;
  p.tiles = tile_plan(out, rows, in, dt, false);
  const bool direct = as_is(dt, in, aligned);
  const double tiles = p.tiles.us + convert_us(out, in, dt, direct) + convert_us(rows, in, dt, direct);
  if (tiles < p.gather.us) p.route = Route::kTiles;
  if (few <= std::min(tiles, p.gather.us)) p.route = Route::kRows;
  return p;
}
struct BackwardPlan {
  Route route;
  GatherPlan gather;
  TilePlan dx, dw;
};
BackwardPlan reckon_backward(int64_t rows, int64_t in, int64_t out, vn_dtype dt, vn_act act, bool aligned) {
  BackwardPlan p;
  const Shape shapes[2] = {{in, rows, out}, {in, out, rows}};
  const int64_t vec = dt == VN_BF16 ? 8 : 4;
  p.gather = gather_plan(shapes, dt, true, aligned && in % vec == 0 && out % vec == 0);
  p.route = Route::kGather;
  if (rows == 0 || in == 0 || out == 0) return p;
  p.dx = tile_plan(in, rows, out, dt, false);
  p.dw = tile_plan(in, out, rows, dt, true);
  const bool direct = as_is(dt, in, aligned), keeps = act != VN_ACT_NONE || !as_is(dt, out, aligned);
  // d, and the bias's sums.
  const double elements = static_cast<double>(rows) * static_cast<double>(out);
  const double delta = 8.0 + (keeps ? 2.0 : 1.0) * elements * (dt == VN_BF16 ? 3 : 7) / 4e6;
  if (p.dx.us + p.dw.us + delta + convert_us(out, in, dt, direct) + convert_us(rows, in, dt, direct) < p.gather.us)
    p.route = Route::kTiles;
  return p;
}

// A call asks for its plan three times (for its workspace, to check that, and to launch), and a program
// for the same sizes again and again: each thread keeps the last one.
struct Sizes {
  int64_t rows, in, out;
  int dt, act, aligned;
  bool operator==(const Sizes& o) const {
    return rows == o.rows && in == o.in && out == o.out && dt == o.dt && act == o.act && aligned == o.aligned;
  }
};
ForwardPlan forward_plan(int64_t rows, int64_t in, int64_t out, vn_dtype dt, bool aligned) {
  thread_local Sizes last = {-1, 0, 0, 0, 0, 0};
  thread_local ForwardPlan plan;
  const Sizes now = {rows, in, out, dt, 0, aligned};
  if (!(now == last)) {
    plan = reckon_forward(rows, in, out, dt, aligned);
    last = now;
  }
  return plan;
}
BackwardPlan backward_plan(int64_t rows, int64_t in, int64_t out, vn_dtype dt, vn_act act, bool aligned) {
  thread_local Sizes last = {-1, 0, 0, 0, 0, 0};
  thread_local BackwardPlan plan;
  const Sizes now = {rows, in, out, dt, act, aligned};
  if (!(now == last)) {
    plan = reckon_backward(rows, in, out, dt, act, aligned);
    last = now;
  }
  return plan;
}

// Row groups that the column sums are split over.
int64_t delta_parts(int64_t rows) { return std::max<int64_t>(1, std::min<int64_t>(64, (rows + 31) / 32)); }

TcOperand operand(const void* p, int64_t rows, int64_t cols, bool mn) {
  return TcOperand{p, rows, cols, cols, rows * cols, 1, mn};
}
// The matrix as the tensor cores take it: itself, or a converted copy at *work (advanced).
cudaError_t prepare(const void* p, vn_dtype dt, int64_t rows, int64_t cols, bool aligned, bool mn, uint8_t** work,
                    TcOperand* o, cudaStream_t stream) {
  *o = operand(p, rows, cols, mn);
  if (as_is(dt, cols, aligned)) return cudaSuccess;
  o->p = *work;
  o->pitch = pitch_of(cols);
  o->plane = rows * o->pitch;
  o->planes = dt == VN_BF16 ? 1 : 3;
  *work += operand_bytes(rows, cols, dt);
  const int64_t grid = (rows * (o->pitch / 8) + 255) / 256;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  const int vec = cols % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
  void* dst = const_cast<void*>(o->p);
  const dim3 ctas(static_cast<unsigned>(grid));
  if (dt == VN_BF16)
    return launch_overlapped(convert_kernel<__nv_bfloat16>, ctas, 256, 0, 0, stream,
                             static_cast<const __nv_bfloat16*>(p), rows, cols, dst, o->pitch, o->plane, vec);
  return launch_overlapped(convert_kernel<float>, ctas, 256, 0, 0, stream, static_cast<const float*>(p), rows, cols, dst,
                           o->pitch, o->plane, vec);
}

}  // namespace

int64_t dense_workspace(int64_t rows, int64_t in, int64_t out, vn_dtype dt, bool aligned) {
  if (rows > kDenseMost)
    return std::max(dense_workspace(kSlice, in, out, dt, aligned), dense_workspace((rows - 1) % kSlice + 1, in, out, dt, aligned));
  if (forward_plan(rows, in, out, dt, aligned).route != Route::kTiles || as_is(dt, in, aligned)) return 0;
  return operand_bytes(rows, in, dt) + operand_bytes(out, in, dt);
}

int64_t dense_backward_workspace(int64_t rows, int64_t in, int64_t out, vn_dtype dt, vn_act act, bool aligned) {
  if (rows > kDenseMost)
    return std::max(dense_backward_workspace(kSlice, in, out, dt, act, aligned),
                    dense_backward_workspace((rows - 1) % kSlice + 1, in, out, dt, act, aligned));
  const Route route = backward_plan(rows, in, out, dt, act, aligned).route;
  const int64_t sums = rounded(delta_parts(rows) * out * 4);
  if (route == Route::kGather) return sums;
  int64_t bytes = sums;
  if (act != VN_ACT_NONE || !as_is(dt, out, aligned)) bytes += operand_bytes(rows, out, dt);
  if (!as_is(dt, in, aligned)) bytes += operand_bytes(rows, in, dt) + operand_bytes(out, in, dt);
  return bytes;
}

cudaError_t launch_dense(const DenseArgs& a, cudaStream_t stream) {
  if (a.rows > kDenseMost) {
    const int64_t es = a.dt == VN_BF16 ? 2 : 4;
    auto at = [&](const void* p, int64_t elements) -> void* {
      return p != nullptr ? static_cast<uint8_t*>(const_cast<void*>(p)) + elements * es : nullptr;
    };
    for (int64_t r = 0; r < a.rows; r += kSlice) {
      DenseArgs one = a;
      one.rows = std::min(kSlice, a.rows - r);
      one.x = at(a.x, r * a.in);
      one.residual = at(a.residual, r * a.out);
      one.y = at(a.y, r * a.out);
      one.preact = at(a.preact, r * a.out);
      const cudaError_t err = launch_dense(one, stream);
      if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
  }
  const bool al = aligned16(a.x) && aligned16(a.w);
  const ForwardPlan plan = forward_plan(a.rows, a.in, a.out, a.dt, al);
  if (plan.route == Route::kRows) return launch_rows_forward(a, stream);
  if (plan.route == Route::kGather) return launch_gather_forward(a, plan.gather, stream);
  uint8_t* work = static_cast<uint8_t*>(a.workspace);
  TcProduct d = {};
  cudaError_t err = prepare(a.w, a.dt, a.out, a.in, al, false, &work, &d.a, stream);
  if (err != cudaSuccess) return err;
  if ((err = prepare(a.x, a.dt, a.rows, a.in, al, false, &work, &d.b, stream)) != cudaSuccess) return err;
  d.np = a.out; d.nq = a.rows; d.nk = a.in;
  d.dt = a.dt;
  d.bias = a.b; d.bias_bf16 = a.b_dt == VN_BF16; d.act = a.act;
  d.residual = a.residual; d.out = a.y; d.preact = a.preact;
  return launch_tc_product(d, plan.tiles, stream);
}

void dense_plan(int64_t rows, int64_t in, int64_t out, vn_dtype dt, vn_act act, bool aligned, bool backward, int32_t (&p)[10]) {
  auto fill = [&](Route route, const GatherPlan& g, const TilePlan& t0, const TilePlan& t1) {
    const int32_t all[10] = {static_cast<int32_t>(route), g.bn, g.log_split[0], g.log_split[1], t0.pair, t0.bn,
                             t0.log_split, t1.pair, t1.bn, t1.log_split};
    std::copy(all, all + 10, p);
  };
  if (backward) {
    const BackwardPlan b = backward_plan(rows, in, out, dt, act, aligned);
    fill(b.route, b.gather, b.dx, b.dw);
  } else {
    const ForwardPlan f = forward_plan(rows, in, out, dt, aligned);
    fill(f.route, f.gather, f.tiles, TilePlan());
  }
}

cudaError_t launch_dense_hook(const DenseArgs& a, int kernel, int at, unsigned long long timeout_ns, cudaStream_t stream) {
  const Withhold hook = {at, timeout_ns};
  if (kernel % 4 == 0) {
    GatherPlan plan;
    plan.log_split[0] = 1;
    return launch_gather_forward(a, plan, stream, &hook);
  }
  TcProduct d = {};
  d.a = operand(a.w, a.out, a.in, false);
  d.b = operand(a.x, a.rows, a.in, false);
  if (a.dt == VN_F32) d.a.planes = d.b.planes = 3;  // given as the tensor cores take them
  d.np = a.out; d.nq = a.rows; d.nk = a.in;
  d.dt = a.dt;
  d.residual = a.residual; d.out = a.y; d.preact = a.preact;
  TilePlan plan;
  plan.pair = kernel % 4 == 2;
  plan.bn = plan.pair ? 128 : 64;
  plan.log_split = plan.pair ? 0 : 1;
  return launch_tc_product(d, plan, stream, &hook);
}

namespace {

// d into `delta` (where given) and the bias's gradient (where asked for) by way of `part`.
cudaError_t delta_pass(const DenseGradArgs& a, const TcOperand* delta, float* part, cudaStream_t stream) {
  const int64_t parts = a.rows > 0 ? delta_parts(a.rows) : 0;
  if (a.rows > 0 && a.out > 0 && (delta != nullptr || a.grad_b != nullptr)) {
    Delta k = {};
    k.g = a.grad; k.z = a.preact;
    k.part = a.grad_b != nullptr ? part : nullptr;
    k.rows = a.rows; k.n = a.out;
    if (delta != nullptr) {
      k.d = const_cast<void*>(delta->p);
      k.pitch = delta->pitch; k.plane = delta->plane;
      k.vec_out = delta->pitch % 8 == 0;
    }
    k.act = a.act;
    k.vec_in = a.out % 8 == 0 && aligned16(a.grad) && (a.act == VN_ACT_NONE || aligned16(a.preact));
    const int64_t tiles = (a.out + 255) / 256;
    if (tiles > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(parts));
    cudaError_t err;
    if (a.dt == VN_BF16) err = launch_overlapped(delta_kernel<__nv_bfloat16, 1>, grid, 256, 0, 0, stream, k);
    else if (delta != nullptr && delta->planes == 3) err = launch_overlapped(delta_kernel<float, 3>, grid, 256, 0, 0, stream, k);
    else err = launch_overlapped(delta_kernel<float, 1>, grid, 256, 0, 0, stream, k);
    if (err != cudaSuccess) return err;
  }
  if (a.grad_b == nullptr || a.out == 0) return cudaSuccess;
  return launch_column_sum(part, parts, a.out, a.out, a.grad_b, nullptr, a.gb_dt, stream);
}

}  // namespace

cudaError_t launch_dense_backward(const DenseGradArgs& a, cudaStream_t stream) {
  if (a.rows > kDenseMost) {  // only grad_x is asked for
    const int64_t es = a.dt == VN_BF16 ? 2 : 4;
    for (int64_t r = 0; r < a.rows; r += kSlice) {
      DenseGradArgs one = a;
      one.rows = std::min(kSlice, a.rows - r);
      one.grad = static_cast<const uint8_t*>(a.grad) + r * a.out * es;
      one.preact = a.preact != nullptr ? static_cast<const uint8_t*>(a.preact) + r * a.out * es : nullptr;
      one.grad_x = static_cast<uint8_t*>(a.grad_x) + r * a.in * es;
      const cudaError_t err = launch_dense_backward(one, stream);
      if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
  }
  const bool al = aligned16(a.grad) && aligned16(a.x) && aligned16(a.w);
  const BackwardPlan plan = backward_plan(a.rows, a.in, a.out, a.dt, a.act, al);
  if (plan.route == Route::kGather) {
    // The gather kernel sums the bias's gradient beside the weight's; alone it is a pass over d.
    DenseGradArgs rest = a;
    if (a.grad_b != nullptr && a.grad_w == nullptr) {
      const cudaError_t err = delta_pass(a, nullptr, static_cast<float*>(a.workspace), stream);
      if (err != cudaSuccess || a.grad_x == nullptr) return err;
      rest.grad_b = nullptr;
    }
    return launch_gather_backward(rest, plan.gather, stream);
  }
  const bool products = a.grad_x != nullptr || a.grad_w != nullptr;
  const bool keep = products && (a.act != VN_ACT_NONE || !as_is(a.dt, a.out, al));  // d has to be stored
  uint8_t* work = static_cast<uint8_t*>(a.workspace);
  cudaError_t err = cudaSuccess;
  float* part = reinterpret_cast<float*>(work);
  work += rounded(delta_parts(a.rows) * a.out * 4);
  TcOperand delta = operand(a.grad, a.rows, a.out, false);
  if (keep) {
    delta.p = work;
    delta.pitch = pitch_of(a.out);
    delta.plane = a.rows * delta.pitch;
    delta.planes = a.dt == VN_BF16 ? 1 : 3;
    work += operand_bytes(a.rows, a.out, a.dt);
  }
  if ((err = delta_pass(a, keep ? &delta : nullptr, part, stream)) != cudaSuccess) return err;
  TcProduct d = {};
  d.dt = a.dt;
  d.b = delta;
  if (a.grad_x != nullptr) {
    if ((err = prepare(a.w, a.dt, a.out, a.in, al, true, &work, &d.a, stream)) != cudaSuccess) return err;
    d.np = a.in; d.nq = a.rows; d.nk = a.out;
    d.out = a.grad_x;
    if ((err = launch_tc_product(d, plan.dx, stream)) != cudaSuccess) return err;
  }
  if (a.grad_w != nullptr) {
    if ((err = prepare(a.x, a.dt, a.rows, a.in, al, true, &work, &d.a, stream)) != cudaSuccess) return err;
    d.b.mn = true;
    d.np = a.in; d.nq = a.out; d.nk = a.rows;
    d.out = a.grad_w;
    err = launch_tc_product(d, plan.dw, stream);
  }
  return err;
}

}  // namespace vn
