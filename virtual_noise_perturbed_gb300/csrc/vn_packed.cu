// vn_packed.cu -- a layer's weights in 4 bits with a scale for each group of a row, and the linear layer on them:
//
//   scale = type(max |w| / 7) of `group` consecutive k,  code = the whole number next to w / scale, -7 .. 7
//   y[r, j] = act(sum_k x[r, k] code[j, k] scale[j, k / group] + b[j]) + residual[r, j]
//
// Codes lie as the tensor cores' warp-level product wants them: a row is blocks of 128 k in 64 bytes, of which lane t of
// four reads the 16 bytes t. Word w of those holds the products 2 w and 2 w + 1, and of product p the k = 16 p + 4 t + 0 .. 3.
// Each code + 8 is a nibble; a pair of neighbouring k lies 16 bits apart, so one mask and one exponent make two
// bf16 values 128 + code + 8 of it, and one subtraction the codes (both exact).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "vn_act.cuh"
#include "vn_internal.h"
#include "vn_launch.cuh"
#include "vn_split.cuh"

namespace vn {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kBlock = 128;            // k of a block
constexpr int kBlockBytes = 64;
constexpr uint32_t kMagic = 0x43004300u;  // 128 in bf16, twice
constexpr uint32_t kNothing = 0x88888888u;

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

__host__ __device__ __forceinline__ int64_t blocks_of(int64_t in) { return (in + kBlock - 1) / kBlock; }

// ---------------------------------------------------------------- packing
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// The whole number next to w / s, halves to even: the quotient's rounding can only miss by one, which the remainder
// (exact: both are multiples of the smaller one's last bit, and it is at most s) tells.
__device__ __forceinline__ int code_of(float w, float s) {
  if (s == 0.f || !(s < INFINITY)) return 0;  // 0 times an infinity or a NaN is a NaN
  float q = rintf(__fdiv_rn(w, s));
  const float r2 = 2.f * __fmaf_rn(-s, q, w);
  const bool odd = (static_cast<int>(q) & 1) != 0;
  if (r2 > s || (r2 == s && odd)) q += 1.f;
  if (r2 < -s || (r2 == -s && odd)) q -= 1.f;
  return static_cast<int>(fminf(fmaxf(q, -7.f), 7.f));
}

// A warp a block of 128 k: lane l has the k 4 l .. 4 l + 3.
template <typename T>
__global__ void __launch_bounds__(kThreads) pack_kernel(const T* w, int64_t out, int64_t in, int group, uint8_t* codes, T* scales, int vec) {
  let_next();
  after_previous();
  const int lane = threadIdx.x & 31;
  const int64_t blocks = blocks_of(in), groups = (in + group - 1) / group;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (at >= out * blocks) return;
  const int64_t row = at / blocks, block = at % blocks;
  const int64_t k = block * kBlock + lane * 4;
  const T* from = w + row * in + k;
  float v[4];
  if (vec && k + 4 <= in) {
    if constexpr (sizeof(T) == 2) {
      const uint2 raw = __ldcs(reinterpret_cast<const uint2*>(from));
      v[0] = __uint_as_float(raw.x << 16); v[1] = __uint_as_float(raw.x & 0xFFFF0000u);
      v[2] = __uint_as_float(raw.y << 16); v[3] = __uint_as_float(raw.y & 0xFFFF0000u);
    } else {
      const float4 raw = __ldcs(reinterpret_cast<const float4*>(from));
      v[0] = raw.x; v[1] = raw.y; v[2] = raw.z; v[3] = raw.w;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = k + q < in ? value(fetch(from + q)) : 0.f;
  }
  float top = max_nan(max_nan(fabsf(v[0]), fabsf(v[1])), max_nan(fabsf(v[2]), fabsf(v[3])));
  for (int o = group / 8; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const T stored = narrow<T>(__fdiv_rn(top, 7.f));
  const float s = value(stored);
  if (lane % (group / 4) == 0 && k < in) scales[row * groups + k / group] = stored;
  uint32_t c[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) c[q] = static_cast<uint32_t>(code_of(v[q], s) + 8);
  // Lane l: word l / 8 of lane l % 4's 16 bytes, its product (l / 4) % 2.
  uint32_t word = c[0] | (c[2] << 4) | (c[1] << 16) | (c[3] << 20);
  if (lane & 4) word <<= 8;
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
  if ((lane & 4) == 0)
    *reinterpret_cast<uint32_t*>(codes + at * kBlockBytes + (lane & 3) * 16 + (lane >> 3) * 4) = word;
}

// The same way back.
template <typename T>
__global__ void __launch_bounds__(kThreads) unpack_kernel(const uint8_t* codes, const T* scales, int64_t out, int64_t in, int group, T* w, int vec) {
  let_next();
  after_previous();
  const int lane = threadIdx.x & 31;
  const int64_t blocks = blocks_of(in), groups = (in + group - 1) / group;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (at >= out * blocks) return;
  const int64_t row = at / blocks, block = at % blocks;
  const int64_t k = block * kBlock + lane * 4;
  if (k >= in) return;
  uint32_t word = fetch(reinterpret_cast<const uint32_t*>(codes + at * kBlockBytes + (lane & 3) * 16 + (lane >> 3) * 4));
  if (lane & 4) word >>= 8;
  const float s = value(fetch(scales + row * groups + k / group));
  const uint32_t c[4] = {word & 15u, (word >> 16) & 15u, (word >> 4) & 15u, (word >> 20) & 15u};
  T v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = narrow<T>(__fmul_rn(static_cast<float>(static_cast<int>(c[q]) - 8), s));
  T* to = w + row * in + k;
  if (vec && k + 4 <= in) {
    if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(v);
    else *reinterpret_cast<float4*>(to) = *reinterpret_cast<const float4*>(v);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (k + q < in) to[q] = v[q];
  }
}

// ---------------------------------------------------------------- the linear layer
// Codes in bf16 of one product: k pairs 0 and 1 of four, from bits `shift` on.
__device__ __forceinline__ uint32_t decode(uint32_t word, int shift) {
  uint32_t v = ((word >> shift) & 0x000F000Fu) | kMagic;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), __floats2bfloat162_rn(136.f, 136.f));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ void product(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr int kFeatures = 16;   // of a CTA
constexpr int kDepth = 4;       // blocks of a warp in flight
constexpr int kPad = 16;        // bf16 elements behind a column in shared memory: columns 32 bytes apart in the banks

template <typename T>
constexpr int kTerms = sizeof(T) == 2 ? 1 : 3;  // bf16 terms of a value of x, each in a column of its own

// A CTA has 16 features, its warps blocks of their k in turn. kTiles: eights of columns (rows of x, times their terms).
template <typename T, int kTiles>
__global__ void __launch_bounds__(kThreads) packed_kernel(const PackedArgs a, int chunk) {
  extern __shared__ __align__(16) uint8_t shared[];
  __nv_bfloat16* const xs = reinterpret_cast<__nv_bfloat16*>(shared);
  let_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rows = static_cast<int>(a.rows), cols = rows * kTerms<T>;
  const int pitch = chunk + kPad;
  const int64_t j0 = static_cast<int64_t>(blockIdx.x) * kFeatures;
  const int64_t blocks = blocks_of(a.in), groups = (a.in + a.group - 1) / a.group;
  const bool there[2] = {j0 + g < a.out, j0 + g + 8 < a.out};
  const uint8_t* const codes = a.codes + (j0 + g) * blocks * kBlockBytes + t * 16;
  const T* const scales = static_cast<const T*>(a.scales) + (j0 + g) * groups;
  after_previous();
  float sum[kTiles][4] = {};
  for (int64_t k0 = 0; k0 < a.in; k0 += chunk) {
    const int64_t first = k0 / kBlock;
    const int count = static_cast<int>(min(static_cast<int64_t>(chunk / kBlock), blocks - first));
    bool staged = false;
    for (int base = 0; base < count; base += kWarps * kDepth) {
      uint4 c[kDepth][2];
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        const int b = base + d * kWarps + warp;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (b < count && there[h])
            c[d][h] = __ldcs(reinterpret_cast<const uint4*>(codes + ((first + b) + h * 8 * blocks) * kBlockBytes));
          else
            c[d][h] = make_uint4(kNothing, kNothing, kNothing, kNothing);
        }
      }
      if (!staged) {
        // The chunk's part of x, while the codes are on their way.
        staged = true;
        __syncthreads();
        const T* const x = static_cast<const T*>(a.x);
        for (int i = threadIdx.x; i < rows * chunk; i += kThreads) {
          const int r = i / chunk, k = i % chunk;
          const T v = k0 + k < a.in ? fetch(x + r * a.in + k0 + k) : narrow<T>(0.f);
          if constexpr (kTerms<T> == 1) {
            xs[r * pitch + k] = v;
          } else {
            uint32_t terms[3];
            split3(v, terms);
#pragma unroll
            for (int q = 0; q < 3; ++q) xs[(r * 3 + q) * pitch + k] = __ushort_as_bfloat16(static_cast<unsigned short>(terms[q] >> 16));
          }
        }
        __syncthreads();
      }
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        const int b = base + d * kWarps + warp;
        if (b >= count) break;
        float part[kTiles][4];
#pragma unroll
        for (int p = 0; p < 8; ++p) {  // products of 16 k
          if (p * 16 % a.group == 0) {
#pragma unroll
            for (int n = 0; n < kTiles; ++n)
#pragma unroll
              for (int q = 0; q < 4; ++q) part[n][q] = 0.f;
          }
          const uint32_t w0[4] = {c[d][0].x, c[d][0].y, c[d][0].z, c[d][0].w}, w1[4] = {c[d][1].x, c[d][1].y, c[d][1].z, c[d][1].w};
          const int shift = (p & 1) * 8;
          const uint32_t op[4] = {decode(w0[p >> 1], shift), decode(w1[p >> 1], shift), decode(w0[p >> 1], shift + 4),
                                  decode(w1[p >> 1], shift + 4)};
#pragma unroll
          for (int n = 0; n < kTiles; ++n) {
            uint2 xv = make_uint2(0u, 0u);
            if (n * 8 + g < cols) xv = *reinterpret_cast<const uint2*>(xs + (n * 8 + g) * pitch + b * kBlock + p * 16 + t * 4);
            product(part[n], op, xv.x, xv.y);
          }
          if ((p * 16 + 16) % a.group == 0) {
            const int64_t at = ((first + b) * kBlock + p * 16) / a.group;
            const float s0 = there[0] && at < groups ? value(fetch(scales + at)) : 0.f;
            const float s1 = there[1] && at < groups ? value(fetch(scales + 8 * groups + at)) : 0.f;
#pragma unroll
            for (int n = 0; n < kTiles; ++n) {
              sum[n][0] = fmaf(part[n][0], s0, sum[n][0]);
              sum[n][1] = fmaf(part[n][1], s0, sum[n][1]);
              sum[n][2] = fmaf(part[n][2], s1, sum[n][2]);
              sum[n][3] = fmaf(part[n][3], s1, sum[n][3]);
            }
          }
        }
      }
    }
  }
  // The warps' sums, in order.
  constexpr int kWide = kTiles * 8 + 1;
  float* const parts = reinterpret_cast<float*>(shared);  // [kWarps][kFeatures][kWide]
  __syncthreads();
#pragma unroll
  for (int n = 0; n < kTiles; ++n)
#pragma unroll
    for (int q = 0; q < 4; ++q) parts[(warp * kFeatures + g + (q >> 1) * 8) * kWide + n * 8 + t * 2 + (q & 1)] = sum[n][q];
  __syncthreads();
  for (int i = threadIdx.x; i < rows * kFeatures; i += kThreads) {
    const int r = i / kFeatures, f = i % kFeatures;
    const int64_t j = j0 + f;
    if (j >= a.out) continue;
    float z[1] = {0.f};
#pragma unroll
    for (int q = kTerms<T> - 1; q >= 0; --q) {  // the smallest terms first
      float v = 0.f;
      for (int w = 0; w < kWarps; ++w) v += parts[(w * kFeatures + f) * kWide + r * kTerms<T> + q];
      z[0] += v;
    }
    if (a.b != nullptr)
      z[0] += a.b_dt == VN_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.b)[j]) : static_cast<const float*>(a.b)[j];
    activate_all<false>(a.act, z);
    const int64_t at = r * a.out + j;
    if (a.residual != nullptr) z[0] += value(static_cast<const T*>(a.residual)[at]);
    static_cast<T*>(a.y)[at] = narrow<T>(z[0]);
  }
}

template <typename T, int kTiles>
cudaError_t run_tiles(const PackedArgs& a, cudaStream_t stream) {
  static SmemRecord record;
  const int cols = static_cast<int>(a.rows) * kTerms<T>;
  // As much of k at once as 96 KB of x take.
  const int64_t fit = (96 * 1024 / (2 * cols) - kPad) / kBlock * kBlock;
  const int chunk = static_cast<int>(std::min(fit, blocks_of(a.in) * kBlock));
  const size_t smem = std::max<size_t>(static_cast<size_t>(cols) * (chunk + kPad) * 2, sizeof(float) * kWarps * kFeatures * (kTiles * 8 + 1));
  const cudaError_t err = ensure_dynamic_smem(reinterpret_cast<const void*>(packed_kernel<T, kTiles>), smem, record);
  if (err != cudaSuccess) return err;
  const int64_t grid = (a.out + kFeatures - 1) / kFeatures;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  return launch_overlapped(packed_kernel<T, kTiles>, dim3(static_cast<unsigned>(grid)), kThreads, 0, smem, stream, a, chunk);
}

template <typename T>
cudaError_t run_packed(const PackedArgs& a, cudaStream_t stream) {
  const int64_t cols = a.rows * kTerms<T>;
  if (cols <= 8) return run_tiles<T, 1>(a, stream);
  if (cols <= 16) return run_tiles<T, 2>(a, stream);
  if (cols <= 32) return run_tiles<T, 4>(a, stream);
  return run_tiles<T, 8>(a, stream);
}

bool fits(const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

template <typename T>
cudaError_t pack_typed(const void* w, int64_t out, int64_t in, int group, uint8_t* codes, void* scales, cudaStream_t stream) {
  const int64_t grid = (out * blocks_of(in) + kWarps - 1) / kWarps;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  const int vec = in % 4 == 0 && fits(w, 4 * sizeof(T));
  return launch_overlapped(pack_kernel<T>, dim3(static_cast<unsigned>(grid)), kThreads, 0, 0, stream, static_cast<const T*>(w), out, in,
                           group, codes, static_cast<T*>(scales), vec);
}
template <typename T>
cudaError_t unpack_typed(const uint8_t* codes, const void* scales, int64_t out, int64_t in, int group, void* w, cudaStream_t stream) {
  const int64_t grid = (out * blocks_of(in) + kWarps - 1) / kWarps;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  const int vec = in % 4 == 0 && fits(w, 4 * sizeof(T));
  return launch_overlapped(unpack_kernel<T>, dim3(static_cast<unsigned>(grid)), kThreads, 0, 0, stream, codes,
                           static_cast<const T*>(scales), out, in, group, static_cast<T*>(w), vec);
}

// The most rows that the kernel on packed weights takes.
int64_t few_rows(vn_dtype dt) { return dt == VN_BF16 ? 64 : 21; }

int64_t padded(int64_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

int64_t packed_row_bytes(int64_t in) { return blocks_of(in) * kBlockBytes; }

cudaError_t launch_pack(const void* w, vn_dtype dt, int64_t out, int64_t in, int group, uint8_t* codes, void* scales, cudaStream_t stream) {
  return dt == VN_BF16 ? pack_typed<__nv_bfloat16>(w, out, in, group, codes, scales, stream)
                       : pack_typed<float>(w, out, in, group, codes, scales, stream);
}
cudaError_t launch_unpack(const uint8_t* codes, const void* scales, vn_dtype dt, int64_t out, int64_t in, int group, void* w,
                          cudaStream_t stream) {
  return dt == VN_BF16 ? unpack_typed<__nv_bfloat16>(codes, scales, out, in, group, w, stream)
                       : unpack_typed<float>(codes, scales, out, in, group, w, stream);
}

int64_t packed_workspace(int64_t rows, int64_t in, int64_t out, vn_dtype dt, bool aligned) {
  if (rows <= few_rows(dt)) return 0;
  return padded(out * in * (dt == VN_BF16 ? 2 : 4)) + dense_workspace(rows, in, out, dt, aligned);
}

// Many rows: the weights' values, then the plain layer.
cudaError_t launch_packed(const PackedArgs& a, cudaStream_t stream) {
  if (a.rows <= few_rows(a.dt)) return a.dt == VN_BF16 ? run_packed<__nv_bfloat16>(a, stream) : run_packed<float>(a, stream);
  const cudaError_t err = launch_unpack(a.codes, a.scales, a.dt, a.out, a.in, a.group, a.workspace, stream);
  if (err != cudaSuccess) return err;
  DenseArgs d = {};
  d.x = a.x; d.w = a.workspace; d.dt = a.dt; d.b = a.b; d.b_dt = a.b_dt; d.residual = a.residual;
  d.rows = a.rows; d.in = a.in; d.out = a.out; d.act = a.act; d.y = a.y;
  d.workspace = static_cast<uint8_t*>(a.workspace) + padded(a.out * a.in * (a.dt == VN_BF16 ? 2 : 4));
  return launch_dense(d, stream);
}

}  // namespace vn
