// vn_packed.cu -- a layer's weights in 4 bits with a scale for each group of a row, and the linear layer on them:
//
//   scale = type(max |w| / 7) of `group` consecutive k,  code = the whole number next to w / scale, -7 .. 7
//   y[r, j] = act(sum_k x[r, k] code[j, k] scale[j, k / group] + b[j]) + residual[r, j]
//
// Codes lie as the tensor cores' warp-level product wants them: a row is blocks of 128 k in 64 bytes, of which lane t of
// four reads the 16 bytes t. Word w of those holds the products 2 w and 2 w + 1, and of product p the k = 16 p + 4 t + 0 .. 3.
// Each code + 8 is a nibble; a pair of neighbouring k lies 16 bits apart, so one mask and one exponent make two
// bf16 values 2^-3 + (code + 8) 2^-10 of it, and one subtraction the codes in units of 2^-10 (both exact). In these units no sum of a
// group, of up to 7 times 128 |x|, passes what fp32 holds; they are taken off at the end (of results, 2^-139 a sum may be lost by it).
//
// The layer on few rows (up to 32, fp32 10) is bound by latency and by the instructions that make operands of codes, 17 for the
// 256 weights of a product, beside reading the codes once: so the rows of x are the product's columns, eight at no
// more cost than one. fp32 rows take three columns each, for the three bf16 terms of their values; a code is exact in
// bf16. The sum of a group is scaled in fp32. 4096 to 4096 in a replayed graph, bf16: one row 4.5 us (8.9 MB: 2.0 TB/s; plain
// weights take 5.2), 8 rows 5.6, 32 13.9; fp32 5.9, 5 rows 8.5, 10 rows 14.4. More rows take unpacked weights, in bf16 as two terms
// each: 64 rows 28 us, 256 43, 1024 60 (32 rows at a time 28, 111 and 445; 64 rows of 1024 to 1024 12.6 and 10.0, of 256 to 256 4.9 and 5.8),
// fp32 16 rows 37 and 64 42 (ten rows at a time 28 and 93).
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
constexpr uint32_t kMagic = 0x3E003E00u;  // 2^-3 in bf16, twice
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
// A group's length as a power of two, and how many a row has.
__host__ __device__ __forceinline__ int digits_of(int group) { return group == 32 ? 5 : group == 64 ? 6 : 7; }
__host__ __device__ __forceinline__ int64_t groups_of(int64_t in, int digits) { return (in + (1 << digits) - 1) >> digits; }

// ---------------------------------------------------------------- packing
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

constexpr int kSegment = 2 * kBlock;  // k of a warp at once: 8 a lane
// Segments of a warp, one after the other in a row, their loads in flight together. 67 M weights in fp32 take 56 us to pack with four,
// 64 with two, and 54 and 46 back; in bf16 44 and 29 with four (one or two, each with a place of its own to find, 66 and 43).
constexpr int kPackRun = 4;
template <typename T>
constexpr int kUnpackRun = sizeof(T) == 2 ? 4 : 2;

// The whole number next to w / s (halves to even), in the lowest four bits of its two's complement; inv: 1 / s to 2^-22.
// bf16: w inv corrected by its remainder is off by less than 2^-40, and not at all where the quotient is a half, as other
// quotients of two bf16 values are 2^-12 away from one.
__device__ __forceinline__ uint32_t code_of(__nv_bfloat16, float w, float s, float inv) {
  const float y = __fmul_rn(w, inv);
  return __float_as_uint(__fadd_rn(__fmaf_rn(__fmaf_rn(-s, y, w), inv, y), 12582912.f));
}
// fp32: the product can miss by one next to a half; the remainder (exact: both of its parts are multiples of the
// smaller one's last bit, and it is at most s) tells.
__device__ __forceinline__ uint32_t code_of(float, float w, float s, float inv) {
  const float t = __fmaf_rn(w, inv, 12582912.f);
  uint32_t q = __float_as_uint(t);
  const float r = __fmaf_rn(-s, __fsub_rn(t, 12582912.f), w);
  // Beyond a half, or at one from an odd number (beyond the value below it), one on towards the remainder.
  const float most = __uint_as_float(__float_as_uint(0.5f * s) - (q & 1u));
  if (fabsf(r) > most) q += static_cast<uint32_t>((__float_as_int(r) >> 31) | 1);
  return q;
}
// The same for scales whose half or reciprocal fp32 does not hold: in 64 bits (the quotient of two fp32 values cannot
// round onto a half in them), and clamped, since such a scale may be far from max / 7.
__device__ __noinline__ uint32_t code_of_tiny(float w, float s) {
  if (s == 0.f || !(s < INFINITY)) return 0;  // 0 times an infinity or a NaN is a NaN
  const double q = rint(static_cast<double>(w) / static_cast<double>(s));
  return static_cast<uint32_t>(static_cast<int>(fmin(fmax(q, -7.0), 7.0)));
}
// max / 7 rounded once: the product with 1/7 corrected by its remainder; the quotient's own rounding where fp32 does not
// hold that. (bf16's second rounding cannot meet a half between two values: seven of those are odd in nine bits.)
__device__ __forceinline__ float seventh(float top) {
  constexpr float inv = 1.f / 7.f;
  const float y = __fmul_rn(top, inv);
  return top >= 0x1p-90f && top < INFINITY ? __fmaf_rn(__fmaf_rn(-7.f, y, top), inv, y) : __fdiv_rn(top, 7.f);
}
__device__ __forceinline__ float largest(const float (&v)[8]) {
  float top = 0.f;
#pragma unroll
  for (int q = 0; q < 8; ++q) top = max_nan(top, fabsf(v[q]));
  return top;
}

// Eight weights as they are in memory.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void gather(const float* p, int left) {
    a = make_float4(left > 0 ? fetch(p) : 0.f, left > 1 ? fetch(p + 1) : 0.f, left > 2 ? fetch(p + 2) : 0.f, left > 3 ? fetch(p + 3) : 0.f);
    b = make_float4(left > 4 ? fetch(p + 4) : 0.f, left > 5 ? fetch(p + 5) : 0.f, left > 6 ? fetch(p + 6) : 0.f, left > 7 ? fetch(p + 7) : 0.f);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
template <>
struct Eight<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 r = __ldcs(reinterpret_cast<const uint4*>(p));
    w[0] = r.x; w[1] = r.y; w[2] = r.z; w[3] = r.w;
  }
  __device__ __forceinline__ void gather(const __nv_bfloat16* p, int left) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t low = left > 2 * q ? __bfloat16_as_ushort(fetch(p + 2 * q)) : 0u;
      const uint32_t high = left > 2 * q + 1 ? __bfloat16_as_ushort(fetch(p + 2 * q + 1)) : 0u;
      w[q] = low | (high << 16);
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = __uint_as_float(w[q] << 16);
      v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
    }
  }
};
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * q], v[2 * q + 1]);
    w[q] = *reinterpret_cast<const uint32_t*>(&b);
  }
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}

// Runs of segments of all rows one after the other, and how a warp finds its row: the quotient by a product with `inverse` (2^64 over
// the runs of a row, rounded up), exact below 2^32 of them; hundreds of instructions for a division beyond.
template <int kRun>
struct Places {
  int64_t out, in, blocks, groups, runs;
  unsigned long long inverse;
  int digits, vec;
  Places(int64_t rows, int64_t k, int group, bool aligned)
      : out(rows), in(k), blocks(blocks_of(k)), groups(groups_of(k, digits_of(group))), runs((k + kRun * kSegment - 1) / (kRun * kSegment)),
        inverse(runs > 1 ? ~0ull / static_cast<unsigned long long>(runs) + 1 : 0), digits(digits_of(group)), vec(aligned) {}
  int64_t items() const { return out * runs; }
  // A run's row, and its first k.
  __device__ __forceinline__ void find(int64_t at, int64_t* row, int64_t* k) const {
    *row = runs == 1 ? at
           : at <= 0xFFFFFFFFll && runs <= 0xFFFFFFFFll
               ? static_cast<int64_t>(__umul64hi(static_cast<unsigned long long>(at), inverse))
               : at / runs;
    *k = (at - *row * runs) * (kRun * kSegment);
  }
};
// Of the 256 k of a segment lane l has 8 l .. 8 l + 7: half a product's, for two of the four lanes that read a
// block. Its word within the codes, once lanes l and l ^ 2 (the products of one word) have exchanged halves.
__device__ __forceinline__ int word_of(int lane) {
  const int p = (lane >> 1) & 7, t = 2 * (lane & 1) + (p & 1);
  return (lane >> 4) * (kBlockBytes / 4) + t * 4 + (p >> 1);
}

// A warp a run of segments of a row; a group's lanes find its largest magnitude by shuffles.
// Bound by instructions next to memory: 67 M weights in bf16 44 us, 3.8 TB/s, in fp32 56, 5.4.
template <typename T>
__global__ void __launch_bounds__(kThreads) pack_kernel(const T* w, uint8_t* codes, T* scales, const Places<kPackRun> at) {
  let_next();
  after_previous();
  const int lane = threadIdx.x & 31, digits = at.digits;
  int64_t row, k0;
  at.find(static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5), &row, &k0);
  if (row >= at.out) return;
  // What is left of the row from this lane's first weight on, as far as the run goes.
  const int left = static_cast<int>(min(at.in - k0, static_cast<int64_t>(kPackRun * kSegment))) - lane * 8;
  const T* const from = w + row * at.in + k0 + lane * 8;
  Eight<T> raw[kPackRun];
#pragma unroll
  for (int u = 0; u < kPackRun; ++u) {
    if (at.vec && left >= u * kSegment + 8) raw[u].load(from + u * kSegment);
    else raw[u].gather(from + u * kSegment, left - u * kSegment);
  }
  T* const to_scales = scales + row * at.groups + ((k0 + lane * 8) >> digits);
  uint32_t* const to = reinterpret_cast<uint32_t*>(codes + (row * at.blocks + k0 / kBlock) * kBlockBytes) + word_of(lane);
  const bool first_of_group = (lane & ((1 << (digits - 3)) - 1)) == 0, odd = (lane & 2) != 0;
#pragma unroll
  for (int u = 0; u < kPackRun; ++u) {
    if (left + lane * 8 <= u * kSegment) break;
    float v[8];
    raw[u].get(v);
    float top = largest(v);
    for (int o = 1 << (digits - 4); o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const T stored = narrow<T>(seventh(top));
    const float s = value(stored);
    if (first_of_group && left > u * kSegment) to_scales[(u * kSegment) >> digits] = stored;
    uint32_t c[8];
    if (s >= 0x1p-100f && s < INFINITY) {
      const float inv = quick_reciprocal(s);
#pragma unroll
      for (int q = 0; q < 8; ++q) c[q] = code_of(T(), v[q], s, inv) & 15u;
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) c[q] = code_of_tiny(v[q], s) & 15u;
    }
    // The four codes for each of two reading lanes, of an even product; an odd one's lie 8 bits higher.
    const uint32_t a = c[0] + c[2] * 16u + c[1] * 65536u + c[3] * 1048576u, b = c[4] + c[6] * 16u + c[5] * 65536u + c[7] * 1048576u;
    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, odd ? a : b, 2);
    const uint32_t word = odd ? other | (b << 8) : a | (other << 8);
    // The last segment of a row may have one block only.
    if (lane < 16 || left + lane * 8 > u * kSegment + kBlock) to[u * (2 * kBlockBytes / 4)] = word ^ kNothing;
  }
}

// The codes of a lane's eight weights, from its word and that of the lane with the other product's.
__device__ __forceinline__ void codes_of(uint32_t word, int lane, float (&v)[8]) {
  const bool odd = (lane & 2) != 0;
  const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, word, 2);
  const uint32_t a = odd ? other >> 8 : word, b = odd ? word >> 8 : other;
  // A nibble as the last bits of 2^23.
  auto code = [](uint32_t n, int shift) { return __uint_as_float(((n >> shift) & 15u) | 0x4B000000u) - 8388616.f; };
  v[0] = code(a, 0); v[1] = code(a, 16); v[2] = code(a, 4); v[3] = code(a, 20);
  v[4] = code(b, 0); v[5] = code(b, 16); v[6] = code(b, 4); v[7] = code(b, 20);
}

// The same way back: 29 us and 5.8 TB/s, in fp32 46 and 6.5. Rows that start off a lane's 16 bytes go through shared
// memory, from where a warp stores neighbours.
template <typename T>
__global__ void __launch_bounds__(kThreads) unpack_kernel(const uint8_t* codes, const T* scales, T* w, const Places<kUnpackRun<T>> at) {
  constexpr int kRun = kUnpackRun<T>;
  __shared__ T staged[kWarps][kSegment];
  let_next();
  after_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t row, k0;
  at.find(static_cast<int64_t>(blockIdx.x) * kWarps + warp, &row, &k0);
  if (row >= at.out) return;
  const int run = static_cast<int>(min(at.in - k0, static_cast<int64_t>(kRun * kSegment))), left = run - lane * 8;
  const uint32_t* const from = reinterpret_cast<const uint32_t*>(codes + (row * at.blocks + k0 / kBlock) * kBlockBytes) + word_of(lane);
  const T* const scale = scales + row * at.groups + ((k0 + lane * 8) >> at.digits);
  uint32_t word[kRun];
  T s[kRun];
#pragma unroll
  for (int u = 0; u < kRun; ++u) {
    word[u] = kNothing;
    s[u] = narrow<T>(0.f);
    if (run > u * kSegment + (lane >> 4) * kBlock) word[u] = __ldcs(from + u * (2 * kBlockBytes / 4));
    if (left > u * kSegment) s[u] = fetch(scale + ((u * kSegment) >> at.digits));
  }
  T* const to = w + row * at.in + k0 + lane * 8;
#pragma unroll
  for (int u = 0; u < kRun; ++u) {
    if (run <= u * kSegment) break;
    float v[8];
    codes_of(word[u], lane, v);
    const float f = value(s[u]);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = __fmul_rn(v[q], f);
    if (at.vec && left >= u * kSegment + 8) {
      store8(to + u * kSegment, v);
    } else if (!at.vec) {
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 8; ++q) staged[warp][lane * 8 + q] = narrow<T>(v[q]);
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (u * kSegment + q * 32 + lane < run) to[u * kSegment + q * 32 + lane - lane * 8] = staged[warp][q * 32 + lane];
    }
  }
}

// ---------------------------------------------------------------- the linear layer
// Codes in units of 2^-10 of one product, in bf16: k pairs 0 and 1 of four, from bits `shift` on.
__device__ __forceinline__ uint32_t decode(uint32_t word, int shift) {
  uint32_t v = ((word >> shift) & 0x000F000Fu) | kMagic;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), __floats2bfloat162_rn(0.1328125f, 0.1328125f));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ void product(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr int kFeatures = 16;   // of a CTA

template <typename T>
constexpr int kTerms = sizeof(T) == 2 ? 1 : 3;  // bf16 terms of a value of x, each in a column of its own

template <typename T>
struct FourOf { using Type = uint2; };
template <>
struct FourOf<float> { using Type = float4; };
// Four values of x from k on, wherever the row starts, and those at or beyond `in` as zeros.
__device__ __forceinline__ uint2 four_of(const __nv_bfloat16* x, int64_t k, int64_t in) {
  uint32_t v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = k + q < in ? static_cast<uint32_t>(__bfloat16_as_ushort(fetch(x + k + q))) : 0u;
  return make_uint2(v[0] | (v[1] << 16), v[2] | (v[3] << 16));
}
__device__ __forceinline__ float4 four_of(const float* x, int64_t k, int64_t in) {
  float v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = k + q < in ? fetch(x + k + q) : 0.f;
  return make_float4(v[0], v[1], v[2], v[3]);
}
// A lane's values of the eight products of a block, from p on, 16 apart: aligned, or (within the row's inside, since
// whole words are read) from any address.
template <typename T>
__device__ __forceinline__ void aligned_block(const T* p, typename FourOf<T>::Type (&to)[8]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) to[q] = fetch(reinterpret_cast<const typename FourOf<T>::Type*>(p + q * 16));
}
__device__ __forceinline__ void shifted_block(const float* p, float4 (&to)[8]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) to[q] = make_float4(fetch(p + q * 16), fetch(p + q * 16 + 1), fetch(p + q * 16 + 2), fetch(p + q * 16 + 3));
}
__device__ __forceinline__ void shifted_block(const __nv_bfloat16* p, uint2 (&to)[8]) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const uint2* w = reinterpret_cast<const uint2*>(at & ~static_cast<uintptr_t>(7));
  const bool word = (at & 4) != 0;
  const uint32_t bits = (at & 2) * 8;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint2 a = fetch(w + q * 4), b = fetch(w + q * 4 + 1);
    const uint32_t v0 = word ? a.y : a.x, v1 = word ? b.x : a.y, v2 = word ? b.y : b.x;
    to[q] = make_uint2(__funnelshift_r(v0, v1, bits), __funnelshift_r(v1, v2, bits));
  }
}
// Their operand: for fp32 the column's term of each, the leading bits taken off once or twice by masks.
__device__ __forceinline__ uint2 operand(const uint2& v, uint32_t, uint32_t) { return v; }
__device__ __forceinline__ uint2 operand(const float4& v, uint32_t once, uint32_t twice) {
  auto one = [&](float x) {
    x -= __uint_as_float(__float_as_uint(x) & once);
    x -= __uint_as_float(__float_as_uint(x) & twice);
    return __float_as_uint(x);
  };
  return make_uint2(join_terms(one(v.x), one(v.y)), join_terms(one(v.z), one(v.w)));
}

// A CTA has 16 features, each warp a stretch of their k. kTiles: eights of columns (rows of x, times their terms);
// columns beyond the last repeat it, and nothing reads their results. Nothing is shared until the end: a warp's lanes read the
// codes, scales and values of x that their fragments take.
template <typename T, int kTiles, int kDigits>
__global__ void __launch_bounds__(kThreads, 2) packed_kernel(const PackedArgs a, int per, int vec) {
  constexpr int kWide = kTiles * 8 + 1;
  constexpr int kPerBlock = kBlock >> kDigits;        // groups of a block
  constexpr int kProducts = 1 << (kDigits - 4);       // products of a group
  __shared__ float parts[kWarps][kFeatures][kWide];
  let_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rows = static_cast<int>(a.rows), cols = rows * kTerms<T>;
  const int64_t j0 = static_cast<int64_t>(blockIdx.x) * kFeatures;
  const int64_t blocks = blocks_of(a.in), groups = groups_of(a.in, kDigits);
  const int64_t first = static_cast<int64_t>(warp) * per;
  const int count = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(per), blocks - first)));
  const bool there[2] = {j0 + g < a.out, j0 + g + 8 < a.out};
  const uint8_t* const codes = a.codes + ((j0 + g) * blocks + first) * kBlockBytes + t * 16;
  const int64_t group0 = first * kPerBlock + (t & (kPerBlock - 1));  // lane t of four reads the scale of group t
  const T* const scales = static_cast<const T*>(a.scales) + (j0 + g) * groups;
  // While the kernel before this one ends, the warp's first codes are asked for into L2 (a hint that reads nothing): a
  // lane takes one of the first two lines of a feature.
  if (j0 + (lane >> 1) < a.out && (lane & 1) * 2 < count)
    prefetch(a.codes + ((j0 + (lane >> 1)) * blocks + first + (lane & 1) * 2) * kBlockBytes);
  const T* from[kTiles];
  uint32_t once[kTiles], twice[kTiles];
#pragma unroll
  for (int n = 0; n < kTiles; ++n) {
    const int col = min(n * 8 + g, cols - 1);
    from[n] = static_cast<const T*>(a.x) + col / kTerms<T> * a.in + first * kBlock + t * 4;
    once[n] = col % kTerms<T> >= 1 ? 0xFFFF0000u : 0u;
    twice[n] = col % kTerms<T> >= 2 ? 0xFFFF0000u : 0u;
  }
  after_previous();
  float sum[kTiles][4] = {};
  constexpr int kInFlight = 2;
  for (int base = 0; base < count; base += kInFlight) {
    uint4 c[kInFlight][2];
    T s[kInFlight][2];
    typename FourOf<T>::Type x[8];
    auto load_x = [&](int d, int n) {
      const int64_t k = (first + base + d) * kBlock;
      const T* const p0 = from[n] + static_cast<int64_t>(base + d) * kBlock;
      if (vec && k + kBlock <= a.in) {
        aligned_block(p0, x);
      } else if (k > 0 && k + kBlock + 4 <= a.in) {
        shifted_block(p0, x);
      } else {
#pragma unroll
        for (int p = 0; p < 8; ++p) x[p] = four_of(p0 - t * 4 - k, k + p * 16 + t * 4, a.in);
      }
    };
#pragma unroll
    for (int d = 0; d < kInFlight; ++d) {
      const bool in = base + d < count;
      const int64_t at = group0 + static_cast<int64_t>(base + d) * kPerBlock;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        c[d][h] = make_uint4(kNothing, kNothing, kNothing, kNothing);
        if (in && there[h]) c[d][h] = __ldcs(reinterpret_cast<const uint4*>(codes + (base + d + h * 8 * blocks) * kBlockBytes));
        s[d][h] = narrow<T>(0.f);
        if (in && there[h] && at < groups) s[d][h] = fetch(scales + h * 8 * groups + at);
      }
    }
#pragma unroll
    for (int d = 0; d < kInFlight; ++d) {
      if (base + d >= count) break;
      const uint32_t w0[4] = {c[d][0].x, c[d][0].y, c[d][0].z, c[d][0].w}, w1[4] = {c[d][1].x, c[d][1].y, c[d][1].z, c[d][1].w};
      auto decoded = [&](int p, uint32_t (&op)[4]) {  // of a product of 16 k
        const int shift = (p & 1) * 8;
        op[0] = decode(w0[p >> 1], shift);
        op[1] = decode(w1[p >> 1], shift);
        op[2] = decode(w0[p >> 1], shift + 4);
        op[3] = decode(w1[p >> 1], shift + 4);
      };
      uint32_t ops[kTiles > 1 ? 8 : 1][4];  // kept where more than one tile takes them
      if constexpr (kTiles > 1) {
#pragma unroll
        for (int p = 0; p < 8; ++p) decoded(p, ops[p]);
      }
      const float s0 = value(s[d][0]), s1 = value(s[d][1]);
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        load_x(d, n);
        float part[4];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          if (p % kProducts == 0) part[0] = part[1] = part[2] = part[3] = 0.f;
          const uint2 b = operand(x[p], once[n], twice[n]);
          if constexpr (kTiles == 1) decoded(p, ops[0]);
          product(part, ops[kTiles > 1 ? p : 0], b.x, b.y);
          if (p % kProducts == kProducts - 1) {
            const float f0 = kPerBlock == 1 ? s0 : __shfl_sync(0xFFFFFFFFu, s0, p / kProducts, 4);
            const float f1 = kPerBlock == 1 ? s1 : __shfl_sync(0xFFFFFFFFu, s1, p / kProducts, 4);
            sum[n][0] = fmaf(part[0], f0, sum[n][0]);
            sum[n][1] = fmaf(part[1], f0, sum[n][1]);
            sum[n][2] = fmaf(part[2], f1, sum[n][2]);
            sum[n][3] = fmaf(part[3], f1, sum[n][3]);
          }
        }
      }
    }
  }
  // The warps' sums, in order.
#pragma unroll
  for (int n = 0; n < kTiles; ++n)
#pragma unroll
    for (int q = 0; q < 4; ++q) parts[warp][g + (q >> 1) * 8][n * 8 + t * 2 + (q & 1)] = sum[n][q];
  __syncthreads();
  for (int i = threadIdx.x; i < rows * kFeatures; i += kThreads) {
    const int r = i / kFeatures, f = i % kFeatures;
    const int64_t j = j0 + f;
    if (j >= a.out) continue;
    float z[1] = {0.f};
#pragma unroll
    for (int q = kTerms<T> - 1; q >= 0; --q) {  // the smallest terms first
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += parts[w][f][r * kTerms<T> + q];
      z[0] += v;
    }
    z[0] *= 1024.f;
    if (a.b != nullptr)
      z[0] += a.b_dt == VN_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.b)[j]) : static_cast<const float*>(a.b)[j];
    activate_all<false>(a.act, z);
    const int64_t at = r * a.out + j;
    if (a.residual != nullptr) z[0] += value(static_cast<const T*>(a.residual)[at]);
    static_cast<T*>(a.y)[at] = narrow<T>(z[0]);
  }
}

bool fits(const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

template <typename T, int kTiles, int kDigits>
cudaError_t run_digits(const PackedArgs& a, cudaStream_t stream) {
  const int64_t grid = (a.out + kFeatures - 1) / kFeatures, per = (blocks_of(a.in) + kWarps - 1) / kWarps;
  if (grid > 0x7FFFFFFFll || per > 0x3FFFFFFFll) return cudaErrorInvalidConfiguration;
  const int vec = a.in % 4 == 0 && fits(a.x, 4 * sizeof(T));
  return launch_overlapped(packed_kernel<T, kTiles, kDigits>, dim3(static_cast<unsigned>(grid)), kThreads, 0, 0, stream, a,
                           static_cast<int>(per), vec);
}
template <typename T, int kTiles>
cudaError_t run_tiles(const PackedArgs& a, cudaStream_t stream) {
  switch (digits_of(a.group)) {
    case 5: return run_digits<T, kTiles, 5>(a, stream);
    case 6: return run_digits<T, kTiles, 6>(a, stream);
    default: return run_digits<T, kTiles, 7>(a, stream);
  }
}

template <typename T>
cudaError_t run_packed(const PackedArgs& a, cudaStream_t stream) {
  const int64_t cols = a.rows * kTerms<T>;
  if (cols <= 8) return run_tiles<T, 1>(a, stream);
  if (cols <= 16) return run_tiles<T, 2>(a, stream);
  return run_tiles<T, 4>(a, stream);
}

template <typename T>
cudaError_t pack_typed(const void* w, int64_t out, int64_t in, int group, uint8_t* codes, void* scales, cudaStream_t stream) {
  const Places<kPackRun> at(out, in, group, in % 8 == 0 && fits(w, 16));
  const int64_t grid = (at.items() + kWarps - 1) / kWarps;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  return launch_overlapped(pack_kernel<T>, dim3(static_cast<unsigned>(grid)), kThreads, 0, 0, stream, static_cast<const T*>(w), codes,
                           static_cast<T*>(scales), at);
}
template <typename T>
cudaError_t unpack_typed(const uint8_t* codes, const void* scales, int64_t out, int64_t in, int group, void* w, cudaStream_t stream) {
  const Places<kUnpackRun<T>> at(out, in, group, in % 8 == 0 && fits(w, 16));
  const int64_t grid = (at.items() + kWarps - 1) / kWarps;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  return launch_overlapped(unpack_kernel<T>, dim3(static_cast<unsigned>(grid)), kThreads, 0, 0, stream, codes,
                           static_cast<const T*>(scales), static_cast<T*>(w), at);
}

// ---------------------------------------------------------------- many rows
// The most rows that the kernel on packed weights takes (both sides at the top of this file).
int64_t few_rows(vn_dtype dt) { return dt == VN_BF16 ? 32 : 10; }

int64_t padded(int64_t bytes) { return (bytes + 255) / 256 * 256; }

// In bf16 a value, code times scale, has up to 11 significant bits and would be rounded to 8: so it is taken as the sum of two bf16
// values, its leading 8 bits and the rest, which is exact (but for a rest below 2^-133). The plain layer runs on rows of twice the length,
//   [x | x] [leading | rest]^T,
// with each half padded by zeros to whole 16 bytes, and adds both up in one accumulator: no value is rounded whatever the rows.
constexpr int64_t kTermRows = 16384;  // rows of x that are laid out at once
constexpr int kTermRun = 2;
int64_t half_of(int64_t in) { return (in + 7) / 8 * 8; }

// The first `weight_ctas` CTAs lay out the weights, a warp a run of segments of a row; the others x, eight elements a
// thread. x's second copy has zeros for infinities (and NaN): the first one's products are theirs, and an infinity times a rest of 0 is none.
__global__ void __launch_bounds__(kThreads)
terms_kernel(const uint8_t* codes, const __nv_bfloat16* scales, uint4* w, const Places<kTermRun> at, int64_t weight_ctas,
             const __nv_bfloat16* x, uint4* xx, int64_t rows, int vec) {
  let_next();
  after_previous();
  const int64_t words = (at.in + 7) / 8;  // 16-byte words of a half
  if (blockIdx.x >= weight_ctas) {
    const int64_t i = (blockIdx.x - weight_ctas) * kThreads + threadIdx.x;
    if (i >= rows * words) return;
    const int64_t row = i / words, word = i - row * words;
    Eight<__nv_bfloat16> v;
    if (vec) v.load(x + row * at.in + word * 8);
    else v.gather(x + row * at.in + word * 8, static_cast<int>(min(at.in - word * 8, static_cast<int64_t>(8))));
    uint32_t finite[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      finite[q] = v.w[q] & (((v.w[q] & 0x7F80u) == 0x7F80u ? 0u : 0xFFFFu) | ((v.w[q] & 0x7F800000u) == 0x7F800000u ? 0u : 0xFFFF0000u));
    uint4* const to = xx + row * 2 * words + word;
    to[0] = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    to[words] = make_uint4(finite[0], finite[1], finite[2], finite[3]);
    return;
  }
  const int lane = threadIdx.x & 31;
  int64_t row, k0;
  at.find(static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5), &row, &k0);
  if (row >= at.out) return;
  const int run = static_cast<int>(min(at.in - k0, static_cast<int64_t>(kTermRun * kSegment))), left = run - lane * 8;
  const uint32_t* const from = reinterpret_cast<const uint32_t*>(codes + (row * at.blocks + k0 / kBlock) * kBlockBytes) + word_of(lane);
  const __nv_bfloat16* const scale = scales + row * at.groups + ((k0 + lane * 8) >> at.digits);
  uint4* const to = w + row * 2 * words + (k0 >> 3) + lane;
  uint32_t word[kTermRun];
  float s[kTermRun];
#pragma unroll
  for (int u = 0; u < kTermRun; ++u) {
    word[u] = run > u * kSegment + (lane >> 4) * kBlock ? __ldcs(from + u * (2 * kBlockBytes / 4)) : kNothing;
    s[u] = left > u * kSegment ? value(fetch(scale + ((u * kSegment) >> at.digits))) : 0.f;
  }
#pragma unroll
  for (int u = 0; u < kTermRun; ++u) {
    if (run <= u * kSegment) break;
    float v[8];
    codes_of(word[u], lane, v);
    if (left <= u * kSegment) continue;
    uint32_t leading[8], rest[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float z = __fmul_rn(v[q], s[u]);  // exact
      const uint32_t upper = __float_as_uint(z) & 0xFFFF0000u;
      leading[q] = upper;
      rest[q] = (upper & 0x7F800000u) == 0x7F800000u ? 0u : __float_as_uint(__fsub_rn(z, __uint_as_float(upper)));
    }
    to[u * (kSegment / 8)] = make_uint4(join_terms(leading[0], leading[1]), join_terms(leading[2], leading[3]),
                                        join_terms(leading[4], leading[5]), join_terms(leading[6], leading[7]));
    to[u * (kSegment / 8) + words] = make_uint4(join_terms(rest[0], rest[1]), join_terms(rest[2], rest[3]),
                                                join_terms(rest[4], rest[5]), join_terms(rest[6], rest[7]));
  }
}

cudaError_t run_terms(const PackedArgs& a, cudaStream_t stream) {
  const int64_t half = half_of(a.in);
  uint8_t* const w = static_cast<uint8_t*>(a.workspace);
  uint8_t* const xx = w + padded(a.out * half * 4);
  const Places<kTermRun> at(a.out, a.in, a.group, true);
  const int vec = a.in % 8 == 0 && fits(a.x, 16);
  for (int64_t r = 0; r < a.rows; r += kTermRows) {
    const int64_t rows = std::min(kTermRows, a.rows - r);
    const int64_t weight_ctas = r == 0 ? (at.items() + kWarps - 1) / kWarps : 0;
    const int64_t grid = weight_ctas + (rows * (half / 8) + kThreads - 1) / kThreads;
    if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    const __nv_bfloat16* const x = static_cast<const __nv_bfloat16*>(a.x) + r * a.in;
    cudaError_t err = launch_overlapped(terms_kernel, dim3(static_cast<unsigned>(grid)), kThreads, 0, 0, stream, a.codes,
                                        static_cast<const __nv_bfloat16*>(a.scales), reinterpret_cast<uint4*>(w), at, weight_ctas, x,
                                        reinterpret_cast<uint4*>(xx), rows, vec);
    if (err != cudaSuccess) return err;
    DenseArgs d = {};
    d.x = xx; d.w = w; d.dt = VN_BF16; d.b = a.b; d.b_dt = a.b_dt;
    d.residual = a.residual != nullptr ? static_cast<const __nv_bfloat16*>(a.residual) + r * a.out : nullptr;
    d.rows = rows; d.in = 2 * half; d.out = a.out; d.act = a.act;
    d.y = static_cast<__nv_bfloat16*>(a.y) + r * a.out;
    if ((err = launch_dense(d, stream)) != cudaSuccess) return err;
  }
  return cudaSuccess;
}

// Rows too long for that: the kernel on packed weights, as many rows as it takes at a time.
cudaError_t run_slices(const PackedArgs& a, cudaStream_t stream) {
  for (int64_t r = 0; r < a.rows; r += few_rows(VN_BF16)) {
    PackedArgs one = a;
    one.rows = std::min(few_rows(VN_BF16), a.rows - r);
    one.x = static_cast<const __nv_bfloat16*>(a.x) + r * a.in;
    if (a.residual != nullptr) one.residual = static_cast<const __nv_bfloat16*>(a.residual) + r * a.out;
    one.y = static_cast<__nv_bfloat16*>(a.y) + r * a.out;
    const cudaError_t err = run_packed<__nv_bfloat16>(one, stream);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}
bool sliced(vn_dtype dt, int64_t in) { return dt == VN_BF16 && 2 * half_of(in) > kDenseMost; }

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
  if (rows <= few_rows(dt) || sliced(dt, in)) return 0;
  if (dt == VN_BF16) {  // out and half are below 2^31 here; rows that are as they are need no workspace in the plain layer
    return padded(out * half_of(in) * 4) + padded(std::min(rows, kTermRows) * half_of(in) * 4);
  }
  return padded(out * in * 4) + dense_workspace(rows, in, out, dt, aligned);
}

// Many rows: the weights' values, then the plain layer.
cudaError_t launch_packed(const PackedArgs& a, cudaStream_t stream) {
  if (a.rows <= few_rows(a.dt)) return a.dt == VN_BF16 ? run_packed<__nv_bfloat16>(a, stream) : run_packed<float>(a, stream);
  if (a.dt == VN_BF16 && a.in > 0) return sliced(a.dt, a.in) ? run_slices(a, stream) : run_terms(a, stream);
  if (a.in > 0) {  // else there is nothing to unpack, and the sums are zeros
    const cudaError_t err = launch_unpack(a.codes, a.scales, a.dt, a.out, a.in, a.group, a.workspace, stream);
    if (err != cudaSuccess) return err;
  }
  DenseArgs d = {};
  d.x = a.x; d.w = a.workspace; d.dt = a.dt; d.b = a.b; d.b_dt = a.b_dt; d.residual = a.residual;
  d.rows = a.rows; d.in = a.in; d.out = a.out; d.act = a.act; d.y = a.y;
  d.workspace = static_cast<uint8_t*>(a.workspace) + padded(a.out * a.in * 4);
  return launch_dense(d, stream);
}

}  // namespace vn
