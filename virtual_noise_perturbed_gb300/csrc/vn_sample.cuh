// vn_sample.cuh -- an index for each row of logits, drawn with a given random number:
//
//   w_i = exp((x_i - max x) / T);   order: x descending, index ascending
//   kept = the first top_k of the order, of those the ones before which less than top_p of the sum lies,
//          and w_i >= min_p                                      (all three are prefixes of the order)
//   index = the smallest i, in index order, with  sum_{j <= i, kept} w_j > u S,  S the sum of all kept w
//
// Which index it is hangs on sums next to a border, so a weight is a whole number: w in units of 2^-42, good
// to 2^-35 of itself and half a unit. Sums of whole numbers are exact in any order, whatever adds them: lanes, CTAs of
// a cluster, atomics. So a sum over a row is good to 2^-35 of itself and n 2^-43 (the largest weight is 1): 2^-24 on the longest
// rows, where all of it lies in a flat tail some 29 T below the largest logit. (With sums of fp32 one row in a hundred of 4,096 would differ from float64's index.)
// Such a weight takes some 45 instructions, so rows beyond 128 logits are decided by coarse weights of 10,
// whose sums' error is bounded, and by whole ones only where a border lies within that bound: one row in
// fifty at 4,096 logits, half of them at 131,072.
//
// A row is read once, into registers or shared memory, and every later pass goes over that copy. Up to 16 logits a part of a warp has
// a row, and each logit looks at all others. Up to 128
// logits (256 where rows are few) a warp has a row in registers, and finds where a prefix ends by bisecting the bits of a logit.
// Beyond, a CTA or a cluster of CTAs has one: each warp holds a contiguous stretch of it and each lane every 32nd 16 bytes of that,
// the ones that it read itself. A histogram over x in units of T tells the bin in which a prefix ends; the logits of that
// bin, some tens, are listed, and each finds its place and what lies before it by a look at all others. With a
// small top_k everything kept is listed, and the rest of the work is done on the list.
//
// Bound by memory in principle (a row once); in fact by instructions, 35 to 70 a logit with what a row costs apart from them, at
// half of the issue rate: 20 to 32 warps an SM that wait for one another's results. 16384 rows of 4096 bf16: 102 us without filters, 134 with
// top_k 50, 233 with top_p 0.9 (20 for reading them); 32 of 131071 fp32: 17 with top_k; 1024 rows of 8: 1.9; one of 4096: 4.1 to 8.2.
// (Compiled once for each type of the logits, vn_sample_f32.cu and vn_sample_bf16.cu, to build in half the time.)
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "vn_act.cuh"
#include "vn_internal.h"
#include "vn_launch.cuh"

namespace cg = cooperative_groups;

namespace vn {
namespace {

using u64 = unsigned long long;
constexpr int kUnit = 42;                // weights are in units of 2^-42
constexpr u64 kOne = 1ull << kUnit;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 256;

// 2^(-j/32) in units of 2^-42.
__constant__ const u64 kPowersInit[32] = {
    4398046511104ull, 4303805443529ull, 4211583767698ull, 4121338212211ull, 4033026432885ull, 3946606992882ull,
    3862039343274ull, 3779283804012ull, 3698301545306ull, 3619054569413ull, 3541505692798ull, 3465618528697ull,
    3391357470036ull, 3318687672730ull, 3247575039328ull, 3177986203020ull, 3109888511975ull, 3043250014027ull,
    2978039441675ull, 2914226197418ull, 2851780339397ull, 2790672567345ull, 2730874208839ull, 2672357205845ull,
    2615094101559ull, 2559058027516ull, 2504222690988ull, 2450562362647ull, 2398051864490ull, 2346666558027ull,
    2296382332721ull, 2247175594673ull};

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <typename T>
__device__ __forceinline__ T lowest() { return narrow<T>(-INFINITY); }

// Bits of a float in its order, -0 as +0; below kLowest for the NaN that stands for no logit (a sign and all
// other bits, in bf16 those of its upper half).
__device__ __forceinline__ uint32_t key_of(float x) {
  uint32_t b = __float_as_uint(x);
  b = b == 0x80000000u ? 0u : b;
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of_key(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ float absent() { return __uint_as_float(0xFFFFFFFFu); }
constexpr uint32_t kLowest = 0x10000;  // below every logit's key

struct Rows {
  const void* x;
  int64_t rows, n;
  const float* u;
  float temperature, min_p;
  u64 top_p;  // a share of 2^64, all ones for everything
  int64_t top_k;
  const float* temperatures;
  const int64_t* top_ks;
  const float* top_ps;
  const float* min_ps;
  int64_t* index;
  float* logprob;
  float ch, cl;   // 32 log2(e) / temperature
  u64 min_units;  // min_p in units, rounded up
};

// p 2^42 rounded up, of p in (0, 1].
__device__ __forceinline__ u64 units_of(float p) {
  const uint32_t b = __float_as_uint(p);
  const int up = static_cast<int>(b >> 23) - 150 + kUnit;  // p = mantissa 2^(up - 42)
  const u64 mantissa = (b & 0x7FFFFFu) | 0x800000u;
  if (up >= 0) return mantissa << min(up, 40);
  return up < -24 ? 1 : (mantissa + (1ull << -up) - 1) >> -up;
}

constexpr u64 kAllOfIt = ~0ull;

// floor(u s) for u of [0, 1), s = 2^64 hi + lo; the last unit of lo for more, 0 for less.
__device__ __forceinline__ u64 share(float u, u64 lo, u64 hi) {
  if (!(u > 0.f)) return 0;
  if (u >= 1.f) return lo - 1;
  const uint32_t b = __float_as_uint(u);
  const int e = static_cast<int>(b >> 23);                               // u = mantissa 2^(e - 150)
  if (e < 64) return 0;                                                  // u s is below 1, and 2^64 u of no account
  const u64 mantissa = (b & 0x7FFFFFu) | 0x800000u;
  const u64 top = __umul64hi(lo, mantissa) + hi * mantissa, bottom = lo * mantissa;
  const int down = 150 - e;                                              // 24 .. 86
  return down < 64 ? (bottom >> down) | (top << (64 - down)) : top >> (down - 64);
}
__device__ __forceinline__ u64 share(float u, u64 s) { return share(u, s, 0); }
// The smallest whole number that is not below p s, one at least; what float64's product would round away (2^-53 of it) is
// taken off first.
__device__ __forceinline__ u64 nucleus(u64 p, u64 s) {
  const u64 hi = __umul64hi(s, p), lo = s * p;
  const u64 rounded = s < (1ull << 53) ? s << 11 : ~0ull;
  const u64 up = hi + (lo > rounded ? 1 : 0);
  return up == 0 ? 1 : up;
}

// What a row asks for.
struct Wish {
  float u, temperature, min_p;
  float ch, cl;    // 32 log2(e) / T in two parts
  u64 top_p;       // a share of 2^64; all ones: everything
  int64_t top_k;
  u64 min_units;   // min_p in units, rounded up
  bool bad;        // a parameter is not a number
};

__device__ __forceinline__ Wish wish_of(const Rows& a, int64_t row) {
  Wish w;
  w.u = fetch(a.u + row);
  w.temperature = a.temperature;
  w.ch = a.ch;
  w.cl = a.cl;
  w.top_p = a.top_p;
  w.min_p = a.min_p;
  w.top_k = a.top_k;
  if (a.temperatures != nullptr) {
    const float t = fetch(a.temperatures + row);
    w.temperature = t;
    constexpr double k = 46.16624130844683;  // 32 log2(e)
    constexpr float kh = static_cast<float>(k), kl = static_cast<float>(k - static_cast<double>(kh));
    w.ch = __fdiv_rn(kh, t);
    w.cl = __fdiv_rn(__fadd_rn(__fmaf_rn(-w.ch, t, kh), kl), t);
    if (!(fabsf(w.cl) < INFINITY)) w.cl = 0.f;  // an infinite temperature, or one whose reciprocal is
  }
  if (a.top_ks != nullptr) w.top_k = fetch(a.top_ks + row);
  bool bad = false;
  if (a.top_ps != nullptr) {
    const float p = fetch(a.top_ps + row);
    bad = p != p;
    w.top_p = p >= 1.f ? kAllOfIt : share(p, 0, 1);
  }
  w.min_units = a.min_units;
  if (a.min_ps != nullptr) {
    w.min_p = fetch(a.min_ps + row);
    w.min_units = units_of(w.min_p);
  }
  w.bad = bad || w.u != w.u || w.temperature != w.temperature || w.min_p != w.min_p;
  if (!(w.temperature > 0.f)) {  // the largest
    w.top_k = 1;
    w.ch = 46.16624130844683f;
    w.cl = 0.f;
  }
  if (w.top_k <= 0 || w.top_k > a.n) w.top_k = a.n;
  if (w.min_p > 1.f) {
    w.min_p = 1.f;
    w.min_units = kOne;
  }
  return w;
}

// (m - x) 32 log2(e) / T in two parts. What both subtractions round off is carried along.
__device__ __forceinline__ float distance(float x, float m, const Wish& w, float* low) {
  const float d = __fsub_rn(m, x), b = __fsub_rn(d, m);
  const float dl = __fsub_rn(__fsub_rn(m, __fsub_rn(d, b)), __fadd_rn(x, b));
  const float p = __fmul_rn(d, w.ch);
  *low = __fmaf_rn(dl, w.ch, __fmaf_rn(d, w.cl, __fmaf_rn(d, w.ch, -p)));
  return p;
}

// exp((x - m) / T) in units of 2^-42: 2^-(k + j / 32) from the table and 2^-(r / 32) - 1, |r| <= 1/2, from its Taylor
// series to r^4 (the next term is 2^-39), whose first term is taken in two parts; in all 2e-11 of the weight.
__device__ __forceinline__ u64 weight(float x, float m, const Wish& w, const u64* powers) {
  if (x == m) return kOne;
  float e;
  const float p = distance(x, m, w, &e);
  if (!(p < 43.f * 32.f)) return 0;  // below half a unit (and no logit, and -inf)
  const float shifted = __fadd_rn(p, 12582912.f);
  const int32_t kj = __float_as_int(shifted) - 0x4B400000;
  const float r0 = __fsub_rn(p, __fsub_rn(shifted, 12582912.f));
  const float r = __fadd_rn(r0, e), rl = __fadd_rn(__fsub_rn(r0, r), e);
  constexpr double b = -0.021660849392498290;  // -ln 2 / 32
  constexpr float bh = static_cast<float>(b), bl = static_cast<float>(b - static_cast<double>(bh));
  constexpr float b2 = static_cast<float>(b * b / 2), b3 = static_cast<float>(b * b * b / 6),
                  b4 = static_cast<float>(b * b * b * b / 24);
  const float first = __fmul_rn(bh, r);
  float rest = __fmaf_rn(bh, rl, __fmaf_rn(bl, r, __fmaf_rn(bh, r, -first)));
  const float s = __fmaf_rn(__fmaf_rn(b4, r, b3), r, b2);
  rest = __fmaf_rn(__fmul_rn(s, r), r, rest);
  // In units of 2^-36: the first part as it is, the rest, below 2^22 of them, by its bits.
  const int32_t q = __float2int_rn(__fmul_rn(first, 0x1p36f)) + __float_as_int(__fmaf_rn(rest, 0x1p36f, 12582912.f)) - 0x4B400000;
  const u64 t = powers[kj & 31];
  const int64_t part = (static_cast<int64_t>(static_cast<int32_t>(t >> 12)) * q) >> 24;
  const u64 v = t + static_cast<u64>(part);
  const int k = kj >> 5;
  return k > 0 ? (v + (1ull << (k - 1))) >> k : v;
}

// The log of a kept logit's share: -(m - x) / T - ln(S), S in units of the largest weight.
__device__ __forceinline__ float logprob_of(float x, float m, const Wish& w, u64 s) {
  float d = 0.f;
  if (x != m) {
    float e;
    const float p = distance(x, m, w, &e);
    d = __fmul_rn(__fadd_rn(p, e), 0.021660849392498290f);
  }
  return -d - log1pf(static_cast<float>(s - kOne) * 0x1p-42f);
}

// Where the min-p prefix ends, for logits next to its border by their weights. The estimate is off by a few
// roundings of |m| and T ln(min_p), `sure` has 2^-20 of them, and by min_p's own rounding to fp32, which is 2^-24 T: `sure` has 2^-23 T.
struct Floor {
  float at, sure;
  __device__ __forceinline__ Floor(float m, const Wish& w) {
    const float drop = logf(w.min_p) * w.temperature;
    at = m + drop;
    sure = 0x1p-20f * (fabsf(m) + fabsf(drop)) + 0x1p-23f * fabsf(w.temperature) + 1e-37f;
  }
  // (At an infinite temperature with a min_p of 1 the estimate is a NaN, and weights decide; so they do for no logit, which has none.)
  __device__ __forceinline__ bool above(float x, float m, const Wish& w, const u64* powers) const {
    if (x == m || x >= at + sure) return true;
    if (x < at - sure) return false;
    return weight(x, m, w, powers) >= w.min_units;
  }
};

// Of sums below 2^59 a lane: three times 27 bits, whose sums over a warp fit 32.
__device__ __forceinline__ u64 warp_sum(u64 v) {
  constexpr uint32_t kPart = (1u << 27) - 1;
  const u64 a = __reduce_add_sync(kAll, static_cast<uint32_t>(v) & kPart), b = __reduce_add_sync(kAll, static_cast<uint32_t>(v >> 27) & kPart),
            c = __reduce_add_sync(kAll, static_cast<uint32_t>(v >> 54));
  return a + (b << 27) + (c << 54);
}
__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 t = __shfl_up_sync(kAll, v, o);
    if (lane >= o) v += t;
  }
  return v;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// The largest logit of 16 bytes, NaN if one is.
template <typename T>
__device__ __forceinline__ float largest_of(const uint4& raw) {
  if constexpr (sizeof(T) == 2) {
    uint32_t a, b;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(raw.x), "r"(raw.y));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(raw.z), "r"(raw.w));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
    return max_nan(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u));
  } else {
    return max_nan(max_nan(__uint_as_float(raw.x), __uint_as_float(raw.y)), max_nan(__uint_as_float(raw.z), __uint_as_float(raw.w)));
  }
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// What is kept so far: keys above `key`, and of those equal to it the ones at an index up to `last`.
struct Kept {
  uint32_t key = kLowest;
  int32_t last = 0x7FFFFFFF;
  __device__ __forceinline__ bool holds(uint32_t k, int32_t at) const { return k > key || (k == key && at <= last); }
};

// ---------------------------------------------------------------- G lanes a row, up to 16 logits
// Of each logit its place in the order and what lies before it come from a look at every other. A policy's handful of actions would leave
// most of a warp idle, and bisection takes a round for each bit: 16384 rows of 8 fp32 take 2.6 us here (with top-p 3.7) and 7.3 (27) with
// a warp a row, of 16 4.2 (7.1) and 7.3 (28); 1024 rows of 8 1.9 (2.3) and 2.3 (5.3).
template <typename T, int G>
__global__ void __launch_bounds__(kThreads) group_kernel(const Rows a) {
  __shared__ u64 powers[32];
  let_next();
  if (threadIdx.x < 32) powers[threadIdx.x] = kPowersInit[threadIdx.x];
  __syncthreads();
  after_previous();
  constexpr int kRows = kThreads / G;
  const int lane = threadIdx.x % G, n = static_cast<int>(a.n);
  const uint32_t group = ((1u << G) - 1u) << (threadIdx.x % 32 - lane);  // other groups of the warp go their own ways
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / G; row < a.rows; row += static_cast<int64_t>(gridDim.x) * kRows) {
    const float v = lane < n ? value(fetch(static_cast<const T*>(a.x) + row * n + lane)) : absent();
    float m = lane < n ? v : -INFINITY;
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(group, m, o));
    const Wish w = wish_of(a, row);
    if (w.bad || m != m || m == -INFINITY) {
      if (lane == 0) {
        a.index[row] = -1;
        if (a.logprob != nullptr) a.logprob[row] = NAN;
      }
      continue;
    }
    u64 mine = weight(v, m, w, powers);
    bool kept = lane < n;
    if (w.top_k < n || w.top_p != kAllOfIt) {
      const uint32_t key = key_of(v);
      int rank = 0;
      u64 before = 0;
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const uint32_t other = __shfl_sync(group, key, j, G);
        const u64 its = __shfl_sync(group, mine, j, G);
        const bool earlier = other > key || (other == key && j < lane);
        rank += earlier;
        before += earlier ? its : 0;
      }
      kept = kept && rank < w.top_k;
      if (w.top_p != kAllOfIt) {
        u64 all = kept ? mine : 0;
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) all += __shfl_xor_sync(group, all, o);
        kept = kept && (rank == 0 || before < nucleus(w.top_p, all));
      }
    }
    if (w.min_p > 0.f) kept = kept && Floor(m, w).above(v, m, w, powers);
    if (!kept) mine = 0;
    u64 scan = mine;
#pragma unroll
    for (int o = 1; o < G; o <<= 1) {
      const u64 t = __shfl_up_sync(group, scan, o, G);
      if (lane >= o) scan += t;
    }
    const u64 s = __shfl_sync(group, scan, G - 1, G), r = share(w.u, s);
    if (scan > r && scan - mine <= r) {
      a.index[row] = lane;
      if (a.logprob != nullptr) a.logprob[row] = logprob_of(v, m, w, s);
    }
  }
}

// ---------------------------------------------------------------- a warp a row
// Lane l holds the logits l, l + 32, ..
template <typename T, int R>
__global__ void __launch_bounds__(kThreads) warp_kernel(const Rows a) {
  __shared__ u64 powers[32];
  let_next();
  if (threadIdx.x < 32) powers[threadIdx.x] = kPowersInit[threadIdx.x];
  __syncthreads();
  after_previous();
  const int lane = threadIdx.x & 31;
  const int n = static_cast<int>(a.n);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); row < a.rows;
       row += static_cast<int64_t>(gridDim.x) * kWarps) {
    const T* x = static_cast<const T*>(a.x) + row * n;
    float v[R];
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      v[j] = j * 32 + lane < n ? value(fetch(x + j * 32 + lane)) : absent();
      if (j * 32 + lane < n) m = max_nan(m, v[j]);
    }
    m = warp_max(m);
    const Wish w = wish_of(a, row);
    if (w.bad || m != m || m == -INFINITY) {
      if (lane == 0) {
        a.index[row] = -1;
        if (a.logprob != nullptr) a.logprob[row] = NAN;
      }
      continue;
    }
    u64 weights[R];
    uint32_t keys[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      keys[j] = key_of(v[j]);
      weights[j] = weight(v[j], m, w, powers);
    }
    Kept kept;
    // The index of the tie number `count` (from 1) of kept.key.
    auto tie = [&](int count) {
      kept.last = 0x7FFFFFFF;
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const uint32_t same = __ballot_sync(kAll, keys[j] == kept.key);
        const bool it = keys[j] == kept.key && __popc(same & ((1u << lane) - 1u)) == count - 1;
        const uint32_t hit = __ballot_sync(kAll, it);
        if (hit != 0) kept.last = j * 32 + __ffs(hit) - 1;
        count -= __popc(same);
      }
    };
    constexpr int kBits = sizeof(T) == 2 ? 16 : 32;
    auto shown = [&](uint32_t k) { return sizeof(T) == 2 ? k >> 16 : k; };
    if (w.top_k < n) {
      // The largest key that at least top_k logits reach.
      uint32_t key = 0;
      if (w.top_k == 1) {
        key = shown(key_of(m));
      } else {
        for (int b = kBits - 1; b >= 0; --b) {
          const uint32_t c = key | (1u << b);
          int count = 0;
#pragma unroll
          for (int j = 0; j < R; ++j) count += shown(keys[j]) >= c;
          if (static_cast<int>(__reduce_add_sync(kAll, static_cast<unsigned>(count))) >= w.top_k) key = c;
        }
      }
      int above = 0;
      uint32_t exact = 0;
#pragma unroll
      for (int j = 0; j < R; ++j) {
        above += shown(keys[j]) > key;
        if (shown(keys[j]) == key) exact = keys[j];
      }
      kept.key = __reduce_max_sync(kAll, exact);
      tie(static_cast<int>(w.top_k) - static_cast<int>(__reduce_add_sync(kAll, static_cast<unsigned>(above))));
    }
    auto sum_of = [&](auto take) {
      u64 s = 0;
#pragma unroll
      for (int j = 0; j < R; ++j) s += take(j) ? weights[j] : 0;
      return warp_sum(s);
    };
    if (w.top_p != kAllOfIt && w.top_k > 1) {
      const Kept before = kept;
      auto in = [&](int j) { return before.holds(keys[j], j * 32 + lane); };
      const u64 p = nucleus(w.top_p, sum_of(in));
      // The largest key whose logits and those above reach the nucleus.
      uint32_t key = 0;
      for (int b = kBits - 1; b >= 0; --b) {
        const uint32_t c = key | (1u << b);
        if (sum_of([&](int j) { return in(j) && shown(keys[j]) >= c; }) >= p) key = c;
      }
      const u64 above = sum_of([&](int j) { return in(j) && shown(keys[j]) > key; });
      uint32_t exact = 0;
      u64 each = 0;
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (in(j) && shown(keys[j]) == key) { exact = keys[j]; each = weights[j]; }
      kept.key = __reduce_max_sync(kAll, exact);
      const int owner = __ffs(__ballot_sync(kAll, each != 0)) - 1;
      each = __shfl_sync(kAll, each, owner < 0 ? 0 : owner);
      const u64 ties = each == 0 ? 1 : (p - above + each - 1) / each;
      tie(ties > static_cast<u64>(n) ? n : static_cast<int>(ties));
      if (kept.key == before.key && before.last < kept.last) kept.last = before.last;
    }
    if (w.min_p > 0.f) {
      const Floor floor(m, w);
      uint32_t least = kAll;
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (floor.above(v[j], m, w, powers)) least = min(least, keys[j]);
      least = __reduce_min_sync(kAll, least);
      if (least > kept.key) {
        kept.key = least;
        kept.last = 0x7FFFFFFF;
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (!kept.holds(keys[j], j * 32 + lane)) weights[j] = 0;
    const u64 s = sum_of([](int) { return true; });
    u64 r = share(w.u, s);
    bool found = false;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (found) continue;
      const u64 scan = warp_scan(weights[j], lane);
      const uint32_t over = __ballot_sync(kAll, scan > r);
      if (over != 0) {
        found = true;
        if (lane == __ffs(over) - 1) {
          a.index[row] = j * 32 + lane;
          if (a.logprob != nullptr) a.logprob[row] = logprob_of(v[j], m, w, s);
        }
      }
      r -= __shfl_sync(kAll, scan, 31);
    }
  }
}

// ---------------------------------------------------------------- a CTA of W warps, or a cluster of them, a row
// What is kept of a row: logits above `edge`, and of those equal to it the ones at an index up to `last`.
struct Prefix {
  float edge = -INFINITY;
  int32_t last = 0x7FFFFFFF;
  __device__ __forceinline__ bool holds(float x, int32_t at) const { return x > edge || (x == edge && at <= last); }
};

// exp((x - m) / T) in a quarter of weight()'s instructions. The difference's rounding is left in: with t = (m - x) / (T ln 2) it
// is t 2^-24 ln 2 of the weight, and the mean of t over the weights of 2^19 logits at most 14.2: 6e-7 of a sum. The
// exponential is good to 2^-22.5, a sum of eight to 2^-22, so two sums differ from the exact ones by less than kSure of all: what is
// decided by them is sure where it is further than that from a border, and else decided by weight(). 0 for the largest
// logits themselves, whose ones would drown a small rest: they are counted.
constexpr float kSure = 2.2e-6f;
__device__ __forceinline__ float coarse(float x, float m, float c, float cl, float* below) {  // c, cl: log2(e) / T in two parts
  const float d = __fsub_rn(m, x), p = __fmul_rn(d, c);
  const float e = __fmaf_rn(d, cl, __fmaf_rn(d, c, -p));
  const float v = quick_exp2(-p);
  const float r = __fmaf_rn(v, e * -0.69314718055994531f, v);
  *below = p;
  return p < 44.f && x != m ? r : 0.f;
}
__device__ __forceinline__ float coarse(float x, float m, float c, float cl) {
  float below;
  return coarse(x, m, c, cl, &below);
}
// In units, rounded down, of a sum below 2^20, by its bits.
__device__ __forceinline__ u64 units(float v) {
  const uint32_t b = __float_as_uint(v);
  const int up = static_cast<int>(b >> 23) - 150 + kUnit;
  const uint32_t mantissa = (b & 0x7FFFFFu) | 0x800000u;
  return up >= 0 ? static_cast<u64>(mantissa) << up : static_cast<u64>(mantissa >> min(-up, 31));
}
// A sum in pairs.
template <int N>
__device__ __forceinline__ float sum_in_pairs(float (&v)[N]) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1)
#pragma unroll
    for (int q = 0; q < o; ++q) v[q] += v[q + o];
  return v[0];
}
// N weights, those not taken as 0, and the largest logits among them.
template <int N, typename F>
__device__ __forceinline__ u64 coarse_sum(const float (&x)[N], float m, float c, float cl, F take) {
  float v[N];
  uint32_t tops = 0;
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const bool in = take(x[q], q);
    v[q] = in ? coarse(x[q], m, c, cl) : 0.f;
    tops += in && x[q] == m;
  }
  return units(sum_in_pairs(v)) + (static_cast<u64>(tops) << kUnit);
}

template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));  // logits of 16 bytes

// Bins of a fraction of a binary order of the weights, over 32 of them, the last bin with all that is below: finer ones for the
// longer rows, so that few logits share the bin of a border (32 rows of 131071 fp32 with top-p, on eight warps: 337 us on 512 bins, 165 on 2048). Padded
// in shared memory, so that lanes with an order each read from different banks.
template <int W>
constexpr int kPerOrder = W < 8 ? 16 : 64;
template <int W>
constexpr int kFine = 32 * kPerOrder<W>;
template <int W>
__device__ __forceinline__ int fine_place(int bin) { return bin + bin / kPerOrder<W>; }
template <int W>
constexpr int kFinePlaces = kFine<W> + 32;
// The most logits that a border is looked for among one by one, and the most that all of the rest is done for so.
template <int W>
constexpr int kCap = W <= 2 ? 256 : 512;
template <int W>
constexpr int kFew = W <= 2 ? 64 : W < 8 ? 128 : 256;

struct Nothing {};
template <int W>
struct MergedBins {
  uint32_t fine[kFinePlaces<W>];
};
// What top_k and top_p need: bins, and a list of the logits next to a border.
template <int W, bool kCluster>
struct Lists {
  union {
    struct {
      u64 list[kCap<W>];          // logits as key and complement of the index: the larger, the earlier in the order
      u64 list_weights[kCap<W>];
    };
    struct {                      // where more logits than that lie next to a border
      u64 sums[kBins];
      uint32_t counts[kBins];
    };
    std::conditional_t<kCluster, MergedBins<W>, Nothing> merged;  // bins over all ranks, in a cluster, until a list is begun
  };
  uint32_t fine[kFinePlaces<W>];  // counts of the bins, or sums
  uint32_t list_count;
  u64 edge[2];                    // the last one kept, by count and by sum: a rank may still read the one when the other is cleared
  u64 few[2][W];
  // Of the bin that a border falls into:
  int bin, last_bin;
  u64 above_sum, target;
  uint32_t above_count, bin_count;
};
// A CTA's shared memory but for its logits.
template <int W, bool kCluster, bool kLists = true>
struct Shared : std::conditional_t<kLists, Lists<W, kCluster>, Nothing> {
  u64 powers[32];
  u64 warps[2][W], warps_too[2][W];  // of the two reductions at work at most
  u64 mine[2], mine_too[2];       // what this CTA hands to the others of its cluster
  int sure;                       // of the draw by coarse sums (rank 0's)
};

// A row's share in a CTA: `vectors` 16-byte words a lane from `mine` on, 32 apart, position = word * kVec + element.
template <typename T>
struct Part {
  const uint4* mine;  // this lane's first word
  int words;          // of a lane
  int first;          // index of this lane's first word's first logit within the row (may be negative)
  __device__ __forceinline__ void unpack(int it, float (&v)[kVec<T>]) const {
    const uint4 raw = mine[it * 32];
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
  __device__ __forceinline__ int index(int it) const { return first + it * 32 * kVec<T>; }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll 1
    for (int it = 0; it < words; ++it) {
      float v[kVec<T>];
      unpack(it, v);
#pragma unroll
      for (int q = 0; q < kVec<T>; ++q) f(v[q], first + it * 32 * kVec<T> + q);
    }
  }
};

template <int W, bool kCluster, bool kLists = true>
struct Team {
  Shared<W, kCluster, kLists>& s;
  int ranks, rank, turn = 0;
  __device__ __forceinline__ Team(Shared<W, kCluster, kLists>& shared) : s(shared) {
    ranks = kCluster ? static_cast<int>(cg::this_cluster().num_blocks()) : 1;
    rank = kCluster ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
  }
  __device__ __forceinline__ void sync() const {
    if constexpr (kCluster) cg::this_cluster().sync(); else __syncthreads();
  }
  template <typename V>
  __device__ __forceinline__ V of_rank(V* p, int r) const {
    if constexpr (kCluster) return *cg::this_cluster().map_shared_rank(p, r);
    return *p;
  }
  // The sum over all threads; *before: over those of the CTAs and warps before this one. Two places taken
  // in turn: none is written again before everyone has read it, as a whole round lies between.
  __device__ __forceinline__ u64 sum(u64 v, u64* before) {
    const int warp = threadIdx.x >> 5;
    const u64 w = warp_sum(v);
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) s.warps[turn][warp] = w;
    __syncthreads();
    u64 mine = 0, ahead = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const u64 t = s.warps[turn][i];
      if (i < warp) ahead += t;
      mine += t;
    }
    if constexpr (!kCluster) {
      *before = ahead;
      return mine;
    }
    if (threadIdx.x == 0) s.mine[turn] = mine;
    sync();
    u64 total = 0;
    for (int r = 0; r < ranks; ++r) {
      const u64 t = of_rank(&s.mine[turn], r);
      if (r < rank) ahead += t;
      total += t;
    }
    *before = ahead;
    return total;
  }
  // The sums over all threads of two values.
  __device__ __forceinline__ void sums(u64 v, u64 w, u64* total_v, u64* total_w) {
    const int warp = threadIdx.x >> 5;
    v = warp_sum(v);
    w = warp_sum(w);
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) {
      s.warps[turn][warp] = v;
      s.warps_too[turn][warp] = w;
    }
    __syncthreads();
    v = w = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      v += s.warps[turn][i];
      w += s.warps_too[turn][i];
    }
    if constexpr (kCluster) {
      if (threadIdx.x == 0) {
        s.mine[turn] = v;
        s.mine_too[turn] = w;
      }
      sync();
      v = w = 0;
      for (int r = 0; r < ranks; ++r) {
        v += of_rank(&s.mine[turn], r);
        w += of_rank(&s.mine_too[turn], r);
      }
    }
    *total_v = v;
    *total_w = w;
  }
  // Of every thread's 32 bits the largest.
  __device__ __forceinline__ uint32_t largest(uint32_t v) {
    v = __reduce_max_sync(kAll, v);
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) s.warps[turn][threadIdx.x >> 5] = v;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) v = max(v, static_cast<uint32_t>(s.warps[turn][i]));
    if constexpr (kCluster) {
      if (threadIdx.x == 0) s.mine[turn] = v;
      sync();
      for (int r = 0; r < ranks; ++r) v = max(v, static_cast<uint32_t>(of_rank(&s.mine[turn], r)));
    }
    return v;
  }
};

// The first logit whose weights up to it pass r, found by the warp that has it; before: the weights ahead of this warp, total:
// its own. found(x, index, up to it, its own weight).
template <typename T, typename S, typename E, typename F>
__device__ __forceinline__ void walk(const Part<T>& part, u64 r, u64 before, u64 total, S word_sum, E each, F found) {
  const int lane = threadIdx.x & 31;
  if (r < before || r >= before + total) return;
#pragma unroll 1
  for (int it = 0; it < part.words; ++it) {
    const u64 own = word_sum(it);
    const u64 scan = warp_scan(own, lane);
    const u64 all = __shfl_sync(kAll, scan, 31);
    if (r < before + all) {
      const uint32_t over = __ballot_sync(kAll, before + scan > r);
      if (lane == __ffs(over) - 1) {
        float v[kVec<T>];
        part.unpack(it, v);
        u64 at = before + scan - own;
        bool done = false;
#pragma unroll
        for (int q = 0; q < kVec<T>; ++q) {
          const u64 t = each(v[q], part.index(it) + q);
          if (!done && (at + t > r || q == kVec<T> - 1)) {
            done = true;
            found(v[q], part.index(it) + q, at + t, t);
          }
          at += t;
        }
      }
      return;
    }
    before += all;
  }
}

// The bin of s.counts and s.sums, over all ranks, that the border falls into: by count, the first whose counts from bin 0
// on reach `target`; by sum likewise.
template <int W, bool kCluster>
__device__ __forceinline__ void find_bin(Team<W, kCluster>& team, bool by_sum, u64 target_count, const u64* top_p) {
  Shared<W, kCluster>& s = team.s;
  team.sync();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    u64 own[kBins / 32], sums[kBins / 32];
    u64 total = 0;
#pragma unroll
    for (int b = 0; b < kBins / 32; ++b) {
      const int bin = lane * (kBins / 32) + b;
      u64 c = 0, w = 0;
      for (int r = 0; r < team.ranks; ++r) {
        c += team.of_rank(&s.counts[bin], r);
        if (by_sum) w += team.of_rank(&s.sums[bin], r);
      }
      own[b] = c;
      sums[b] = w;
      total += by_sum ? w : c;
    }
    const u64 scan = warp_scan(total, lane);
    u64 target = target_count;
    if (top_p != nullptr) target = nucleus(*top_p, __shfl_sync(kAll, scan, 31));
    const uint32_t reach = __ballot_sync(kAll, scan >= target);
    if (reach != 0 && lane == __ffs(reach) - 1) {
      u64 at = scan - total;
      int hit = -1;
#pragma unroll
      for (int b = 0; b < kBins / 32; ++b) {
        const u64 step = by_sum ? sums[b] : own[b];
        if (hit < 0) {
          if (at + step >= target) {
            hit = b;
            s.bin = lane * (kBins / 32) + b;
            s.bin_count = static_cast<uint32_t>(own[b]);
            s.above_sum = at;
          } else {
            at += step;
          }
        }
      }
      s.target = target;
    }
  }
  team.sync();
}

template <int W, bool kCluster>
__device__ __forceinline__ void clear_bins(Shared<W, kCluster>& s) {
  for (int b = threadIdx.x; b < kBins; b += W * 32) {
    s.counts[b] = 0;
    s.sums[b] = 0;
  }
  __syncthreads();
}

// Cuts `kept` to its first `count` logits, or (by_sum) to those before which less than top_p of its sum lies.
// Out of line: it is the way for more logits next to a border than kCap<W>, many equal ones above all.
template <typename T, int W, bool kCluster>
__device__ __noinline__ Prefix cut(Shared<W, kCluster>& s, const Part<T> part, float m, const Wish w, bool by_sum, u64 count) {
  Team<W, kCluster> team(s);
  __syncthreads();  // its reductions take their places from the first again
  Prefix kept;
  uint32_t low = kLowest, high = kAll;  // keys of the bin
  u64 target = count, above = 0;        // still to be reached within it, and ahead of it
  {
    // Bins of an eighth of a binary order of the weights, the last one with all that is below.
    const float scale = w.ch * 0.25f;
    auto bin_of = [&](float x) { return min(kBins - 1, __float2int_rd((m - x) * scale)); };
    clear_bins(s);
    part.each([&](float x, int) {
      const int b = bin_of(x);
      atomicAdd(&s.counts[b], 1u);
      if (by_sum) atomicAdd(&s.sums[b], weight(x, m, w, s.powers));
    });
    find_bin(team, by_sum, target, by_sum ? &w.top_p : nullptr);
    int bin = s.bin;
    above = s.above_sum;
    target = s.target;
    // The keys of its logits.
    uint32_t most = 0, least = 0;  // the smallest as its complement's largest
    part.each([&](float x, int) {
      const uint32_t k = key_of(x);
      if (bin_of(x) == bin) {
        most = max(most, k);
        least = max(least, ~k);
      }
    });
    high = team.largest(most);
    low = ~team.largest(least);
    while (low < high) {
      const int shift = max(0, 32 - __clz(high - low) - 8);
      clear_bins(s);
      part.each([&](float x, int) {
        const uint32_t k = key_of(x);
        if (k < low || k > high) return;
        atomicAdd(&s.counts[(high - k) >> shift], 1u);
        if (by_sum) atomicAdd(&s.sums[(high - k) >> shift], weight(x, m, w, s.powers));
      });
      find_bin(team, by_sum, target - above, nullptr);
      bin = s.bin;
      above += s.above_sum;
      const uint32_t top = high - (static_cast<uint32_t>(bin) << shift);
      if (shift == 0) {
        low = high = top;
      } else {
        const uint32_t span = (1u << shift) - 1, bottom = top - low > span ? top - span : low;
        most = least = 0;
        part.each([&](float x, int) {
          const uint32_t k = key_of(x);
          if (k <= top && k >= bottom) {
            most = max(most, k);
            least = max(least, ~k);
          }
        });
        high = team.largest(most);
        low = ~team.largest(least);
      }
    }
  }
  // Of the logits with that key, how many, and the index of the last one.
  const float edge = value_of_key(high);
  kept.edge = edge;
  u64 ties = target - above;
  if (by_sum) {
    const u64 each = weight(edge, m, w, s.powers);
    ties = each == 0 ? 1 : (ties + each - 1) / each;
  }
  u64 mine = 0, before;
  auto tied = [&](float x, int) -> u64 { return x == edge; };
  part.each([&](float x, int) { mine += x == edge; });
  const u64 all = team.sum(mine, &before);
  if (ties < all) {
    walk(
        part, ties - 1, before, warp_sum(mine),
        [&](int it) {
          float v[kVec<T>];
          part.unpack(it, v);
          u64 t = 0;
#pragma unroll
          for (int q = 0; q < kVec<T>; ++q) t += tied(v[q], part.index(it) + q);
          return t;
        },
        tied,
        [&](float, int at, u64, u64) {
          for (int r = 0; r < team.ranks; ++r) {
            if constexpr (kCluster) *cg::this_cluster().map_shared_rank(&s.bin, r) = at;
            else s.bin = at;
          }
        });
    team.sync();
    kept.last = s.bin;
  }
  team.sync();
  return kept;
}

// How many bins a logit lies below the largest, and its bin.
template <int W>
struct Fine {
  float m, scale;
  __device__ __forceinline__ Fine(float top, const Wish& w) : m(top), scale(w.ch * (kPerOrder<W> * 0.03125f)) {}
  __device__ __forceinline__ float at(float x) const { return __fmul_rn(__fsub_rn(m, x), scale); }
  __device__ __forceinline__ int bin(float f) const { return min(kFine<W> - 1, __float2int_rd(f)); }
};
__device__ __forceinline__ u64 item_of(uint32_t key, int at) { return static_cast<u64>(key) << 32 | static_cast<uint32_t>(~at); }
__device__ __forceinline__ uint32_t item_key(u64 item) { return static_cast<uint32_t>(item >> 32); }
__device__ __forceinline__ int item_index(u64 item) { return static_cast<int>(~static_cast<uint32_t>(item)); }

template <int W, bool kCluster>
__device__ __forceinline__ uint32_t* bins_of(Shared<W, kCluster>& s) {
  if constexpr (kCluster) return s.merged.fine; else return s.fine;
}

// Counts of the logits, or (kSums) their weights, over all ranks, in bins_of(s): sums in units of 2^-bits of the largest
// weight of their bin, good to 2^-12, in 32 bits.
template <bool kSums, typename T, int W, bool kCluster>
__device__ __forceinline__ void fill_bins(Team<W, kCluster>& team, const Part<T>& part, const Fine<W>& fine, int bits) {
  Shared<W, kCluster>& s = team.s;
  for (int b = threadIdx.x; b < kFinePlaces<W>; b += W * 32) s.fine[b] = 0;
  if (threadIdx.x == 0) {
    s.list_count = 0;
    s.edge[kSums] = 0;
  }
  __syncthreads();
  const float unit = static_cast<float>(1 << bits);
  part.each([&](float x, int) {
    const float f = fine.at(x);
    const int b = fine.bin(f);
    uint32_t add = 1u;
    if (kSums) add = static_cast<uint32_t>(__float2int_rn(unit * quick_exp2((f - static_cast<float>(b)) * (-1.f / kPerOrder<W>))));
    atomicAdd(&s.fine[fine_place<W>(b)], add);
  });
  team.sync();
  if constexpr (kCluster) {
    for (int b = threadIdx.x; b < kFine<W>; b += W * 32) {
      uint32_t count = 0;
      for (int r = 0; r < team.ranks; ++r) count += team.of_rank(&s.fine[fine_place<W>(b)], r);
      s.merged.fine[fine_place<W>(b)] = count;
    }
    __syncthreads();
  }
}

template <typename V>
__device__ __forceinline__ V scan_of(V v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V t = __shfl_up_sync(kAll, v, o);
    if (lane >= o) v += t;
  }
  return v;
}
// Where the sum over bins reaches `target`, by a warp: first the binary order, whose sums the lanes hold (up to it: scan), then its
// bins, one or a few a lane. The bin, what lies before it, and it itself; -1 if it is not reached.
template <int W, typename V, typename F>
__device__ __forceinline__ int reached(V scan, V total, V target, F bin_sum, V* before, V* itself) {
  const int lane = threadIdx.x & 31;
  const uint32_t orders = __ballot_sync(kAll, scan >= target);
  if (orders == 0) return -1;
  const int order = __ffs(orders) - 1;
  const V ahead = __shfl_sync(kAll, scan - total, order);
  constexpr int kEach = kPerOrder<W> > 32 ? kPerOrder<W> / 32 : 1;
  V own[kEach], sum = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    own[e] = lane * kEach + e < kPerOrder<W> ? bin_sum(order, lane * kEach + e) : V(0);
    sum += own[e];
  }
  V at = ahead + (scan_of(sum, lane) - sum);
  int mine = kPerOrder<W>;
  V mine_before = 0, mine_itself = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    if (mine == kPerOrder<W> && at + own[e] >= target) {
      mine = lane * kEach + e;
      mine_before = at;
      mine_itself = own[e];
    }
    at += own[e];
  }
  // By rounding it may seem to be reached in the order and in none of its bins: the last one then.
  const uint32_t bins = __ballot_sync(kAll, mine < kPerOrder<W>);
  const int holder = bins != 0 ? __ffs(bins) - 1 : 31;
  *before = __shfl_sync(kAll, mine_before, holder);
  *itself = __shfl_sync(kAll, mine_itself, holder);
  mine = __shfl_sync(kAll, mine, holder);
  return order * kPerOrder<W> + min(mine, kPerOrder<W> - 1);
}

// By count: the bin that the logit number `target` (from 1) of the order is in. A lane has the bins of one binary order.
template <int W, bool kCluster>
__device__ __forceinline__ void find_count(Team<W, kCluster>& team, uint32_t target) {
  Shared<W, kCluster>& s = team.s;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const uint32_t* const bins = bins_of(s);
    uint32_t total = 0, before = 0, itself = 0;
#pragma unroll 16
    for (int b = 0; b < kPerOrder<W>; ++b) total += bins[lane * (kPerOrder<W> + 1) + b];
    const int bin = reached<W>(
        scan_of(total, lane), total, target, [&](int order, int b) { return bins[order * (kPerOrder<W> + 1) + b]; }, &before, &itself);
    if (lane == 0) {
      s.bin = s.last_bin = bin;
      s.above_count = before;
      s.bin_count = itself;
    }
  }
  team.sync();
}
// By sum: the bins that the border of top_p is in, whatever their sums' error does to it: that of what lies beyond the border
// counts, not that of all.
template <int W, bool kCluster>
__device__ __forceinline__ void find_sum(Team<W, kCluster>& team, u64 top_p) {
  Shared<W, kCluster>& s = team.s;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const uint32_t* const bins = bins_of(s);
    auto bin_sum = [&](int order, int b) {
      return static_cast<float>(bins[order * (kPerOrder<W> + 1) + b]) *
             (quick_exp2(static_cast<float>(b) * (-1.f / kPerOrder<W>)) * quick_exp2(static_cast<float>(-order)));
    };
    float total = 0.f, before, itself;
#pragma unroll 16
    for (int b = 0; b < kPerOrder<W>; ++b) total += bin_sum(lane, b);
    const float scan = scan_of(total, lane);
    const float all = __shfl_sync(kAll, scan, 31), border = all * (static_cast<float>(static_cast<uint32_t>(top_p >> 32)) * 0x1p-32f);
    const float off = (all - border) * 0x1p-11f + all * 0x1p-19f;
    const int first = reached<W>(scan, total, border - off, bin_sum, &before, &itself);
    const int last = reached<W>(scan, total, border + off, bin_sum, &before, &itself);
    if (lane == 0) {
      s.bin = first < 0 ? kFine<W> - 1 : first;
      s.last_bin = last < 0 ? kFine<W> - 1 : last;
    }
  }
  team.sync();
}

// A logit into rank 0's list, if it is not full; the list counts on.
template <int W, bool kCluster>
__device__ __forceinline__ void enlist(Team<W, kCluster>& team, float x, int at) {
  Shared<W, kCluster>* s = &team.s;
  if constexpr (kCluster) s = cg::this_cluster().map_shared_rank(&team.s, 0);
  const uint32_t to = atomicAdd(&s->list_count, 1u);
  if (to < kCap<W>) s->list[to] = item_of(key_of(x), at);
}
// The logits of bins first .. last.
template <typename T, int W, bool kCluster>
__device__ __forceinline__ void collect(Team<W, kCluster>& team, const Part<T>& part, const Fine<W>& fine, int first, int last) {
  part.each([&](float x, int at) {
    const int b = fine.bin(fine.at(x));
    if (b >= first && b <= last) enlist(team, x, at);
  });
  team.sync();
}

// The sum over a CTA's threads (not over its cluster).
template <int W, bool kCluster>
__device__ __forceinline__ u64 cta_sum(Shared<W, kCluster>& s, int place, u64 v) {
  v = warp_sum(v);
  if constexpr (W == 1) {
    __syncwarp();
    return v;
  }
  if ((threadIdx.x & 31) == 0) s.few[place][threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) v += s.few[place][i];
  return v;
}

// All of the rest for at most kFew<W> logits that s.list holds, the first top_k of the order among them: of each its place in
// either order, and what lies before it, come from a look at every other.
template <int W, bool kCluster>
__device__ __noinline__ void few(Shared<W, kCluster>& s, const Rows& a, int64_t row, float m, const Wish w, int count) {
  constexpr int kEach = kFew<W> > W * 32 ? kFew<W> / (W * 32) : 1;  // logits of a thread
  for (int i = threadIdx.x; i < count; i += W * 32)
    s.list_weights[i] = weight(value_of_key(item_key(s.list[i])), m, w, s.powers);
  __syncthreads();
  int rank[kEach];
  u64 before[kEach], all = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = threadIdx.x + e * W * 32;
    rank[e] = 0;
    before[e] = 0;
    if (i < count) {
      const u64 item = s.list[i];
      for (int j = 0; j < count; ++j) {
        const bool earlier = s.list[j] > item;
        rank[e] += earlier;
        before[e] += earlier ? s.list_weights[j] : 0;
      }
      if (rank[e] < w.top_k) all += s.list_weights[i];
    }
  }
  all = cta_sum(s, 0, all);  // everyone is past the reading of the weights
  const u64 target = w.top_p != kAllOfIt ? nucleus(w.top_p, all) : ~0ull;
  u64 total = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = threadIdx.x + e * W * 32;
    if (i >= count) break;
    const float x = value_of_key(item_key(s.list[i]));
    const bool kept = rank[e] < w.top_k && (rank[e] == 0 || before[e] < target) &&
                      (!(w.min_p > 0.f) || Floor(m, w).above(x, m, w, s.powers));
    if (kept) total += s.list_weights[i];
    else s.list_weights[i] = 0;
  }
  total = cta_sum(s, 1, total);
  const u64 r = share(w.u, total);
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = threadIdx.x + e * W * 32;
    if (i >= count) break;
    const u64 mine = s.list_weights[i];
    if (mine == 0) continue;
    const int index = item_index(s.list[i]);
    u64 up_to = 0;
    for (int j = 0; j < count; ++j)
      if (item_index(s.list[j]) <= index) up_to += s.list_weights[j];
    if (up_to > r && up_to - mine <= r) {
      a.index[row] = index;
      if (a.logprob != nullptr) a.logprob[row] = logprob_of(value_of_key(item_key(s.list[i])), m, w, total);
    }
  }
}

// Of `count` logits in rank 0's list the one with `rank` others before it: where a prefix of so many ends.
template <int W, bool kCluster>
__device__ __forceinline__ u64 edge_by_count(Team<W, kCluster>& team, int count, uint32_t rank) {
  Shared<W, kCluster>& s = team.s;
  if (team.rank == 0) {
    for (int i = threadIdx.x; i < count; i += W * 32) {
      const u64 item = s.list[i];
      uint32_t place = 0;
      for (int j = 0; j < count; ++j) place += s.list[j] > item;
      if (place == rank) s.edge[0] = item;
    }
  }
  team.sync();
  return team.of_rank(&s.edge[0], 0);
}
// The one in which the sum passes `target`, `above` lying before all of the list. With weigh's weights known to `sure`: 0 if
// the border is no further than that from one of its sides. 0 too if there is none.
template <int W, bool kCluster, typename F>
__device__ __forceinline__ u64 edge_by_sum(Team<W, kCluster>& team, int count, u64 above, u64 target, u64 sure, F weigh) {
  Shared<W, kCluster>& s = team.s;
  if (team.rank == 0) {
    for (int i = threadIdx.x; i < count; i += W * 32) s.list_weights[i] = weigh(value_of_key(item_key(s.list[i])));
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += W * 32) {
      const u64 item = s.list[i];
      u64 before = above;
      for (int j = 0; j < count; ++j) before += s.list[j] > item ? s.list_weights[j] : 0;
      const u64 up_to = before + s.list_weights[i];
      if (before < target && up_to >= target && (before == 0 || target - before >= sure) && up_to - target >= sure) s.edge[1] = item;
    }
  }
  team.sync();
  return team.of_rank(&s.edge[1], 0);
}

// What is kept of a nucleus whose border coarse sums cannot tell, by the list of the logits next to it if it holds them.
template <typename T, int W, bool kCluster>
__device__ __noinline__ Prefix exact_nucleus(Shared<W, kCluster>& s, const Part<T> part, float m, const Wish w, int first, int count) {
  if (count <= kCap<W>) {
    Team<W, kCluster> team(s);
    team.sync();  // its reductions take their places from the first again
    const Fine<W> fine(m, w);
    u64 own = 0, rest = 0, before;
    part.each([&](float v, int) {
      const u64 t = weight(v, m, w, s.powers);
      if (fine.bin(fine.at(v)) < first) own += t; else rest += t;
    });
    const u64 above = team.sum(own, &before);
    const u64 target = nucleus(w.top_p, above + team.sum(rest, &before));
    const u64 edge = edge_by_sum(team, count, above, target, 0, [&](float v) { return weight(v, m, w, s.powers); });
    team.sync();
    if (edge != 0) return {value_of_key(item_key(edge)), item_index(edge)};
  }
  return cut<T, W, kCluster>(s, part, m, w, true, 0);
}

// The draw by weight().
template <typename T, int W, bool kCluster, bool kLists>
__device__ __noinline__ void exact_draw(Shared<W, kCluster, kLists>& s, const Part<T> part, const Rows& a, int64_t row, float m, const Wish w,
                                        const Prefix kept) {
  Team<W, kCluster, kLists> team(s);
  team.sync();
  auto weigh = [&](float v, int at) { return kept.holds(v, at) ? weight(v, m, w, s.powers) : 0; };
  u64 own = 0, before;
  part.each([&](float v, int at) { own += weigh(v, at); });
  const u64 total = team.sum(own, &before);
  walk(
      part, share(w.u, total), before, warp_sum(own),
      [&](int it) {
        float v[kVec<T>];
        part.unpack(it, v);
        u64 t = 0;
#pragma unroll
        for (int q = 0; q < kVec<T>; ++q) t += weigh(v[q], part.index(it) + q);
        return t;
      },
      weigh,
      [&](float v, int at, u64, u64) {
        a.index[row] = at;
        if (a.logprob != nullptr) a.logprob[row] = logprob_of(v, m, w, total);
      });
  team.sync();
}

// per: 16-byte words of a warp's lane; the CTA's logits take W * 32 * per of them. kCuts: 1 if top_k may be asked for, 2 if top_p.
template <typename T, int W, bool kCluster, int kCuts>
__global__ void __launch_bounds__(W * 32, (kCuts != 0 ? 24 : 32) / W) cta_kernel(const Rows a, int per) {
  extern __shared__ uint4 logits[];
  constexpr bool kLists = kCuts != 0;
  __shared__ Shared<W, kCluster, kLists> s;
  let_next();
  if (threadIdx.x < 32) s.powers[threadIdx.x] = kPowersInit[threadIdx.x];
  Team<W, kCluster, kLists> team(s);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = static_cast<int>(a.n);
  // So that no bin's sum passes 32 bits.
  const int bits = min(16, __clz(per * W * 32 * kVec<T> * team.ranks) - 1);
  // Behind the logits a sum for each of their words: this lane's first, the next ones 32 on.
  u64* const word_sums = reinterpret_cast<u64*>(logits + W * 32 * per);
  u64* const sums = word_sums + warp * 32 * per + lane;
  after_previous();
  for (int64_t row = blockIdx.x / team.ranks; row < a.rows; row += gridDim.x / team.ranks) {
    const T* x = static_cast<const T*>(a.x) + row * n;
    // Words are those of memory: the first starts up to 15 bytes before the row.
    const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(x) % 16 / sizeof(T));
    uint4* mine = logits + warp * 32 * per + lane;
    Part<T> part;
    part.mine = mine;
    part.words = per;
    part.first = ((team.rank * W + warp) * per * 32 + lane) * kVec<T> - shift;
    float m = -INFINITY;
    constexpr int kBatch = 4;  // words of a lane in flight
    for (int it0 = 0; it0 < per; it0 += kBatch) {
      uint4 raw[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int at = part.first + (it0 + u) * 32 * kVec<T>;
        if (it0 + u < per && at >= 0 && at + kVec<T> <= n) raw[u] = __ldcs(reinterpret_cast<const uint4*>(x + at));
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int at = part.first + (it0 + u) * 32 * kVec<T>;
        if (it0 + u >= per) break;
        if (at >= 0 && at + kVec<T> <= n) {
          mine[(it0 + u) * 32] = raw[u];
          m = max_nan(m, largest_of<T>(raw[u]));
        } else {
          T* to = reinterpret_cast<T*>(mine + (it0 + u) * 32);
          for (int q = 0; q < kVec<T>; ++q) {
            // No logit there: one that is never drawn, and after all others in the order.
            const T v = at + q >= 0 && at + q < n ? fetch(x + at + q) : lowest<T>();
            to[q] = v;
            m = max_nan(m, value(v));
          }
        }
      }
    }
    const Wish w = wish_of(a, row);
    {
      const uint32_t top = team.largest(m != m ? kAll : key_of(m));  // (and the powers are there)
      m = top == kAll ? NAN : value_of_key(top);
    }
    if (w.bad || m != m || m == -INFINITY) {
      if (threadIdx.x == 0 && team.rank == 0) {
        a.index[row] = -1;
        if (a.logprob != nullptr) a.logprob[row] = NAN;
      }
      continue;
    }
    if (m == INFINITY) {
      // All of the probability is the infinite ones': as if they were 0, and the others -infinity.
#pragma unroll 1
      for (int it = 0; it < per; ++it) {
        T* to = reinterpret_cast<T*>(mine + it * 32);
        for (int q = 0; q < kVec<T>; ++q) to[q] = value(to[q]) == INFINITY ? narrow<T>(0.f) : lowest<T>();
      }
      m = 0.f;
    }
    if (w.top_k == 1) {
      // The first of the largest.
      uint32_t first = 0;
      part.each([&](float v, int at) {
        if (v == m) first = max(first, static_cast<uint32_t>(~at));
      });
      first = team.largest(first);
      if (threadIdx.x == 0 && team.rank == 0) {
        a.index[row] = static_cast<int>(~first);
        if (a.logprob != nullptr) a.logprob[row] = 0.f;
      }
      continue;
    }
    const float c = w.ch * 0.03125f, cl = w.cl * 0.03125f;
    Prefix kept;
    bool summed = false;  // the words' sums are those of what is kept
    [[maybe_unused]] const Fine<W> fine(m, w);
    if constexpr ((kCuts & 1) != 0) {
      if (w.top_k < n) {
        fill_bins<false>(team, part, fine, 0);
        find_count(team, static_cast<uint32_t>(w.top_k));
        const int bin = s.bin;
        const uint32_t above = s.above_count, inside = s.bin_count;
        if (above + inside <= kFew<W>) {
          collect(team, part, fine, 0, bin);
          if (team.rank == 0) few(s, a, row, m, w, static_cast<int>(above + inside));
          continue;
        }
        Prefix first;
        if (inside <= kCap<W>) {
          collect(team, part, fine, bin, bin);
          const u64 edge = edge_by_count(team, static_cast<int>(inside), static_cast<uint32_t>(w.top_k) - above - 1);
          first = {value_of_key(item_key(edge)), item_index(edge)};
        } else {
          first = cut<T, W, kCluster>(s, part, m, w, false, static_cast<u64>(w.top_k));
        }
        // The others are out for good.
#pragma unroll 1
        for (int it = 0; it < per; ++it) {
          float v[kVec<T>];
          part.unpack(it, v);
          T* to = reinterpret_cast<T*>(mine + it * 32);
#pragma unroll
          for (int q = 0; q < kVec<T>; ++q)
            if (!first.holds(v[q], part.index(it) + q)) to[q] = lowest<T>();
        }
      }
    }
    if constexpr ((kCuts & 2) != 0) {
      if (w.top_p != kAllOfIt) {
        fill_bins<true>(team, part, fine, bits);
        find_sum(team, w.top_p);
        const int first = s.bin, last = s.last_bin;
        // The same borders in units of coarse()'s distance.
        const float from = static_cast<float>(first) * (1.f / kPerOrder<W>);
        const float to = last == kFine<W> - 1 ? INFINITY : static_cast<float>(last + 1) * (1.f / kPerOrder<W>);
        u64 own = 0, late = 0, above, rest;
#pragma unroll 1
        for (int it = 0; it < per; ++it) {
          float v[kVec<T>], early[kVec<T>];
          part.unpack(it, v);
          uint32_t tops = 0;
#pragma unroll
          for (int q = 0; q < kVec<T>; ++q) {
            float below;
            const float t = coarse(v[q], m, c, cl, &below);
            if (below >= from && below < to) enlist(team, v[q], part.index(it) + q);
            tops += v[q] == m;
            early[q] = below < from ? t : 0.f;
            v[q] = below < from ? 0.f : t;
          }
          const u64 ones = static_cast<u64>(tops) << kUnit;
          const u64 sum = units(sum_in_pairs(early)) + (first > 0 ? ones : 0);
          sums[it * 32] = sum;
          own += sum;
          late += units(sum_in_pairs(v)) + (first > 0 ? 0 : ones);
        }
        team.sums(own, late, &above, &rest);
        const u64 target = nucleus(w.top_p, above + rest);
        const int count = static_cast<int>(team.of_rank(&s.list_count, 0));
        u64 edge = 0;
        // How far a logit's `before` is from the target: (1 - p) above + those of the list - p rest. So what counts is the error of
        // what lies beyond the border and next to it, and not that of all.
        if (count <= kCap<W>)
          edge = edge_by_sum(team, count, above, target, static_cast<u64>(static_cast<float>(above + rest - target + rest) * kSure) + 1,
                             [&](float v) { return v == m ? kOne : units(coarse(v, m, c, cl)); });
        if (edge != 0) {
          kept = {value_of_key(item_key(edge)), item_index(edge)};
          summed = true;
          // The list's part of what is kept, to its words' sums.
          if (team.rank == 0) {
            for (int i = threadIdx.x; i < count; i += W * 32) {
              if (s.list[i] < edge) continue;
              const int word = (item_index(s.list[i]) + shift) / kVec<T>, lanes = W * 32 * per;
              u64* at = word_sums + word % lanes;
              if constexpr (kCluster) at = cg::this_cluster().map_shared_rank(word_sums, word / lanes) + word % lanes;
              atomicAdd(at, s.list_weights[i]);
            }
          }
          team.sync();
        } else {
          kept = exact_nucleus<T, W, kCluster>(s, part, m, w, first, count);
        }
      }
    }
    if (w.min_p > 0.f) {
      const Floor floor(m, w);
      uint32_t least = 0;
      part.each([&](float v, int) {
        if (floor.above(v, m, w, s.powers)) least = max(least, ~key_of(v));
      });
      const float edge = value_of_key(~team.largest(least));
      if (edge > kept.edge) {
        kept = {edge, 0x7FFFFFFF};
        summed = false;
      }
    }
    const bool whole = kept.edge == -INFINITY;
    u64 own = 0, before;
#pragma unroll 1
    for (int it = 0; it < per; ++it) {
      if (!summed) {
        float v[kVec<T>];
        part.unpack(it, v);
        sums[it * 32] = whole ? coarse_sum(v, m, c, cl, [](float, int) { return true; })
                              : coarse_sum(v, m, c, cl, [&](float x, int q) { return kept.holds(x, part.index(it) + q); });
      }
      own += sums[it * 32];
    }
    if (threadIdx.x == 0 && team.rank == 0) s.sure = 0;
    const u64 total = team.sum(own, &before);
    const u64 r = share(w.u, total), margin = static_cast<u64>(static_cast<float>(total) * kSure) + 1;
    walk(
        part, r, before, warp_sum(own),
        [&](int it) { return sums[it * 32]; },
        [&](float v, int at) -> u64 { return !kept.holds(v, at) ? 0 : v == m ? kOne : units(coarse(v, m, c, cl)); },
        [&](float v, int at, u64 up_to, u64 its) {
          if (up_to <= r + margin || r < up_to - its + margin) return;
          if constexpr (kCluster) *cg::this_cluster().map_shared_rank(&s.sure, 0) = 1;
          else s.sure = 1;
          a.index[row] = at;
          if (a.logprob != nullptr) a.logprob[row] = logprob_of(v, m, w, total);
        });
    team.sync();
    if (team.of_rank(&s.sure, 0) == 0) exact_draw<T, W, kCluster, kLists>(s, part, a, row, m, w, kept);
  }
  if constexpr (kCluster) team.sync();  // no CTA ends while another may read its shared memory
}

template <typename T, int R>
cudaError_t run_warp(const Rows& a, cudaStream_t stream) {
  const int64_t grid = std::min<int64_t>((a.rows + kWarps - 1) / kWarps, 0x7FFFFFFFll);
  return launch_overlapped(warp_kernel<T, R>, dim3(static_cast<unsigned>(grid)), kThreads, 0, 0, stream, a);
}

template <typename T, int G>
cudaError_t run_group(const Rows& a, cudaStream_t stream) {
  const int64_t grid = std::min<int64_t>((a.rows + kThreads / G - 1) / (kThreads / G), 0x7FFFFFFFll);
  return launch_overlapped(group_kernel<T, G>, dim3(static_cast<unsigned>(grid)), kThreads, 0, 0, stream, a);
}

// The 16-byte words of a row: one more where rows start within one.
template <typename T>
int64_t words_of(const Rows& a) {
  const bool aligned = a.n % kVec<T> == 0 && reinterpret_cast<uintptr_t>(a.x) % 16 == 0;
  return (a.n + kVec<T> - 1) / kVec<T> + (aligned ? 0 : 1);
}

constexpr int kLongRow = 512;  // threads of a CTA for long rows
// Shared memory of a CTA for its words and their sums; the rest is for Shared.
constexpr size_t kMostWords = 204 * 1024;
static_assert(sizeof(Shared<16, true>) + kMostWords <= 227 * 1024 && sizeof(Shared<16, false>) + kMostWords <= 227 * 1024, "shared memory of a CTA");
static_assert(24 * (kSampleMost / 4 + 16 * kLongRow) / 16 <= static_cast<int64_t>(kMostWords), "the longest rows fit a cluster of 16 CTAs");

template <typename T, int W, bool kCluster, int kCuts>
cudaError_t run_cuts(const Rows& a, int cluster, cudaStream_t stream) {
  static SmemRecord record, wide;
  const int64_t words = words_of<T>(a);
  const int64_t lanes = static_cast<int64_t>(cluster) * W * 32;
  const int per = static_cast<int>((words + lanes - 1) / lanes);
  const size_t smem = static_cast<size_t>(per) * W * 32 * (16 + 8);
  const void* fn = reinterpret_cast<const void*>(cta_kernel<T, W, kCluster, kCuts>);
  cudaError_t err = ensure_dynamic_smem(fn, smem, record);
  if (err == cudaSuccess && cluster > 8) err = allow_wide_clusters(fn, wide);
  if (err != cudaSuccess) return err;
  const int64_t rows = std::min<int64_t>(a.rows, (int64_t{1} << 30) / cluster);
  return launch_overlapped(cta_kernel<T, W, kCluster, kCuts>, dim3(static_cast<unsigned>(rows * cluster)), W * 32, kCluster ? cluster : 0, smem,
                           stream, a, per);
}

// A kernel for each set of cuts that may be asked for: code, registers and shared memory that a call does not need cost it rows at once. With
// four warps a row 16384 rows of 4096 bf16 without any took 105 us for 133, with min_p 134 for 197, with top_k 166 for 170, with top_p 244
// for 258; without the lists' shared memory as many of fp32 111 for 124.
template <typename T, int W, bool kCluster>
cudaError_t run_cta(const Rows& a, int cluster, cudaStream_t stream) {
  const int cuts = (a.top_ks != nullptr || (a.top_k > 0 && a.top_k < a.n) ? 1 : 0) + (a.top_ps != nullptr || a.top_p != kAllOfIt ? 2 : 0);
  switch (cuts) {
    case 0: return run_cuts<T, W, kCluster, 0>(a, cluster, stream);
    case 1: return run_cuts<T, W, kCluster, 1>(a, cluster, stream);
    case 2: return run_cuts<T, W, kCluster, 2>(a, cluster, stream);
    default: return run_cuts<T, W, kCluster, 3>(a, cluster, stream);
  }
}

template <typename T>
cudaError_t run(const Rows& a, cudaStream_t stream) {
  if (a.n <= 4) return run_group<T, 4>(a, stream);
  if (a.n <= 8) return run_group<T, 8>(a, stream);
  if (a.n <= 16) return run_group<T, 16>(a, stream);
  if (a.n <= 32) return run_warp<T, 1>(a, stream);
  if (a.n <= 64) return run_warp<T, 2>(a, stream);
  if (a.n <= 128) return run_warp<T, 4>(a, stream);
  DeviceInfo dev;
  const cudaError_t err = device_info(&dev);
  if (err != cudaSuccess) return err;
  // Up to 256 logits where a warp a row does not fill the GPU anyhow: 1024 rows of 256 bf16 take 5.4 us here (13.4 with top-p, 7.2 with
  // top-k) and 10.0 (10.0, 12.6) by a histogram, 16384 rows 31 (84, 44) and 22 (41, 53).
  const bool many = a.rows >= 24 * static_cast<int64_t>(dev.sm_count);
  if (a.n <= 256 && !many) return run_warp<T, 8>(a, stream);
  // CTAs a row: until the rows fill the SMs, while a lane has eight words or more; at least what holds the row. Beyond eight a cluster's
  // barriers and the merging of bins cost more: 8 rows of 131072 fp32 with top_k take 13 us on eight CTAs each and 30 on sixteen (with
  // top-p 54 and 63, without filters 20 and 18); one row of 131071 bf16 with four words a lane 16.9 (41.7, 15.7), with eight 13.9 (43.5,
  // 17.2), with sixteen 14.8 (49, 23.6).
  const int64_t words = words_of<T>(a);
  auto bytes = [&](int64_t cluster) {
    const int64_t lanes = cluster * kLongRow;
    return (words + lanes - 1) / lanes * kLongRow * 24;
  };
  int cluster = 1;
  while (cluster < 8 && a.rows * cluster * 2 <= dev.sm_count && words >= static_cast<int64_t>(cluster) * kLongRow * 8) cluster *= 2;
  while (cluster < 16 && bytes(cluster) > static_cast<int64_t>(kMostWords)) cluster *= 2;
  // Sixteen warps where a CTA has an SM to itself: 32 rows of 131071 fp32 with top_k 17 us, with top-p 137, on eight 25 and 212; 100 rows of
  // 4096 bf16 6.0 and 11.7, on eight 6.9 and 12.7; of 32768 10.3 and 40, on eight 14.7 and 60; one row of 4096 with all filters 6.2 and 6.4.
  if (cluster > 1) return run_cta<T, kLongRow / 32, true>(a, cluster, stream);
  if (a.rows <= dev.sm_count && words >= kLongRow) return run_cta<T, kLongRow / 32, false>(a, 1, stream);
  // Warps a row. Many rows side by side run best on few warps each, long rows and few of them on more. 16384 rows with top-p, on one,
  // two and four warps: of 1000 bf16 86, 91, 131 us; of 1000 fp32 92, 90, 122; of 2048 bf16 150, 134, 165; of 4096 bf16 327, 233, 241,
  // with top_k 186, 134, 164; of 4096 fp32 442, 279, 245; 1024 rows of 16384 139 on four, 105 on eight; 1024 rows of 1000 24 on one, 17
  // on four, 24 on eight; 200 rows of 4096 20 on four, 16 on eight; one row of 1000 6.5 and 8.2.
  if (words <= 160 && many) return run_cta<T, 1, false>(a, 1, stream);
  if (words <= 512 && many) return run_cta<T, 2, false>(a, 1, stream);
  if (words <= (a.rows >= 2 * static_cast<int64_t>(dev.sm_count) ? 1024 : 256)) return run_cta<T, 4, false>(a, 1, stream);
  return run_cta<T, 8, false>(a, 1, stream);
}

template <typename T>
cudaError_t sample_rows(const SampleArgs& g, cudaStream_t stream) {
  Rows a;
  a.x = g.logits; a.rows = g.rows; a.n = g.n; a.u = g.u;
  a.temperature = static_cast<float>(g.temperature); a.min_p = static_cast<float>(g.min_p); a.top_k = g.top_k;
  a.temperatures = g.temperatures; a.top_ks = g.top_ks; a.top_ps = g.top_ps; a.min_ps = g.min_ps;
  a.index = g.index; a.logprob = g.logprob;
  a.top_p = g.top_p >= 1.0 ? kAllOfIt : static_cast<u64>(std::ldexp(std::max(g.top_p, 0.0), 64));
  a.min_units = static_cast<u64>(std::ceil(std::min(std::max(g.min_p, 0.0), 1.0) * 0x1p42));
  const double c = g.temperature > 0.0 ? 46.16624130844683 / g.temperature : 46.16624130844683;
  a.ch = static_cast<float>(c);
  a.cl = static_cast<float>(c - static_cast<double>(a.ch));
  return run<T>(a, stream);
}

}  // namespace
}  // namespace vn
