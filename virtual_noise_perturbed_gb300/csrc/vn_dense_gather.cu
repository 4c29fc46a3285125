// vn_dense_gather.cu -- the centre network's products for problems that do not fill the GPU, and
// for operands that TMA cannot take: one launch for a layer, one for all its gradients.
//
// The form is that of vn_dense_tc.cu, D[q, p] = sum_k A(p, k) B(q, k) on 128 x BN tiles of one
// CTA, but the operands are gathered by threads: loaded from memory in their own type and
// layout (any alignment), turned into what the tensor cores take on the way, and stored in the
// 128-byte-swizzled layout of the MMA's operands. Turned into means:
//   - fp32 into three bf16 planes; each stage then takes the six products of planes that
//     reach fp32's precision (8 + 8 + 8 significant bits);
//   - d = g act'(z), in the gradients, from g and z: no d is ever stored, and the bias's
//     gradient is summed from the same registers, unrounded.
// What a conversion pass and its planes in memory would cost is paid per tile instead, which is less
// as long as tiles are few; launches, which bound such sizes, are one instead of three to five
// (grads of 1021 x 256 x 256 in fp32: 13.9 us, latency of loads, MMAs and instruction fetches; in
// single launches on tiles 30).
//
// The k loop is split over the CTAs of a cluster of up to 16; partial sums are added through
// distributed shared memory in rank order. Warps 0..7 gather, then run the epilogue; warp 8
// allocates TMEM and issues the MMAs. Waits are bounded as in vn_dense_tc.cu.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "vn_act.cuh"
#include "vn_dense.h"
#include "vn_internal.h"
#include "vn_split.cuh"
#include "vn_tc.cuh"

namespace vn {
namespace {

constexpr int kGatherThreads = 256;
constexpr int kThreads = kGatherThreads + 32;

struct Source {
  const void* p;
  const void* z;       // the operand is p act'(z) where act says so
  int64_t rows, cols;  // in memory
  int vec;             // 16-byte loads
};
struct Part {
  Source a, b;
  int64_t np, nq;
  int p_tiles, units;
  int chunks;  // of 64 k
  int log_split;  // log2 of the CTAs that share a tile's chunks; a cluster may hold several tiles
  int blocks;  // CTAs of this part
  int slope;   // act of B's slope
  const void* bias;
  int bias_bf16, act;
  const void* residual;
  void* out;
  void* preact;
  void* sum;  // sums of B over k, or NULL
  int sum_bf16;
};
struct GatherParams {
  Part part[2];
  int cluster;
  int withhold;  // test hook: the chunk that CTA 0's first warp never hands over; beyond its last, the final commit
  unsigned long long timeout_ns;
  unsigned int* status;
};

// Eight consecutive elements of an operand as they are in memory.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
template <>
struct Eight<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ uint4 words() const { return a; }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = __uint_as_float(w[q] << 16);
      v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
    }
  }
};
__device__ __forceinline__ Eight<float> load8(const float* base, int64_t rows, int64_t cols, int64_t r, int64_t c, int vec) {
  Eight<float> e;
  e.a = e.b = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r >= rows) return e;
  const float* p = base + r * cols + c;
  const int left = static_cast<int>(min(static_cast<int64_t>(8), cols - c));
  if (vec) {
    if (left > 0) e.a = fetch(reinterpret_cast<const float4*>(p));
    if (left > 4) e.b = fetch(reinterpret_cast<const float4*>(p) + 1);
  } else {
    if (left > 0) e.a.x = fetch(p);
    if (left > 1) e.a.y = fetch(p + 1);
    if (left > 2) e.a.z = fetch(p + 2);
    if (left > 3) e.a.w = fetch(p + 3);
    if (left > 4) e.b.x = fetch(p + 4);
    if (left > 5) e.b.y = fetch(p + 5);
    if (left > 6) e.b.z = fetch(p + 6);
    if (left > 7) e.b.w = fetch(p + 7);
  }
  return e;
}
__device__ __forceinline__ Eight<__nv_bfloat16> load8(const __nv_bfloat16* base, int64_t rows, int64_t cols, int64_t r,
                                                      int64_t c, int) {
  Eight<__nv_bfloat16> e;
  e.a = make_uint4(0u, 0u, 0u, 0u);
  if (r < rows && c < cols) e.a = fetch(reinterpret_cast<const uint4*>(base + r * cols + c));
  return e;
}
// Eight bf16 elements that start anywhere, as the two aligned 16-byte words that hold them (where those
// lie within the matrix; else the elements one by one): put in place when they are used, so
// that the loads of a chunk are all on their way at once. In the gradients 64 of k take 2.9 us a CTA,
// where loads of single elements took 4.4 (1.2 where rows start on 16 bytes).
struct Shifted {
  uint4 a, b;
  uint32_t how;  // elements of a before the first, and 16 times the number of elements (8: all)
  __device__ __forceinline__ uint4 words() const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t x[6], y[5], z[4];
#pragma unroll
    for (int i = 0; i < 6; ++i) x[i] = how & 4 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) y[i] = how & 2 ? x[i + 1] : x[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = __funnelshift_r(y[i], y[i + 1], (how & 1) * 16);
    const int left = static_cast<int>(how >> 4);
    if (left < 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] = left >= 2 * i + 2 ? z[i] : left > 2 * i ? z[i] & 0xFFFFu : 0u;
    }
    return make_uint4(z[0], z[1], z[2], z[3]);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const { Eight<__nv_bfloat16>{words()}.get(v); }
};
__device__ __forceinline__ Shifted load_shifted(const __nv_bfloat16* base, int64_t rows, int64_t cols, int64_t r, int64_t c) {
  Shifted e;
  e.a = e.b = make_uint4(0u, 0u, 0u, 0u);
  e.how = 0;
  if (r >= rows || c >= cols) return e;
  const int left = static_cast<int>(min(static_cast<int64_t>(8), cols - c));
  const int64_t at = r * cols + c;
  const __nv_bfloat16* p = base + at;
  const int before = static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16 / 2);
  if (at >= before && at - before + (before > 0 ? 16 : 8) <= rows * cols) {
    const uint4* q = reinterpret_cast<const uint4*>(p - before);
    e.a = fetch(q);
    if (before > 0) e.b = fetch(q + 1);
    e.how = static_cast<uint32_t>(before | (left << 4));
  } else {
    const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
    auto one = [&](int q) { return q < left ? static_cast<uint32_t>(fetch(h + q)) : 0u; };
    e.a = make_uint4(one(0) | (one(1) << 16), one(2) | (one(3) << 16), one(4) | (one(5) << 16), one(6) | (one(7) << 16));
    e.how = 8u << 4;
  }
  return e;
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// Eight values to their place in a stage: one plane of bf16, or three.
template <typename T>
__device__ __forceinline__ void store_planes(uint32_t addr, uint32_t plane, const float (&v)[8]) {
  uint32_t w[3][4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (sizeof(T) == 4) {
      uint32_t a[3], b[3];
      split3(v[2 * q], a);
      split3(v[2 * q + 1], b);
#pragma unroll
      for (int k = 0; k < 3; ++k) w[k][q] = join_terms(a[k], b[k]);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * q], v[2 * q + 1]);
      w[0][q] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  st_shared16(addr, w[0][0], w[0][1], w[0][2], w[0][3]);
  if constexpr (sizeof(T) == 4) {
    st_shared16(addr + plane, w[1][0], w[1][1], w[1][2], w[1][3]);
    st_shared16(addr + 2 * plane, w[2][0], w[2][1], w[2][2], w[2][3]);
  }
}

// A group as it was loaded: in bf16 a copy.
template <typename T, typename E>
__device__ __forceinline__ void store_group(uint32_t addr, uint32_t plane, const E& e) {
  if constexpr (sizeof(T) == 2) {
    const uint4 w = e.words();
    st_shared16(addr, w.x, w.y, w.z, w.w);
  } else {
    float v[8];
    e.get(v);
    store_planes<T>(addr, plane, v);
  }
}

__device__ __forceinline__ Eight<float> load8(const float* p) {
  Eight<float> e;
  e.a = fetch(reinterpret_cast<const float4*>(p));
  e.b = fetch(reinterpret_cast<const float4*>(p) + 1);
  return e;
}
__device__ __forceinline__ Eight<__nv_bfloat16> load8(const __nv_bfloat16* p) {
  Eight<__nv_bfloat16> e;
  e.a = fetch(reinterpret_cast<const uint4*>(p));
  return e;
}

// A tile's operand of kRows rows x 64 k, gathered by 256 threads, kCount groups of eight each.
// Group g of thread t is number g * 256 + t; eight lanes take one 128-byte row of the tile
// (16 lanes 128 elements of p or q).
template <typename T, bool kMn, int kRows, bool kShift>
struct Gather {
  static constexpr int kCount = kRows * 8 / kGatherThreads > 0 ? kRows * 8 / kGatherThreads : 1;
  static constexpr bool kAll = kRows * 8 >= kGatherThreads;  // every thread has a group
  static constexpr int kAcross = kMn ? kRows / 8 : 8;        // groups along the contiguous dimension
  static constexpr int kNext = kGatherThreads / kAcross;     // tile rows from one group of a thread to its next
  static_assert(kGatherThreads % kAcross == 0, "a thread's groups share their place along a row");
  std::conditional_t<kShift, Shifted, Eight<T>> v[kCount];

  // All of the tile's rows, and all of its 64 k, lie inside: plain vector loads.
  static __device__ __forceinline__ bool inside(const Source& s, int64_t base, int64_t k0) {
    return s.vec && (kMn ? base + kRows <= s.cols && k0 + kK <= s.rows : base + kRows <= s.rows && k0 + kK <= s.cols);
  }
  __device__ __forceinline__ void load(const T* p, const Source& s, int64_t base, int64_t k0, int t) {
    if (!kAll && t >= kRows * 8) return;
    const int row = t / kAcross, col = t % kAcross;
    const int64_t r = (kMn ? k0 : base) + row, c = (kMn ? base : k0) + col * 8;
    if constexpr (kShift) {
#pragma unroll
      for (int g = 0; g < kCount; ++g) v[g] = load_shifted(p, s.rows, s.cols, r + g * kNext, c);
    } else if (inside(s, base, k0)) {
      const T* at = p + r * s.cols + c;
      const int64_t next = kNext * s.cols;
#pragma unroll
      for (int g = 0; g < kCount; ++g) v[g] = load8(at + g * next);
    } else {
#pragma unroll
      for (int g = 0; g < kCount; ++g) v[g] = load8(p, s.rows, s.cols, r + g * kNext, c, s.vec);
    }
  }
  static __device__ __forceinline__ uint32_t offset(int g, int t) {
    const int row = t / kAcross + g * kNext, col = t % kAcross;
    const uint32_t block = kMn ? static_cast<uint32_t>(col >> 3) * kBlockBytes : 0u;
    return block + row * 128u + (static_cast<uint32_t>((col & 7) ^ (row & 7)) << 4);
  }
};

template <typename T>
constexpr int kPlanes = sizeof(T) == 4 ? 3 : 1;
template <int BN>
constexpr uint32_t kBBytes = BN * 128;
template <typename T, int BN>
constexpr uint32_t kStageBytes = kPlanes<T> * (kABytes + kBBytes<BN>);
// Stages: in bf16 so that two CTAs share an SM.
template <typename T, int BN>
constexpr int kStages = static_cast<int>((sizeof(T) == 4 ? 221184 : 106496) / kStageBytes<T, BN>);

// Accumulators of a tile. MMAs into one accumulator follow each other at the latency of an MMA (about 100
// cycles, three times what one with 64 columns takes), and each rounds its sum towards zero: n steps
// shrink it by about n 2^-25. So the leading products of a chunk's four steps of k rotate over
// kLead accumulators and the five smaller products of fp32 over kRest; the epilogue adds them up.
// In fp32 sums over more than kShort chunks are taken in pieces (kPieces), whose sums a further accumulator
// holds, rounded to nearest: the leading accumulators are added to it after 32 steps each, the others, below
// 2^-6 of the result, after at most 427, so that what is lost does not grow with k (sums of one sign over
// 262,144 rows: 4e-7 of the result, where one piece lost 9e-6). The MMAs stand still meanwhile: 2.3 us for
// each 8 chunks of 128 columns, 0.3 for each 32 of 64. Shorter sums have kernels without it, whose code is
// what small calls wait for (gradients of 1021 x 256 to 256 13.8 us, 14.3 with it).
template <typename T, int BN>
constexpr int kShort = sizeof(T) == 2 ? INT_MAX : BN == 128 ? 16 : 32;
template <typename T, int BN, bool kPieces>
constexpr int kLead = sizeof(T) == 2 ? 2 : BN == 128 ? (kPieces ? 1 : 2) : 4;
template <typename T, int BN>
constexpr int kRest = sizeof(T) == 2 ? 0 : BN == 128 ? 2 : 3;
template <typename T, int BN, bool kPieces>
constexpr int kAccumulators = kLead<T, BN, kPieces> + kRest<T, BN>;
template <typename T, int BN, bool kPieces>
constexpr uint32_t kTmemNeed = (kAccumulators<T, BN, kPieces> + kPieces) * BN;
template <typename T, int BN, bool kPieces>
constexpr uint32_t kTmemCols = kTmemNeed<T, BN, kPieces> <= 32    ? 32
                               : kTmemNeed<T, BN, kPieces> <= 128 ? 128
                               : kTmemNeed<T, BN, kPieces> <= 256 ? 256
                                                                  : 512;
template <int BN>
constexpr int kPiece = BN == 128 ? 8 : 32;  // chunks
template <int BN>
constexpr int kLongPiece = BN == 128 ? 32 : 64;  // of the smaller products

// The sums of 16 columns from `at` on in the first `count` accumulators, and in column `total` on, if any.
template <int BN>
__device__ __forceinline__ void sums_of(uint32_t at, int count, int total, float (&z)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
#pragma unroll 1
  for (int acc = count - (total > 0 ? 0 : 1); acc >= 0; --acc) {  // the smaller products' first
    uint32_t v[16];
    __syncwarp();
    tmem_load16(at + (acc == count ? total : acc * BN), v);
    tmem_wait_load(v);
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] += __uint_as_float(v[i]);
  }
}
// A piece's end: this warp's columns of the first `count` accumulators into those from `total` on.
template <int BN>
__device__ __forceinline__ void end_piece(uint32_t at, int count, int total, bool more) {
#pragma unroll 1
  for (int c = static_cast<int>(threadIdx.x >> 7) * 16; c < BN; c += 32) {
    float z[16];
    sums_of<BN>(at + c, count, more ? total : 0, z);
    tmem_store16(at + total + c, z);
  }
  tmem_wait_store();
}

// One product's tile. kSum: also the sums of B over k (the bias's gradient), by the tiles of p's
// first 128. Called by every thread of the CTA.
template <typename T, int BN, bool kShift, bool kAMn, bool kBMn, bool kSum, bool kPieces, bool kHook>
__device__ __forceinline__ void tile(const Part& d, const GatherParams& g, uint8_t* smem, uint64_t* bars, uint32_t tmem,
                                     volatile Control* ctl, int block, int cta) {
  constexpr int S = kStages<T, BN>;
  constexpr uint32_t kStage = kStageBytes<T, BN>;
  const uint32_t stage0 = smem_u32(smem), bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (S + s); };
  const uint32_t done = bar0 + 8u * (2 * S);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  // `cta` is this CTA's rank in the cluster, `base` that of the first CTA on the same tile.
  const int split = 1 << d.log_split, rank = cta & (split - 1), base = cta - rank;
  const int unit = ((block - cta) >> d.log_split) + (cta >> d.log_split);
  const bool idle = unit >= d.units;  // the last cluster's spare CTAs only keep the cluster's barriers
  const int tp = idle ? 0 : unit % d.p_tiles, tq = idle ? 0 : unit / d.p_tiles;
  const int64_t p0 = static_cast<int64_t>(tp) * 128, q0 = static_cast<int64_t>(tq) * BN;
  // The CTAs' shares of the chunks: the first ones take one more where it does not divide.
  const int share = d.chunks >> d.log_split, more = d.chunks & (split - 1);
  const int first = rank * share + min(rank, more);
  const int last = idle ? first : first + share + (rank < more ? 1 : 0);
  const bool sums = kSum && d.sum != nullptr && tp == 0 && !idle;
  float sum[8] = {};
  // Warp w has p from 32 (w % 4) on, and of 32 columns the first or the last 16.
  const uint32_t tmem_row = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  constexpr int kAccs = kAccumulators<T, BN, kPieces>, kTotal = kAccs * BN;

  if (warp < 8) {
    const int t = threadIdx.x;
    Gather<T, kAMn, 128, kShift> ga;
    Gather<T, kBMn, BN, kShift> gb, gz;
    const T* ap = static_cast<const T*>(d.a.p);
    const T* bp = static_cast<const T*>(d.b.p);
    const T* zp = static_cast<const T*>(d.b.z);
    const bool sloped = d.slope != VN_ACT_NONE;
    Ring rg;
    bool ok = true;
    // Iteration `it` stores chunk it - 1, which the one before loaded, and loads chunk it: one
    // copy of the code for either, since fetching instructions is what small calls wait for.
    // fp32: the iterations after which a piece's MMAs are waited for and added up, ahead of the next chunk.
    int it = first, halt = kPieces ? min(last, first + kPiece<BN>) : last;
#pragma unroll 1
    for (;;) {
#pragma unroll 1
      for (; it <= halt; ++it) {
        const bool have = it > first;
        if (have) {
          if (lane == 0) ok = mbar_wait(empty(rg.s), rg.ph ^ 1u, ctl);
          ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
          if (!ok) break;
          const uint32_t stage = stage0 + rg.s * kStage;
#pragma unroll
          for (int i = 0; i < ga.kCount; ++i) {
            store_group<T>(stage + ga.offset(i, t), kABytes, ga.v[i]);
          }
          if (gb.kAll || t < BN * 8) {
#pragma unroll
            for (int i = 0; i < gb.kCount; ++i) {
              const uint32_t at = stage + kPlanes<T> * kABytes + gb.offset(i, t);
              if (!kSum && !sloped) {
                store_group<T>(at, kBBytes<BN>, gb.v[i]);
                continue;
              }
              float v[8];
              gb.v[i].get(v);
              if (sloped) {
                float z[8];
                gz.v[i].get(z);
                slope_all<true>(d.slope, z, v);
              }
              if (kSum) {
#pragma unroll
                for (int q = 0; q < 8; ++q) sum[q] += v[q];
              }
              store_planes<T>(at, kBBytes<BN>, v);
            }
          }
        }
        if (it < last) {
          const int64_t k = static_cast<int64_t>(it) * kK;
          ga.load(ap, d.a, p0, k, t);
          gb.load(bp, d.b, q0, k, t);
          if (sloped) gz.load(zp, d.b, q0, k, t);
        }
        if (have) {
          fence_async_smem();
          __syncwarp();
          if (lane == 0 && !(kHook && block == 0 && warp == 0 && it - 1 - first == g.withhold)) mbar_arrive(full(rg.s));
          rg.next(S);
        }
      }
      if (!kPieces || !ok || halt == last) break;
      // The chunk stored last was a piece's last: its MMAs have to be complete.
      const bool wrapped = rg.s == 0;
      ok = mbar_wait(empty(wrapped ? S - 1 : rg.s - 1), wrapped ? rg.ph ^ 1u : rg.ph, ctl);
      if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
      fence_after();
      const int count = (halt - first) % kLongPiece<BN> == 0 ? kAccs : kLead<T, BN, kPieces>;
      end_piece<BN>(tmem_row, count, kTotal, halt - first > kPiece<BN>);
      fence_before();
      __syncwarp();
      halt = min(last, halt + kPiece<BN>);
    }
  } else if (elect_one()) {
    const uint32_t idesc = idesc_of(128, BN, kAMn, kBMn);
    Ring rg;
    for (int it = first; it < last; ++it, rg.next(S)) {
      if (!mbar_wait(full(rg.s), rg.ph, ctl)) break;
      fence_after();
      const uint32_t a0 = stage0 + rg.s * kStage, b0 = a0 + kPlanes<T> * kABytes;
      const uint64_t a = descriptor<kAMn>(a0), b = descriptor<kBMn>(b0);
      const bool fresh = kPieces ? (it - first) % kPiece<BN> == 0 : it == first;
      const bool fresh_rest = kPieces ? (it - first) % kLongPiece<BN> == 0 : it == first;
#pragma unroll
      for (int ks = 0; ks < kK / 16; ++ks) {
#pragma unroll
        for (int pr = sizeof(T) == 4 ? 0 : 5; pr < 6; ++pr) {
          const int step = pr == 5 ? ks : ks * 5 + pr;  // among its accumulators' steps of this chunk
          const int ring = pr == 5 ? kLead<T, BN, kPieces> : (kRest<T, BN> > 0 ? kRest<T, BN> : 1);
          const int acc = (pr == 5 ? 0 : kLead<T, BN, kPieces>) + step % ring;
          mma<false>(tmem + acc * BN, further(a, plane_a(pr) * kABytes + ks * kStepBytes<kAMn>),
                     further(b, plane_b(pr) * kBBytes<BN> + ks * kStepBytes<kBMn>), idesc,
                     !(pr == 5 ? fresh : fresh_rest) || step >= ring);
        }
      }
      mma_commit<false>(empty(rg.s));
    }
    if (!(kHook && block == 0 && last - first <= g.withhold)) mma_commit<false>(done);  // also after an abort
    // The epilogue's sums depend on this wait: one that runs out is recorded and skips them. What was issued
    // still gets its time to complete.
    if (!mbar_wait(done, 0, ctl)) settle(done, 0, g.timeout_ns);
  }
  __syncwarp();
  fence_before();
  __syncthreads();  // every MMA is complete: the stages are free
  fence_after();

  // Epilogue. Warp w has p from 32 (w % 4) on. First the accumulators' sums to shared memory, in 16
  // columns at a time of which every other are the upper warps'; then each CTA of the split adds up
  // its share of the columns over all of them, four a step, all loads of a step at once.
  const int row = (warp & 3) * 32 + lane;
  const int64_t pp = p0 + row;
  const int cols = static_cast<int>(min(static_cast<int64_t>(BN), d.nq - q0));
  constexpr int kPitch = BN + 4;  // 16-byte accesses of a row's columns by 32 rows at once
  float* part = reinterpret_cast<float*>(smem);                 // [128][kPitch]
  float* s_sum = reinterpret_cast<float*>(smem) + 128 * kPitch;  // [256][8], then [BN]
  const bool stop = ctl->abort != 0 || idle;
  const bool mine = warp < 8 && !stop && pp < d.np;
  float bias = 0.f;
  if (mine && d.bias != nullptr)
    bias = d.bias_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(d.bias)[pp])
                       : static_cast<const float*>(d.bias)[pp];
  if (warp < 8 && !stop) {
#pragma unroll 1
    for (int c = (warp >> 2) * 16; c < cols; c += 32) {
      float z[16] = {};
      if (first < last) sums_of<BN>(tmem_row + c, kAccs, kPieces && last - first > kPiece<BN> ? kTotal : 0, z);
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4*>(part + row * kPitch + c + i) = make_float4(z[i], z[i + 1], z[i + 2], z[i + 3]);
    }
    if (kSum && sums) {
#pragma unroll
      for (int q = 0; q < 8; ++q) s_sum[threadIdx.x * 8 + q] = sum[q];
    }
  }
  if (kSum && sums) {  // the same for the whole CTA, and for the split
    // Group `col` of eight columns was gathered by the threads t with t % (BN / 8) == col.
    __syncthreads();
    float v = 0.f;
    if (threadIdx.x < BN) {
#pragma unroll 8
      for (int t = threadIdx.x / 8; t < kGatherThreads; t += BN / 8) v += s_sum[t * 8 + threadIdx.x % 8];
    }
    __syncthreads();
    if (threadIdx.x < BN) s_sum[threadIdx.x] = v;
  }
  __syncwarp();
  if (g.cluster > 1) cluster_sync(); else __syncthreads();
  // This CTA's columns: whole steps of four, so that the reads are aligned.
  const int quads = (cols + 3) >> 2;
  const int c0 = ((quads * rank) >> d.log_split) * 4, c1 = min(cols, ((quads * (rank + 1)) >> d.log_split) * 4);
  if (mine) {
    T* const out = static_cast<T*>(d.out);
    T* const pre = static_cast<T*>(d.preact);
    const T* const res = static_cast<const T*>(d.residual);
#pragma unroll 1
    for (int c = c0 + (warp >> 2) * 4; c < c1; c += 8) {
      const int64_t o = (q0 + c) * d.np + pp;
      float r[4] = {}, z[4];
      float4 v[8];
      if (res != nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c + i < c1) r[i] = value(res[o + i * d.np]);
      }
      // Of a last step's columns beyond c1, whatever lies there: they are not stored.
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < split) v[k] = load_cluster4(map_rank(stage0 + (row * kPitch + c) * 4, base + k));
      z[0] = v[0].x; z[1] = v[0].y; z[2] = v[0].z; z[3] = v[0].w;
#pragma unroll
      for (int k = 1; k < 8; ++k)
        if (k < split) {
          z[0] += v[k].x; z[1] += v[k].y; z[2] += v[k].z; z[3] += v[k].w;
        }
      if constexpr (kSum) {  // only these are split 16 ways
        if (split > 8) {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = load_cluster4(map_rank(stage0 + (row * kPitch + c) * 4, base + 8 + k));
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            z[0] += v[k].x; z[1] += v[k].y; z[2] += v[k].z; z[3] += v[k].w;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] += bias;
      if (pre != nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c + i < c1) pre[o + i * d.np] = narrow<T>(z[i]);
      }
      activate_all<true>(d.act, z);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < c1) out[o + i * d.np] = narrow<T>(z[i] + r[i]);
    }
  }
  if (kSum && sums && rank == 0 && !stop && threadIdx.x < cols) {
    float v = 0.f;
    for (int k = 0; k < split; ++k) v += load_cluster(map_rank(smem_u32(s_sum + threadIdx.x), base + k));
    if (d.sum_bf16) static_cast<__nv_bfloat16*>(d.sum)[q0 + threadIdx.x] = __float2bfloat16_rn(v);
    else static_cast<float*>(d.sum)[q0 + threadIdx.x] = v;
  }
  __syncwarp();
  if (g.cluster > 1) cluster_sync();  // no CTA's partial sums go while another may read them
}

// kBackward: parts 0 and 1 are dx (A = W, B = d) and dw (A = x, B = d^T, with the bias's sums);
// otherwise part 0 is the forward product.
// In bf16 the registers of two CTAs fit an SM, as their stages do.
// kHook: the instance whose waits a test makes run out.
template <typename T, int BN, bool kBackward, bool kShift, bool kPieces = false, bool kHook = false>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1)
gather_kernel(const __grid_constant__ GatherParams g) {
  constexpr int S = kStages<T, BN>;
  constexpr uint32_t kCols = kTmemCols<T, BN, kPieces>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * kStageBytes<T, BN>);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 2 * S + 1);
  volatile Control* ctl = reinterpret_cast<volatile Control*>(bars + 2 * S + 2);
  const int warp = threadIdx.x >> 5;
  {
    // Every warp reads one 64-byte line of the parameters: their misses in the constant cache
    // then overlap each other and the setup, instead of meeting the epilogue one by one.
    static_assert(sizeof(GatherParams) <= 9 * 64, "a line of the parameters for each of 9 warps");
    const int at = min(warp * 16, static_cast<int>(sizeof(GatherParams) / 4) - 1);
    asm volatile("" ::"r"(reinterpret_cast<const uint32_t*>(&g)[at]));
  }
  if (threadIdx.x == 0) {
    const uint32_t bar0 = smem_u32(bars);
    for (int s = 0; s < S; ++s) {
      mbar_init(bar0 + 8u * s, kGatherThreads / 32);
      mbar_init(bar0 + 8u * (S + s), 1);
    }
    mbar_init(bar0 + 8u * (2 * S), 1);
    ctl->abort = 0;
    ctl->timeout_ns = g.timeout_ns;
    ctl->status = g.status;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8) tmem_alloc<false>(smem_u32(s_tmem), kCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *s_tmem;
  let_next();
  after_previous();
  const int cta = g.cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int block = static_cast<int>(blockIdx.x);
  if constexpr (kBackward) {
    // The weight's gradient first: its k loop, over the rows, tends to be the longer one.
    if (block < g.part[1].blocks)
      tile<T, BN, kShift, true, true, true, kPieces, kHook>(g.part[1], g, smem, bars, tmem, ctl, block, cta);
    else
      tile<T, BN, kShift, true, false, false, kPieces, kHook>(g.part[0], g, smem, bars, tmem, ctl, block - g.part[1].blocks, cta);
  } else {
    tile<T, BN, kShift, false, false, false, kPieces, kHook>(g.part[0], g, smem, bars, tmem, ctl, block, cta);
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == 8) {
    fence_after();
    tmem_free<false>(tmem, kCols);
  }
}

// ---------------------------------------------------------------- host
template <typename T, int BN, bool kBackward>
constexpr size_t kSmemBytes = 1024 + kStages<T, BN> * kStageBytes<T, BN> + 8 * (2 * kStages<T, BN> + 2) + sizeof(Control);

template <typename T, int BN, bool kBackward, bool kShift, bool kPieces = false, bool kHook = false>
cudaError_t run(GatherParams& g, const int (&log_split)[2], cudaStream_t stream) {
  int64_t blocks = 0;
  g.cluster = 1 << std::max(log_split[0], log_split[1]);
  for (int i = 0; i < 2; ++i) {
    Part& d = g.part[i];
    d.log_split = log_split[i];
    d.p_tiles = static_cast<int>((d.np + 127) / 128);
    const int64_t units = d.p_tiles * ((d.nq + BN - 1) / BN);
    const int64_t all = ((units << log_split[i]) + g.cluster - 1) / g.cluster * g.cluster;
    blocks += all;
    if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    d.units = static_cast<int>(units);
    d.blocks = static_cast<int>(all);
  }
  if (blocks == 0) return cudaSuccess;
  if (!kHook) g.timeout_ns = kTimeoutNs;
  const cudaError_t err = device_status_word(&g.status);
  if (err != cudaSuccess) return err;
  constexpr int S = kStages<T, BN>;
  static_assert(S >= 2 && S * kStageBytes<T, BN> >= (BN + 4) * 512 + 8192, "the partial sums lie in the stages");
  static SmemRecord record;
  if (g.cluster > 8) {
    static SmemRecord wide;  // per device: clusters beyond the portable size are allowed
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (wide[dev].load(std::memory_order_acquire) == 0) {
      err = cudaFuncSetAttribute(reinterpret_cast<const void*>(gather_kernel<T, BN, kBackward, kShift, kPieces, kHook>),
                                 cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (err != cudaSuccess) return err;
      wide[dev].store(1, std::memory_order_release);
    }
  }
  return launch_cluster(gather_kernel<T, BN, kBackward, kShift, kPieces, kHook>, record, static_cast<int>(blocks), kThreads, g.cluster,
                        kSmemBytes<T, BN, kBackward>, stream, g);
}

// fp32: with pieces where a CTA's share of k is long.
template <typename T, int BN, bool kBackward, bool kShift>
cudaError_t run_columns(GatherParams& g, const GatherPlan& plan, cudaStream_t stream) {
  if constexpr (sizeof(T) == 4) {
    for (int i = 0; i < 2; ++i)
      if (((g.part[i].chunks - 1) >> plan.log_split[i]) + 1 > kShort<T, BN>)
        return run<T, BN, kBackward, kShift, true>(g, plan.log_split, stream);
  }
  return run<T, BN, kBackward, kShift>(g, plan.log_split, stream);
}
template <typename T, bool kBackward, bool kShift>
cudaError_t run_tile(GatherParams& g, const GatherPlan& plan, cudaStream_t stream) {
  if constexpr (!kBackward) {
    if (plan.bn == 16) return run_columns<T, 16, kBackward, kShift>(g, plan, stream);
  }
  // In bf16: gradients of 128 columns would hold 108 registers of shifted groups; no forward product is
  // planned on 128 columns, nor on 64 where its rows start on 16 bytes.
  if constexpr (sizeof(T) == 4 || (kBackward && !kShift)) {
    if (plan.bn == 128) return run_columns<T, 128, kBackward, kShift>(g, plan, stream);
  }
  if constexpr (sizeof(T) == 2 && !kBackward && !kShift) return cudaErrorInvalidValue;
  else return run_columns<T, 64, kBackward, kShift>(g, plan, stream);
}
template <typename T, bool kBackward>
cudaError_t run_plan(GatherParams& g, const GatherPlan& plan, cudaStream_t stream) {
  if constexpr (sizeof(T) == 2) {
    bool vec = true;
    for (const Part& d : g.part) vec = vec && (d.np == 0 || d.nq == 0 || (d.a.vec && d.b.vec));
    if (!vec) return run_tile<T, kBackward, true>(g, plan, stream);
  }
  return run_tile<T, kBackward, false>(g, plan, stream);
}

Source source(const void* p, const void* z, int64_t rows, int64_t cols, vn_dtype dt) {
  const bool fits = reinterpret_cast<uintptr_t>(p) % 16 == 0 && reinterpret_cast<uintptr_t>(z) % 16 == 0;
  return Source{p, z, rows, cols, fits && cols % (dt == VN_BF16 ? 8 : 4) == 0};
}
int chunks_of(int64_t nk) { return static_cast<int>((nk + kK - 1) / kK); }

}  // namespace

cudaError_t launch_gather_forward(const DenseArgs& a, const GatherPlan& plan, cudaStream_t stream, const Withhold* hook) {
  GatherParams g = {};
  Part& d = g.part[0];
  d.a = source(a.w, nullptr, a.out, a.in, a.dt);
  d.b = source(a.x, nullptr, a.rows, a.in, a.dt);
  d.np = a.out; d.nq = a.rows; d.chunks = chunks_of(a.in);
  d.bias = a.b; d.bias_bf16 = a.b_dt == VN_BF16; d.act = a.act;
  d.residual = a.residual; d.out = a.y; d.preact = a.preact;
  if (hook != nullptr) {
    g.withhold = hook->at;
    g.timeout_ns = hook->timeout_ns;
    return a.dt == VN_BF16 ? run<__nv_bfloat16, 16, false, false, false, true>(g, plan.log_split, stream)
                           : run<float, 16, false, false, true, true>(g, plan.log_split, stream);
  }
  return a.dt == VN_BF16 ? run_plan<__nv_bfloat16, false>(g, plan, stream)
                         : run_plan<float, false>(g, plan, stream);
}

cudaError_t launch_gather_backward(const DenseGradArgs& a, const GatherPlan& plan, cudaStream_t stream) {
  GatherParams g = {};
  const void* z = a.act != VN_ACT_NONE ? a.preact : nullptr;
  if (a.grad_x != nullptr) {
    Part& d = g.part[0];
    d.a = source(a.w, nullptr, a.out, a.in, a.dt);
    d.b = source(a.grad, z, a.rows, a.out, a.dt);
    d.np = a.in; d.nq = a.rows; d.chunks = chunks_of(a.out);
    d.slope = a.act;
    d.out = a.grad_x;
  }
  if (a.grad_w != nullptr) {
    Part& d = g.part[1];
    d.a = source(a.x, nullptr, a.rows, a.in, a.dt);
    d.b = source(a.grad, z, a.rows, a.out, a.dt);
    d.np = a.in; d.nq = a.out; d.chunks = chunks_of(a.rows);
    d.slope = a.act;
    d.out = a.grad_w;
    d.sum = a.grad_b; d.sum_bf16 = a.gb_dt == VN_BF16;
  }
  return a.dt == VN_BF16 ? run_plan<__nv_bfloat16, true>(g, plan, stream)
                         : run_plan<float, true>(g, plan, stream);
}

}  // namespace vn
