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
// (grads of 1021 x 256 x 256 in fp32: 109 us before, of which 97 in two products of 16 and 64
// CTAs without tensor cores).
//
// The k loop is split over the CTAs of a cluster of up to 8; partial sums are added through
// distributed shared memory in rank order. Warps 0..7 gather, then run the epilogue; warp 8
// allocates TMEM and issues the MMAs. Waits are bounded as in vn_dense_tc.cu.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

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
  int split;   // CTAs that share a tile's chunks: a cluster holds cluster / split tiles
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
  unsigned long long timeout_ns;
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
    if (left > 0) e.a = __ldg(reinterpret_cast<const float4*>(p));
    if (left > 4) e.b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  } else {
    if (left > 0) e.a.x = __ldg(p);
    if (left > 1) e.a.y = __ldg(p + 1);
    if (left > 2) e.a.z = __ldg(p + 2);
    if (left > 3) e.a.w = __ldg(p + 3);
    if (left > 4) e.b.x = __ldg(p + 4);
    if (left > 5) e.b.y = __ldg(p + 5);
    if (left > 6) e.b.z = __ldg(p + 6);
    if (left > 7) e.b.w = __ldg(p + 7);
  }
  return e;
}
__device__ __forceinline__ Eight<__nv_bfloat16> load8(const __nv_bfloat16* base, int64_t rows, int64_t cols, int64_t r,
                                                      int64_t c, int vec) {
  Eight<__nv_bfloat16> e;
  e.a = make_uint4(0u, 0u, 0u, 0u);
  if (r >= rows) return e;
  const int left = static_cast<int>(min(static_cast<int64_t>(8), cols - c));
  if (vec) {
    if (left > 0) e.a = __ldg(reinterpret_cast<const uint4*>(base + r * cols + c));
  } else {
    const unsigned short* p = reinterpret_cast<const unsigned short*>(base) + r * cols + c;
    uint32_t h[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) h[q] = q < left ? __ldg(p + q) : 0u;
    e.a = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
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

__device__ __forceinline__ Eight<float> load8(const float* p) {
  Eight<float> e;
  e.a = __ldg(reinterpret_cast<const float4*>(p));
  e.b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  return e;
}
__device__ __forceinline__ Eight<__nv_bfloat16> load8(const __nv_bfloat16* p) {
  Eight<__nv_bfloat16> e;
  e.a = __ldg(reinterpret_cast<const uint4*>(p));
  return e;
}

// A tile's operand of kRows rows x 64 k, gathered by 256 threads, kCount groups of eight each.
// Group g of thread t is number g * 256 + t; eight lanes take one 128-byte row of the tile
// (16 lanes 128 elements of p or q).
template <typename T, bool kMn, int kRows>
struct Gather {
  static constexpr int kCount = kRows * 8 / kGatherThreads > 0 ? kRows * 8 / kGatherThreads : 1;
  static constexpr bool kAll = kRows * 8 >= kGatherThreads;  // every thread has a group
  static constexpr int kAcross = kMn ? kRows / 8 : 8;        // groups along the contiguous dimension
  static constexpr int kNext = kGatherThreads / kAcross;     // tile rows from one group of a thread to its next
  static_assert(kGatherThreads % kAcross == 0, "a thread's groups share their place along a row");
  Eight<T> v[kCount];

  // All of the tile's rows, and all of its 64 k, lie inside: plain vector loads.
  static __device__ __forceinline__ bool inside(const Source& s, int64_t base, int64_t k0) {
    return s.vec && (kMn ? base + kRows <= s.cols && k0 + kK <= s.rows : base + kRows <= s.rows && k0 + kK <= s.cols);
  }
  __device__ __forceinline__ void load(const T* p, const Source& s, int64_t base, int64_t k0, int t) {
    if (!kAll && t >= kRows * 8) return;
    const int row = t / kAcross, col = t % kAcross;
    const int64_t r = (kMn ? k0 : base) + row, c = (kMn ? base : k0) + col * 8;
    if (inside(s, base, k0)) {
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
constexpr uint32_t kBBytes = BN < 64 ? BN * 128 : BN * 128;
template <typename T, int BN>
constexpr uint32_t kStageBytes = kPlanes<T> * (kABytes + kBBytes<BN>);
// Stages: in bf16 so that two CTAs share an SM.
template <typename T, int BN>
constexpr int kStages = sizeof(T) == 4 ? static_cast<int>(221184 / kStageBytes<T, BN>) : static_cast<int>(106496 / kStageBytes<T, BN>);

// The tensor cores round each step's sum towards zero: n steps into one accumulator shrink it by
// about n 2^-25. In fp32 the leading products therefore rotate over all accumulators that
// TMEM holds but one, which takes the five smaller ones; the epilogue adds them up.
template <typename T, int BN>
constexpr int kMain = sizeof(T) == 2 ? 1 : (512 / BN > 8 ? 7 : 512 / BN - 1);
template <typename T, int BN>
constexpr uint32_t kTmemCols = sizeof(T) == 2 ? (BN < 32 ? 32 : BN) : (kMain<T, BN> + 1) * BN;

// One product's tile. kSum: also the sums of B over k (the bias's gradient), by the tiles of p's
// first 128. Called by every thread of the CTA.
template <typename T, int BN, bool kAMn, bool kBMn, bool kSum>
__device__ __forceinline__ void tile(const Part& d, const GatherParams& g, uint8_t* smem, uint64_t* bars, uint32_t tmem,
                                     volatile Control* ctl, int block, int cta) {
  constexpr int S = kStages<T, BN>;
  constexpr uint32_t kStage = kStageBytes<T, BN>;
  const uint32_t stage0 = smem_u32(smem), bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (S + s); };
  const uint32_t done = bar0 + 8u * (2 * S);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // `cta` is this CTA's rank in the cluster, `base` that of the first CTA on the same tile.
  const int split = d.split, rank = cta % split, base = cta - rank;
  const int unit = (block - cta) / split + cta / split;
  const bool idle = unit >= d.units;  // the last cluster's spare CTAs only keep the cluster's barriers
  const int tp = idle ? 0 : unit % d.p_tiles, tq = idle ? 0 : unit / d.p_tiles;
  const int64_t p0 = static_cast<int64_t>(tp) * 128, q0 = static_cast<int64_t>(tq) * BN;
  const int first = static_cast<int>(static_cast<int64_t>(d.chunks) * rank / split);
  const int last = idle ? first : static_cast<int>(static_cast<int64_t>(d.chunks) * (rank + 1) / split);
  const bool sums = kSum && d.sum != nullptr && tp == 0 && !idle;
  float sum[8] = {};

  if (warp < 8) {
    const int t = threadIdx.x;
    Gather<T, kAMn, 128> ga;
    Gather<T, kBMn, BN> gb, gz;
    const T* ap = static_cast<const T*>(d.a.p);
    const T* bp = static_cast<const T*>(d.b.p);
    const T* zp = static_cast<const T*>(d.b.z);
    const bool sloped = d.slope != VN_ACT_NONE;
    Ring rg;
    bool ok = true;
    if (first < last) {
      ga.load(ap, d.a, p0, static_cast<int64_t>(first) * kK, t);
      gb.load(bp, d.b, q0, static_cast<int64_t>(first) * kK, t);
      if (sloped) gz.load(zp, d.b, q0, static_cast<int64_t>(first) * kK, t);
    }
    for (int it = first; it < last; ++it, rg.next(S)) {
      if (lane == 0) ok = mbar_wait(empty(rg.s), rg.ph ^ 1u, ctl);
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if (!ok) break;
      const uint32_t stage = stage0 + rg.s * kStage;
#pragma unroll
      for (int i = 0; i < ga.kCount; ++i) {
        float v[8];
        ga.v[i].get(v);
        store_planes<T>(stage + ga.offset(i, t), kABytes, v);
      }
      if (gb.kAll || t < BN * 8) {
#pragma unroll
        for (int i = 0; i < gb.kCount; ++i) {
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
          store_planes<T>(stage + kPlanes<T> * kABytes + gb.offset(i, t), kBBytes<BN>, v);
        }
      }
      if (it + 1 < last) {
        const int64_t k = static_cast<int64_t>(it + 1) * kK;
        ga.load(ap, d.a, p0, k, t);
        gb.load(bp, d.b, q0, k, t);
        if (sloped) gz.load(zp, d.b, q0, k, t);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full(rg.s));
    }
  } else if (lane == 0) {
    const uint32_t idesc = idesc_of(128, BN, kAMn, kBMn);
    Ring rg;
    uint32_t main = 0;
    for (int it = first; it < last; ++it, rg.next(S)) {
      if (!mbar_wait(full(rg.s), rg.ph, ctl)) break;
      fence_after();
      const uint32_t a0 = stage0 + rg.s * kStage, b0 = a0 + kPlanes<T> * kABytes;
#pragma unroll
      for (int pr = sizeof(T) == 4 ? 0 : 5; pr < 6; ++pr) {
        const uint32_t a = a0 + plane_a(pr) * kABytes, b = b0 + plane_b(pr) * kBBytes<BN>;
        const bool lead = pr == 5;
        const uint32_t acc = tmem + (lead ? main * BN : kMain<T, BN> * BN);
        const bool fresh = lead ? it - first < kMain<T, BN> : it == first && pr == 0;
#pragma unroll
        for (int ks = 0; ks < kK / 16; ++ks)
          mma<false>(acc, descriptor<kAMn>(a + ks * kStepBytes<kAMn>), descriptor<kBMn>(b + ks * kStepBytes<kBMn>),
                     idesc, !fresh || ks != 0);
      }
      if (++main == kMain<T, BN>) main = 0;
      mma_commit<false>(empty(rg.s));
    }
    mma_commit<false>(done);  // also after an abort: what was issued completes
    const uint64_t t0 = global_ns();
    while (!mbar_try(done, 0) && global_ns() - t0 < g.timeout_ns) {
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();  // every MMA is complete: the stages are free
  fence_after();

  // Epilogue: warp w has lanes 32 (w % 4) .. of p and every other 16 columns from 16 (w / 4).
  const int row = (warp & 3) * 32 + lane;
  const int64_t pp = p0 + row;
  const int cols = static_cast<int>(min(static_cast<int64_t>(BN), d.nq - q0));
  float* part = reinterpret_cast<float*>(smem);              // [BN][128]
  float* s_sum = reinterpret_cast<float*>(smem) + BN * 128;  // [256][8], then [BN]
  const bool stop = ctl->abort != 0 || idle;
  Epilogue e;
  e.bias = d.bias; e.bias_bf16 = d.bias_bf16; e.act = d.act; e.residual = d.residual; e.out = d.out; e.preact = d.preact;
  e.np = d.np;
  const float bias = warp < 8 ? bias_of(e, pp) : 0.f;
  if (warp < 8 && !stop) {
    const uint32_t at = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    for (int c = (warp >> 2) * 16; c < cols; c += 32) {
      Residual<T> r;
      if (split == 1) load_residual(e, q0 + c, pp, cols - c, &r);
      float z[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) z[i] = 0.f;
      if (first < last) {
        const int mains = min(kMain<T, BN>, last - first);
        auto add = [&](int acc) {
          uint32_t v[16];
          __syncwarp();
          tmem_load16(at + acc * BN + c, v);
          tmem_wait_load();
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] += __uint_as_float(v[i]);
        };
        if constexpr (sizeof(T) == 4) add(kMain<T, BN>);
#pragma unroll 1
        for (int acc = 0; acc < mains; ++acc) add(acc);
      }
      if (split == 1) {
        if (pp < d.np) finish<T>(e, z, r, q0 + c, pp, cols - c, bias);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(c + i) * 128 + row] = z[i];
      }
    }
    if (kSum && sums) {
#pragma unroll
      for (int q = 0; q < 8; ++q) s_sum[threadIdx.x * 8 + q] = sum[q];
    }
  }
  if (kSum && sums) {  // the same for the whole CTA, and for the cluster
    // Group `col` of eight columns was gathered by the threads t with t % (BN / 8) == col.
    __syncthreads();
    float v = 0.f;
    if (threadIdx.x < BN)
      for (int t = threadIdx.x / 8; t < kGatherThreads; t += BN / 8) v += s_sum[t * 8 + threadIdx.x % 8];
    __syncthreads();
    if (threadIdx.x < BN) s_sum[threadIdx.x] = v;
    if (split == 1 && threadIdx.x < cols && !stop) {
      if (d.sum_bf16) static_cast<__nv_bfloat16*>(d.sum)[q0 + threadIdx.x] = __float2bfloat16_rn(v);
      else static_cast<float*>(d.sum)[q0 + threadIdx.x] = v;
    }
  }
  if (g.cluster > 1) {
    __syncwarp();
    cluster_sync();
    if (warp < 8 && !stop && split > 1) {
      const int c0 = cols * rank / split, c1 = cols * (rank + 1) / split;
      if (pp < d.np) {
        for (int c = c0 + (warp >> 2) * 8; c < c1; c += 16) {
          float z[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] = 0.f;
          const int count = min(8, c1 - c);
          Residual<T> r;
          load_residual(e, q0 + c, pp, count, &r);
          for (int k = 0; k < split; ++k) {
            const uint32_t from = map_rank(stage0 + (c * 128 + row) * 4, base + k);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i < count) z[i] += load_cluster(from + i * 512);
          }
          finish<T>(e, z, r, q0 + c, pp, count, bias);
        }
      }
      if (kSum && sums && rank == 0 && threadIdx.x < cols) {
        float v = 0.f;
        for (int k = 0; k < split; ++k) v += load_cluster(map_rank(smem_u32(s_sum + threadIdx.x), base + k));
        if (d.sum_bf16) static_cast<__nv_bfloat16*>(d.sum)[q0 + threadIdx.x] = __float2bfloat16_rn(v);
        else static_cast<float*>(d.sum)[q0 + threadIdx.x] = v;
      }
    }
    __syncwarp();
    cluster_sync();
  }
}

// kBackward: parts 0 and 1 are dx (A = W, B = d) and dw (A = x, B = d^T, with the bias's sums);
// otherwise part 0 is the forward product.
template <typename T, int BN, bool kBackward>
__global__ void __launch_bounds__(kThreads) gather_kernel(const __grid_constant__ GatherParams g) {
  constexpr int S = kStages<T, BN>;
  constexpr uint32_t kCols = kTmemCols<T, BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * kStageBytes<T, BN>);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 2 * S + 1);
  volatile Control* ctl = reinterpret_cast<volatile Control*>(bars + 2 * S + 2);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    const uint32_t bar0 = smem_u32(bars);
    for (int s = 0; s < S; ++s) {
      mbar_init(bar0 + 8u * s, kGatherThreads / 32);
      mbar_init(bar0 + 8u * (S + s), 1);
    }
    mbar_init(bar0 + 8u * (2 * S), 1);
    ctl->abort = 0;
    ctl->timeout_ns = g.timeout_ns;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8) tmem_alloc<false>(smem_u32(s_tmem), kCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *s_tmem;
  const int cta = g.cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int block = static_cast<int>(blockIdx.x);
  if constexpr (kBackward) {
    // The weight's gradient first: its k loop, over the rows, tends to be the longer one.
    if (block < g.part[1].blocks)
      tile<T, BN, true, true, true>(g.part[1], g, smem, bars, tmem, ctl, block, cta);
    else
      tile<T, BN, true, false, false>(g.part[0], g, smem, bars, tmem, ctl, block - g.part[1].blocks, cta);
  } else {
    tile<T, BN, false, false, false>(g.part[0], g, smem, bars, tmem, ctl, block, cta);
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
cudaError_t run(GatherParams& g, const int (&split)[2], cudaStream_t stream) {
  int64_t blocks = 0;
  g.cluster = std::max(split[0], split[1]);
  for (int i = 0; i < 2; ++i) {
    Part& d = g.part[i];
    d.split = split[i];
    d.p_tiles = static_cast<int>((d.np + 127) / 128);
    const int64_t units = d.p_tiles * ((d.nq + BN - 1) / BN);
    const int64_t all = (units * d.split + g.cluster - 1) / g.cluster * g.cluster;
    blocks += all;
    if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    d.units = static_cast<int>(units);
    d.blocks = static_cast<int>(all);
  }
  if (blocks == 0) return cudaSuccess;
  g.timeout_ns = kTimeoutNs;
  constexpr int S = kStages<T, BN>;
  static_assert(S >= 2 && S * kStageBytes<T, BN> >= BN * 512 + 8192, "the partial sums lie in the stages");
  static SmemRecord record;
  return launch_cluster(gather_kernel<T, BN, kBackward>, record, static_cast<int>(blocks), kThreads, g.cluster,
                        1024 + S * kStageBytes<T, BN> + 8 * (2 * S + 2) + sizeof(Control), stream, g);
}

// Tile width and splits by the time they take: rounds of CTAs over the GPU x (stages the longest
// CTA walks x a stage's time + what a CTA takes besides).
template <typename T, bool kBackward>
cudaError_t choose(GatherParams& g, int sms, cudaStream_t stream) {
  int best_bn = 64, best_split[2] = {1, 1};
  double best = 1e30;
  const int wide[3] = {16, 64, 128};
  for (int w = kBackward ? 1 : 0; w < 3; ++w) {
    const int bn = wide[w];
    const double stage = sizeof(T) == 4 ? (bn == 128 ? 1.9 : bn == 64 ? 1.5 : 1.2) : (bn == 128 ? 1.0 : 0.9);
    const double room = sms * (sizeof(T) == 2 ? 2 : 1);
    for (int s0 = 1; s0 <= 8; s0 *= 2)
      for (int s1 = 1; s1 <= 8; s1 *= 2) {
        const int split[2] = {s0, s1};
        double work = 0, longest = 0, ctas = 0;  // in stages, of all CTAs and of the longest
        for (int i = 0; i < 2; ++i) {
          const Part& d = g.part[i];
          if (d.np == 0 || d.nq == 0) continue;
          const double n = static_cast<double>((d.np + 127) / 128) * ((d.nq + bn - 1) / bn) * split[i];
          const double t = ((d.chunks + split[i] - 1) / split[i]) * stage + 3.0 + (split[i] > 1 ? 1.0 : 0.0);
          ctas += n;
          work += n * t;
          longest = std::max(longest, t);
        }
        const double t = std::max(longest, ctas > room ? work / room + 0.5 * longest : 0.0);
        if (t < best) { best = t; best_bn = bn; best_split[0] = s0; best_split[1] = s1; }
      }
  }
  if constexpr (!kBackward) {
    if (best_bn == 16) return run<T, 16, kBackward>(g, best_split, stream);
  }
  return best_bn == 64 ? run<T, 64, kBackward>(g, best_split, stream) : run<T, 128, kBackward>(g, best_split, stream);
}

Source source(const void* p, const void* z, int64_t rows, int64_t cols, vn_dtype dt) {
  const bool fits = reinterpret_cast<uintptr_t>(p) % 16 == 0 && reinterpret_cast<uintptr_t>(z) % 16 == 0;
  return Source{p, z, rows, cols, fits && cols % (dt == VN_BF16 ? 8 : 4) == 0};
}
int chunks_of(int64_t nk) { return static_cast<int>((nk + kK - 1) / kK); }

}  // namespace

cudaError_t launch_gather_forward(const DenseArgs& a, cudaStream_t stream) {
  DeviceInfo dev;
  const cudaError_t err = device_info(&dev);
  if (err != cudaSuccess) return err;
  GatherParams g = {};
  Part& d = g.part[0];
  d.a = source(a.w, nullptr, a.out, a.in, a.dt);
  d.b = source(a.x, nullptr, a.rows, a.in, a.dt);
  d.np = a.out; d.nq = a.rows; d.chunks = chunks_of(a.in);
  d.bias = a.b; d.bias_bf16 = a.b_dt == VN_BF16; d.act = a.act;
  d.residual = a.residual; d.out = a.y; d.preact = a.preact;
  return a.dt == VN_BF16 ? choose<__nv_bfloat16, false>(g, dev.sm_count, stream)
                         : choose<float, false>(g, dev.sm_count, stream);
}

cudaError_t launch_gather_backward(const DenseGradArgs& a, cudaStream_t stream) {
  DeviceInfo dev;
  const cudaError_t err = device_info(&dev);
  if (err != cudaSuccess) return err;
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
  return a.dt == VN_BF16 ? choose<__nv_bfloat16, true>(g, dev.sm_count, stream)
                         : choose<float, true>(g, dev.sm_count, stream);
}

cudaError_t take_gather_status(unsigned int* status, cudaStream_t stream) { return take_wait_status(status, stream); }

}  // namespace vn
