// vn_dense_tc.cu -- the centre network's products on the 5th-generation tensor cores.
//
//   D[q, p] = sum_k A(p, k) B(q, k), p the contiguous dimension of the result (see
//   vn_dense.cu for the three products that take this form)
//
// MMA rows are p (128 TMEM lanes), MMA columns are q: lane l of a warp then holds output
// p0 + l of every q, so a warp's stores are contiguous, straight from registers. A and B
// are bf16 in memory, either with k contiguous or with p (q) contiguous: TMA writes
// 128-byte-swizzled tiles of 64 elements of the contiguous dimension, and the MMA's
// descriptors and transpose bits say which dimension that is, so no operand is ever transposed
// by a pass of its own.
//
// fp32 operands come as three bf16 planes (8 + 8 + 8 significant bits); the k loop then runs over the
// six products of planes that reach fp32's precision, the smallest first, and no accumulator takes more
// of it than a short piece before it is added to sums in registers.
//
// Two kernels:
//   pair   256 x 256 tiles, one per pair of CTAs (cta_group::2): each CTA stages 128 rows of
//          A and of B, half of what single CTAs would stage for as many products, and L2
//          carries half as much. Persistent; two accumulators of 256 columns in TMEM, so that a
//          tile's epilogue runs under the next tile's products.
//   single 128 x 16, 64 or 128 tiles of one CTA, two CTAs an SM, for problems that do not fill the
//          GPU with pairs: the k loop is split over the CTAs of a cluster of up to 8, whose
//          partial sums are added through distributed shared memory in rank order.
// What bounds the pairs (8192 x 4096 to 4096 in bf16, 141 us, cuBLAS 138): the tensor cores, at 519 cycles
// for 64 k of a 256 x 256 tile where its MMAs take 512, under the power cap's clock of 1.75 GHz. With a
// GELU, a residual and the pre-activation (180 us) the epilogue's copies and instructions
// get in the way of the operands' and the MMAs': 620 cycles.
//
// Warp roles: 0 TMA producer, 1 TMEM allocation and MMA issue, from 2 on epilogue (one or two
// per TMEM lane quarter). Every barrier wait is bounded; one that runs out records a status word,
// stops the other roles, and the kernel drains what it has issued, frees TMEM and returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "vn_act.cuh"
#include "vn_dense.h"
#include "vn_internal.h"
#include "vn_tc.cuh"

namespace vn {

namespace {

constexpr int kThreads = 6 * 32;      // single: 4 epilogue warps
constexpr int kPairThreads = 10 * 32;  // pair: 8, two for each lane quarter, 128 columns each
constexpr int kMaxStages = 8;

struct Params : Epilogue {
  int64_t nq;
  int p_tiles, q_tiles;
  int bn;  // pair: columns of a tile, a multiple of 16
  int64_t units;
  uint32_t staging_bytes;  // pair: the epilogue's chunks, both halves
  int k_chunks, iters;  // iterations of the k loop: k_chunks x pairs of planes
  int stages;
  uint32_t idesc;
  int withhold;  // test hook: the stage of the first CTA that expects more bytes than its copies bring
  unsigned long long timeout_ns;
  unsigned int* status;
};

// Tile of a unit: groups of 8 tiles along q, p fastest between them, so that the CTAs at
// work at one time share few rows of A and of B.
__device__ __forceinline__ void tile_of(const Params& p, int64_t unit, int* tp, int* tq) {
  const int64_t band = static_cast<int64_t>(p.p_tiles) * 8;
  const int64_t g = unit / band, r = unit - g * band;
  const int rows = static_cast<int>(min(static_cast<int64_t>(8), p.q_tiles - g * 8));
  *tp = static_cast<int>(r / rows);
  *tq = static_cast<int>(g * 8 + r % rows);
}

// One stage: A's 128 rows and B's rows of this CTA (one box, or `blocks` 64-wide blocks) of
// 64 k.
template <bool kAMn, bool kBMn, bool kPair>
__device__ __forceinline__ void load_stage(uint32_t dst, const CUtensorMap* am, const CUtensorMap* bm, uint32_t bar,
                                           int p0, int q0, int k0, int pa, int pb, int blocks) {
  if constexpr (kAMn) {
    tma_load<kPair>(dst, am, bar, p0, k0, pa);
    tma_load<kPair>(dst + kBlockBytes, am, bar, p0 + 64, k0, pa);
  } else {
    tma_load<kPair>(dst, am, bar, k0, p0, pa);
  }
  dst += kABytes;
  if constexpr (kBMn) {
    for (int b = 0; b < blocks; ++b) tma_load<kPair>(dst + b * kBlockBytes, bm, bar, q0 + b * 64, k0, pb);
  } else {
    tma_load<kPair>(dst, bm, bar, k0, q0, pb);
  }
}

template <bool kAMn, bool kBMn, bool kPair>
__device__ __forceinline__ void issue_stage(uint32_t d, uint32_t stage, uint32_t idesc, bool first) {
  const uint64_t a = descriptor<kAMn>(stage), b = descriptor<kBMn>(stage + kABytes);
#pragma unroll
  for (int ks = 0; ks < kK / 16; ++ks)
    mma<kPair>(d, further(a, ks * kStepBytes<kAMn>), further(b, ks * kStepBytes<kBMn>), idesc, !(first && ks == 0));
}

// ---------------------------------------------------------------- pairs of CTAs
// Staged epilogue: each half of the epilogue warps (128 threads, half the tile's columns)
// moves 16 columns x 128 p at a time through shared memory, residual in and outputs out by
// TMA: whole 256-byte rows travel, and no warp waits on a load of its own. With GELU, residual and
// pre-activation in bf16: 8192 x 1024 to 4096 80 us, and 132 to 4095, whose rows TMA cannot take and
// whose epilogue is straight 2-byte loads and stores. A chunk has one of three buffers, where an output
// takes its residual's place, and there are three for the pre-activation: with two, a chunk took
// as long as its predecessor's copy out of shared memory.
constexpr int kBuffers = 3;
template <typename T>
constexpr uint32_t kChunkBytes = 16 * 128 * sizeof(T);
constexpr uint32_t kPairStageBytes = kABytes + 128 * 128;

// fp32: the accumulator rounds each step's sum towards zero, which over n steps of one sign shrinks it by
// about n 2^-25 (8e-6 of the result at k = 4096, 2e-4 at 65,536). So an accumulator takes one piece of the
// k loop, kDrain stages of 4 steps; then the epilogue's warps add it to sums in their registers while the
// MMAs go on in the other one. The five smaller products' sums are below 2^-6 of the result and take
// longer pieces. An accumulator is read in about 3,000 cycles beside MMAs, 8 stages of 256 columns take
// 4,150: 4096 cubed 482 us (without pieces 477, and off by 8e-6 of sums of one sign where it is now off by
// 3.4e-7; pieces of 6 stages 497 us and 2.6e-7, of 4 513 us and 1.3e-7).
constexpr int kDrain = 8, kLongDrain = 128;
// Where the piece ends that begins with iteration `at`.
__device__ __forceinline__ int piece_end(const Params& p, int at) {
  const int leading = 5 * p.k_chunks;
  return at < leading ? min(at + kLongDrain, leading) : min(at + kDrain, p.iters);
}

// Barriers: full[S] (leader's, armed for both CTAs' bytes), empty[S], tmem_full[2],
// tmem_empty[2] (leader's, both CTAs' epilogues), drain, residual[2 halves][kBuffers].
// kHook: the instance whose waits a test makes run out.
template <typename T, bool kAMn, bool kBMn, bool kStaged, bool kHook = false>
__global__ void __launch_bounds__(kPairThreads, 1)
pair_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
            const __grid_constant__ CUtensorMap ymap, const __grid_constant__ CUtensorMap zmap,
            const __grid_constant__ CUtensorMap rmap, const Params p) {
  const int S = p.stages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* staging = smem + S * kPairStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + p.staging_bytes);
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (S + s); };
  auto tmem_full = [&](int b) { return bar0 + 8u * (2 * S + b); };
  auto tmem_empty = [&](int b) { return bar0 + 8u * (2 * S + 2 + b); };
  const uint32_t drain = bar0 + 8u * (2 * S + 4);
  auto arrived = [&](int h, int b) { return bar0 + 8u * (2 * S + 5 + kBuffers * h + b); };
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 2 * S + 5 + 2 * kBuffers);
  // Whether the half's leader saw its wait for the tile through: [half][accumulator].
  volatile int* s_go = reinterpret_cast<volatile int*>(bars + 2 * S + 6 + 2 * kBuffers);
  volatile Control* ctl = reinterpret_cast<volatile Control*>(bars + 2 * S + 8 + 2 * kBuffers);
  const uint32_t stage0 = smem_u32(smem);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tmem_full(b), 1);
      mbar_init(tmem_empty(b), 2 * 8);
    }
    mbar_init(drain, 1);
    for (int b = 0; b < 2 * kBuffers; ++b) mbar_init(arrived(0, b), 1);
    ctl->abort = 0;
    ctl->timeout_ns = p.timeout_ns;
    ctl->status = p.status;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<true>(smem_u32(s_tmem), 512);
  fence_before();
  __syncthreads();
  cluster_sync();
  fence_after();
  const uint32_t tmem = *s_tmem;
  let_next();
  after_previous();
  // The peer waits here from its start, so for the whole run of the leader's waits.
  const unsigned long long drain_ns = 4 * p.timeout_ns;
  const int half_q = p.bn / 2;  // rows of B in each CTA

  if (warp == 0) {
    if (elect_one()) {
      Ring rg;
      bool ok = true;
      const int blocks = (half_q + 63) / 64;
      const uint32_t bytes = 2 * (kABytes + (kBMn ? blocks * kBlockBytes : half_q * 128u));
      for (int64_t u = pair; ok && u < p.units; u += pairs) {
        int tp, tq;
        tile_of(p, u, &tp, &tq);
        const int p0 = tp * 256 + static_cast<int>(rank) * 128, q0 = tq * p.bn + static_cast<int>(rank) * half_q;
        int kc = 0, pr = p.iters == p.k_chunks ? 5 : 0;
        for (int it = 0; it < p.iters; ++it, rg.next(S)) {
          if (!(ok = mbar_wait(empty(rg.s), rg.ph ^ 1u, ctl))) break;
          if (rank == 0) mbar_expect_tx(full(rg.s), bytes + (kHook && pair == 0 && it == p.withhold ? 16 : 0));
          load_stage<kAMn, kBMn, true>(stage0 + rg.s * kPairStageBytes, &amap, &bmap, map_rank(full(rg.s), 0), p0, q0,
                                       kc * kK, plane_a(pr), plane_b(pr), blocks);
          if (++kc == p.k_chunks) { kc = 0; ++pr; }
        }
      }
      // The leader's last commits arrive on this CTA's barriers: be there for them.
      for (int s = 0; ok && s < S; ++s, rg.next(S)) ok = mbar_wait(empty(rg.s), rg.ph ^ 1u, ctl);
      if (!ok) {
        // The copies in flight complete on the leader's barriers, which only the leader
        // could wait on and may not have armed: give them far longer than a copy takes.
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < 2000000) __nanosleep(1000);
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      Ring rg, tb;
      bool ok = true, ready = false;
      int at = 0;  // of a tile's iterations, where its next piece begins
      for (int64_t u = pair; ok && u < p.units; tb.next(2)) {
        if (!(ok = mbar_wait(tmem_empty(tb.s), tb.ph ^ 1u, ctl))) break;
        fence_after();
        const int end = sizeof(T) == 4 ? piece_end(p, at) : p.iters;
        for (int it = at; it < end; ++it) {
          if (!ready && !(ok = mbar_wait(full(rg.s), rg.ph, ctl))) break;
          fence_after();
          const int s = rg.s;
          rg.next(S);
          ready = mbar_done(full(rg.s), rg.ph);  // the next stage, while this one's MMAs are issued
          issue_stage<kAMn, kBMn, true>(tmem + tb.s * 256, stage0 + s * kPairStageBytes, p.idesc, it == at);
          mma_commit<true>(empty(s));
        }
        if (ok) mma_commit<true>(tmem_full(tb.s));
        at = end;
        if (end == p.iters) {
          at = 0;
          u += pairs;
        }
      }
      mma_commit<true>(drain);
    }
    __syncwarp();
    if (elect_one()) {  // both CTAs: every MMA of the pair is complete
      settle(drain, 0, drain_ns);
    }
  } else {
    const int quarter = warp & 3;
    const int h = warp < 6 ? 0 : 1;
    const int half = (p.bn / 16 + 1) / 2 * 16;  // columns of half 0
    const int c0 = h * half, width = h ? p.bn - half : half;
    const bool leader = quarter == 2 && lane == 0;  // warps 2 and 6
    // The chunks' buffers, then the pre-activation's.
    T* const buf = reinterpret_cast<T*>(staging + h * (p.staging_bytes / 2));
    const uint32_t buf0 = smem_u32(buf);
    constexpr int kChunk = 16 * 128;
    const bool has_r = p.residual != nullptr, has_z = p.preact != nullptr;
    Ring tb, ck;  // accumulators, chunks' buffers
    constexpr bool kPieces = sizeof(T) == 4;
    float sum[kPieces ? 128 : 1];  // fp32: this lane's sums of the tile
    // All pieces of a tile into `sum`; false after a wait that ran out.
    auto add_pieces = [&](int cols) {
#pragma unroll
      for (int i = 0; i < (kPieces ? 128 : 1); ++i) sum[i] = 0.f;
      for (int at = 0; at < p.iters; at = piece_end(p, at), tb.next(2)) {
        const bool ok = mbar_wait(tmem_full(tb.s), tb.ph, ctl);
        if (!__all_sync(0xFFFFFFFFu, ok)) return false;
        fence_after();
        const uint32_t from = tmem + tb.s * 256 + c0 + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll
        for (int c = 0; c < (kPieces ? 128 : 0); c += 16)
          if (c < cols) {
            uint32_t v[16];
            tmem_load16(from + c, v);
            tmem_wait_load(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[c + i] += __uint_as_float(v[i]);
          }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_rank(tmem_empty(tb.s), 0));
      }
      return true;
    };
    // The first 16 sums, which the others move up to replace.
    auto next_sums = [&](float (&z)[16]) {
#pragma unroll
      for (int i = 0; i < (kPieces ? 16 : 0); ++i) z[i] = sum[i];
#pragma unroll
      for (int i = 0; i < (kPieces ? 112 : 0); ++i) sum[i] = sum[i + 16];
    };
    for (int64_t u = pair; u < p.units; u += pairs) {
      int tp, tq;
      tile_of(p, u, &tp, &tq);
      const int p0 = tp * 256 + static_cast<int>(rank) * 128;
      const int64_t pp = static_cast<int64_t>(p0) + quarter * 32 + lane;
      const int64_t q0 = static_cast<int64_t>(tq) * p.bn + c0;
      const float bias = bias_of(p, pp);
      const int cols = static_cast<int>(min(static_cast<int64_t>(width), p.nq - q0));
      const uint32_t d = tmem + tb.s * 256 + c0 + (static_cast<uint32_t>(quarter * 32) << 16);
      if constexpr (kStaged) {
        auto fetch = [&](int b, int c) {
          mbar_expect_tx(arrived(h, b), kChunkBytes<T>);
          tma_load_2d(buf0 + b * kChunkBytes<T>, &rmap, arrived(h, b), p0, static_cast<int>(q0) + c);
        };
        Ring second = ck;
        second.next(kBuffers);
        if (leader) {
          if (has_r) {  // the outputs that were in these buffers have left
            bulk_wait_read<1>();
            if (cols > 0) fetch(ck.s, 0);
            if (cols > 16) fetch(second.s, 16);
          }
          if (!kPieces) s_go[2 * h + tb.s] = mbar_wait(tmem_full(tb.s), tb.ph, ctl);
        }
        bool go;
        if constexpr (kPieces) {
          __syncwarp();
          go = named_barrier_and(1 + h, 128, add_pieces(cols));
        } else {
          named_barrier(1 + h, 128);
          go = s_go[2 * h + tb.s] != 0;
        }
        if (!go) {  // the residual on its way has to land before the CTA ends
          if (leader && has_r && cols > 0) settle(arrived(h, ck.s), ck.ph, p.timeout_ns);
          if (leader && has_r && cols > 16) settle(arrived(h, second.s), second.ph, p.timeout_ns);
          break;
        }
        fence_after();
        __syncwarp();
        uint32_t v[16];
        if (!kPieces && cols > 0) tmem_load16(d, v);
#pragma unroll 1
        for (int c = 0; c < cols; c += 16, ck.next(kBuffers)) {
          float z[16];
          T pre[kPieces ? 1 : 16];
          if constexpr (kPieces) {
            next_sums(z);
          } else {
            __syncwarp();
            tmem_wait_load(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = __uint_as_float(v[i]);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            z[i] += bias;
            if constexpr (!kPieces) pre[i] = narrow<T>(z[i]);
          }
          __syncwarp();
          if (!kPieces && c + 16 < cols) tmem_load16(d + c + 16, v);
          T* const y = buf + ck.s * kChunk + quarter * 32 + lane;
          if (kPieces && has_z) {  // at once: the sums leave no registers to keep it in
#pragma unroll
            for (int i = 0; i < 16; ++i) y[kBuffers * kChunk + i * 128] = narrow<T>(z[i]);
          }
          activate_all<sizeof(T) == 2>(p.act, z);
          if (has_r) {
            // A wait that ran out ends no thread here, where the others would miss it at the
            // barrier: the products have ended with it, and the next tile's wait is the last.
            mbar_wait(arrived(h, ck.s), ck.ph, ctl);
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] += value(y[i * 128]);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i * 128] = narrow<T>(z[i]);
          if (!kPieces && has_z) {
#pragma unroll
            for (int i = 0; i < 16; ++i) y[kBuffers * kChunk + i * 128] = pre[kPieces ? 0 : i];
          }
          fence_async_smem();
          // One barrier a chunk: it is written, and the next one's buffers have been read out (the
          // leader waits for all copies but the last one's here).
          if (leader) bulk_wait_read<1>();
          named_barrier(1 + h, 128);
          if (leader) {
            const uint32_t from = buf0 + ck.s * kChunkBytes<T>;
            tma_store_2d(&ymap, from, p0, static_cast<int>(q0) + c);
            if (has_z) tma_store_2d(&zmap, from + kBuffers * kChunkBytes<T>, p0, static_cast<int>(q0) + c);
            bulk_commit();
            if (has_r && c + 32 < cols) {
              bulk_wait_read<1>();  // the chunk before this one, whose buffer it is
              fetch(ck.s == 0 ? kBuffers - 1 : ck.s - 1, c + 32);
            }
          }
        }
      } else {
        if constexpr (kPieces) {
          if (!add_pieces(cols)) break;
#pragma unroll 1
          for (int c = 0; c < cols; c += 16) {
            float z[16];
            next_sums(z);
#pragma unroll
            for (int g = 0; g < 16; g += 4) {  // few at a time, beside the sums
              Residual<T, 4> r;
              float some[4] = {z[g], z[g + 1], z[g + 2], z[g + 3]};
              load_residual(p, q0 + c + g, pp, cols - c - g, &r);
              if (pp < p.np) finish<T>(p, some, r, q0 + c + g, pp, cols - c - g, bias);
            }
          }
        } else {
          // The residual's loads run two chunks ahead, from three sets of registers: one that was moved to
          // another would be waited for.
          Residual<T> r0, r1, r2;
          load_residual(p, q0, pp, cols, &r0);
          load_residual(p, q0 + 16, pp, cols - 16, &r1);
          const bool ok = mbar_wait(tmem_full(tb.s), tb.ph, ctl);
          if (!__all_sync(0xFFFFFFFFu, ok)) break;
          fence_after();
          auto chunk = [&](int c, const Residual<T>& r, Residual<T>* ahead) {
            if (c >= cols) return;
            uint32_t v[16];
            tmem_load16(d + c, v);
            load_residual(p, q0 + c + 32, pp, cols - c - 32, ahead);
            tmem_wait_load(v);
            float z[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = __uint_as_float(v[i]);
            if (pp < p.np) finish<T>(p, z, r, q0 + c, pp, cols - c, bias);
            __syncwarp();
          };
#pragma unroll 1
          for (int c = 0; c < cols; c += 48) {
            chunk(c, r0, &r2);
            chunk(c + 16, r1, &r0);
            chunk(c + 32, r2, &r1);
          }
        }
      }
      if constexpr (!kPieces) {
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_rank(tmem_empty(tb.s), 0));
        tb.next(2);
      }
    }
    if (kStaged && leader) bulk_wait_read<0>();
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA's shared memory or TMEM goes while the other may use it
  if (warp == 1) {
    fence_after();
    tmem_free<true>(tmem, 512);
  }
}

// ---------------------------------------------------------------- single CTAs, k split
// The unit's k iterations are split over the cluster's CTAs. Barriers: full[S], empty[S],
// tmem_full[2], tmem_empty[2] (fp32's pieces, in two accumulators), drain.
template <typename T, int BN, bool kAMn, bool kBMn, bool kHook = false>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 2 : 1)
single_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap, const Params p,
              const int split) {
  constexpr uint32_t kStageBytes = kABytes + BN * 128;
  constexpr bool kPieces = sizeof(T) == 4;
  constexpr uint32_t kCols = kPieces ? 2 * BN : BN < 32 ? 32 : BN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int S = p.stages;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(S) * kStageBytes);
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (S + s); };
  auto tmem_full = [&](int b) { return bar0 + 8u * (2 * S + b); };
  auto tmem_empty = [&](int b) { return bar0 + 8u * (2 * S + 2 + b); };
  const uint32_t drain = bar0 + 8u * (2 * S + 4);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 2 * S + 5);
  volatile Control* ctl = reinterpret_cast<volatile Control*>(bars + 2 * S + 6);
  const uint32_t stage0 = smem_u32(smem);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int rank = split > 1 ? static_cast<int>(cluster_rank()) : 0;
  int tp, tq;
  tile_of(p, blockIdx.x / split, &tp, &tq);
  const int first = static_cast<int>(static_cast<int64_t>(p.iters) * rank / split);
  const int last = static_cast<int>(static_cast<int64_t>(p.iters) * (rank + 1) / split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tmem_full(b), 1);
      mbar_init(tmem_empty(b), 4);
    }
    mbar_init(drain, 1);
    ctl->abort = 0;
    ctl->timeout_ns = p.timeout_ns;
    ctl->status = p.status;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<false>(smem_u32(s_tmem), kCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *s_tmem;
  let_next();
  after_previous();
  bool ok = true;

  if (warp == 0) {
    if (elect_one()) {
      Ring rg;
      uint32_t issued = 0;
      const bool planes = p.iters != p.k_chunks;
      int pr = planes ? first / p.k_chunks : 5, kc = planes ? first % p.k_chunks : first;
      for (int it = first; it < last; ++it, rg.next(S)) {
        if (!(ok = mbar_wait(empty(rg.s), rg.ph ^ 1u, ctl))) break;
        mbar_expect_tx(full(rg.s), kStageBytes + (kHook && blockIdx.x == 0 && it - first == p.withhold ? 16 : 0));
        load_stage<kAMn, kBMn, false>(stage0 + rg.s * kStageBytes, &amap, &bmap, full(rg.s), tp * 128, tq * BN, kc * kK,
                                      plane_a(pr), plane_b(pr), BN / 64);
        ++issued;
        if (++kc == p.k_chunks) { kc = 0; ++pr; }
      }
      if (!ok) {  // wait, bounded, for the copies in flight
        for (uint32_t k = 0; k < static_cast<uint32_t>(S) && k < issued; ++k) {
          const uint32_t j = issued - 1 - k;
          settle(full(static_cast<int>(j % S)), (j / S) & 1u, p.timeout_ns);
        }
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      Ring rg, tb;
      for (int at = first; ok && at < last; tb.next(2)) {
        if (kPieces) {
          if (!(ok = mbar_wait(tmem_empty(tb.s), tb.ph ^ 1u, ctl))) break;
          fence_after();
        }
        const int end = kPieces ? min(piece_end(p, at), last) : last;
        for (int it = at; it < end; ++it, rg.next(S)) {
          if (!(ok = mbar_wait(full(rg.s), rg.ph, ctl))) break;
          fence_after();
          issue_stage<kAMn, kBMn, false>(tmem + tb.s * BN, stage0 + rg.s * kStageBytes, p.idesc, it == at);
          mma_commit<false>(empty(rg.s));
        }
        if (ok) mma_commit<false>(tmem_full(tb.s));
        at = end;
      }
      mma_commit<false>(drain);  // also after an abort: what was issued completes
      settle(drain, 0, p.timeout_ns);
    }
  } else {
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const int64_t pp = static_cast<int64_t>(tp) * 128 + row;
    const int64_t q0 = static_cast<int64_t>(tq) * BN;
    const uint32_t d = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const int cols = static_cast<int>(min(static_cast<int64_t>(BN), p.nq - q0));
    const float bias = bias_of(p, pp);
    if constexpr (kPieces) {
      // fp32: pieces as in the pairs' kernel.
      float sum[BN];
#pragma unroll
      for (int i = 0; i < BN; ++i) sum[i] = 0.f;
      Ring tb;
      for (int at = first; ok && at < last; at = piece_end(p, at), tb.next(2)) {
        ok = mbar_wait(tmem_full(tb.s), tb.ph, ctl);
        if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
        fence_after();
#pragma unroll
        for (int c = 0; c < BN; c += 16)
          if (c < cols) {
            uint32_t v[16];
            tmem_load16(d + tb.s * BN + c, v);
            tmem_wait_load(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[c + i] += __uint_as_float(v[i]);
          }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tmem_empty(tb.s));
      }
      if (ok) {
        // Every copy has landed and every MMA has read it: the stages hold the sums now, and the registers
        // are free for the epilogue.
        float* part = reinterpret_cast<float*>(smem) + row;
        Residual<T> r;
        if (split == 1) load_residual(p, q0, pp, cols, &r);
#pragma unroll
        for (int c = 0; c < BN; c += 16)
          if (c < cols) {
#pragma unroll
            for (int i = 0; i < 16; ++i) part[(c + i) * 128] = sum[c + i];
          }
        if (split == 1) {
#pragma unroll 1
          for (int c = 0; c < cols; c += 16) {
            float z[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = part[(c + i) * 128];
            Residual<T> ahead;
            load_residual(p, q0 + c + 16, pp, cols - c - 16, &ahead);
            if (pp < p.np) finish<T>(p, z, r, q0 + c, pp, cols - c, bias);
            r = ahead;
          }
        }
      }
    } else {
      Residual<T> r;
      if (split == 1) load_residual(p, q0, pp, cols, &r);
      if (first < last) ok = mbar_wait(tmem_full(0), 0, ctl);
      ok = __all_sync(0xFFFFFFFFu, ok) && !ctl->abort;
      if (ok) {
        fence_after();
#pragma unroll 1
        for (int c = 0; c < cols; c += 16) {
          uint32_t v[16] = {};  // of a CTA without a share of k
          if (first < last) {
            tmem_load16(d + c, v);
            tmem_wait_load(v);
          }
          if (split == 1) {
            float z[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = __uint_as_float(v[i]);
            Residual<T> ahead;
            load_residual(p, q0 + c + 16, pp, cols - c - 16, &ahead);
            if (pp < p.np) finish<T>(p, z, r, q0 + c, pp, cols - c, bias);
            r = ahead;
          } else {
            // Every copy has landed and every MMA has read it: the stages hold the partial sums now.
            float* part = reinterpret_cast<float*>(smem) + row;
#pragma unroll
            for (int i = 0; i < 16; ++i) part[(c + i) * 128] = __uint_as_float(v[i]);
          }
        }
        fence_before();
      }
    }
  }
  if (split > 1) {
    __syncwarp();
    cluster_sync();
    if (warp >= 2 && !ctl->abort) {
      const int row = (warp & 3) * 32 + lane;
      const int64_t pp = static_cast<int64_t>(tp) * 128 + row;
      const int64_t q0 = static_cast<int64_t>(tq) * BN;
      const int cols = static_cast<int>(min(static_cast<int64_t>(BN), p.nq - q0));
      const int c0 = cols * rank / split, c1 = cols * (rank + 1) / split;
      const float bias = bias_of(p, pp);
      if (pp < p.np) {
        for (int c = c0; c < c1; c += 16) {
          float z[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] = 0.f;
          Residual<T> res;
          load_residual(p, q0 + c, pp, c1 - c, &res);
          for (int r = 0; r < split; ++r) {
            const uint32_t from = map_rank(stage0 + (c * 128 + row) * 4, r);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (c + i < c1) z[i] += load_cluster(from + i * 512);
          }
          finish<T>(p, z, res, q0 + c, pp, c1 - c, bias);
        }
      }
    }
    __syncwarp();
    cluster_sync();
  }
  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tmem_free<false>(tmem, kCols);
  }
}

// ---------------------------------------------------------------- host
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// [planes][rows][cols] of bf16, `pitch` elements a row; boxes of 64 x `box` rows.
bool make_map(CUtensorMap* map, const TcOperand& o, int box) {
  std::memset(map, 0, sizeof(*map));
  const PFN_cuTensorMapEncodeTiled_v12000 encode = encode_fn();
  if (encode == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(o.cols), static_cast<cuuint64_t>(o.rows),
                              static_cast<cuuint64_t>(o.planes)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(o.pitch) * 2, static_cast<cuuint64_t>(o.plane) * 2};
  const cuuint32_t boxes[3] = {64, static_cast<cuuint32_t>(box), 1};
  const cuuint32_t ones[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(o.p), dims, strides, boxes, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [nq][np] of the results' type, boxes of 128 x 16.
bool make_result_map(CUtensorMap* map, const void* p, vn_dtype dt, int64_t np, int64_t nq) {
  std::memset(map, 0, sizeof(*map));
  if (p == nullptr) return true;
  const PFN_cuTensorMapEncodeTiled_v12000 encode = encode_fn();
  if (encode == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(np), static_cast<cuuint64_t>(nq)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(np) * (dt == VN_BF16 ? 2 : 4)};
  const cuuint32_t boxes[2] = {128, 16};
  const cuuint32_t ones[2] = {1, 1};
  return encode(map, dt == VN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
                const_cast<void*>(p), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kFixed = 1024 + 8 * (2 * kMaxStages + 8 + 2 * kBuffers) + sizeof(Control);

template <typename T, bool kAMn, bool kBMn, bool kStaged, bool kHook = false>
cudaError_t run_pair_typed(const TcProduct& d, Params p, int sms, int bn, cudaStream_t stream) {
  const int pairs = sms / 2;
  p.bn = bn;
  CUtensorMap am, bm, ym, zm, rm;
  if (!make_map(&am, d.a, kAMn ? 64 : 128) || !make_map(&bm, d.b, kBMn ? 64 : p.bn / 2)) return cudaErrorInvalidValue;
  if (!make_result_map(&ym, kStaged ? d.out : nullptr, d.dt, d.np, d.nq) ||
      !make_result_map(&zm, kStaged ? d.preact : nullptr, d.dt, d.np, d.nq) ||
      !make_result_map(&rm, kStaged ? d.residual : nullptr, d.dt, d.np, d.nq))
    return cudaErrorInvalidValue;
  p.p_tiles = static_cast<int>((d.np + 255) / 256);
  p.q_tiles = static_cast<int>((d.nq + p.bn - 1) / p.bn);
  p.units = static_cast<int64_t>(p.p_tiles) * p.q_tiles;
  p.idesc = idesc_of(256, p.bn, kAMn, kBMn);
  const int grid = static_cast<int>(std::min<int64_t>(2 * p.units, 2 * pairs));
  const int chunks = kStaged ? kBuffers * (d.preact != nullptr ? 2 : 1) : 0;
  p.staging_bytes = 2 * chunks * kChunkBytes<T>;
  // As many stages as the rest of the 227 KB holds: 4 to 6 (in bf16 6, or 5 with a pre-activation). 4
  // instead of 6 cost 5 to 12 per cent.
  p.stages = std::min<int>(kMaxStages, static_cast<int>((232448 - kFixed - p.staging_bytes) / kPairStageBytes));
  static SmemRecord record;
  return launch_cluster(pair_kernel<T, kAMn, kBMn, kStaged, kHook>, record, grid, kPairThreads, 2,
                        kFixed + p.stages * kPairStageBytes + p.staging_bytes, stream, am, bm, ym, zm, rm, p);
}
template <typename T, bool kAMn, bool kBMn>
cudaError_t run_pair(const TcProduct& d, const Params& p, int sms, int bn, cudaStream_t stream) {
  auto fits = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
  const bool staged = d.np * sizeof(T) % 16 == 0 && fits(d.out) && fits(d.preact) && fits(d.residual);
  return staged ? run_pair_typed<T, kAMn, kBMn, true>(d, p, sms, bn, stream)
                : run_pair_typed<T, kAMn, kBMn, false>(d, p, sms, bn, stream);
}

template <typename T, int BN, bool kAMn, bool kBMn, bool kHook = false>
cudaError_t run_single(const TcProduct& d, Params p, int split, cudaStream_t stream) {
  constexpr uint32_t kStage = kABytes + BN * 128;
  CUtensorMap am, bm;
  if (!make_map(&am, d.a, kAMn ? 64 : 128) || !make_map(&bm, d.b, kBMn ? 64 : BN)) return cudaErrorInvalidValue;
  p.p_tiles = static_cast<int>((d.np + 127) / 128);
  p.q_tiles = static_cast<int>((d.nq + BN - 1) / BN);
  p.units = static_cast<int64_t>(p.p_tiles) * p.q_tiles;
  p.stages = static_cast<int>(std::min<uint32_t>(kMaxStages, 106496 / kStage));  // two CTAs an SM
  p.idesc = idesc_of(128, BN, kAMn, kBMn);
  if (p.units * split > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  static SmemRecord record;
  return launch_cluster(single_kernel<T, BN, kAMn, kBMn, kHook>, record, static_cast<int>(p.units * split), kThreads, split,
                        kFixed + static_cast<size_t>(p.stages) * kStage, stream, am, bm, p, split);
}

template <typename T, bool kAMn, bool kBMn>
cudaError_t run(const TcProduct& d, const TilePlan& plan, cudaStream_t stream, const Withhold* hook) {
  DeviceInfo dev;
  cudaError_t err = device_info(&dev);
  if (err != cudaSuccess) return err;
  Params p = {};
  p.bias = d.bias; p.bias_bf16 = d.bias_bf16; p.act = d.act;
  p.residual = d.residual; p.out = d.out; p.preact = d.preact;
  p.np = d.np; p.nq = d.nq;
  p.k_chunks = static_cast<int>((d.nk + kK - 1) / kK);
  p.iters = p.k_chunks * (d.a.planes == 3 ? 6 : 1);
  p.timeout_ns = kTimeoutNs;
  if ((err = device_status_word(&p.status)) != cudaSuccess) return err;
  if constexpr (!kAMn && !kBMn) {
    if (hook != nullptr) {
      p.withhold = hook->at;
      p.timeout_ns = hook->timeout_ns;
      return plan.pair ? run_pair_typed<T, false, false, true, true>(d, p, dev.sm_count, plan.bn, stream)
                       : run_single<T, 64, false, false, true>(d, p, 1 << plan.log_split, stream);
    }
  }
  if (plan.pair) return run_pair<T, kAMn, kBMn>(d, p, dev.sm_count, plan.bn, stream);
  const int split = 1 << plan.log_split;
  if constexpr (!kBMn) {
    if (plan.bn == 16) return run_single<T, 16, kAMn, kBMn>(d, p, split, stream);
  }
  if (plan.bn == 64) return run_single<T, 64, kAMn, kBMn>(d, p, split, stream);
  return run_single<T, 128, kAMn, kBMn>(d, p, split, stream);
}

template <typename T>
cudaError_t run_layout(const TcProduct& d, const TilePlan& plan, cudaStream_t stream, const Withhold* hook) {
  if (!d.a.mn) return run<T, false, false>(d, plan, stream, hook);
  return d.b.mn ? run<T, true, true>(d, plan, stream, hook) : run<T, true, false>(d, plan, stream, hook);
}

}  // namespace

cudaError_t launch_tc_product(const TcProduct& d, const TilePlan& plan, cudaStream_t stream, const Withhold* hook) {
  return d.dt == VN_BF16 ? run_layout<__nv_bfloat16>(d, plan, stream, hook) : run_layout<float>(d, plan, stream, hook);
}

}  // namespace vn
