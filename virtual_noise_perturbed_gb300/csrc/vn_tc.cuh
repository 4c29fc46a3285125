// vn_tc.cuh -- what the tensor-core kernels of the centre network share: the PTX they issue,
// bounded barrier waits, operand descriptors, the epilogue's types and cluster launches.
//
// Everything here has internal linkage.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "vn_act.cuh"
#include "vn_internal.h"
#include "vn_launch.cuh"

namespace vn {
namespace {

constexpr int kK = 64;                          // k of a stage: 128 bytes of bf16, one swizzle atom
constexpr uint32_t kABytes = 128 * 128;         // 128 rows (or 64 k x 2 blocks of 64 p)
constexpr uint32_t kBlockBytes = kK * 128;      // one 64-wide block of a p- or q-contiguous operand
constexpr unsigned long long kTimeoutNs = 4000000000ull;

struct Control {
  int abort;
  int pad;
  unsigned long long timeout_ns;
  unsigned int* status;  // the device's status word, which a wait that ran out sets
};

// ---------------------------------------------------------------- PTX
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The shared::cluster address of `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float load_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 load_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Whether the phase of this parity is complete, without waiting.
__device__ __forceinline__ bool mbar_done(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait for the phase of this parity: false when it ran out (status and abort flag are
// then set) or when another role of the CTA has aborted.
__device__ __noinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, volatile Control* c) {
  const uint64_t t0 = global_ns();
  const unsigned long long limit = c->timeout_ns;
  for (uint32_t n = 1;; ++n) {
    if (mbar_try(bar, parity)) return true;
    if ((n & 63) == 0) {
      if (c->abort) return false;
      if (global_ns() - t0 > limit) {
        atomicOr(c->status, 1u);
        c->abort = 1;
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile Control* c) {
  return mbar_try(bar, parity) || mbar_wait_slow(bar, parity, c);
}
// A wait for what is in flight before the CTA ends, aborted or not: bounded by `ns` alone.
__device__ __forceinline__ void settle(uint32_t bar, uint32_t parity, unsigned long long ns) {
  const uint64_t t0 = global_ns();
  while (!mbar_try(bar, parity) && global_ns() - t0 < ns) {
  }
}
template <bool kPair>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("barrier.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// The same, and whether `value` held in all of the threads.
__device__ __forceinline__ bool named_barrier_and(int id, int threads, bool value) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "barrier.red.and.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(value))
      : "memory");
  return all != 0;
}
template <bool kPair>
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t cols) {
  if constexpr (kPair) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}
template <bool kPair>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  if constexpr (kPair)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// One thread of a converged warp, as an election: after a comparison of lane numbers the compiler does
// not know that a single thread is left, and every operand of an MMA or a copy (they are uniform
// registers) costs a vote over the lanes. 8192 x 4096 to 4096 in bf16 161 us for 171, 1024 cubed
// 8.2 for 10.5. The warp's number by warp_index() is uniform for the same reason.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0); }
template <bool kPair>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on the barrier (of both CTAs of a pair) once every MMA issued so far is complete.
template <bool kPair>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  if constexpr (kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// 32 lanes x 16 consecutive columns: thread t gets lane base + t.
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Waits for the loads so far; v, the last one's registers, pass through it, so that no use of them can
// be moved ahead.
__device__ __forceinline__ void tmem_wait_load(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}

// Shared-memory descriptor of a 128-byte-swizzled operand. k contiguous: rows of 128 bytes,
// 8-row groups 1024 bytes apart; the leading offset is unused. p (q) contiguous: a
// 64-wide block holds one 128-byte row per k, 8-k groups 1024 bytes apart (stride), and
// the next 64 elements start kBlockBytes on (leading).
template <bool kMn>
__device__ __forceinline__ uint64_t descriptor(uint32_t addr) {
  uint64_t d = static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(kMn ? kBlockBytes >> 4 : 1) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
// An operand `bytes` further on (a multiple of 16): one addition, since no address carries out of
// the descriptor's field. MMAs are issued by one thread, which building each descriptor
// anew kept busy for longer than the MMAs take (3,100 cycles for the 24 of an fp32 chunk).
__device__ __forceinline__ uint64_t further(uint64_t descriptor, uint32_t bytes) { return descriptor + (bytes >> 4); }
// Bytes from one MMA's 16 k to the next within a stage.
template <bool kMn>
constexpr uint32_t kStepBytes = kMn ? 16 * 128 : 32;

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// The planes of A and B in the i-th of the six products: (2,0) (0,2) (1,1) (1,0) (0,1) (0,0).
__device__ __forceinline__ constexpr int plane_a(int i) { return (0b000001010010 >> (2 * i)) & 3; }
__device__ __forceinline__ constexpr int plane_b(int i) { return (0b000100011000 >> (2 * i)) & 3; }

struct Ring {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int n) {
    if (++s == n) { s = 0; ph ^= 1u; }
  }
};

// What is done to a product's sums: out = act(sum + bias) + residual, preact before act.
struct Epilogue {
  const void* bias;      // [np] or NULL
  const void* residual;  // [nq, np] or NULL
  void* out;             // [nq, np]
  void* preact;          // [nq, np] or NULL
  int64_t np;
  int bias_bf16, act;
};

// N outputs of one p, columns q .. q + N - 1 (the first `count` of them), in two steps: the
// residual's loads, which the caller issues ahead of the sums, and the rest of the epilogue.
template <typename T, int N = 16>
struct Residual {
  T v[N];
};
template <typename T, int N>
__device__ __forceinline__ void load_residual(const Epilogue& p, int64_t q, int64_t pp, int count, Residual<T, N>* r) {
  if (p.residual == nullptr || pp >= p.np) return;
  const T* at = static_cast<const T*>(p.residual) + q * p.np + pp;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < count) r->v[i] = at[i * p.np];
}
template <typename T, int N>
__device__ __forceinline__ void finish(const Epilogue& p, float (&z)[N], const Residual<T, N>& r, int64_t q, int64_t pp,
                                       int count, float bias) {
  const int64_t at = q * p.np + pp;
#pragma unroll
  for (int i = 0; i < N; ++i) z[i] += bias;
  if (p.preact != nullptr) {
    T* pre = static_cast<T*>(p.preact) + at;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < count) pre[i * p.np] = narrow<T>(z[i]);
  }
  activate_all<sizeof(T) == 2>(p.act, z);
  if (p.residual != nullptr) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] += value(r.v[i]);
  }
  T* out = static_cast<T*>(p.out) + at;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < count) out[i * p.np] = narrow<T>(z[i]);
}
__device__ __forceinline__ float bias_of(const Epilogue& p, int64_t pp) {
  if (p.bias == nullptr || pp >= p.np) return 0.f;
  return p.bias_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[pp])
                     : static_cast<const float*>(p.bias)[pp];
}


// ---------------------------------------------------------------- host
__host__ __device__ __forceinline__ uint32_t idesc_of(int m, int n, bool a_mn, bool b_mn) {
  // fp32 accumulator, bf16 operands, transpose bits, N / 8, M / 16
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*fn)(KArgs...), SmemRecord& record, int grid, int threads, int cluster, size_t smem,
                           cudaStream_t stream, Args... args) {
  const cudaError_t err = ensure_dynamic_smem(reinterpret_cast<const void*>(fn), smem, record);
  if (err != cudaSuccess) return err;
  return launch_overlapped(fn, dim3(static_cast<unsigned>(grid)), threads, cluster, smem, stream, args...);
}

}  // namespace
}  // namespace vn
