// vn_launch.cuh -- launches that overlap the end of the kernel before them on their stream.
//
// A kernel launched here may start while its predecessor still runs: it sets itself up, and
// after_previous() then holds it until every kernel before it on the stream is complete and its
// writes are visible. Every thread that reads or writes memory calls it first. let_next() allows the
// successor to start likewise, once every CTA has called it or ended; a kernel that allocates tensor
// memory calls it after the allocation (a successor that took the columns first would wait for this
// kernel, and this kernel for the columns). Kernels launched in the plain way, before or after, see
// nothing of it. Calls one after the other on a stream, with and without: a linear of 1024 x 256 to 256
// in fp32 9.4 us for 12.3, one row of 4096 to 4096 in bf16 8.0 for 9.6, layer norm's gradients of
// 4099 x 1021 17.4 for 22.5, AdamW over a small policy's tensors 3.1 for 4.1, a linear of 8192 x 4096
// to 4096 200 for 201.
#pragma once

#include <cuda_runtime.h>

#include "vn_smem.h"

namespace vn {

__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A line on its way to L2, which may be asked for before after_previous(): it is no read.
__device__ __forceinline__ void prefetch(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// A load of what a kernel before this one may have written: never through the read-only path, whose
// data has to stay as it is from the launch on (so none of these kernels' pointers is __restrict__
// either).
template <typename T>
__device__ __forceinline__ T fetch(const T* p) { return *p; }

template <typename... KArgs, typename... Args>
cudaError_t launch_overlapped(void (*fn)(KArgs...), dim3 grid, int threads, int cluster, size_t smem, cudaStream_t stream,
                              Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fn, static_cast<KArgs>(args)...);
}

// Lets `fn` run in clusters of more than the portable 8 CTAs on the current device (once a device: done).
inline cudaError_t allow_wide_clusters(const void* fn, SmemRecord& done) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (done[dev].load(std::memory_order_acquire) != 0) return cudaSuccess;
  err = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (err == cudaSuccess) done[dev].store(1, std::memory_order_release);
  return err;
}

}  // namespace vn
