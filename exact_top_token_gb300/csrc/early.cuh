// early.cuh -- launches that begin while the stream's kernel before still runs.
//
// A short kernel's time is mostly its launch and set-up. A kernel launched with
// launch_early may be brought onto the multiprocessors once every CTA of the kernel
// before it has called allow_next (or ended); it calls wait_for_earlier before its first
// access to global memory, which returns when everything launched before is complete
// and visible. So only set-up overlaps (barriers, tensor memory, index arithmetic), and
// results are those of a plain stream. After anything but such a kernel, it is a plain
// launch. Calls in a row, plain -> early: a write of a few rows 4.1 -> 2.4 us (the host's
// time), attention of a single token over 2048 rows 14.3 -> 11.1, of a small batch with
// its gradients 29.7 -> 24.6.
#pragma once

#include <cuda_runtime.h>

namespace hytopk {

__device__ __forceinline__ void wait_for_earlier() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void allow_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// A load of what an earlier kernel may have written. The read-only path (__ldg, ld.global.nc)
// is for data that nobody writes while the kernel lives, and a kernel launched early
// lives while the one before it still writes: its lines are not kept coherent, and one that
// a kernel two launches back read would do as well as the new one.
template <typename T>
__device__ __forceinline__ T ld_after(const T* p) {
  return *p;
}

// cluster: CTAs of a cluster (1: none)
template <class... P>
cudaError_t launch_early(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem,
                         cudaStream_t st, unsigned cluster, const P&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace hytopk
