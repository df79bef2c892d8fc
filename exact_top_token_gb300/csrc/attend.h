// attend.h -- arguments of the attention over selected rows (internal).
#pragma once

#include "common.cuh"

namespace hytopk {
namespace att {

struct Args {
  const void* q;       // [n, Hq, d] bf16
  int64_t q_row;       // elements between queries
  const void* k;       // [L, Hkv, d]
  const void* v;
  int64_t k_row, v_row;
  const float* k_scale;  // e4m3: [L, Hkv]
  const float* v_scale;
  const int32_t* idx;  // [n, k_top]
  int n, L, Hkv, G, d, k_top;
  float scale;
  void* out;           // [n, Hq, d] bf16 or fp32
  float* lse;          // [n, Hq] (forward: or NULL)
  uint32_t* status;
  // backward
  const void* grad;    // [n, Hq, d] bf16
  float* dq;
  float* dk;
  float* dv;
  int zero;            // dk and dv are set to zero first
};

// attend.cu: zeros to x and y (nx floats each) and z (nz), whole and aligned float4s
cudaError_t launch_zero(float* x, float* y, size_t nx, float* z, size_t nz, int sms,
                        cudaStream_t st);

// Opt in to `bytes` of dynamic shared memory, once per kernel and device: the call
// takes longer than a launch, and single-token calls are bound by the host. `done` is the
// kernel's own.
inline cudaError_t opt_in(const void* kernel, int bytes, int dev, unsigned long long* done,
                          bool anew) {
  const unsigned long long bit = 1ull << (dev & 63);
  if (!anew && dev < 64 && (__atomic_load_n(done, __ATOMIC_RELAXED) & bit)) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) __atomic_fetch_or(done, bit, __ATOMIC_RELAXED);
  return e;
}

// A launch after that. A context that was reset forgets it: a launch that fails is tried
// again after setting it anew.
template <class Launch>
cudaError_t launch_opted_in(const void* kernel, int bytes, unsigned long long* done,
                            Launch&& launch) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  for (int attempt = 0; e == cudaSuccess && attempt < 2; ++attempt) {
    e = opt_in(kernel, bytes, dev, done, attempt > 0);
    if (e != cudaSuccess) break;
    e = launch();
    if (e != cudaErrorInvalidValue || attempt) break;
    cudaGetLastError();  // of the refused launch
    e = cudaSuccess;
  }
  return e;
}

// Clusters of `size` (2, 4 or 8) CTAs that the device runs at once, asked for once per
// kernel, device and size; 0 if it cannot be told.
inline int clusters_at_once(const void* kernel, int threads, int bytes, int size,
                            unsigned long long* done, int (*known)[4]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  int* at = &known[dev & 63][size == 2 ? 0 : size == 4 ? 1 : 2];
  const int have = dev < 64 ? __atomic_load_n(at, __ATOMIC_RELAXED) : 0;
  if (have) return have - 1;
  int n = 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)size);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = bytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (opt_in(kernel, bytes, dev, done, false) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  __atomic_store_n(at, n + 1, __ATOMIC_RELAXED);
  return n;
}

}  // namespace att
}  // namespace hytopk
