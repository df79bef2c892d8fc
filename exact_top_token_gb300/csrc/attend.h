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
};

// Opt in to `bytes` of dynamic shared memory, once per kernel and device: the call
// takes longer than a launch, and single-token calls are bound by the host. `done` is the
// kernel's own. A context that was reset forgets it: a launch that fails is
// tried again after setting it anew.
template <class Launch>
cudaError_t launch_opted_in(const void* kernel, int bytes, unsigned long long* done,
                            Launch&& launch) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  for (int attempt = 0; attempt < 2; ++attempt) {
    if (attempt || !(__atomic_load_n(done, __ATOMIC_RELAXED) & bit) || dev > 63) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
      if (e != cudaSuccess) return e;
      __atomic_fetch_or(done, bit, __ATOMIC_RELAXED);
      attempt = 1;
    }
    e = launch();
    if (e != cudaErrorInvalidValue || attempt) break;
    cudaGetLastError();  // of the refused launch
  }
  return e;
}

}  // namespace att
}  // namespace hytopk
