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

}  // namespace att
}  // namespace hytopk
