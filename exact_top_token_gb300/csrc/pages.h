// pages.h -- what the operators of a cache in pages share (internal).
#pragma once

#include <cuda_runtime.h>

#include "hytopk.h"

namespace hytopk {
namespace pages {

// Rows of a page. Whole groups of 16 rows, so that 16 neighbouring keys have one scale.
inline bool page_rows_ok(int P) { return P == 16 || P == 32 || P == 64 || P == 128 || P == 256; }

// Host checks of the sequences of a call (the numbers on the device are the kernels').
inline hytopk_status check_paged(const hytopk_paged* s, int n) {
  if (!s || s->B < 0 || s->columns < 1 || s->N < 1 || n < 0) return HYTOPK_INVALID_ARG;
  if (!s->cu_q && n != s->B) return HYTOPK_INVALID_ARG;
  if (!page_rows_ok(s->P) || (int64_t)s->columns * s->P >= (int64_t)1 << 31)
    return HYTOPK_UNSUPPORTED;
  if (s->B > 0 && (!s->table || !s->lengths)) return HYTOPK_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(s->table), static_cast<const void*>(s->lengths),
                        static_cast<const void*>(s->cu_q)})
    if (reinterpret_cast<uintptr_t>(p) & 3) return HYTOPK_MISALIGNED;
  return HYTOPK_OK;
}

#ifdef __CUDACC__
// Sequence b as a call sees it: rows [row0, row0 + m) at the end of a context of `length`.
struct Seq {
  int row0, m, length;
  bool bad;  // brought back into the range
};
__device__ __forceinline__ Seq seq_of(const hytopk_paged& s, int n, int b) {
  Seq q{};
  int lo = b, hi = b + 1;
  if (s.cu_q) {
    lo = s.cu_q[b];
    hi = s.cu_q[b + 1];
  }
  const int most = s.columns * s.P, length = s.lengths[b];
  q.row0 = min(max(lo, 0), n);
  q.m = max(min(max(hi, 0), n) - q.row0, 0);
  q.length = min(max(length, 0), most);
  q.bad = lo < 0 || hi < lo || hi > n || q.length != length;
  return q;
}
#endif

}  // namespace pages
}  // namespace hytopk
