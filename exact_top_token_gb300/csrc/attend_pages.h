// attend_pages.h -- arguments of the attention over a cache in pages (internal).
#pragma once

#include <cuda_bf16.h>

#include "pages.h"

namespace hytopk {
namespace pages {

constexpr int kMaxCtas = 160;  // shares of a call's work

struct AttendArgs {
  const __nv_bfloat16* q;
  int64_t q_row;
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  hytopk_paged s;
  int n, Hkv, G;
  int tokens;  // of a block of 128 rows: 128 / G
  int shift;   // log2 of a page's rows
  int box;     // rows that a page and a tile of 128 share
  float scale;
  __nv_bfloat16* out;
  float* lse;
  uint32_t* status;
  float* part;   // [2 * ctas][rows][d] results, each divided by its own sum
  float2* ml;    // [2 * ctas][rows] sums and -m of them
  int4* record;  // [ctas][2]: what each is a part of
  int rows;      // of a part
  // both kernels are launched: the first tells here whether some sequence has several rows, which
  // are the second's; NULL: one alone
  int* several;
  int groups;    // of CTAs, by cache heads: divides Hkv and the number of CTAs
};

}  // namespace pages
}  // namespace hytopk
