// attend_pages.cu -- hytopk_attend_pages: host checks and dispatch; instances in
// attend_pages_d*.cu.
#include <cmath>
#include <numeric>

#include "attend_pages.h"
#include "launch.h"

namespace hytopk {
namespace pages {

// attend_pages_d*.cu
cudaError_t launch_attend_pages_d64(const AttendArgs& a, int ctas, cudaStream_t st);
cudaError_t launch_attend_pages_d128(const AttendArgs& a, int ctas, cudaStream_t st);
// attend_pages_t*.cu: one row of a sequence, at most kTokenHeads heads on a cache head
cudaError_t launch_attend_tokens_d64(const AttendArgs& a, int ctas, bool join, cudaStream_t st);
cudaError_t launch_attend_tokens_d128(const AttendArgs& a, int ctas, bool join, cudaStream_t st);

constexpr int kTokenHeads = 16;
// The kernel of single rows is taken where at most that many heads share a cache head, no more
// rows are given than there are sequences, and contexts may be as long as kTokenTiles tiles of
// 128 keys a multiprocessor: 64 rows over up to 16384 keys, 8 cache heads of 128 columns, take
// 167 us with it and 221 with the general one, over 256 keys each (7 tiles) 29 and 37. A cu_q
// may hold several rows of a sequence all the same, so with one both are launched and the
// second mostly ends at once, which takes 2 to 3 us: 16 rows over 100 keys (0.8 tiles) 17 us
// either way, 32 (1.7 tiles) 19 and 23, one row over 500 keys 17 and 16. Without a cu_q the
// kernel of single rows is ahead at any size (that row 14 and 16, 64 over 100 keys, 3.4 tiles,
// 24 and 36), so that the rule, one for both, is cautious.
constexpr int kTokenTiles = 4;

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Rows of a part in the workspace: of one block, unless some item may have more tokens.
int part_rows(int n, int G) { return n > 128 / G ? 256 : 128; }

size_t part_bytes(int rows, int d) { return (size_t)2 * kMaxCtas * rows * d * sizeof(float); }
constexpr size_t kRecordBytes = 2 * kMaxCtas * sizeof(int4);
size_t ml_bytes(int rows) { return (size_t)2 * kMaxCtas * rows * sizeof(float2); }

}  // namespace
}  // namespace pages
}  // namespace hytopk

using namespace hytopk;
using namespace hytopk::pages;

extern "C" size_t hytopk_attend_pages_workspace_size(int n, int Hq, int Hkv, int d) {
  if (n < 0 || Hkv < 1 || Hq < Hkv || Hq % Hkv || Hq / Hkv > 128 || (d != 64 && d != 128)) return 0;
  const int rows = part_rows(n, Hq / Hkv);
  return part_bytes(rows, d) + ml_bytes(rows) + kRecordBytes + 256;
}

extern "C" hytopk_status hytopk_attend_pages(const void* q, int64_t q_row, const void* k_pages,
                                             const float* k_scale, const void* v_pages,
                                             const float* v_scale, const hytopk_paged* paged,
                                             int n, int Hq, int Hkv, int d, float scale, void* out,
                                             float* lse, void* workspace, size_t workspace_bytes,
                                             uint32_t* dev_status, cudaStream_t stream) {
  const hytopk_status s = check_paged(paged, n);
  if (s != HYTOPK_OK) return s;
  if (Hkv < 1 || Hq < 1 || Hq % Hkv || !std::isfinite(scale)) return HYTOPK_INVALID_ARG;
  if (Hq / Hkv > 128 || (d != 64 && d != 128) || (int64_t)n * Hq >= (int64_t)1 << 31)
    return HYTOPK_UNSUPPORTED;
  // rows of a pool are numbered in 32 bits, one past the last included
  if ((int64_t)paged->N * paged->P >= ((int64_t)1 << 31) - 16) return HYTOPK_UNSUPPORTED;
  if (n == 0 || paged->B == 0) return HYTOPK_OK;
  if (!q || !k_pages || !v_pages || !k_scale || !v_scale || !out || !workspace)
    return HYTOPK_INVALID_ARG;
  if (workspace_bytes < hytopk_attend_pages_workspace_size(n, Hq, Hkv, d))
    return HYTOPK_WORKSPACE_TOO_SMALL;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(lse, 4) ||
      !aligned(workspace, 256) || q_row % 8)
    return HYTOPK_MISALIGNED;
  AttendArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_row = q_row;
  a.k = static_cast<const uint8_t*>(k_pages);
  a.v = static_cast<const uint8_t*>(v_pages);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.s = *paged;
  a.n = n;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.scale = scale;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.status = dev_status;
  a.tokens = 128 / a.G;
  a.shift = __builtin_ctz((unsigned)paged->P);
  a.box = paged->P < 128 ? paged->P : 128;
  a.rows = part_rows(n, a.G);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.part = reinterpret_cast<float*>(ws);
  a.ml = reinterpret_cast<float2*>(ws + part_bytes(a.rows, d));
  a.record = reinterpret_cast<int4*>(ws + part_bytes(a.rows, d) + ml_bytes(a.rows));
  const int sms = num_sms(), ctas = sms < kMaxCtas ? sms : kMaxCtas;
  a.groups = std::gcd(Hkv, ctas);
  cudaError_t e;
  const int64_t tiles = ((int64_t)paged->columns * paged->P + 127) / 128 * paged->B * Hkv;
  const bool tokens = n <= paged->B && a.G <= kTokenHeads && tiles >= (int64_t)kTokenTiles * ctas;
  if (tokens && paged->cu_q)
    a.several = reinterpret_cast<int*>(ws + part_bytes(a.rows, d) + ml_bytes(a.rows) + kRecordBytes);
  e = cudaSuccess;
  if (tokens)
    e = d == 64 ? launch_attend_tokens_d64(a, ctas, !a.several, stream)
                : launch_attend_tokens_d128(a, ctas, !a.several, stream);
  if (e == cudaSuccess && (!tokens || a.several))
    e = d == 64 ? launch_attend_pages_d64(a, ctas, stream) : launch_attend_pages_d128(a, ctas, stream);
  return e == cudaSuccess ? HYTOPK_OK : HYTOPK_CUDA_ERROR;
}
