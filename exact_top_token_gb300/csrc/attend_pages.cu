// attend_pages.cu -- attention over a cache in pages (hytopk_attend_pages).
#include <cuda_bf16.h>

#include "early.cuh"
#include "launch.h"
#include "pages.h"

namespace hytopk {
namespace pages {
namespace {

struct AttendArgs {
  const __nv_bfloat16* q;
  int64_t q_row;
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  hytopk_paged s;
  int n, Hkv, G;
  float scale;
  __nv_bfloat16* out;
  float* lse;
  uint32_t* status;
};

__device__ __forceinline__ float2 two_of(uint16_t codes) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h2));
}

// A warp a (row, head), the running maximum and sum in every lane.
template <int D>
__global__ void __launch_bounds__(128) k_attend_pages(const AttendArgs a) {
  allow_next();
  wait_for_earlier();
  constexpr int E = D / 32;  // columns of a lane
  const int lane = threadIdx.x & 31, Hq = a.Hkv * a.G;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (item >= (int64_t)a.n * Hq) return;
  const int t = (int)(item / Hq), h = (int)(item % Hq), hk = h / a.G;
  int b = 0;
  Seq s{};
  for (; b < a.s.B; ++b) {
    s = seq_of(a.s, a.n, b);
    if (s.bad && lane == 0 && a.status) atomicOr(a.status, HYTOPK_DEV_BAD_POSITION);
    if (t >= s.row0 && t < s.row0 + s.m) break;
  }
  if (b == a.s.B) return;
  const int last = s.length - s.m + (t - s.row0), P = a.s.P;
  float q[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(a.q[(size_t)t * a.q_row + (size_t)h * D + lane * E + e]) * 0x1p-40f;
    o[e] = 0.0f;
  }
  for (int j = 0; j <= last; ++j) {
    const int page = a.s.table[(size_t)b * a.s.columns + j / P];
    if (page < 0 || page >= a.s.N) {
      if (page != -1 && lane == 0 && a.status) atomicOr(a.status, HYTOPK_DEV_BAD_INDEX);
      continue;
    }
    float ks = a.k_scale[(size_t)page * a.Hkv + hk], vs = a.v_scale[(size_t)page * a.Hkv + hk];
    if (!(ks > 0.0f && ks < INFINITY) || !(vs > 0.0f && vs < INFINITY)) {
      ks = vs = __int_as_float(0x7fc00000);
      if (lane == 0 && a.status) atomicOr(a.status, HYTOPK_DEV_BAD_SCALE);
    }
    const size_t at = (((size_t)page * P + j % P) * a.Hkv + hk) * D + lane * E;
    float x = 0.0f, v[E];
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 k2 = two_of(*reinterpret_cast<const uint16_t*>(a.k + at + e));
      const float2 v2 = two_of(*reinterpret_cast<const uint16_t*>(a.v + at + e));
      x += q[e] * k2.x + q[e + 1] * k2.y;
      v[e] = v2.x;
      v[e + 1] = v2.y;
    }
    for (int i = 16; i; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
    x *= a.scale * ks * 0x1p40f;
    if (x == -INFINITY) continue;
    const float top = fmaxf(m, x), f = m == -INFINITY ? 0.0f : expf(m - top), p = expf(x - top);
    m = top;
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * vs * v[e];
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    a.out[((size_t)t * Hq + h) * D + lane * E + e] =
        __float2bfloat16_rn(l == 0.0f ? 0.0f : o[e] / l);
  if (a.lse && lane == 0) a.lse[(size_t)t * Hq + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace pages
}  // namespace hytopk

using namespace hytopk;
using namespace hytopk::pages;

extern "C" size_t hytopk_attend_pages_workspace_size(int Hq, int Hkv, int d) {
  if (Hkv < 1 || Hq < Hkv || Hq % Hkv || Hq / Hkv > 128 || (d != 64 && d != 128)) return 0;
  return 256;
}

extern "C" hytopk_status hytopk_attend_pages(const void* q, int64_t q_row, const void* k_pages,
                                             const float* k_scale, const void* v_pages,
                                             const float* v_scale, const hytopk_paged* paged,
                                             int n, int Hq, int Hkv, int d, float scale, void* out,
                                             float* lse, void* workspace, size_t workspace_bytes,
                                             uint32_t* dev_status, cudaStream_t stream) {
  const hytopk_status s = check_paged(paged, n);
  if (s != HYTOPK_OK) return s;
  if (Hkv < 1 || Hq < 1 || Hq % Hkv) return HYTOPK_INVALID_ARG;
  if (Hq / Hkv > 128 || (d != 64 && d != 128) || (int64_t)n * Hq >= (int64_t)1 << 31)
    return HYTOPK_UNSUPPORTED;
  if (n == 0 || paged->B == 0) return HYTOPK_OK;
  if (!q || !k_pages || !v_pages || !k_scale || !v_scale || !out || !workspace)
    return HYTOPK_INVALID_ARG;
  if (workspace_bytes < hytopk_attend_pages_workspace_size(Hq, Hkv, d))
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
  const unsigned grid = (unsigned)(((int64_t)n * Hq + 3) / 4);
  const cudaError_t e = launch_early(d == 64 ? k_attend_pages<64> : k_attend_pages<128>, grid, 128,
                                     0, stream, 1, a);
  return e == cudaSuccess ? HYTOPK_OK : HYTOPK_CUDA_ERROR;
}
