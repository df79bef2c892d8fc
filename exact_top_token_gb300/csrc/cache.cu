// cache.cu -- rotary positions (hytopk_rope) and cache rows: quantised as they
// are written, with the rotation fused in (hytopk_cache_write), and read back
// (hytopk_cache_read). All three move each row once and are bound by memory.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "launch.h"
#include "rope.cuh"

namespace hytopk {
namespace {

struct RowArgs {
  const void* x;
  int64_t x_row, x_head;
  void* out;
  int64_t out_row, out_head;
  float* scale;  // e4m3 output: [L, H]
  const int32_t* slots;
  const int32_t* positions;
  const float* inv_freq;
  int n, H, d, L;
  int rot, first, interleaved, inverse;
  float mscale;
  uint32_t* status;
};

__device__ __forceinline__ float load_elem(const float* p) { return *p; }
__device__ __forceinline__ float load_elem(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// One (row, head) per warp: values in shared memory, then rotated, then stored.
constexpr int kWarps = 4;

template <typename T>
__device__ __forceinline__ void load_rotated(const RowArgs& a, int t, int h, float* row, int lane) {
  const T* x = static_cast<const T*>(a.x) + (size_t)t * a.x_row + (size_t)h * a.x_head;
  for (int j = lane; j < a.d; j += 32) row[j] = load_elem(x + j);
  __syncwarp();
  if (!a.positions) return;
  const int pos = a.positions[t];
  const bool bad = pos < 0 || pos >= kMaxPosition;
  if (bad && lane == 0 && a.status) atomicOr(a.status, HYTOPK_DEV_BAD_POSITION);
  for (int i = lane; i < a.rot / 2; i += 32) {
    const int j1 = a.first + (a.interleaved ? 2 * i : i);
    const int j2 = a.interleaved ? j1 + 1 : j1 + a.rot / 2;
    float c, s;
    rope_turn((float)pos, a.inv_freq[i], c, s);
    c *= a.mscale;
    s *= a.inverse ? -a.mscale : a.mscale;
    if (bad) c = s = __int_as_float(0x7fc00000);
    const float x1 = row[j1], x2 = row[j2];
    row[j1] = x1 * c - x2 * s;
    row[j2] = x1 * s + x2 * c;
  }
  __syncwarp();
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) k_rope(const RowArgs a) {
  extern __shared__ float rows[];
  const int lane = threadIdx.x & 31;
  float* row = rows + (threadIdx.x >> 5) * a.d;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (item >= (int64_t)a.n * a.H) return;
  const int t = (int)(item / a.H), h = (int)(item % a.H);
  load_rotated<T>(a, t, h, row, lane);
  T* y = static_cast<T*>(a.out) + (size_t)t * a.out_row + (size_t)h * a.out_head;
  for (int j = lane; j < a.d; j += 32) y[j] = (T)row[j];
}

template <typename T, bool E4M3>
__global__ void __launch_bounds__(32 * kWarps) k_cache_write(const RowArgs a) {
  extern __shared__ float rows[];
  const int lane = threadIdx.x & 31;
  float* row = rows + (threadIdx.x >> 5) * a.d;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (item >= (int64_t)a.n * a.H) return;
  const int t = (int)(item / a.H), h = (int)(item % a.H);
  const int slot = a.slots ? a.slots[t] : t;
  if (slot < 0 || slot >= a.L) {
    if (slot != -1 && lane == 0 && a.status) atomicOr(a.status, HYTOPK_DEV_BAD_INDEX);
    return;
  }
  load_rotated<T>(a, t, h, row, lane);
  const size_t at = ((size_t)slot * a.H + h) * a.d;
  if constexpr (!E4M3) {
    for (int j = lane; j < a.d; j += 32)
      static_cast<__nv_bfloat16*>(a.out)[at + j] = __float2bfloat16_rn(row[j]);
  } else {
    float amax = 0.0f;
    bool bad = false;
    for (int j = lane; j < a.d; j += 32) {
      const float v = fabsf(row[j]);
      if (v <= 3.402823466e38f) amax = fmaxf(amax, v);
      else bad = true;
    }
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (bad && a.status) atomicOr(a.status, HYTOPK_DEV_NONFINITE);
    const float scale = amax > 0.0f ? fmaxf(__fdiv_rn(amax, 448.0f), 1.17549435e-38f) : 1.0f;
    for (int j = lane; j < a.d; j += 32) {
      const float v = __fdiv_rn(row[j], scale);
      uint8_t code = __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
      if (!(fabsf(row[j]) <= 3.402823466e38f)) code = 0x7F;
      static_cast<uint8_t*>(a.out)[at + j] = code;
    }
    if (lane == 0) a.scale[(size_t)slot * a.H + h] = scale;
  }
}

struct ReadArgs {
  const void* cache;
  const float* scale;
  const int32_t* slots;
  void* out;
  int n, H, d, L;
  uint32_t* status;
};

template <bool E4M3, typename T>
__global__ void __launch_bounds__(32 * kWarps) k_cache_read(const ReadArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (item >= (int64_t)a.n * a.H) return;
  const int t = (int)(item / a.H), h = (int)(item % a.H);
  const int slot = a.slots ? a.slots[t] : t;
  const bool in = slot >= 0 && slot < a.L;
  if (!in && slot != -1 && lane == 0 && a.status) atomicOr(a.status, HYTOPK_DEV_BAD_INDEX);
  const size_t at = in ? ((size_t)slot * a.H + h) * a.d : 0;
  const float scale = (E4M3 && in) ? a.scale[(size_t)slot * a.H + h] : 1.0f;
  T* y = static_cast<T*>(a.out) + (size_t)item * a.d;
  for (int j = lane; j < a.d; j += 32) {
    float v = slot == -1 ? 0.0f : __int_as_float(0x7fc00000);
    if (in) {
      if constexpr (E4M3) {
        const __half_raw r =
            __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(a.cache)[at + j], __NV_E4M3);
        v = __half2float(__half(r)) * scale;
      } else {
        v = __bfloat162float(static_cast<const __nv_bfloat16*>(a.cache)[at + j]);
      }
    }
    y[j] = (T)v;
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
int elem_bytes(hytopk_elem e) { return e == HYTOPK_ELEM_F32 ? 4 : (e == HYTOPK_ELEM_BF16 ? 2 : 1); }
bool stride_ok(int64_t s, hytopk_elem e) { return (s * elem_bytes(e)) % 16 == 0; }

// Shape, type and alignment checks that hytopk_rope and hytopk_cache_write share.
hytopk_status check_rows(const void* x, int64_t x_row, int64_t x_head, hytopk_elem type, int n,
                         int H, int d, const hytopk_rope_params* r) {
  if (n < 0 || H < 1) return HYTOPK_INVALID_ARG;
  if (type != HYTOPK_ELEM_BF16 && type != HYTOPK_ELEM_F32) return HYTOPK_INVALID_ARG;
  if (d < 8 || d > 1024 || d % 8) return HYTOPK_UNSUPPORTED;
  if (r) {
    if (r->rot < 2 || r->first < 0 || (int64_t)r->first + r->rot > d) return HYTOPK_INVALID_ARG;
    if (r->rot % 16 || r->first % 8) return HYTOPK_UNSUPPORTED;
  }
  if ((int64_t)n * H >= (int64_t)1 << 31) return HYTOPK_UNSUPPORTED;
  if (n == 0) return HYTOPK_OK;
  if (!x || (r && (!r->positions || !r->inv_freq))) return HYTOPK_INVALID_ARG;
  if (!aligned16(x) || !stride_ok(x_row, type) || !stride_ok(x_head, type))
    return HYTOPK_MISALIGNED;
  if (r && (!aligned4(r->positions) || !aligned4(r->inv_freq))) return HYTOPK_MISALIGNED;
  return HYTOPK_OK;
}

RowArgs row_args(const void* x, int64_t x_row, int64_t x_head, int n, int H, int d,
                 const hytopk_rope_params* r, uint32_t* status) {
  RowArgs a{};
  a.x = x;
  a.x_row = x_row;
  a.x_head = x_head;
  a.n = n;
  a.H = H;
  a.d = d;
  a.status = status;
  if (r) {
    a.positions = r->positions;
    a.inv_freq = r->inv_freq;
    a.rot = r->rot;
    a.first = r->first;
    a.interleaved = r->interleaved;
    a.inverse = r->inverse;
    a.mscale = r->mscale;
  }
  return a;
}

hytopk_status launched() {
  return cudaGetLastError() == cudaSuccess ? HYTOPK_OK : HYTOPK_CUDA_ERROR;
}

}  // namespace
}  // namespace hytopk

using namespace hytopk;

extern "C" hytopk_status hytopk_rope(const void* x, int64_t x_row, int64_t x_head,
                                     hytopk_elem type, int n, int H, int d,
                                     const hytopk_rope_params* rope, void* out, int64_t out_row,
                                     int64_t out_head, uint32_t* dev_status, cudaStream_t stream) {
  if (!rope) return HYTOPK_INVALID_ARG;
  hytopk_status s = check_rows(x, x_row, x_head, type, n, H, d, rope);
  if (s != HYTOPK_OK || n == 0) return s;
  if (!out) return HYTOPK_INVALID_ARG;
  if (!aligned16(out) || !stride_ok(out_row, type) || !stride_ok(out_head, type))
    return HYTOPK_MISALIGNED;
  if (out == x && (out_row != x_row || out_head != x_head)) return HYTOPK_INVALID_ARG;
  RowArgs a = row_args(x, x_row, x_head, n, H, d, rope, dev_status);
  a.out = out;
  a.out_row = out_row;
  a.out_head = out_head;
  const unsigned grid = (unsigned)(((int64_t)n * H + kWarps - 1) / kWarps);
  const size_t smem = sizeof(float) * kWarps * d;
  if (type == HYTOPK_ELEM_F32) k_rope<float><<<grid, 32 * kWarps, smem, stream>>>(a);
  else k_rope<__nv_bfloat16><<<grid, 32 * kWarps, smem, stream>>>(a);
  return launched();
}

extern "C" hytopk_status hytopk_cache_write(const void* x, int64_t x_row, int64_t x_head,
                                            hytopk_elem x_type, int n, int H, int d,
                                            const hytopk_rope_params* rope, const int32_t* slots,
                                            void* cache, hytopk_elem cache_type,
                                            float* cache_scale, int L, uint32_t* dev_status,
                                            cudaStream_t stream) {
  hytopk_status s = check_rows(x, x_row, x_head, x_type, n, H, d, rope);
  if (s != HYTOPK_OK) return s;
  const bool e4 = cache_type == HYTOPK_ELEM_E4M3;
  if (!e4 && cache_type != HYTOPK_ELEM_BF16) return HYTOPK_INVALID_ARG;
  if (L < 1 || (!slots && n > L)) return HYTOPK_INVALID_ARG;
  if (e4 && d % 16) return HYTOPK_UNSUPPORTED;
  if (n == 0) return HYTOPK_OK;
  if (!cache || e4 != (cache_scale != nullptr)) return HYTOPK_INVALID_ARG;
  if (!aligned16(cache) || !aligned4(cache_scale) || !aligned4(slots)) return HYTOPK_MISALIGNED;
  RowArgs a = row_args(x, x_row, x_head, n, H, d, rope, dev_status);
  a.out = cache;
  a.scale = cache_scale;
  a.slots = slots;
  a.L = L;
  const unsigned grid = (unsigned)(((int64_t)n * H + kWarps - 1) / kWarps);
  const size_t smem = sizeof(float) * kWarps * d;
  if (x_type == HYTOPK_ELEM_F32) {
    if (e4) k_cache_write<float, true><<<grid, 32 * kWarps, smem, stream>>>(a);
    else k_cache_write<float, false><<<grid, 32 * kWarps, smem, stream>>>(a);
  } else {
    if (e4) k_cache_write<__nv_bfloat16, true><<<grid, 32 * kWarps, smem, stream>>>(a);
    else k_cache_write<__nv_bfloat16, false><<<grid, 32 * kWarps, smem, stream>>>(a);
  }
  return launched();
}

extern "C" hytopk_status hytopk_cache_read(const void* cache, hytopk_elem cache_type,
                                           const float* cache_scale, int L, const int32_t* slots,
                                           int n, int H, int d, void* out, hytopk_elem out_type,
                                           uint32_t* dev_status, cudaStream_t stream) {
  const bool e4 = cache_type == HYTOPK_ELEM_E4M3;
  if (n < 0 || H < 1 || L < 1 || (!slots && n > L)) return HYTOPK_INVALID_ARG;
  if (!e4 && cache_type != HYTOPK_ELEM_BF16) return HYTOPK_INVALID_ARG;
  if (out_type != HYTOPK_ELEM_BF16 && out_type != HYTOPK_ELEM_F32) return HYTOPK_INVALID_ARG;
  if (d < 8 || d > 1024 || d % (e4 ? 16 : 8)) return HYTOPK_UNSUPPORTED;
  if ((int64_t)n * H >= (int64_t)1 << 31) return HYTOPK_UNSUPPORTED;
  if (n == 0) return HYTOPK_OK;
  if (!cache || !out || e4 != (cache_scale != nullptr)) return HYTOPK_INVALID_ARG;
  if (!aligned16(cache) || !aligned16(out) || !aligned4(cache_scale) || !aligned4(slots))
    return HYTOPK_MISALIGNED;
  const ReadArgs a{cache, cache_scale, slots, out, n, H, d, L, dev_status};
  const unsigned grid = (unsigned)(((int64_t)n * H + kWarps - 1) / kWarps);
  if (out_type == HYTOPK_ELEM_F32) {
    if (e4) k_cache_read<true, float><<<grid, 32 * kWarps, 0, stream>>>(a);
    else k_cache_read<false, float><<<grid, 32 * kWarps, 0, stream>>>(a);
  } else {
    if (e4) k_cache_read<true, __nv_bfloat16><<<grid, 32 * kWarps, 0, stream>>>(a);
    else k_cache_read<false, __nv_bfloat16><<<grid, 32 * kWarps, 0, stream>>>(a);
  }
  return launched();
}
