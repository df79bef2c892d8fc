// attend.cu -- hytopk_attend and hytopk_attend_backward: attention of each
// query over its own selected cache rows, and its gradients.
#include "attend.h"

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "launch.h"

namespace hytopk {

// attend_d*.cu
cudaError_t launch_attend_d64_bf16(const att::Args& a, bool f32, int sms, cudaStream_t st);
cudaError_t launch_attend_d64_e4m3(const att::Args& a, bool f32, int sms, cudaStream_t st);
cudaError_t launch_attend_d128_bf16(const att::Args& a, bool f32, int sms, cudaStream_t st);
cudaError_t launch_attend_d128_e4m3(const att::Args& a, bool f32, int sms, cudaStream_t st);
cudaError_t launch_attend_d256_bf16(const att::Args& a, bool f32, int sms, cudaStream_t st);
cudaError_t launch_attend_d256_e4m3(const att::Args& a, bool f32, int sms, cudaStream_t st);

namespace att {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float block_reduce(float v, bool maximum, float* red) {
  for (int o = 16; o; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = maximum ? fmaxf(v, w) : v + w;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int i = 1; i < kThreads / 32; ++i) v = maximum ? fmaxf(v, red[i]) : v + red[i];
  return v;
}

template <bool E4M3>
__device__ __forceinline__ float row_elem(const void* base, int64_t row, int s, int hk, int d, int j) {
  const size_t at = (size_t)s * row + (size_t)hk * d + j;
  if constexpr (E4M3) {
    const __half_raw r = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(base)[at], __NV_E4M3);
    return __half2float(__half(r));
  } else {
    return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at]);
  }
}

__device__ __forceinline__ int checked_row(const Args& a, int t, int j) {
  const int s = a.idx[(size_t)t * a.k_top + j];
  if (s >= 0 && s < a.L) return s;
  if (s != -1 && a.status) atomicOr(a.status, HYTOPK_DEV_BAD_INDEX);
  return -1;
}

// One query head per CTA: a warp per selected row.
__global__ void __launch_bounds__(kThreads) k_attend_backward_simple(const Args a, int out_f32) {
  extern __shared__ float sh[];
  float* qs = sh;
  float* dos = qs + a.d;
  float* dqs = dos + a.d;
  __shared__ float red[4];
  const int Hq = a.Hkv * a.G;
  const int t = blockIdx.x / Hq, h = blockIdx.x % Hq, hk = h / a.G;
  const size_t at = ((size_t)t * Hq + h) * a.d;
  float delta = 0.0f;
  for (int i = threadIdx.x; i < a.d; i += kThreads) {
    qs[i] = __bfloat162float(
        static_cast<const __nv_bfloat16*>(a.q)[(size_t)t * a.q_row + (size_t)h * a.d + i]);
    dos[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.grad)[at + i]);
    const float o = out_f32 ? static_cast<const float*>(a.out)[at + i]
                            : __bfloat162float(static_cast<const __nv_bfloat16*>(a.out)[at + i]);
    delta += dos[i] * o;
    dqs[i] = 0.0f;
  }
  delta = block_reduce(delta, false, red);
  const float lse = a.lse[(size_t)t * Hq + h];
  const int lane = threadIdx.x & 31;
  for (int j = threadIdx.x >> 5; j < a.k_top; j += kThreads / 32) {
    const int s = checked_row(a, t, j);
    if (s < 0 || lse == -INFINITY) continue;
    float x = 0.0f, dp = 0.0f;
    for (int i = lane; i < a.d; i += 32) {
      x += qs[i] * row_elem<false>(a.k, a.k_row, s, hk, a.d, i);
      dp += dos[i] * row_elem<false>(a.v, a.v_row, s, hk, a.d, i);
    }
    for (int o = 16; o; o >>= 1) {
      x += __shfl_xor_sync(0xffffffffu, x, o);
      dp += __shfl_xor_sync(0xffffffffu, dp, o);
    }
    const float p = __expf(x * a.scale - lse);
    const float ds = p * (dp - delta) * a.scale;
    const size_t row = ((size_t)s * a.Hkv + hk) * a.d;
    for (int i = lane; i < a.d; i += 32) {
      atomicAdd(a.dv + row + i, p * dos[i]);
      atomicAdd(a.dk + row + i, ds * qs[i]);
      atomicAdd(dqs + i, ds * row_elem<false>(a.k, a.k_row, s, hk, a.d, i));
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.d; i += kThreads) a.dq[at + i] = dqs[i];
}

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

hytopk_status check(int n, int L, int Hq, int Hkv, int d, int k_top, hytopk_elem out_type,
                    bool wide) {
  if (n < 0 || L < 1 || Hkv < 1 || Hq < 1 || k_top < 1) return HYTOPK_INVALID_ARG;
  if (Hq % Hkv) return HYTOPK_INVALID_ARG;
  if (out_type != HYTOPK_ELEM_BF16 && out_type != HYTOPK_ELEM_F32) return HYTOPK_INVALID_ARG;
  if (Hq / Hkv > 128 || k_top > kMaxTopK) return HYTOPK_UNSUPPORTED;
  if (d != 64 && d != 128 && !(wide && d == 256)) return HYTOPK_UNSUPPORTED;
  if ((int64_t)n * Hq >= (int64_t)1 << 31) return HYTOPK_UNSUPPORTED;
  return HYTOPK_OK;
}

}  // namespace
}  // namespace att
}  // namespace hytopk

using namespace hytopk;

extern "C" hytopk_status hytopk_attend(const void* q, int64_t q_row, const void* k, int64_t k_row,
                                       const float* k_scale, const void* v, int64_t v_row,
                                       const float* v_scale, const int32_t* idx, int n, int L,
                                       int Hq, int Hkv, int d, int k_top, hytopk_elem cache_type,
                                       float scale, void* out, hytopk_elem out_type, float* lse,
                                       uint32_t* dev_status, cudaStream_t stream) {
  const bool e4 = cache_type == HYTOPK_ELEM_E4M3;
  if (!e4 && cache_type != HYTOPK_ELEM_BF16) return HYTOPK_INVALID_ARG;
  hytopk_status s =
      att::check(n, L, Hq, Hkv, d, k_top, out_type, out_type != HYTOPK_ELEM_F32);
  if (s != HYTOPK_OK) return s;
  if (n == 0) return HYTOPK_OK;
  if (!q || !k || !v || !idx || !out) return HYTOPK_INVALID_ARG;
  if (e4 != (k_scale != nullptr) || e4 != (v_scale != nullptr)) return HYTOPK_INVALID_ARG;
  const int per16 = e4 ? 16 : 8;
  if (!att::aligned(q, 16) || !att::aligned(k, 16) || !att::aligned(v, 16) ||
      !att::aligned(out, 16) || !att::aligned(idx, 4) || !att::aligned(lse, 4) ||
      !att::aligned(k_scale, 4) || !att::aligned(v_scale, 4) || q_row % 8 || k_row % per16 ||
      v_row % per16)
    return HYTOPK_MISALIGNED;
  att::Args a{};
  a.q = q;
  a.q_row = q_row;
  a.k = k;
  a.v = v;
  a.k_row = k_row;
  a.v_row = v_row;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.idx = idx;
  a.n = n;
  a.L = L;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.d = d;
  a.k_top = k_top;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.status = dev_status;
  const bool f32 = out_type == HYTOPK_ELEM_F32;
  auto launch = d == 64    ? (e4 ? launch_attend_d64_e4m3 : launch_attend_d64_bf16)
                : d == 128 ? (e4 ? launch_attend_d128_e4m3 : launch_attend_d128_bf16)
                           : (e4 ? launch_attend_d256_e4m3 : launch_attend_d256_bf16);
  return launch(a, f32, num_sms(), stream) == cudaSuccess ? HYTOPK_OK : HYTOPK_CUDA_ERROR;
}

extern "C" hytopk_status hytopk_attend_backward(const void* q, int64_t q_row, const void* k,
                                                int64_t k_row, const void* v, int64_t v_row,
                                                const int32_t* idx, const void* out,
                                                hytopk_elem out_type, const float* lse,
                                                const void* grad, int n, int L, int Hq, int Hkv,
                                                int d, int k_top, float scale, float* dq,
                                                float* dk, float* dv, uint32_t* dev_status,
                                                cudaStream_t stream) {
  hytopk_status s = att::check(n, L, Hq, Hkv, d, k_top, out_type, false);
  if (s != HYTOPK_OK) return s;
  if (n == 0) return HYTOPK_OK;
  if (!q || !k || !v || !idx || !out || !lse || !grad || !dq || !dk || !dv)
    return HYTOPK_INVALID_ARG;
  if (!att::aligned(q, 16) || !att::aligned(k, 16) || !att::aligned(v, 16) ||
      !att::aligned(out, 16) || !att::aligned(grad, 16) || !att::aligned(dq, 16) ||
      !att::aligned(dk, 16) || !att::aligned(dv, 16) || !att::aligned(idx, 4) ||
      !att::aligned(lse, 4) || q_row % 8 || k_row % 8 || v_row % 8)
    return HYTOPK_MISALIGNED;
  att::Args a{};
  a.q = q;
  a.q_row = q_row;
  a.k = k;
  a.v = v;
  a.k_row = k_row;
  a.v_row = v_row;
  a.idx = idx;
  a.n = n;
  a.L = L;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.d = d;
  a.k_top = k_top;
  a.scale = scale;
  a.out = const_cast<void*>(out);
  a.lse = const_cast<float*>(lse);
  a.status = dev_status;
  a.grad = grad;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  att::k_attend_backward_simple<<<(unsigned)n * Hq, att::kThreads, sizeof(float) * 3 * d, stream>>>(
      a, out_type == HYTOPK_ELEM_F32);
  return cudaGetLastError() == cudaSuccess ? HYTOPK_OK : HYTOPK_CUDA_ERROR;
}
