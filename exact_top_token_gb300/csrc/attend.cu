// attend.cu -- hytopk_attend and hytopk_attend_backward: attention of each
// query over its own selected cache rows, and its gradients.
#include "attend.h"
#include "early.cuh"

#include "launch.h"

namespace hytopk {

// attend_d*.cu
cudaError_t launch_attend_d64_bf16(const att::Args& a, bool f32, int sms, cudaStream_t st);
cudaError_t launch_attend_d64_e4m3(const att::Args& a, bool f32, int sms, cudaStream_t st);
cudaError_t launch_attend_d128_bf16(const att::Args& a, bool f32, int sms, cudaStream_t st);
cudaError_t launch_attend_d128_e4m3(const att::Args& a, bool f32, int sms, cudaStream_t st);
cudaError_t launch_attend_d256_bf16(const att::Args& a, bool f32, int sms, cudaStream_t st);
cudaError_t launch_attend_d256_e4m3(const att::Args& a, bool f32, int sms, cudaStream_t st);
// attend_backward_d*.cu
cudaError_t launch_attend_backward_d64(const att::Args& a, bool out_f32, int sms, cudaStream_t st);
cudaError_t launch_attend_backward_d128(const att::Args& a, bool out_f32, int sms, cudaStream_t st);

namespace att {
namespace {

// One kernel for all that is zeroed: two clearing calls took 4 us of a small step, and
// the kernel after them cannot be launched early.
constexpr int kZeroThreads = 512;
__global__ void __launch_bounds__(kZeroThreads) k_zero(float4* x, float4* y, size_t nx, float4* z,
                                                       size_t nz) {
  allow_next();
  wait_for_earlier();
  const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const size_t step = (size_t)gridDim.x * kZeroThreads;
  const size_t i0 = (size_t)blockIdx.x * kZeroThreads + threadIdx.x;
  for (size_t i = i0; i < nx; i += step) {
    x[i] = zero;
    y[i] = zero;
  }
  for (size_t i = i0; i < nz; i += step) z[i] = zero;
}

// Byte offsets of cache rows are 64-bit products of two 32-bit factors.
hytopk_status check_row(int64_t row, int bytes) {
  if (row < 0) return HYTOPK_INVALID_ARG;
  return row >= ((int64_t)1 << 32) / bytes ? HYTOPK_UNSUPPORTED : HYTOPK_OK;
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

cudaError_t launch_zero(float* x, float* y, size_t nx, float* z, size_t nz, int sms,
                        cudaStream_t st) {
  const size_t most = (nx > nz ? nx : nz) / 4, blocks = (most + kZeroThreads - 1) / kZeroThreads;
  if (blocks == 0) return cudaSuccess;
  return launch_early(k_zero, (unsigned)(blocks < 4 * (size_t)sms ? blocks : 4 * (size_t)sms),
                      kZeroThreads, 0, st, 1, reinterpret_cast<float4*>(x),
                      reinterpret_cast<float4*>(y), nx / 4, reinterpret_cast<float4*>(z), nz / 4);
}

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
  s = att::check_row(k_row, e4 ? 1 : 2);
  if (s == HYTOPK_OK) s = att::check_row(v_row, e4 ? 1 : 2);
  if (s != HYTOPK_OK) return s;
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
                                                float* dk, float* dv, int accumulate,
                                                uint32_t* dev_status, cudaStream_t stream) {
  hytopk_status s = att::check(n, L, Hq, Hkv, d, k_top, out_type, false);
  if (s != HYTOPK_OK) return s;
  s = att::check_row(k_row, 2);
  if (s == HYTOPK_OK) s = att::check_row(v_row, 2);
  if (s == HYTOPK_OK) s = att::check_row((int64_t)Hkv * d, sizeof(float));
  if (s != HYTOPK_OK) return s;
  if (n == 0 && accumulate) return HYTOPK_OK;
  if (!dk || !dv) return HYTOPK_INVALID_ARG;
  if (n > 0 && (!q || !k || !v || !idx || !out || !lse || !grad || !dq)) return HYTOPK_INVALID_ARG;
  if (!att::aligned(q, 16) || !att::aligned(k, 16) || !att::aligned(v, 16) ||
      !att::aligned(out, 16) || !att::aligned(grad, 16) || !att::aligned(dq, 16) ||
      !att::aligned(dk, 16) || !att::aligned(dv, 16) || !att::aligned(idx, 4) ||
      !att::aligned(lse, 4) || q_row % 8 || k_row % 8 || v_row % 8)
    return HYTOPK_MISALIGNED;
  if (n == 0)
    return att::launch_zero(dk, dv, (size_t)L * Hkv * d, nullptr, 0, num_sms(), stream) ==
                   cudaSuccess
               ? HYTOPK_OK
               : HYTOPK_CUDA_ERROR;
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
  a.zero = !accumulate;
  auto launch = d == 64 ? launch_attend_backward_d64 : launch_attend_backward_d128;
  return launch(a, out_type == HYTOPK_ELEM_F32, num_sms(), stream) == cudaSuccess
             ? HYTOPK_OK
             : HYTOPK_CUDA_ERROR;
}
