// rows.cuh -- eight neighbouring columns of a row in a thread: loads, stores and the steps of
// quantising them (rows of a cache and of its pages).
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace hytopk {

template <typename T>
__device__ __forceinline__ void load8(const T* p, uint32_t (&raw)[sizeof(T) * 2]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  raw[0] = a.x, raw[1] = a.y, raw[2] = a.z, raw[3] = a.w;
  if constexpr (sizeof(T) == 4) {
    const uint4 b = *(reinterpret_cast<const uint4*>(p) + 1);
    raw[4] = b.x, raw[5] = b.y, raw[6] = b.z, raw[7] = b.w;
  }
}
template <int W>
__device__ __forceinline__ void unpack8(const uint32_t (&raw)[W], float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if constexpr (W == 8) {
      v[i] = __uint_as_float(raw[i]);
    } else {
      v[2 * i] = __uint_as_float(raw[i] << 16);
      v[2 * i + 1] = __uint_as_float(raw[i] & 0xFFFF0000u);
    }
  }
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]),
                                              bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
  }
}
// two values as e4m3 codes, round to nearest even, saturating
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two quotients y / -scale from ninv = -1 / scale: q = y ninv, then q + (y + q scale) ninv.
__device__ __forceinline__ void quotient2(float y0, float y1, float scale, float ninv, float& c0,
                                          float& c1) {
  asm("{\n .reg .b64 y, s, n, q, e;\n mov.b64 y, {%2, %3};\n mov.b64 s, {%4, %4};\n"
      " mov.b64 n, {%5, %5};\n mul.rn.f32x2 q, y, n;\n fma.rn.f32x2 e, q, s, y;\n"
      " fma.rn.f32x2 q, e, n, q;\n mov.b64 {%0, %1}, q;\n}\n"
      : "=f"(c0), "=f"(c1)
      : "f"(y0), "f"(y1), "f"(scale), "f"(ninv));
}

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Rows whose largest magnitude lies between these bits (1e-18 and 2^127) divide by a
// reciprocal.
constexpr uint32_t kTinyRow = 0x219392EFu, kHugeRow = 0x7F000000u;

}  // namespace hytopk
