// rope.cuh -- rotary angles: cos and sin of position * frequency, accurate to
// about an ulp of 1 at every position below 2^24.
//
// The product of a 24-bit position and a 24-bit frequency needs 48 bits; at a
// million tokens its fp32 rounding alone is 0.03 rad. So the product is kept as
// hi + lo (lo is the exact remainder, from a fused multiply-add) and reduced by
// a multiple of pi / 2 = C1 + C2 + C3 in fp32 parts (the reduction by constants
// in parts of Cody and Waite, "Software Manual for the Elementary Functions",
// 1980). The multiple comes from the rounded product. Below 2^20 it is the
// nearest one or off by so little that the rest stays within 0.91, where the
// Taylor series of sin and cos to x^9 and x^10 are off by less than 1e-8; up to
// 2^22 the rest reaches 1.27 and is reduced once more; past that in 64 bits. The
// result is off by at most 1.3 x 2^-24 (56 million angles of the whole range, in
// the same operations on the host).
#pragma once

#include "common.cuh"

namespace hytopk {

constexpr int kMaxPosition = 1 << 24;  // positions below this are exact in fp32

// The same reduction in 64 bits, for angles past 2^22 (a call, so that its 64-bit
// arithmetic is not run ahead of the branch).
static __device__ __noinline__ float2 rope_reduce_far(float pos, float freq) {
  constexpr double kHalfPi = 1.5707963267948966192313216916398;
  const double x = (double)pos * (double)freq;
  const double n = rint(x * (1.0 / kHalfPi));
  return make_float2((float)(x - n * kHalfPi), __int_as_float((int)(long long)n));
}

__device__ __forceinline__ void rope_turn(float pos, float freq, float& c, float& s) {
  constexpr double kHalfPi = 1.5707963267948966192313216916398;
  constexpr float C1 = (float)kHalfPi;
  constexpr float C2 = (float)(kHalfPi - (double)C1);
  constexpr float C3 = (float)(kHalfPi - (double)C1 - (double)C2);
  const float hi = __fmul_rn(pos, freq);
  float r;
  int q;
  if (fabsf(hi) < 1048576.0f) {
    const float lo = __fmaf_rn(pos, freq, -hi);
    const float n = rintf(hi * (float)(1.0 / kHalfPi));
    r = __fmaf_rn(-n, C1, hi);
    r = __fmaf_rn(-n, C2, r);
    r = __fmaf_rn(-n, C3, r) + lo;
    q = (int)n;
  } else if (fabsf(hi) < 4194304.0f) {
    // (200000 rows written, 64 columns rotated: 41 us, 37 of smaller angles, 107 of larger)
    const float n = rintf(hi * (float)(1.0 / kHalfPi));
    float x = __fmaf_rn(-n, C1, hi);  // exact, as is the second one
    float y = __fmaf_rn(-n, C3, __fmaf_rn(-n, C2, __fmaf_rn(pos, freq, -hi)));
    const float k = rintf((x + y) * (float)(1.0 / kHalfPi));
    x = __fmaf_rn(-k, C1, x);
    y = __fmaf_rn(-k, C2, y);
    r = x + y;
    q = (int)n + (int)k;
  } else {  // past 2^22 the multiple is no longer exact in fp32
    const float2 far = rope_reduce_far(pos, freq);
    r = far.x;
    q = __float_as_int(far.y);
  }
  const float z = r * r;
  float sn = __fmaf_rn(z, 1.0f / 362880.0f, -1.0f / 5040.0f);
  sn = __fmaf_rn(sn, z, 1.0f / 120.0f);
  sn = __fmaf_rn(sn, z, -1.0f / 6.0f);
  sn = __fmaf_rn(sn * z, r, r);
  float cs = __fmaf_rn(z, -1.0f / 3628800.0f, 1.0f / 40320.0f);
  cs = __fmaf_rn(cs, z, -1.0f / 720.0f);
  cs = __fmaf_rn(cs, z, 1.0f / 24.0f);
  cs = __fmaf_rn(cs, z, -0.5f);
  cs = __fmaf_rn(cs, z, 1.0f);
  // quadrant: (c, s) -> (-s, c) for each quarter turn
  const float a = (q & 1) ? sn : cs, b = (q & 1) ? cs : sn;
  c = ((q + 1) & 2) ? -a : a;
  s = (q & 2) ? -b : b;
}

}  // namespace hytopk
