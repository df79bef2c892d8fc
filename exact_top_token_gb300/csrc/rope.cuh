// rope.cuh -- rotary angles: cos and sin of position * frequency, accurate at
// every position below 2^24.
//
// The product of a 24-bit position and a 24-bit frequency needs 48 bits; at a
// million tokens its fp32 rounding alone is 0.03 rad. So the product is kept as
// hi + lo (lo is the exact remainder, from a fused multiply-add) and reduced by
// the nearest multiple of 2 pi with 2 pi = C1 + C2 + C3 in fp32 parts (the
// reduction by constants in parts of Cody and Waite, "Software Manual for the
// Elementary Functions", 1980), which leaves an angle in [-pi, pi] that is
// good to about 2^-23.
#pragma once

#include "common.cuh"

namespace hytopk {

constexpr int kMaxPosition = 1 << 24;  // positions below this are exact in fp32

__device__ __forceinline__ void rope_turn(float pos, float freq, float& c, float& s) {
  const float hi = __fmul_rn(pos, freq);
  const float lo = __fmaf_rn(pos, freq, -hi);
  // 2 pi = 6.28318548202514648 - 1.74845553146951715e-7 - ... (fp32 parts)
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  constexpr float C1 = (float)kTwoPi;
  constexpr float C2 = (float)(kTwoPi - (double)C1);
  constexpr float C3 = (float)(kTwoPi - (double)C1 - (double)C2);
  const float turns = rintf(hi * (float)(1.0 / kTwoPi));
  float r = __fmaf_rn(-turns, C1, hi);
  r = __fmaf_rn(-turns, C2, r);
  r = __fmaf_rn(-turns, C3, r);
  sincosf(r + lo, &s, &c);
}

}  // namespace hytopk
