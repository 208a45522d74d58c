// Rotations by angles that change from token to token or from block to
// block, shared by the rope (rope.hip) and the attention (attend.hip).
#pragma once

#include <math.h>

#include "hkv_device.h"

namespace hkv {

// theta = rope_base^(-2 f / 128) in quarter turns: an angle is then its
// whole number of quarter turns, which picks the quadrant, and a remainder.
inline double quarter_turns(double rope_base, int freq) {
  return 0.63661977236758134308 / pow(rope_base, static_cast<double>(2 * freq) / kHeadDim);
}

// cos and sin of pos * theta, theta in quarter turns.  The product's whole
// part k and remainder pos * theta - k (one fused step) are taken in double,
// so the remainder is off by what theta is (a constant, a power and their
// quotient, each rounded): some 2^-51 of the angle.  The Taylor series of sin
// (to x^9) and cos (to x^10) on |x| <= pi/4 leave out less than 2e-9 and 2e-11
// and run in fp32, within about one step of the exact values.  k < 2^31 for
// |pos * theta| < 2^31.
__device__ __forceinline__ void cos_sin(int pos, double theta, float* c, float* s) {
  const double p = static_cast<double>(pos);
  const double k = rint(p * theta);
  const float x = static_cast<float>(fma(p, theta, -k) * 1.57079632679489661923);
  const float x2 = x * x;
  float ps = __builtin_fmaf(x2, 1.0f / 362880.0f, -1.0f / 5040.0f);
  ps = __builtin_fmaf(ps, x2, 1.0f / 120.0f);
  ps = __builtin_fmaf(ps, x2, -1.0f / 6.0f);
  const float sr = __builtin_fmaf(x * x2, ps, x);
  float pc = __builtin_fmaf(x2, -1.0f / 3628800.0f, 1.0f / 40320.0f);
  pc = __builtin_fmaf(pc, x2, -1.0f / 720.0f);
  pc = __builtin_fmaf(pc, x2, 1.0f / 24.0f);
  pc = __builtin_fmaf(pc, x2, -0.5f);
  const float cr = __builtin_fmaf(x2, pc, 1.0f);
  const int q = static_cast<int>(k) & 3;
  const float a = (q & 1) ? sr : cr;
  const float b = (q & 1) ? cr : sr;
  *c = (q == 1 || q == 2) ? -a : a;
  *s = (q & 2) ? -b : b;
}

// The pair that element-run position j of a lane belongs to (lane layout of
// hkv_device.h: 8 lanes per vector, lane sub owns elements 8 sub .. 8 sub + 7
// and the same of the upper half).
__device__ __forceinline__ int lane_pair(int pairs, int sub, int j) {
  if (pairs == kInterleaved) return j < 4 ? 4 * sub + j : 28 + 4 * sub + j;
  return 8 * sub + j;
}

// (a, b) turned by the angle whose cosine and sine are c and s.  s = 0 only
// for whole half turns, where c = 1 or -1: either value then keeps its size
// whatever its partner holds.
__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
  const float x = s == 0.0f ? a * c : a * c - b * s;
  const float y = s == 0.0f ? b * c : a * s + b * c;
  a = x;
  b = y;
}

// The 8 pairs of a lane's two runs.
template <int PAIRS>
__device__ __forceinline__ void turn_runs(float (&a)[8], float (&b)[8], const float (&cs)[8],
                                          const float (&sn)[8]) {
  if constexpr (PAIRS == kInterleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      turn_pair(a[2 * j], a[2 * j + 1], cs[j], sn[j]);
      turn_pair(b[2 * j], b[2 * j + 1], cs[4 + j], sn[4 + j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) turn_pair(a[j], b[j], cs[j], sn[j]);
  }
}

}  // namespace hkv
