// When a step of the 4-bit decode (int4_decode.cu) sets a head's reference and lift again, and to
// what.  On its own, so that it also compiles for the host, where a test sees that a correction always
// leads to values that the same step does not vote on again: it costs a step as much again, so it has
// to be seldom.
//
// A lane has four probabilities p of its head, relative to 2^R, and their weights y = p vs lift and
// z = p vl lift.
#pragma once

namespace pkv {

constexpr float kMostSum = 8.f;              // of a lane's p: none passes R + 3
constexpr float kMostWeights = 0x1.ffp15f;   // of its y, which enter the MMAs as fp16 (to 65504)
constexpr float kMostWeight = 0x1p13f;       // of all y, and z / 16, behind a correction: four are half of that sum
constexpr float kMostMinima = 0x1p60f;       // of its z, which stay in fp32

// The vote, on sums that a step needs anyway (the scales of V are not negative, so the sum is at least
// the largest; NaN votes too).
__device__ __forceinline__ bool i4_votes(float p, float y, float z) {
  return !(p <= kMostSum) || !(fabsf(y) <= kMostWeights) || !(fabsf(z) <= kMostMinima);
}

// The reference for scores up to `top`: no p is above 1, so that four are half of their sum's limit.
__device__ __forceinline__ float i4_reference(float ref, float top) { return top > ref ? ceilf(top) : ref; }

// The lift for weights p max(vs, |vl| / 16) up to `most`.  (A vote for weights has one at 2^14 - 32 at
// least, so that the lift falls; it rises with the reference only.)
__device__ __forceinline__ float i4_lift(float lift, float most) {
  if (!(most * lift >= kMostWeight)) return lift;
  // 2^12 up to 2^13; the largest weight is at least 2^-113
  const int e = 127 + 12 + 127 - (int)(__float_as_uint(most) >> 23);
  return __uint_as_float((unsigned)(e > 1 ? e : 1) << 23);
}

}  // namespace pkv
