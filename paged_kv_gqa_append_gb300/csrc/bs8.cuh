// 8-bit codes of the block-scaled pages: int8 or e4m3, one fp32 scale per
// block (16 slots x 64 dims of one page, K or V, and KV head).
//
//   scale = amax / top,  code = round-half-even(x / scale)   (IEEE fp32 divisions)
//
// with top = 127 (int8; codes clamped to [-127, 127]) or 448 (e4m3; the
// conversion rounds to nearest even and saturates).  scale 0 gives zero codes.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "pkv.h"

namespace pkv {

constexpr int kBs8BlockBytes = PKV_PAGE_TOKENS * PKV_HEAD_DIM;   // 1024
constexpr int kBs8PageBytes = PKV_BS8_PAGE_BYTES;                 // 16384
static_assert(kBs8PageBytes == 2 * PKV_NUM_KV_HEADS * kBs8BlockBytes, "page layout");

// the byte of x under `scale`
template <bool kE4m3>
__device__ __forceinline__ uint32_t bs8_encode(float x, float scale) {
  if (scale == 0.f) return 0u;
  const float y = __fdiv_rn(x, scale);
  if (kE4m3) return (uint32_t)__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
  return (uint32_t)(uint8_t)(int8_t)max(-127, min(127, __float2int_rn(y)));
}

// the value of a byte's code
template <bool kE4m3>
__device__ __forceinline__ float bs8_decode(uint32_t byte) {
  if (kE4m3) return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
  return (float)(int8_t)(uint8_t)byte;
}

// Eight codes in two words, the definition's way.
template <bool kE4m3>
__device__ __noinline__ uint2 bs8_encode8_exact(float x0, float x1, float x2, float x3, float x4, float x5, float x6,
                                                float x7, float scale) {
  const uint32_t lo = bs8_encode<kE4m3>(x0, scale) | bs8_encode<kE4m3>(x1, scale) << 8 |
                      bs8_encode<kE4m3>(x2, scale) << 16 | bs8_encode<kE4m3>(x3, scale) << 24;
  const uint32_t hi = bs8_encode<kE4m3>(x4, scale) | bs8_encode<kE4m3>(x5, scale) << 8 |
                      bs8_encode<kE4m3>(x6, scale) << 16 | bs8_encode<kE4m3>(x7, scale) << 24;
  return make_uint2(lo, hi);
}

// The codes of four products x * inv, unclamped (|x * inv| stays below 128 or
// saturates): adding 1.5 * 2^23 rounds the exact product to the nearest even
// integer in the low bits.
template <bool kE4m3>
__device__ __forceinline__ uint32_t bs8_round4(const float* x, float inv) {
  if (kE4m3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0] * inv, x[1] * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2] * inv, x[3] * inv), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
  }
  constexpr float kRound = 12582912.f;
  const uint32_t a = __byte_perm(__float_as_uint(fmaf(x[0], inv, kRound)), __float_as_uint(fmaf(x[1], inv, kRound)), 0x0040);
  const uint32_t b = __byte_perm(__float_as_uint(fmaf(x[2], inv, kRound)), __float_as_uint(fmaf(x[3], inv, kRound)), 0x0040);
  return __byte_perm(a, b, 0x5410);
}

// The codes of |x| <= top * scale without 32 divisions: a quotient lies between
// x * inv (1 - 2^-21) and x * inv (1 + 2^-21), with inv = 1 / scale rounded; where
// both give the same codes (rounding is monotonic) they are the quotients', and
// elsewhere -- one value in about 10^4 -- the divisions are done.
struct Bs8Inverse {
  float lo, hi;  // 0: no short way (scale 0 or near the subnormals)
};
__device__ __forceinline__ Bs8Inverse bs8_inverse(float scale) {
  if (!(scale > 7.9e-31f && scale < 1e30f)) return {0.f, 0.f};  // 2^-100 .. 2^100
  const float inv = __frcp_rn(scale);
  return {inv * (1.f - 4.76837158203125e-7f), inv * (1.f + 4.76837158203125e-7f)};
}
template <bool kE4m3>
__device__ __forceinline__ uint2 bs8_encode8(const float (&x)[8], float scale, Bs8Inverse inv) {
  const uint2 a = make_uint2(bs8_round4<kE4m3>(x, inv.lo), bs8_round4<kE4m3>(x + 4, inv.lo));
  const uint2 b = make_uint2(bs8_round4<kE4m3>(x, inv.hi), bs8_round4<kE4m3>(x + 4, inv.hi));
  if (a.x == b.x && a.y == b.y && inv.lo > 0.f) return a;
  return bs8_encode8_exact<kE4m3>(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], scale);
}

template <bool kE4m3>
__device__ __forceinline__ void bs8_decode8(uint2 u, float (&x)[8]) {
  const uint32_t w[2] = {u.x, u.y};
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = bs8_decode<kE4m3>((w[e >> 2] >> (8 * (e & 3))) & 0xFFu);
}

}  // namespace pkv
