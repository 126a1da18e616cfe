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
#include "ptx.cuh"

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

// Eight codes of values |x| <= top * scale without divisions, inv = 1 / scale
// rounded: the quotient from the product x * inv by corrections with its remainder
// (Markstein, IBM J. Res. Dev. 34, 1990).  A second one makes any quotient the IEEE
// one, the first having brought it within a unit in the last place.  For bf16
// values one is enough: with their 8-bit significands it equals the IEEE quotient
// beside every point where a code changes, for all 2^23 significands of the scale.
// The scale is in [2^-100, 2^100], so that nothing that a code depends on
// underflows.  The remainder is taken as q * scale - x: -0 stays -0.  Adding
// 1.5 * 2^23 rounds to the nearest even integer in the low bits.
// kAny: values of codes held before, which also may be -128.
template <bool kE4m3, bool kAny = false>
__device__ __forceinline__ uint2 bs8_encode8(const float2 (&x)[4], float scale, float inv) {
  const float2 s = make_float2(scale, scale), v = make_float2(inv, inv), minus = make_float2(-inv, -inv);
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float2 q = mul2(x[e], v);
#pragma unroll
    for (int c = 0; c < (kAny ? 2 : 1); ++c) q = fma2(fma2(q, s, make_float2(-x[e].x, -x[e].y)), minus, q);
    if (kE4m3) {
      w[e] = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
    } else {
      float2 r = add2(q, make_float2(12582912.f, 12582912.f));
      if (kAny) r = make_float2(fmaxf(r.x, 12582785.f), fmaxf(r.y, 12582785.f));
      w[e] = __byte_perm(__float_as_uint(r.x), __float_as_uint(r.y), 0x0040);
    }
  }
  return make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
}
__device__ __forceinline__ bool bs8_has_inverse(float scale) { return scale > 7.9e-31f && scale < 1e30f; }

template <bool kE4m3>
__device__ __forceinline__ void bs8_decode8(uint2 u, float (&x)[8]) {
  const uint32_t w[2] = {u.x, u.y};
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = bs8_decode<kE4m3>((w[e >> 2] >> (8 * (e & 3))) & 0xFFu);
}

}  // namespace pkv
