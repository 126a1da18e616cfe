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

// eight bytes in two words
template <bool kE4m3>
__device__ __forceinline__ uint2 bs8_encode8(const float (&x)[8], float scale) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e >> 2] |= bs8_encode<kE4m3>(x[e], scale) << (8 * (e & 3));
  return make_uint2(w[0], w[1]);
}

template <bool kE4m3>
__device__ __forceinline__ void bs8_decode8(uint2 u, float (&x)[8]) {
  const uint32_t w[2] = {u.x, u.y};
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = bs8_decode<kE4m3>((w[e >> 2] >> (8 * (e & 3))) & 0xFFu);
}

}  // namespace pkv
