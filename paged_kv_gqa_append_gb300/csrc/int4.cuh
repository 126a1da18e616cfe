// 4-bit pages: the block of a (page, KV head) and the codes of a row.
//
//   scale = bf16((hi / 2 - lo / 2) / 7.5) (0 below 2^-126),  inv = 2 / scale
//   code  = round-half-even((x / 2 - lo / 2) * inv),  value = lo + code * scale
//
// in IEEE fp32, lo and hi the row's smallest and largest value.  The halves keep
// rows that reach from one end of bf16 to the other from overflowing.
//
// A block holds K and V in the order of the matrix instructions' fragments
// (int4_decode.cu): lane (g, t) = 4 g + t of a warp takes 16 bytes of K -- 16 dims
// from 16 t on of slots g and g + 8 -- and 16 of V -- 8 dims from 8 g on of slots 2 t,
// 2 t + 1, 2 t + 8, 2 t + 9 --, and 16 bytes of scales, of slots g and g + 8 of both.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "pkv.h"
#include "ptx.cuh"

namespace pkv {

constexpr int kI4BlockBytes = PKV_I4_BLOCK_BYTES;  // 1152
constexpr int kI4PageBytes = PKV_I4_PAGE_BYTES;    // 9216
constexpr int kI4V = 512, kI4Scales = 1024;        // where V and the scales begin

// Byte of four dims' codes, dims 4 e .. 4 e + 3 (e < 16) of slot r.
__device__ __forceinline__ int i4_k_at(int r, int e) { return 16 * (4 * (r & 7) + (e >> 2)) + 8 * (r >> 3) + 2 * (e & 3); }
__device__ __forceinline__ int i4_v_at(int r, int e) {
  return kI4V + 16 * (4 * (e >> 1) + ((r & 7) >> 1)) + 8 * (r >> 3) + 4 * (e & 1) + 2 * (r & 1);
}
// Byte of a row's (scale, minimum).
__device__ __forceinline__ int i4_scale_at(int r, int kv) { return kI4Scales + 16 * (r & 7) + 8 * kv + 4 * (r >> 3); }

// A row's scale and what multiplies (x / 2 - lo / 2), of bf16 lo and hi as floats; a row that is
// not finite gets a NaN scale.
struct I4Row {
  uint32_t word;   // scale and minimum, as stored
  float half, inv;  // lo / 2, 2 / scale (0: all codes are 0)
};
__device__ __forceinline__ I4Row i4_row(float lo, float hi) {
  I4Row r;
  r.half = 0.5f * lo;
  const float range = __fsub_rn(0.5f * hi, r.half);
  if (!(range < INFINITY)) {  // infinities and NaN
    r.word = 0x7FC07FC0u;
    r.half = r.inv = 0.f;
    return r;
  }
  const uint32_t bits = __bfloat16_as_ushort(__float2bfloat16_rn(__fdiv_rn(range, 7.5f)));
  const float scale = __uint_as_float(bits << 16);
  const bool flat = scale < 0x1p-126f;
  r.word = (flat ? 0u : bits) | (__float_as_uint(lo) & 0xFFFF0000u);
  r.inv = flat ? 0.f : __fdiv_rn(2.f, scale);
  return r;
}

// The codes of four dims, the first in the lowest bits.  The quotient is at most 15.04
// (the rounding of the scale), so that no code passes 15; adding 1.5 2^23 rounds to the
// nearest even whole number in the lowest bits.  (x of a row with inv = 0 may be anything.)
__device__ __forceinline__ uint32_t i4_codes4(const float (&x)[4], const I4Row& r) {
  uint32_t c = 0;
  if (r.inv == 0.f) return c;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float y = __fmul_rn(__fmaf_rn(x[e], 0.5f, -r.half), r.inv);
    c |= (__float_as_uint(__fadd_rn(y, 12582912.f)) & 15u) << (4 * e);
  }
  return c;
}

}  // namespace pkv
