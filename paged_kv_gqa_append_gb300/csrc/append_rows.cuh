// What the appends of ragged rows into quantised pages share (bs8_append.cu,
// int4_append.cu): where a row goes, the runs of rows that fall into one page, the
// rotation of K and q, and how the rows are shared out.
//
// A CTA of 16 warps (8 heads x {K, V}) looks at `chunk` consecutive tokens and
// handles the runs that begin among them; a warp holds its head's K or V rows of a
// run, 16 x 64 values, in registers: a row over 8 lanes, each with four dims and
// their four rotation partners, four rows per step.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "append_place.cuh"
#include "pkv.h"
#include "ptx.cuh"

namespace pkv {

constexpr int kAppendWarps = 16;
constexpr int kRow = PKV_HEAD_DIM;
constexpr int kChunkMany = 16;
// By chunks: 16 tokens a sequence or more, and at least 3 per SM in all; or 4 and 20.
// With less there are few runs, and each finds a CTA at once if every token has one,
// while a chunk's runs follow one another: 16 of one token, as beside a prompt, take 25
// us (300 x 1 and a prompt of 1600: 20, 32).  By tokens and by chunks (us): 316 tokens of
// six sequences 5.6, 6.9; 1029 of four 10.2, 5.9; 38 x 16 7.8, 5.3; 57 x 8 6.9, 6.1; 512
// x 8 40, 16; 114 x 4 7.0, 9.3; 1024 x 4 43, 21; 400 x 2 12, 17; 1000 x 2 28, 26; 1000 x 1
// 14, 25; 3000 x 1 and a prompt of 14000 182, 60.
constexpr int kManyPerSequence = 16, kManyTokensPerSm = 3;
constexpr int kMorePerSequence = 4, kMoreTokensPerSm = 20;
inline int append_chunk_tokens(int T, int num_seqs, int sms) {
  const bool many = (T / num_seqs >= kManyPerSequence && T >= kManyTokensPerSm * sms) ||
                    (T / num_seqs >= kMorePerSequence && T >= kMoreTokensPerSm * sms);
  return many ? kChunkMany : 1;
}

// What an append of ragged rows is given.
struct AppendRows {
  const uint16_t *k, *v, *q_in;
  long long k_stride, v_stride, q_stride;  // elements between tokens
  const int32_t *cu_new, *seq_lens, *block_tables;
  const float *cos, *sin;                  // [max_pos][32] or null: k is taken as it is
  uint16_t* q_out;
  int* d_err;
  int T, num_seqs, bt_stride, num_pages, chunk;
  int most;  // tokens that the tables, of pages and of rotations, have room for
};

// The last sequence s with cu[s] <= t (cu ascending, n = number of sequences),
// or -1: the count of such entries among n + 1, minus 1; a result of n means
// that t lies behind the last sequence.  All lanes of a warp.
__device__ inline int find_sequence(const int32_t* __restrict__ cu, int n, int t) {
  const int lane = threadIdx.x & 31;
  int base = 0, size = n + 1;
  while (size > 0) {
    const int step = (size + 31) >> 5;
    const int at = base + (lane + 1) * step - 1;
    const bool below = at < base + size && __ldg(cu + at) <= t;
    const int full = __popc(__ballot_sync(0xffffffffu, below));
    base += full * step;
    if (step == 1) break;
    size = min(step - 1, size - full * step);
  }
  return base - 1;
}

__device__ __forceinline__ Place place_of(const AppendRows& p, int t) {
  Place a{-1, 0, t + 1, false, false, false};
  int lo = 0, hi = 0, len = 0;
  bool found = false;
  if (p.T == p.num_seqs) {  // a step of one token each, most likely: row t is sequence t's
    lo = __ldg(p.cu_new + t);
    hi = __ldg(p.cu_new + t + 1);
    len = __ldg(p.seq_lens + t);
    found = lo == t && hi == t + 1;
    a.seq = t;
  }
  if (!found) {
    a.seq = find_sequence(p.cu_new, p.num_seqs, t);
    if (a.seq >= p.num_seqs) {  // rows behind the last sequence are left alone
      a.end = p.T;
      return a;
    }
    a.live = true;
    if (a.seq < 0) return a;
    lo = __ldg(p.cu_new + a.seq);
    hi = __ldg(p.cu_new + a.seq + 1);
    len = __ldg(p.seq_lens + a.seq);
  }
  a.live = true;
  set_place(a, t, p.T, lo, hi, len, p.most);
  return a;
}

// Four dims and their partners rotated in place, in kv_append_rope's order of
// operations: x[0], x[1] with x[2], x[3].
__device__ __forceinline__ void rotate8(float2 (&x)[4], const float4& c4, const float4& s4) {
  const float2 c[2] = {make_float2(c4.x, c4.y), make_float2(c4.z, c4.w)};
  const float2 s[2] = {make_float2(s4.x, s4.y), make_float2(s4.z, s4.w)};
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float2 a = x[e], b = x[e + 2];
    // (each product and each sum rounded: mul2 with add2 would not do)
    const float2 ac = mul2(a, c[e]), bs = mul2(b, s[e]), as = mul2(a, s[e]), bc = mul2(b, c[e]);
    x[e] = make_float2(__fsub_rn(ac.x, bs.x), __fsub_rn(ac.y, bs.y));
    x[e + 2] = make_float2(__fadd_rn(as.x, bc.x), __fadd_rn(as.y, bc.y));
  }
}

// dims 4 j .. 4 j + 3 and 32 + 4 j .. of a row
__device__ __forceinline__ uint4 load_halves(const uint16_t* row, int j) {
  const uint2 a = __ldcs(reinterpret_cast<const uint2*>(row + 4 * j));
  const uint2 b = __ldcs(reinterpret_cast<const uint2*>(row + 32 + 4 * j));
  return make_uint4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void widen8(const uint4& u, float2 (&x)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = make_float2(bf16lo_to_f32(w[e]), bf16hi_to_f32(w[e]));
}
__device__ __forceinline__ uint4 narrow8(const float2 (&x)[4]) {
  return make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y), pack_bf16x2(x[2].x, x[2].y),
                    pack_bf16x2(x[3].x, x[3].y));
}

// K and V of the runs that begin in the CTA's chunk of tokens.
// append(t, pos, n, entry, kv, head): the run's first row and position, its length and table entry.
template <class Append>
__device__ __forceinline__ void append_chunk(const AppendRows& p, int t0, int t1, const Append& append) {
  const int warp = threadIdx.x >> 5;
  Place a = place_of(p, t0);
  for (int t = t0; t < t1;) {
    if (!a.live) break;
    if (!a.ok) {
      if (threadIdx.x == 0) report_error(p.d_err, PKV_ERR_DEVICE_INDEX);
      t = max(t + 1, min(a.end, t1));
      if (t < t1) a = place_of(p, t);
      continue;
    }
    const int slot = a.pos % PKV_PAGE_TOKENS;
    const int n = min(PKV_PAGE_TOKENS - slot, a.end - t);
    if (a.first || slot == 0)  // else it began in an earlier chunk
      append(t, a.pos, n, p.block_tables + (size_t)a.seq * p.bt_stride + a.pos / PKV_PAGE_TOKENS, warp >> 3, warp & 7);
    t += n;
    if (t < a.end) {  // the same sequence's next page
      a.pos += n;
      a.first = false;
    } else if (t < t1) {
      a = place_of(p, t);
    }
  }
}

// q of the chunk's tokens, four heads per warp and step: one token by 8 warps,
// or one token by each warp, whose rows are loaded before its place is known.
__device__ __forceinline__ void rotate_chunk(const AppendRows& p, int t0, int t1) {
  static_assert(kChunkMany == kAppendWarps && kAppendWarps >= PKV_NUM_Q_HEADS / 4, "tokens and q heads over the warps");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane >> 3, j = lane & 7;
  const bool many = p.chunk > 1;
  const int t = many ? t0 + warp : t0;
  if (t >= t1 || (!many && warp >= PKV_NUM_Q_HEADS / 4)) return;
  constexpr int kSteps = PKV_NUM_Q_HEADS / 4;
  uint4 raw[kSteps];
  const uint16_t* src = p.q_in + (long long)t * p.q_stride;
#pragma unroll
  for (int u = 0; u < kSteps; ++u)
    if (many || u == 0) raw[u] = load_halves(src + ((many ? 4 * u : 4 * warp) + sub) * kRow, j);
  const Place a = place_of(p, t);
  if (!a.live) return;
  bool ok = a.ok;
  float4 c = make_float4(0.f, 0.f, 0.f, 0.f), s = c;
  if (ok) {
    const int page = __ldg(p.block_tables + (size_t)a.seq * p.bt_stride + a.pos / PKV_PAGE_TOKENS);
    const size_t row = (size_t)a.pos * PKV_ROPE_PAIRS + 4 * j;
    c = __ldg(reinterpret_cast<const float4*>(p.cos + row));
    s = __ldg(reinterpret_cast<const float4*>(p.sin + row));
    ok = page >= 0 && page < p.num_pages;
  }
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    if (!many && u) break;
    uint16_t* dst = p.q_out + ((size_t)t * PKV_NUM_Q_HEADS + (many ? 4 * u : 4 * warp) + sub) * kRow;
    uint4 res = make_uint4(0, 0, 0, 0);
    if (ok) {
      float2 x[4];
      widen8(raw[u], x);
      rotate8(x, c, s);
      res = narrow8(x);
    }
    *reinterpret_cast<uint2*>(dst + 4 * j) = make_uint2(res.x, res.y);
    *reinterpret_cast<uint2*>(dst + 32 + 4 * j) = make_uint2(res.z, res.w);
  }
}

}  // namespace pkv
