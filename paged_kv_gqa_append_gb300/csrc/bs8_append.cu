// RoPE + append into pages of 8-bit codes with one scale per block (16 slots
// of one page, K or V, and KV head), and the pages read back as bf16, for
// sm_103a.
//
// A block's scale covers every token in it, so the tokens that go to the same
// page are handled together: the unit of work is a run -- the new tokens of
// one sequence that fall into one page -- and its K or V rows of one head,
// 16 x 64 values in the registers of one warp (a row over 8 lanes, each with
// four dims and their four rotation partners; four rows per step).  A run that
// starts at slot 0 sets the block's scale to amax / top; a later one keeps the
// larger of that and the scale found, and when the scale grows the codes held by
// the earlier slots are decoded under the old scale and encoded under the new
// one.  The earlier slots are read only then.
//
// A CTA of 16 warps (8 heads x {K, V}) looks at `chunk` consecutive tokens
// and handles the runs that begin among them: one token per CTA for decode
// steps and few tokens, 16 per CTA when sequences bring several tokens each, so
// that most begin no run.  The chunk's q heads are rotated by another CTA, so
// that neither waits for the other.
//
// Bound: memory, 3 KiB per token for K and V, and 8 KiB for q.  Codes without a
// division per value (bs8.cuh), rotations without shuffles and products by pairs
// took 14400 tokens of eight prompts from 65 us to 31 us (K and V alone 13 us).  A step of few tokens is latency: the
// token's place (without a search where a step has one token per sequence; else
// one round of a 32-way search for up to 1023 sequences), then the table entry,
// the rows and the rotations together, then the old scale.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "append_place.cuh"
#include "bs8.cuh"
#include "internal.h"
#include "pkv.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 16;
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

struct Bs8AppendParams {
  const uint16_t *k, *v, *q_in;
  long long k_stride, v_stride, q_stride;  // elements between tokens
  const int32_t *cu_new, *seq_lens, *block_tables;
  const float *cos, *sin;                  // [max_pos][32] or null: k is taken as it is
  uint16_t* q_out;
  uint8_t* pool;
  float* scales;
  int* d_err;
  int T, num_seqs, bt_stride, num_pages, chunk;
  int most;  // tokens that the tables, of pages and of rotations, have room for
};

// The last sequence s with cu[s] <= t (cu ascending, n = number of sequences),
// or -1: the count of such entries among n + 1, minus 1; a result of n means
// that t lies behind the last sequence.  All lanes of a warp.
__device__ int find_sequence(const int32_t* __restrict__ cu, int n, int t) {
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

__device__ __forceinline__ Place place_of(const Bs8AppendParams& p, int t) {
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

// K (kv = 0) or V rows of one head of a run: slots [slot, slot + n) of the page
// that `entry` of the block table names.  The page is needed last: its entry, the
// rows and the rotations are under way together.
template <bool kE4m3>
__device__ __forceinline__ void append_run(const Bs8AppendParams& p, int t, int pos, int n, const int32_t* entry,
                                           int kv, int head) {
  const int lane = threadIdx.x & 31, sub = lane >> 3, j = lane & 7;
  const int slot = pos % PKV_PAGE_TOKENS;
  const uint16_t* src = kv ? p.v : p.k;
  const long long stride = kv ? p.v_stride : p.k_stride;
  const int page = __ldg(entry);

  uint4 raw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * i + sub - slot;  // row of the run
    raw[i] = make_uint4(0, 0, 0, 0);
    if (r >= 0 && r < n) raw[i] = load_halves(src + (long long)(t + r) * stride + head * kRow, j);
  }
  const bool turn = kv == 0 && p.cos;
  float4 c[4], s[4];  // rows beside the run (of zeros) take its first entry
  if (turn) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * i + sub - slot;
      const size_t row = (size_t)(r >= 0 && r < n ? pos + r : pos) * PKV_ROPE_PAIRS + 4 * j;
      c[i] = __ldg(reinterpret_cast<const float4*>(p.cos + row));
      s[i] = __ldg(reinterpret_cast<const float4*>(p.sin + row));
    }
  }
  if (page < 0 || page >= p.num_pages) {
    if (threadIdx.x == 0) report_error(p.d_err, PKV_ERR_DEVICE_INDEX);
    return;
  }
  uint8_t* block = p.pool + ((size_t)page * 2 + kv) * (PKV_NUM_KV_HEADS * kBs8BlockBytes) +
                   (size_t)head * kBs8BlockBytes;
  float* scale = p.scales + ((size_t)page * 2 + kv) * PKV_NUM_KV_HEADS + head;
  float old = 0.f;
  if (slot && lane == 0) old = *scale;
  if (turn) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (4 * i + 4 <= slot || 4 * i >= slot + n) continue;  // none of the warp's four rows
      float2 x[4];
      widen8(raw[i], x);
      rotate8(x, c[i], s[i]);
      raw[i] = narrow8(x);
    }
  }
  // largest |x| of the run: bf16 magnitudes order as their bits
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) top = __vmaxu2(top, w[e] & 0x7FFF7FFFu);
  }
  const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, max(top & 0xFFFF0000u, top << 16)));
  old = __shfl_sync(0xffffffffu, old, 0);
  const float fresh = __fdiv_rn(amax, kE4m3 ? 448.f : 127.f);
  // (a NaN among the rows becomes the block's scale and stays it, so that it shows)
  const bool grown = slot > 0 && (fresh > old || fresh != fresh);
  const float now = slot == 0 || grown ? fresh : old;
  if (lane == 0 && (slot == 0 || grown)) *scale = now;
  const auto write = [&](int r, const uint2& codes) {
    uint32_t* to = reinterpret_cast<uint32_t*>(block + r * kRow + 4 * j);
    to[0] = codes.x;
    to[8] = codes.y;
  };
  const bool by_inverse = bs8_has_inverse(now);
  const float inv = by_inverse ? __frcp_rn(now) : 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * i + sub;
    if (4 * i + 4 <= slot || 4 * i >= slot + n) continue;
    float2 x[4];
    widen8(raw[i], x);
    const uint2 codes = by_inverse ? bs8_encode8<kE4m3>(x, now, inv)
                                   : bs8_encode8_exact<kE4m3>(x[0].x, x[0].y, x[1].x, x[1].y, x[2].x, x[2].y, x[3].x,
                                                              x[3].y, now);
    if (r >= slot && r < slot + n) write(r, codes);
  }
  if (grown) {  // the earlier rows' codes, all under way together
    uint2 held[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t* from = reinterpret_cast<const uint32_t*>(block + (4 * i + sub) * kRow + 4 * j);
      held[i] = make_uint2(0, 0);
      if (4 * i + sub < slot) held[i] = make_uint2(from[0], from[8]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (4 * i >= slot) break;
      float x[8];
      bs8_decode8<kE4m3>(held[i], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(x[e], old);
      const float2 pairs[4] = {make_float2(x[0], x[1]), make_float2(x[2], x[3]), make_float2(x[4], x[5]),
                               make_float2(x[6], x[7])};
      const uint2 codes = by_inverse ? bs8_encode8<kE4m3, true>(pairs, now, inv)
                                     : bs8_encode8_exact<kE4m3>(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], now);
      if (4 * i + sub < slot) write(4 * i + sub, codes);
    }
  }
}

// K and V of the runs that begin in the CTA's chunk of tokens.
template <bool kE4m3>
__device__ __forceinline__ void append_chunk(const Bs8AppendParams& p, int t0, int t1) {
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
      append_run<kE4m3>(p, t, a.pos, n, p.block_tables + (size_t)a.seq * p.bt_stride + a.pos / PKV_PAGE_TOKENS,
                        warp >> 3, warp & 7);
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
__device__ __forceinline__ void rotate_chunk(const Bs8AppendParams& p, int t0, int t1) {
  static_assert(kChunkMany == kWarps && kWarps >= PKV_NUM_Q_HEADS / 4, "tokens and q heads over the warps");
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

template <bool kE4m3>
__global__ void __launch_bounds__(kWarps * 32, 2) bs8_append_kernel(const Bs8AppendParams p) {
  pdl_wait();
  pdl_launch_dependents();
  // with q, the two kinds of CTA take turns, so that both kinds are on every SM
  const int kinds = p.q_in ? 2 : 1;
  const int t0 = blockIdx.x / kinds * p.chunk, t1 = min(p.T, t0 + p.chunk);
  if (blockIdx.x % kinds == 0)
    append_chunk<kE4m3>(p, t0, t1);
  else
    rotate_chunk(p, t0, t1);
}

// out[i] = the page page_ids[i] as bf16: code * scale, rounded once.  One CTA
// per page, 16 codes per thread and step; bound by memory (16 KiB read,
// 32 KiB written per page) and, for the usual few hundred pages, by its start and
// end: 906 pages take 9.8 us with 512 threads and 11.9 us with 256, 32 pages 2.6
// and 2.4 us, so that a grid of one CTA per SM at most takes 256.
template <bool kE4m3, int kReadThreads>
__global__ void __launch_bounds__(kReadThreads) bs8_read_kernel(const uint8_t* __restrict__ pool,
                                                       const float* __restrict__ scales, int num_pages,
                                                       const int32_t* __restrict__ page_ids,
                                                       uint16_t* __restrict__ out, int* d_err) {
  pdl_wait();
  pdl_launch_dependents();
  const int page = __ldg(page_ids + blockIdx.x);
  const bool ok = page >= 0 && page < num_pages;
  if (!ok && threadIdx.x == 0) report_error(d_err, PKV_ERR_DEVICE_INDEX);
  uint16_t* dst = out + (size_t)blockIdx.x * kBs8PageBytes;
  const uint8_t* src = pool + (size_t)(ok ? page : 0) * kBs8PageBytes;
  constexpr int kSteps = kBs8PageBytes / (kReadThreads * 16);
  uint4 raw[kSteps];
  float scale[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int at = (i * kReadThreads + threadIdx.x) * 16;
    raw[i] = make_uint4(0, 0, 0, 0);
    scale[i] = 0.f;
    if (ok) {
      raw[i] = __ldcs(reinterpret_cast<const uint4*>(src + at));
      scale[i] = __ldg(scales + (size_t)page * 2 * PKV_NUM_KV_HEADS + at / kBs8BlockBytes);
    }
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int at = (i * kReadThreads + threadIdx.x) * 16;
    const uint2 half[2] = {make_uint2(raw[i].x, raw[i].y), make_uint2(raw[i].z, raw[i].w)};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float x[8];
      bs8_decode8<kE4m3>(half[h], x);
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = pack_bf16x2(__fmul_rn(x[2 * e], scale[i]), __fmul_rn(x[2 * e + 1], scale[i]));
      *reinterpret_cast<uint4*>(dst + at + 8 * h) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int kv_append_rope_bs8(const void* k, long long k_stride, const void* v, long long v_stride,
                                  const int32_t* cu_new, const int32_t* seq_lens, int T,
                                  const int32_t* block_tables, int num_seqs, int bt_row_stride,
                                  int max_blocks, void* kv_pool, float* kv_scales, int num_pages,
                                  int code_type, const float* rope_cos, const float* rope_sin, int max_pos,
                                  const void* q_in, long long q_stride, void* q_out, int* d_err,
                                  void* stream) {
  if (T < 0 || num_seqs < 1 || max_blocks < 1 || bt_row_stride < max_blocks || num_pages < 1 ||
      (code_type != PKV_BS8_INT8 && code_type != PKV_BS8_E4M3))
    return PKV_ERR_INVALID_ARGUMENT;
  if ((rope_cos == nullptr) != (rope_sin == nullptr) || (q_in == nullptr) != (q_out == nullptr) ||
      (q_in && !rope_cos) || (rope_cos && max_pos < 1))
    return PKV_ERR_INVALID_ARGUMENT;
  if (T == 0) return PKV_OK;
  if (!k || !v || !cu_new || !seq_lens || !block_tables || !kv_pool || !kv_scales)
    return PKV_ERR_INVALID_ARGUMENT;
  if (k_stride < PKV_NUM_KV_HEADS * PKV_HEAD_DIM || v_stride < PKV_NUM_KV_HEADS * PKV_HEAD_DIM ||
      (q_in && q_stride < PKV_NUM_Q_HEADS * PKV_HEAD_DIM))
    return PKV_ERR_INVALID_ARGUMENT;
  if (!aligned16(k) || !aligned16(v) || !aligned16(kv_pool) || !aligned16(q_in) || !aligned16(q_out) ||
      !aligned16(rope_cos) || !aligned16(rope_sin) || (k_stride & 7) || (v_stride & 7) || (q_in && (q_stride & 7)))
    return PKV_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(cu_new) | reinterpret_cast<uintptr_t>(seq_lens) |
       reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(kv_scales) |
       reinterpret_cast<uintptr_t>(d_err)) & 3u)
    return PKV_ERR_MISALIGNED;
  if (T > (1 << 29) || num_seqs > (1 << 30) || max_blocks > (1 << 26))
    return PKV_ERR_UNSUPPORTED_SHAPE;
  int dev = 0;
  const int rc = bind_stream_device(stream, &dev);
  if (rc != PKV_OK) return rc;

  Bs8AppendParams p;
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_in = static_cast<const uint16_t*>(q_in);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_stride = q_stride;
  p.cu_new = cu_new;
  p.seq_lens = seq_lens;
  p.block_tables = block_tables;
  p.cos = rope_cos;
  p.sin = rope_sin;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.pool = static_cast<uint8_t*>(kv_pool);
  p.scales = kv_scales;
  p.d_err = d_err;
  p.T = T;
  p.num_seqs = num_seqs;
  p.bt_stride = bt_row_stride;
  p.most = max_blocks * PKV_PAGE_TOKENS;
  if (rope_cos && max_pos < p.most) p.most = max_pos;
  p.num_pages = num_pages;
  const int sms = sm_count(dev);
  const bool many = (T / num_seqs >= kManyPerSequence && T >= kManyTokensPerSm * sms) ||
                    (T / num_seqs >= kMorePerSequence && T >= kMoreTokensPerSm * sms);
  p.chunk = many ? kChunkMany : 1;

  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)T + p.chunk - 1) / p.chunk) * (q_in ? 2 : 1));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(code_type == PKV_BS8_E4M3 ? cudaLaunchKernelEx(&cfg, bs8_append_kernel<true>, p)
                                               : cudaLaunchKernelEx(&cfg, bs8_append_kernel<false>, p),
                     "cudaLaunchKernelEx(append bs8)");
}

extern "C" int kv_read_bs8(const void* kv_pool, const float* kv_scales, int num_pages, int code_type,
                           const int32_t* page_ids, int count, void* out, int* d_err, void* stream) {
  if (count < 0 || num_pages < 1 || (code_type != PKV_BS8_INT8 && code_type != PKV_BS8_E4M3))
    return PKV_ERR_INVALID_ARGUMENT;
  if (count == 0) return PKV_OK;
  if (!kv_pool || !kv_scales || !page_ids || !out) return PKV_ERR_INVALID_ARGUMENT;
  if (!aligned16(kv_pool) || !aligned16(out) ||
      ((reinterpret_cast<uintptr_t>(kv_scales) | reinterpret_cast<uintptr_t>(page_ids) |
        reinterpret_cast<uintptr_t>(d_err)) & 3u))
    return PKV_ERR_MISALIGNED;
  int dev = 0;
  const int rc = bind_stream_device(stream, &dev);
  if (rc != PKV_OK) return rc;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)count);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool few = count <= sm_count(dev);
  cfg.blockDim = dim3(few ? 256 : 512);
  auto* kernel = code_type == PKV_BS8_E4M3 ? (few ? bs8_read_kernel<true, 256> : bs8_read_kernel<true, 512>)
                                           : (few ? bs8_read_kernel<false, 256> : bs8_read_kernel<false, 512>);
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, static_cast<const uint8_t*>(kv_pool), kv_scales, num_pages, page_ids,
                                        static_cast<uint16_t*>(out), d_err),
                     "cudaLaunchKernelEx(read bs8)");
}
