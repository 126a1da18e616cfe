// RoPE + append into pages of 8-bit codes with one scale per block (16 slots
// of one page, K or V, and KV head), and the pages read back as bf16, for
// sm_103a.
//
// A block's scale covers every token in it, so the tokens that go to the same
// page are handled together: the unit of work is a run -- the new tokens of
// one sequence that fall into one page -- and its K or V rows of one head,
// 16 x 64 values in the registers of one warp (a row over 8 lanes of 8 dims,
// four rows per step).  A run that starts at slot 0 sets the block's scale to
// amax / top; a later one keeps the larger of that and the scale found, and
// when the scale grows the codes held by the earlier slots are decoded under
// the old scale and encoded under the new one.  The earlier slots are read
// only then.
//
// A CTA of 16 warps (8 heads x {K, V}) looks at `chunk` consecutive tokens
// and handles the runs that begin among them: one token per CTA for decode
// steps, 16 per CTA when sequences bring 16 tokens or more on average, where
// most tokens begin no run.  The chunk's q heads are rotated by all warps.
//
// Bound: memory, 3 KiB per token for K and V, and 8 KiB for q.  A step of few
// tokens is latency: the sequence search (one round of a 32-way search for up
// to 1023 sequences), the table entry, the rows, the old scale.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bs8.cuh"
#include "internal.h"
#include "pkv.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 16;
constexpr int kRow = PKV_HEAD_DIM;
constexpr int kChunkMany = 16;

struct Bs8AppendParams {
  const uint16_t *k, *v, *q_in;
  long long k_stride, v_stride, q_stride;  // elements between tokens
  const int32_t *cu_new, *seq_lens, *block_tables;
  const float *cos, *sin;                  // [max_pos][32] or null: k is taken as it is
  uint16_t* q_out;
  uint8_t* pool;
  float* scales;
  int* d_err;
  int T, num_seqs, bt_stride, max_blocks, num_pages, max_pos, chunk;
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

// A token's place: its sequence and position; ok only if both can be used.
struct Place {
  int seq, pos, end;  // end: the row behind the sequence's last new token
  bool live, ok;      // live: the token belongs to a sequence
};

__device__ __forceinline__ Place place_of(const Bs8AppendParams& p, int t) {
  Place a{-1, 0, t + 1, false, false};
  a.seq = find_sequence(p.cu_new, p.num_seqs, t);
  if (a.seq >= p.num_seqs) {  // rows behind the last sequence are left alone
    a.end = p.T;
    return a;
  }
  a.live = true;
  if (a.seq < 0) return a;
  const int lo = __ldg(p.cu_new + a.seq), hi = __ldg(p.cu_new + a.seq + 1);
  const int len = __ldg(p.seq_lens + a.seq);
  const int fresh = hi - lo;
  if (hi <= t || hi > p.T || lo < 0) return a;  // not ascending, or beyond the rows given
  a.end = hi;
  if (len < fresh || len > (long long)p.max_blocks * PKV_PAGE_TOKENS || (p.cos && len > p.max_pos)) return a;
  a.pos = len - fresh + (t - lo);
  a.ok = true;
  return a;
}

// K (kv = 0) or V rows of one head of a run: slots [slot, slot + n) of the page.
template <bool kE4m3>
__device__ __forceinline__ void append_run(const Bs8AppendParams& p, int t, int pos, int n, int page, int kv,
                                           int head) {
  const int lane = threadIdx.x & 31, sub = lane >> 3, j = lane & 7;
  const int slot = pos % PKV_PAGE_TOKENS;
  const uint16_t* src = kv ? p.v : p.k;
  const long long stride = kv ? p.v_stride : p.k_stride;
  uint8_t* block = p.pool + ((size_t)page * 2 + kv) * (PKV_NUM_KV_HEADS * kBs8BlockBytes) +
                   (size_t)head * kBs8BlockBytes;
  float* scale = p.scales + ((size_t)page * 2 + kv) * PKV_NUM_KV_HEADS + head;

  uint4 raw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * i + sub - slot;  // row of the run
    raw[i] = make_uint4(0, 0, 0, 0);
    if (r >= 0 && r < n)
      raw[i] = __ldcs(reinterpret_cast<const uint4*>(src + (long long)(t + r) * stride + head * kRow + 8 * j));
  }
  float old = 0.f;
  if (slot && lane == 0) old = *scale;
  old = __shfl_sync(0xffffffffu, old, 0);
  if (kv == 0 && p.cos) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * i + sub - slot;
      const uint32_t mine[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      uint32_t res[4];
      alignas(16) float c[8], s[8];
      const size_t row = (size_t)(r >= 0 && r < n ? pos + r : pos) * PKV_ROPE_PAIRS + 8 * (j & 3);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        *reinterpret_cast<float4*>(c + 4 * h) = __ldg(reinterpret_cast<const float4*>(p.cos + row) + h);
        *reinterpret_cast<float4*>(s + 4 * h) = __ldg(reinterpret_cast<const float4*>(p.sin + row) + h);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, mine[e], 4);
        const uint32_t a = j < 4 ? mine[e] : other, b = j < 4 ? other : mine[e];
        uint16_t lo0, lo1, hi0, hi1;
        rope_pair((uint16_t)a, (uint16_t)b, c[2 * e], s[2 * e], lo0, lo1);
        rope_pair((uint16_t)(a >> 16), (uint16_t)(b >> 16), c[2 * e + 1], s[2 * e + 1], hi0, hi1);
        res[e] = j < 4 ? (uint32_t)lo0 | ((uint32_t)hi0 << 16) : (uint32_t)lo1 | ((uint32_t)hi1 << 16);
      }
      raw[i] = make_uint4(res[0], res[1], res[2], res[3]);
    }
  }
  // largest |x| of the run: bf16 magnitudes order as their bits
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max(top, max((w[e] << 16) & 0x7FFF0000u, w[e] & 0x7FFF0000u));
  }
  const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, top));
  const float fresh = __fdiv_rn(amax, kE4m3 ? 448.f : 127.f);
  const bool grown = slot > 0 && fresh > old;
  const float now = slot == 0 || grown ? fresh : old;
  if (lane == 0 && (slot == 0 || grown)) *scale = now;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * i + sub;
    uint2* at = reinterpret_cast<uint2*>(block + r * kRow + 8 * j);
    float x[8];
    if (r >= slot && r < slot + n) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = bf16lo_to_f32(w[e]);
        x[2 * e + 1] = bf16hi_to_f32(w[e]);
      }
      *at = bs8_encode8<kE4m3>(x, now);
    } else if (r < slot && grown) {
      bs8_decode8<kE4m3>(*at, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(x[e], old);
      *at = bs8_encode8<kE4m3>(x, now);
    }
  }
}

template <bool kE4m3>
__global__ void __launch_bounds__(kWarps * 32) bs8_append_kernel(const Bs8AppendParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * p.chunk, t1 = min(p.T, t0 + p.chunk);

  // K and V of the runs that begin in the chunk
  for (int t = t0; t < t1;) {
    const Place a = place_of(p, t);
    if (!a.live) break;
    if (!a.ok) {
      if (threadIdx.x == 0) report_error(p.d_err, PKV_ERR_DEVICE_INDEX);
      t = max(t + 1, min(a.end, t1));
      continue;
    }
    const int slot = a.pos % PKV_PAGE_TOKENS;
    const int n = min(PKV_PAGE_TOKENS - slot, a.end - t);
    if (t == __ldg(p.cu_new + a.seq) || slot == 0) {
      const int page = __ldg(p.block_tables + (size_t)a.seq * p.bt_stride + a.pos / PKV_PAGE_TOKENS);
      if (page >= 0 && page < p.num_pages)
        append_run<kE4m3>(p, t, a.pos, n, page, warp >> 3, warp & 7);
      else if (threadIdx.x == 0)
        report_error(p.d_err, PKV_ERR_DEVICE_INDEX);
    }
    t += n;
  }

  // q of the chunk's tokens, two heads per warp and step, 16 lanes of 4 dims
  // each: one token by all warps, or one token by each warp
  if (p.q_in == nullptr) return;
  const int t = p.chunk == 1 ? t0 : t0 + warp;
  if (t >= t1) return;
  const Place a = place_of(p, t);
  if (!a.live) return;
  bool ok = a.ok;
  if (ok) {
    const int page = __ldg(p.block_tables + (size_t)a.seq * p.bt_stride + a.pos / PKV_PAGE_TOKENS);
    ok = page >= 0 && page < p.num_pages;
  }
  const int l16 = lane & 15;
  const bool first = l16 < 8;  // dims 0..31: the pairs' first halves
  float4 c = make_float4(0.f, 0.f, 0.f, 0.f), s = c;
  if (ok) {
    const size_t row = (size_t)a.pos * PKV_ROPE_PAIRS + 4 * (l16 & 7);
    c = __ldg(reinterpret_cast<const float4*>(p.cos + row));
    s = __ldg(reinterpret_cast<const float4*>(p.sin + row));
  }
  const int u0 = p.chunk == 1 ? warp : 0, u1 = p.chunk == 1 ? warp + 1 : kWarps;
  static_assert(kWarps * 2 == PKV_NUM_Q_HEADS && kChunkMany == kWarps, "q heads and tokens over the warps");
#pragma unroll 4
  for (int u = u0; u < u1; ++u) {
    const int head = 2 * u + (lane >> 4);
    uint2 res = make_uint2(0, 0);
    if (ok) {
      const uint2 x = *reinterpret_cast<const uint2*>(p.q_in + (long long)t * p.q_stride + head * kRow + 4 * l16);
      const uint32_t mine[2] = {x.x, x.y};
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
      uint32_t w[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, mine[e], 8);
        const uint32_t x0 = first ? mine[e] : other, x1 = first ? other : mine[e];
        uint16_t lo0, lo1, hi0, hi1;
        rope_pair((uint16_t)x0, (uint16_t)x1, cc[2 * e], ss[2 * e], lo0, lo1);
        rope_pair((uint16_t)(x0 >> 16), (uint16_t)(x1 >> 16), cc[2 * e + 1], ss[2 * e + 1], hi0, hi1);
        w[e] = first ? (uint32_t)lo0 | ((uint32_t)hi0 << 16) : (uint32_t)lo1 | ((uint32_t)hi1 << 16);
      }
      res = make_uint2(w[0], w[1]);
    }
    *reinterpret_cast<uint2*>(p.q_out + ((size_t)t * PKV_NUM_Q_HEADS + head) * kRow + 4 * l16) = res;
  }
}

// out[i] = the page page_ids[i] as bf16: code * scale, rounded once.  One CTA
// per page, 16 codes per thread and step; bound by memory (16 KiB read,
// 32 KiB written per page).
template <bool kE4m3>
__global__ void __launch_bounds__(256) bs8_read_kernel(const uint8_t* __restrict__ pool,
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
  constexpr int kSteps = kBs8PageBytes / (256 * 16);
  uint4 raw[kSteps];
  float scale[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int at = (i * 256 + threadIdx.x) * 16;
    raw[i] = make_uint4(0, 0, 0, 0);
    scale[i] = 0.f;
    if (ok) {
      raw[i] = __ldcs(reinterpret_cast<const uint4*>(src + at));
      scale[i] = __ldg(scales + (size_t)page * 2 * PKV_NUM_KV_HEADS + at / kBs8BlockBytes);
    }
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int at = (i * 256 + threadIdx.x) * 16;
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
  if (T > (1 << 30) || num_seqs > (1 << 30) || max_blocks > (1 << 26))
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
  p.max_blocks = max_blocks;
  p.num_pages = num_pages;
  p.max_pos = max_pos;
  p.chunk = T / num_seqs >= kChunkMany ? kChunkMany : 1;

  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)T + p.chunk - 1) / p.chunk));
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
  cfg.blockDim = dim3(256);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const uint8_t* pool = static_cast<const uint8_t*>(kv_pool);
  uint16_t* dst = static_cast<uint16_t*>(out);
  return cuda_status(
      code_type == PKV_BS8_E4M3
          ? cudaLaunchKernelEx(&cfg, bs8_read_kernel<true>, pool, kv_scales, num_pages, page_ids, dst, d_err)
          : cudaLaunchKernelEx(&cfg, bs8_read_kernel<false>, pool, kv_scales, num_pages, page_ids, dst, d_err),
      "cudaLaunchKernelEx(read bs8)");
}
