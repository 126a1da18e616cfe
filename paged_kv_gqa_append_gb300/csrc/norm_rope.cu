// RMS norm of the q and k heads and their rotation in one pass, optionally
// with the append of k and v into bf16 pages, for sm_103a.
//
// For a head row x of 64 bf16 values and weights w (no norm without w):
//   y_d = x_d * r * w_d,  r = 1 / sqrt(mean(x^2) + eps)        (fp32)
// then the first 2 P dims are rotated by the table row of the token's
// position, P = rope_pairs: pairs (i, i + P), or (2 i, 2 i + 1) when
// interleaved,
//   (a, b) -> (a c_i - b s_i, a s_i + b c_i)
// each operation rounded to nearest in fp32, and every dim is rounded to bf16
// once, at the end.  Without a norm and with P = 32 in the half layout these
// are exactly kv_append_rope's operations, and its bytes.
//
// Work: one warp per token and part -- two parts of 16 q heads and one of the
// k (and v) heads, so a part is 16 head rows = four 512-byte loads that are
// all in flight before anything else is read.  A row is spread over 8 lanes
// of 8 dims (one 16-byte load each): the sum of squares is three shuffles,
// and the half layout's partner dims sit at the same place of lane +-P/8 when
// P is a multiple of 8.  Other P go through a row buffer in shared memory;
// interleaved pairs never leave their lane.
//
// Bound: memory.  A token moves 12 KiB (32 + 8 + 8 rows read and written)
// and one table row.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "pkv.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 12;       // a multiple of 1, 2 and 3: a CTA holds whole tokens
constexpr int kGroups = 4;       // 4-row groups of a part
constexpr int kRow = PKV_HEAD_DIM;

enum Layout { kHalfAligned = 0, kHalfAny = 1, kInterleaved = 2 };

struct NormRopeParams {
  const uint16_t *q, *k, *v;             // token rows of [heads][64] bf16
  long long q_stride, k_stride, v_stride;  // elements between tokens
  const void *q_weight, *k_weight;       // [64] or null
  const float *cos, *sin;                // [max_pos][pairs]
  const int32_t *positions, *token_seq, *block_tables;
  uint16_t *q_out, *k_out, *pool;        // [T][32][64], [T][8][64] or null, pages or null
  int* d_err;
  float eps;
  int weight_f32, T, pairs, max_pos, num_seqs, bt_stride, max_blocks, num_pages;
  int q_parts;                           // parts of q heads per token: 2, or 0 without q
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16lo_to_f32(w[i]);
    x[2 * i + 1] = bf16hi_to_f32(w[i]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

template <int kLayout>
__global__ void __launch_bounds__(kWarps * 32) norm_rope_kernel(const NormRopeParams p) {
  __shared__ float rows[kLayout == kHalfAny ? kWarps : 1][4][kRow + 4];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane >> 3, j = lane & 7;  // row of a group, and which 8 dims of it
  const int parts = p.q_parts + 1;
  const long long unit = (long long)blockIdx.x * kWarps + warp;
  const int t = (int)(unit / parts), part = (int)(unit - (long long)t * parts);
  if (t >= p.T) return;
  const bool is_q = part < p.q_parts;

  // all of the part's rows: groups 0..3 are 16 q heads, or 8 k heads and 8 v heads
  uint4 raw[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const uint16_t* src;
    if (is_q)
      src = p.q + (long long)t * p.q_stride + (part * 16 + g * 4 + sub) * kRow;
    else if (g < 2)
      src = p.k + (long long)t * p.k_stride + (g * 4 + sub) * kRow;
    else
      src = p.v + (long long)t * p.v_stride + ((g - 2) * 4 + sub) * kRow;
    if (is_q || g < 2 || p.pool) raw[g] = __ldcs(reinterpret_cast<const uint4*>(src + j * 8));
  }

  const int pos = __ldg(p.positions + t);
  bool ok = pos >= 0 && pos < p.max_pos;
  int page = -1;
  if (p.pool) {
    const int s = p.token_seq ? __ldg(p.token_seq + t) : t;
    ok = ok && s >= 0 && s < p.num_seqs && pos / PKV_PAGE_TOKENS < p.max_blocks;
    if (ok) {
      page = __ldg(p.block_tables + (size_t)s * p.bt_stride + pos / PKV_PAGE_TOKENS);
      ok = page >= 0 && page < p.num_pages;
    }
  }
  uint16_t* out = is_q ? p.q_out + ((size_t)t * PKV_NUM_Q_HEADS + part * 16) * kRow
                       : p.k_out ? p.k_out + (size_t)t * PKV_NUM_KV_HEADS * kRow : nullptr;
  if (!ok) {
    if (lane == 0) report_error(p.d_err, PKV_ERR_DEVICE_INDEX);
    if (out) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
        if (is_q || g < 2)
          *reinterpret_cast<uint4*>(out + (g * 4 + sub) * kRow + j * 8) = make_uint4(0, 0, 0, 0);
    }
    return;
  }

  // this lane's table entries: of dims 8 j .. 8 j + 7 (half), or of its 4 pairs
  constexpr int kTab = kLayout == kInterleaved ? 4 : 8;
  float c[kTab], s[kTab];
  {
    const float* cr = p.cos + (size_t)pos * p.pairs;
    const float* sr = p.sin + (size_t)pos * p.pairs;
    if (kLayout == kHalfAligned) {
      const int at = 8 * j < p.pairs ? 8 * j : 8 * j - p.pairs;
      if (8 * j < 2 * p.pairs) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 a = __ldg(reinterpret_cast<const float4*>(cr + at) + h);
          const float4 b = __ldg(reinterpret_cast<const float4*>(sr + at) + h);
          c[4 * h] = a.x; c[4 * h + 1] = a.y; c[4 * h + 2] = a.z; c[4 * h + 3] = a.w;
          s[4 * h] = b.x; s[4 * h + 1] = b.y; s[4 * h + 2] = b.z; s[4 * h + 3] = b.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) { c[e] = 1.f; s[e] = 0.f; }
      }
    } else {
#pragma unroll
      for (int e = 0; e < kTab; ++e) {
        const int i = kLayout == kInterleaved ? 4 * j + e : 8 * j + e - (8 * j + e < p.pairs ? 0 : p.pairs);
        const bool turned = i < p.pairs;
        c[e] = turned ? __ldg(cr + i) : 1.f;
        s[e] = turned ? __ldg(sr + i) : 0.f;
      }
    }
  }
  float w[8];
  const void* weight = is_q ? p.q_weight : p.k_weight;
  if (weight) {
    if (p.weight_f32) {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = __ldg(static_cast<const float*>(weight) + 8 * j + e);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[e] = __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(weight) + 8 * j + e) << 16);
    }
  }

#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    if (!is_q && g >= 2) break;  // V rows are copied below
    float x[8], y[8];
    unpack8(raw[g], x);
    if (weight) {
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float r = __frsqrt_rn(fmaf(sum, 1.f / kRow, p.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(__fmul_rn(x[e], r), w[e]);
    }
    if (kLayout == kInterleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool turned = 4 * j + e < p.pairs;
        const float a = x[2 * e], b = x[2 * e + 1];
        y[2 * e] = turned ? __fsub_rn(__fmul_rn(a, c[e]), __fmul_rn(b, s[e])) : a;
        y[2 * e + 1] = turned ? __fadd_rn(__fmul_rn(a, s[e]), __fmul_rn(b, c[e])) : b;
      }
    } else if (kLayout == kHalfAligned) {
      const int step = p.pairs >> 3;
      const bool first = j < step, turned = j < 2 * step;
      const int src = (lane & ~7) | (first ? j + step : turned ? j - step : j);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float b = __shfl_sync(0xffffffffu, x[e], src);
        const float xc = __fmul_rn(x[e], c[e]), bs = __fmul_rn(b, s[e]);
        // first half: a c - b s; second half (x is the pair's b, b its a): a s + b c
        y[e] = !turned ? x[e] : first ? __fsub_rn(xc, bs) : __fadd_rn(bs, xc);
      }
    } else {
      float* buf = rows[warp][sub];
      *reinterpret_cast<float4*>(buf + 8 * j) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4*>(buf + 8 * j + 4) = make_float4(x[4], x[5], x[6], x[7]);
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = 8 * j + e;
        const bool first = d < p.pairs, turned = d < 2 * p.pairs;
        const float b = buf[first ? d + p.pairs : turned ? d - p.pairs : d];
        const float xc = __fmul_rn(x[e], c[e]), bs = __fmul_rn(b, s[e]);
        y[e] = !turned ? x[e] : first ? __fsub_rn(xc, bs) : __fadd_rn(bs, xc);
      }
      __syncwarp();  // the next group writes the buffer again
    }
    const uint4 res = pack8(y);
    if (out) *reinterpret_cast<uint4*>(out + (g * 4 + sub) * kRow + j * 8) = res;
    if (!is_q && p.pool) raw[g] = res;
  }
  if (!is_q && p.pool) {
    const int slot = pos % PKV_PAGE_TOKENS;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int kv = g >> 1, head = (g & 1) * 4 + sub;
      uint16_t* dst = p.pool + ((((size_t)page * 2 + kv) * PKV_NUM_KV_HEADS + head) * PKV_PAGE_TOKENS + slot) * kRow;
      *reinterpret_cast<uint4*>(dst + j * 8) = raw[g];
    }
  }
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int kv_append_norm_rope(const void* q, long long q_stride, const void* k, long long k_stride,
                                   const void* v, long long v_stride, const void* q_weight,
                                   const void* k_weight, int weight_f32, float eps,
                                   const float* rope_cos, const float* rope_sin, int max_pos,
                                   int rope_pairs, int interleaved, const int32_t* positions,
                                   const int32_t* token_seq, int T, const int32_t* block_tables,
                                   int num_seqs, int bt_row_stride, int max_blocks, void* kv_pool,
                                   int num_pages, void* q_out, void* k_out, int* d_err, void* stream) {
  if (T < 0 || max_pos < 1 || rope_pairs < 1 || rope_pairs > PKV_ROPE_PAIRS ||
      (weight_f32 != 0 && weight_f32 != 1) || (interleaved != 0 && interleaved != 1))
    return PKV_ERR_INVALID_ARGUMENT;
  if (kv_pool && (num_seqs < 1 || max_blocks < 1 || bt_row_stride < max_blocks || num_pages < 1))
    return PKV_ERR_INVALID_ARGUMENT;
  if (T == 0) return PKV_OK;
  if (!k || !positions || !rope_cos || !rope_sin) return PKV_ERR_INVALID_ARGUMENT;
  if ((q == nullptr) != (q_out == nullptr) || (kv_pool != nullptr && (!v || !block_tables)) ||
      (!kv_pool && !k_out) || (!q && q_weight))
    return PKV_ERR_INVALID_ARGUMENT;
  if ((q_weight || k_weight) && !(eps >= 0.f && isfinite(eps))) return PKV_ERR_INVALID_ARGUMENT;
  if (k_stride < PKV_NUM_KV_HEADS * PKV_HEAD_DIM || (q && q_stride < PKV_NUM_Q_HEADS * PKV_HEAD_DIM) ||
      (kv_pool && v_stride < PKV_NUM_KV_HEADS * PKV_HEAD_DIM))
    return PKV_ERR_INVALID_ARGUMENT;
  // rows are read and written 16 bytes at a time
  if (!aligned16(q) || !aligned16(k) || (kv_pool && !aligned16(v)) || !aligned16(q_out) ||
      !aligned16(k_out) || !aligned16(kv_pool) || (k_stride & 7) || (q && (q_stride & 7)) ||
      (kv_pool && (v_stride & 7)))
    return PKV_ERR_MISALIGNED;
  const uintptr_t words = reinterpret_cast<uintptr_t>(rope_cos) | reinterpret_cast<uintptr_t>(rope_sin) |
                          reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(token_seq) |
                          reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(d_err);
  const uintptr_t weights = reinterpret_cast<uintptr_t>(q_weight) | reinterpret_cast<uintptr_t>(k_weight);
  if ((words & 3u) || (weights & (weight_f32 ? 3u : 1u))) return PKV_ERR_MISALIGNED;
  if (T > (1 << 30) || (kv_pool && (long long)num_pages * PKV_PAGE_ELEMS >= (1ll << 40)))
    return PKV_ERR_UNSUPPORTED_SHAPE;
  int dev = 0;
  const int rc = bind_stream_device(stream, &dev);
  if (rc != PKV_OK) return rc;

  NormRopeParams p;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.cos = rope_cos;
  p.sin = rope_sin;
  p.positions = positions;
  p.token_seq = token_seq;
  p.block_tables = block_tables;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_out = static_cast<uint16_t*>(k_out);
  p.pool = static_cast<uint16_t*>(kv_pool);
  p.d_err = d_err;
  p.eps = eps;
  p.weight_f32 = weight_f32;
  p.T = T;
  p.pairs = rope_pairs;
  p.max_pos = max_pos;
  p.num_seqs = num_seqs;
  p.bt_stride = bt_row_stride;
  p.max_blocks = max_blocks;
  p.num_pages = num_pages;
  p.q_parts = q ? 2 : 0;

  const long long units = (long long)T * (p.q_parts + 1);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((units + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // lane-aligned partners and 16-byte table loads, where the pairs and the tables allow them
  const bool by_lane = rope_pairs % 8 == 0 && aligned16(rope_cos) && aligned16(rope_sin);
  cudaError_t e = interleaved ? cudaLaunchKernelEx(&cfg, norm_rope_kernel<kInterleaved>, p)
                  : by_lane   ? cudaLaunchKernelEx(&cfg, norm_rope_kernel<kHalfAligned>, p)
                              : cudaLaunchKernelEx(&cfg, norm_rope_kernel<kHalfAny>, p);
  return cuda_status(e, "cudaLaunchKernelEx(norm_rope)");
}
