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
// Work: a row is spread over 8 lanes of 8 dims, and a warp has four rows at a
// time (a group).  In the half layout, where the pairs are a multiple of 4, a
// lane holds four dims and their four partners, two 8-byte loads, so that the
// rotation needs no exchange and a lane only four table entries; interleaved
// pairs are neighbours in one 16-byte load.  Other half layouts go through a
// row buffer in shared memory.  The norm's sum of squares is three shuffles.
//   many tokens: one warp per token, all of its 12 groups -- 8 of q, 2 of k, 2
//     of v -- in flight before anything else is read;
//   few tokens, or no q: one warp per token and part of 4 groups (16 q heads,
//     or k and v), for the shorter way through.
//
// Bound: memory.  A token moves 12 KiB (32 + 8 + 8 rows read and written)
// and one table row.  24 warps per SM (80 registers) keep 144 KB in flight;
// with 16 warps 32768 tokens took 87 us, not 74.  With 16 contiguous bytes per
// lane and the partners fetched by shuffles, and three warps per token, they
// took 131 us: 2450 instructions a token, half of the issue slots; with two
// 16-byte loads per lane and four lanes per row, 79 us.  With later rows on their
// way into the L2 they take 67.7 us (89 % of the measured copy rate), interleaved
// pairs 63.8 us, the layouts through the row buffer 80.4 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "pkv.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kRow = PKV_HEAD_DIM;
constexpr int kGroups = 4;       // groups of a part
constexpr int kAllGroups = 12;   // of a token: 8 of q, 2 of k, 2 of v
constexpr int kQGroups = 8;

enum Layout { kHalf4 = 0, kHalfAny = 1, kInterleaved = 2 };

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
  int ahead;                             // tokens between the one read and the one fetched into the L2
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

// Where a lane's 8 dims of a row are: dims[0 .. 3] at `lo`, dims[4 .. 7] at `hi`.
// Half layout by fours: chunk j and its partner behind `pairs` dims, then the
// chunks that are not rotated, two by two.  Else 8 neighbours.
template <int kLayout>
__device__ __forceinline__ void places(int j, int pairs, int& lo, int& hi, bool& turned) {
  if (kLayout == kHalf4) {
    const int chunks = pairs >> 2;
    turned = j < chunks;
    lo = turned ? 4 * j : 4 * (2 * chunks + 2 * (j - chunks));
    hi = turned ? lo + pairs : lo + 4;
  } else {
    turned = true;
    lo = 8 * j;
    hi = lo + 4;
  }
}

template <int kLayout>
__device__ __forceinline__ uint4 load_row(const uint16_t* row, int lo, int hi) {
  if (kLayout != kHalf4) return __ldcs(reinterpret_cast<const uint4*>(row + lo));
  const uint2 a = __ldcs(reinterpret_cast<const uint2*>(row + lo)), b = __ldcs(reinterpret_cast<const uint2*>(row + hi));
  return make_uint4(a.x, a.y, b.x, b.y);
}

template <int kLayout>
__device__ __forceinline__ void store_row(uint16_t* row, int lo, int hi, const uint4& v) {
  if (kLayout != kHalf4) {
    *reinterpret_cast<uint4*>(row + lo) = v;
  } else {
    *reinterpret_cast<uint2*>(row + lo) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2*>(row + hi) = make_uint2(v.z, v.w);
  }
}

// kWhole: a warp has a whole token, else a part of it.
template <int kLayout, bool kWhole, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, kWhole ? 24 / kWarps : 1) norm_rope_kernel(const NormRopeParams p) {
  constexpr int kMine = kWhole ? kAllGroups : kGroups;
  // of any half layout; dim d at d + 4 (d / 32), so that 32 lanes -- four rows, every 8th dim --
  // find 32 banks
  __shared__ float rows[kLayout == kHalfAny ? kWarps : 1][4][kRow + 5];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane >> 3, j = lane & 7;  // row of a group, and which dims of it
  const int parts = kWhole ? 1 : p.q_parts + 1;
  const long long unit = (long long)blockIdx.x * kWarps + warp;
  const int t = (int)(unit / parts);
  if (t >= p.T) return;
  // this warp's groups g0 .. g0 + kMine - 1 of the token's 12; q is the first 8
  const int part = (int)(unit - (long long)t * parts);
  const int g0 = kWhole ? 0 : part < p.q_parts ? part * kGroups : kQGroups;
  const auto is_q = [&](int g) { return kWhole ? g < kQGroups : g0 < kQGroups; };
  const auto is_v = [&](int g) { return !is_q(g) && (kWhole ? g >= kQGroups + 2 : g >= 2); };
  const auto head_of = [&](int g) {  // of q, or of k or v
    const int n = g0 + g;
    return (n < kQGroups ? n : (n - kQGroups) & 1) * 4 + sub;
  };
  int lo, hi;
  bool turned;
  places<kLayout>(j, p.pairs, lo, hi, turned);

  // the way to the table and page entries starts first, then everything else is under way
  const int pos = __ldg(p.positions + t);
  const int row = p.pool && p.token_seq ? __ldg(p.token_seq + t) : t;
  uint4 raw[kMine];
  const uint16_t* q = p.q + (long long)t * p.q_stride;
  const uint16_t* k = p.k + (long long)t * p.k_stride;
  const uint16_t* v = p.v + (long long)t * p.v_stride;
#pragma unroll
  for (int g = 0; g < kMine; ++g)
    if (!is_v(g) || p.pool)
      raw[g] = load_row<kLayout>((is_q(g) ? q : is_v(g) ? v : k) + head_of(g) * kRow, lo, hi);

  if (kWhole && lane < 3 && t < p.T - p.ahead) {  // rows that a later warp reads
    const uint16_t* r = lane == 0 ? q + p.ahead * p.q_stride : lane == 1 ? k + p.ahead * p.k_stride : v + p.ahead * p.v_stride;
    if (lane < 2 || p.pool) prefetch_l2(r, (lane ? PKV_NUM_KV_HEADS : PKV_NUM_Q_HEADS) * kRow * 2);
  }
  bool ok = pos >= 0 && pos < p.max_pos;
  int page = -1;
  if (p.pool) {
    ok = ok && row >= 0 && row < p.num_seqs && pos / PKV_PAGE_TOKENS < p.max_blocks;
    if (ok) {
      page = __ldg(p.block_tables + (size_t)row * p.bt_stride + pos / PKV_PAGE_TOKENS);
      ok = page >= 0 && page < p.num_pages;
    }
  }
  uint16_t* q_out = p.q_out + (size_t)t * PKV_NUM_Q_HEADS * kRow;
  uint16_t* k_out = p.k_out ? p.k_out + (size_t)t * PKV_NUM_KV_HEADS * kRow : nullptr;
  if (!ok) {
    if (lane == 0) report_error(p.d_err, PKV_ERR_DEVICE_INDEX);
#pragma unroll
    for (int g = 0; g < kMine; ++g)
      if (!is_v(g) && (is_q(g) || k_out))
        store_row<kLayout>((is_q(g) ? q_out : k_out) + head_of(g) * kRow, lo, hi, make_uint4(0, 0, 0, 0));
    return;
  }

  // table entries: of this lane's four pairs, or (any half layout) of its 8 dims
  constexpr int kTab = kLayout == kHalfAny ? 8 : 4;
  float c[kTab], s[kTab];
  {
    const float* cr = p.cos + (size_t)pos * p.pairs;
    const float* sr = p.sin + (size_t)pos * p.pairs;
    if (kLayout == kHalf4) {
      const float4 a = turned ? __ldg(reinterpret_cast<const float4*>(cr + lo)) : make_float4(1.f, 1.f, 1.f, 1.f);
      const float4 b = turned ? __ldg(reinterpret_cast<const float4*>(sr + lo)) : make_float4(0.f, 0.f, 0.f, 0.f);
      c[0] = a.x; c[1] = a.y; c[2] = a.z; c[3] = a.w;
      s[0] = b.x; s[1] = b.y; s[2] = b.z; s[3] = b.w;
    } else {
#pragma unroll
      for (int e = 0; e < kTab; ++e) {
        const int i = kLayout == kInterleaved ? 4 * j + e : 8 * j + e - (8 * j + e < p.pairs ? 0 : p.pairs);
        const bool in = i < p.pairs;
        c[e] = in ? __ldg(cr + i) : 1.f;
        s[e] = in ? __ldg(sr + i) : 0.f;
      }
    }
  }
  const auto row_of = [](int d) { return d + 4 * (d >> 5); };
  int partner[kTab];  // any half layout: where the other dim of each pair is; s gets its sign
  if (kLayout == kHalfAny) {
#pragma unroll
    for (int e = 0; e < kTab; ++e) {
      const int d = 8 * j + e;
      partner[e] = row_of(d < p.pairs ? d + p.pairs : d < 2 * p.pairs ? d - p.pairs : d);
      if (d < p.pairs) s[e] = -s[e];
    }
  }
  const auto load_weights = [&](const void* weight, float (&w)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = (e < 4 ? lo : hi - 4) + e;
      w[e] = p.weight_f32 ? __ldg(static_cast<const float*>(weight) + d)
                          : __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(weight) + d) << 16);
    }
  };
  float w[8];
  const bool first_is_q = g0 < kQGroups;
  const void* weight = first_is_q ? p.q_weight : p.k_weight;
  if (weight) load_weights(weight, w);

#pragma unroll
  for (int g = 0; g < kMine; ++g) {
    if (is_v(g)) break;  // V rows are copied below
    if (kWhole && g == kQGroups) {
      weight = p.k_weight;
      if (weight) load_weights(weight, w);
    }
    float x[8], y[8];
    unpack8(raw[g], x);
    if (weight) {
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float r = rsqrtf(fmaf(sum, 1.f / kRow, p.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(__fmul_rn(x[e], r), w[e]);
    }
    if (kLayout == kHalf4) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // (1, 0) entries leave dims that are not rotated as they are
        y[e] = turned ? __fsub_rn(__fmul_rn(x[e], c[e]), __fmul_rn(x[e + 4], s[e])) : x[e];
        y[e + 4] = turned ? __fadd_rn(__fmul_rn(x[e], s[e]), __fmul_rn(x[e + 4], c[e])) : x[e + 4];
      }
    } else if (kLayout == kInterleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool in = 4 * j + e < p.pairs;
        const float a = x[2 * e], b = x[2 * e + 1];
        y[2 * e] = in ? __fsub_rn(__fmul_rn(a, c[e]), __fmul_rn(b, s[e])) : a;
        y[2 * e + 1] = in ? __fadd_rn(__fmul_rn(a, s[e]), __fmul_rn(b, c[e])) : b;
      }
    } else {
      float* buf = rows[warp][sub];
#pragma unroll
      for (int e = 0; e < 8; ++e) buf[row_of(8 * j) + e] = x[e];
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // a c + b (-s) in the first half; in the second x is the pair's b, and its a is multiplied by s
        const float turned_e = __fadd_rn(__fmul_rn(x[e], c[e]), __fmul_rn(buf[partner[e]], s[e]));
        y[e] = 8 * j + e < 2 * p.pairs ? turned_e : x[e];
      }
      __syncwarp();  // the next group writes the buffer again
    }
    raw[g] = pack8(y);
    if (is_q(g))
      store_row<kLayout>(q_out + head_of(g) * kRow, lo, hi, raw[g]);
    else if (k_out)
      store_row<kLayout>(k_out + head_of(g) * kRow, lo, hi, raw[g]);
  }
  if (p.pool && (kWhole || !first_is_q)) {
    const int slot = pos % PKV_PAGE_TOKENS;
#pragma unroll
    for (int g = 0; g < kMine; ++g)
      if (!is_q(g))
        store_row<kLayout>(p.pool + ((((size_t)page * 2 + (is_v(g) ? 1 : 0)) * PKV_NUM_KV_HEADS + head_of(g)) *
                                         PKV_PAGE_TOKENS + slot) * kRow,
                           lo, hi, raw[g]);
  }
}

// Where one warp per token has enough warps to fill the GPU (about 16 on each
// SM): 32768 tokens take 68 us whole and 100 us in parts, 2432 tokens 7.6 and
// 7.8 us; 257 tokens take 4.0 us whole and 3.1 us in parts, one token 3.6 and
// 2.7 us.
constexpr int kWholeTokensPerSm = 16;
// A warp fetches the rows half a wave behind its own into the L2: 32768 tokens
// 67.7 us, without 75.6 us; 6, 24 and 36 tokens per SM ahead take 0.8, 1 and 4 us more.
constexpr int kAheadPerSm = 12;

template <int kLayout>
cudaError_t launch_norm_rope(NormRopeParams p, int sms, cudaLaunchConfig_t& cfg) {
  p.ahead = sms * kAheadPerSm;
  if (p.q_parts && p.T >= sms * kWholeTokensPerSm) {
    constexpr int kWarps = 4;
    cfg.gridDim = dim3((unsigned)((p.T + kWarps - 1) / kWarps));
    cfg.blockDim = dim3(kWarps * 32);
    return cudaLaunchKernelEx(&cfg, norm_rope_kernel<kLayout, true, kWarps>, p);
  }
  constexpr int kWarps = 6;
  cfg.gridDim = dim3((unsigned)(((long long)p.T * (p.q_parts + 1) + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kWarps * 32);
  return cudaLaunchKernelEx(&cfg, norm_rope_kernel<kLayout, false, kWarps>, p);
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

  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // 16-byte table loads by fours, where the pairs and the tables allow them
  const bool by_fours = rope_pairs % 4 == 0 && aligned16(rope_cos) && aligned16(rope_sin);
  const int sms = sm_count(dev);
  const cudaError_t e = interleaved ? launch_norm_rope<kInterleaved>(p, sms, cfg)
                        : by_fours  ? launch_norm_rope<kHalf4>(p, sms, cfg)
                                    : launch_norm_rope<kHalfAny>(p, sms, cfg);
  return cuda_status(e, "cudaLaunchKernelEx(norm_rope)");
}
