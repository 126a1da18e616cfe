// One decode step of grouped-query attention over pages of 8-bit codes with
// one scale per block (16 slots of one page, K or V, and KV head), sm_103a.
//
// For sequence s with n tokens, KV head g and its query heads h (flash
// decoding, one pass with a running maximum, exponentials in base 2):
//   x_j = scale log2(e) ks(page of j) (q_h . ck_j),  p_j = 2^(x_j - m)
//   out_h = sum_pages vs(page) sum_{j in page} p_j cv_j / sum_j p_j
// The scales are one number per page and head, so they multiply a page's
// four scores and its finished P V product, and the codes themselves enter
// the MMAs.
//
// Work: sequences that are short by the caller's bound have a CTA each.  Else the
// pages of all sequences, one after another, are one long list; every CTA takes an
// equal share of it (an even number of pages), whatever the lengths.  A share that ends inside a sequence leaves a partial (o, m, l)
// in the workspace, and a second kernel merges the parts of such sequences.
// One CTA is a producer warp and 8 consumer warps, one per KV head: the
// producer copies whole pages -- 16 KiB, all heads, one TMA box each -- into a
// ring of stages of two pages, under the 64-byte swizzle, and every consumer
// reads its head's 2 KiB of each page from there.
//
// A consumer's page: S = q K^T as m16n8k16 with the four query heads in rows
// 0..3 and again in 4..7 (two n-tiles of 8 tokens, four k-steps), whose
// accumulator layout is the B operand's of O^T = V^T P^T, so the probabilities
// never leave their lanes.  fp16 holds 11 bits of a probability: columns 0..3 of
// P^T are p rounded, columns 4..7 what the rounding left of it, in products that
// the tile has room for, and their sums are added at the end.  V^T is loaded by ldmatrix.trans on byte pairs, which puts the codes
// of two tokens and two dims into one register.  Codes become fp16 exactly:
// e4m3 by conversion, int8 by placing code + 128 into the mantissa of 1024
// and subtracting 1152.  A head's q is scaled by the power of two that brings its
// largest value into [2^14, 2^15): exact in fp16 unless smaller by 2^-31.
// Probabilities carry a factor 2^14 that cancels in the division; the two
// columns together are within 2^-22 of one, and within 2^-39 of the largest for
// the smallest of them.  Their sum is over the unrounded ones.  The output's sums
// are kept 2^20 times smaller than they are, so that a million values next to
// fp32's largest do not overflow.
//
// Bound: memory, 1 KiB + 4 B of scales per token.  Of 32 sequences of 2048 tokens
// (19.6 us, 51 % of the measured copy rate) the pages take 9 us at 7.5 TB/s; 2.3
// us go by before the first copy is issued (lengths, their sums, the table
// entries: loads that wait for one another), 3 us at the end, where SMs of larger
// GPCs get less bandwidth each and finish their equal shares later, and 2.8 us
// for the merge.  97 sequences of up to 8191 tokens run at 80 %.  A page holds
// one warp for about 210 instructions, everything around it included (58 % of the
// issue slots); the tensor pipe is busy 26 % of the time.  The second column of the
// probabilities costs 0.4 us of the 19.6 and the lowered sums 0.2; the ragged 97 take
// the same time without both, 4096 sequences of 64 tokens 54 instead of 58 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "bs8.cuh"
#include "internal.h"
#include "pkv.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kHeads = PKV_NUM_KV_HEADS;
constexpr int kConsumers = kHeads;                      // one warp per KV head
constexpr int kThreads = (kConsumers + 1) * 32;
constexpr int kStages = 3;
constexpr int kStagePages = 2;
constexpr int kScaleBytes = 2 * kHeads * 4;             // of one page
constexpr int kStageBytes = kStagePages * kBs8PageBytes;
constexpr int kSmemBytes = 1024 + kStages * (kStageBytes + kStagePages * kScaleBytes);
constexpr int kCtasPerSm = 2;
constexpr int kMaxSeqsBs8 = 4096;
constexpr int kMinPages = 4;                            // least share of a CTA
// Short sequences stay whole, one CTA's each: nothing to merge, nothing to add up
// first.  Short is up to 8 pages, and one more per 8 sequences up to 24: one
// sequence of 8 pages takes 6.5 us, by shares 7.1 us, of 12 pages 8.3 and 7.1 us; 64
// of 8 pages 6.7 and 9.2 us, of 16 10.4 and 9.3 us (ragged 10.5 and 11.5 us), of 24
// 14.4 and 11.1 us; 152 of 24 pages 16.6 and 21.7 us; 1000 ragged ones to 24 pages 57
// and 53 us; 4096 of 4 pages 58 and 72 us.
constexpr int kWholePages = 8, kWholePagesMost = 24;
// Up to this many sequences the merge looks at every sequence; beyond it at every
// CTA, in each of which one split sequence begins at most (4096 sequences of 64
// tokens in shares: 72 us, by sequence 93 us; 1000 ragged ones to 300: 46 and 51 us;
// 256 of 2048: 95.5 us both; 97 ragged ones to 8191: 73.7 and 72.6 us).
constexpr int kBySequence = 128;
constexpr uint32_t kWaitUs = 2000000;                   // limit of every wait
constexpr float kLift = 14.f;                           // probabilities carry 2^14
// 2^-34 on a page's product, with them, to the output's sums (in the page's scale it would
// cost bits where values are below 1e-27).
constexpr float kLower = 0x1p-34f;
constexpr float kRaise = 0x1p34f;                       // with the final division
constexpr float kNothing = -1.f;                        // l of a part with a bad page

// Workspace: per CTA two parts (of a sequence begun in an earlier CTA, and of
// one that goes on in the next) of 32 heads, o [64] then (m, l) pairs; then
// which CTAs a split sequence lies in, by sequence or by CTA.
constexpr int kPartFloats = PKV_NUM_Q_HEADS * (PKV_HEAD_DIM + 2);

struct Bs8DecodeParams {
  const uint16_t* q;
  const float* scales;
  const int32_t *block_tables, *seq_lens;
  uint16_t* out;
  float* parts;
  int2* span;  // by sequence: first and last CTA of a split one; by CTA: the split sequence that begins
               // there and its last CTA; else (-1, -1)
  int* d_err;
  float scale;
  int num_pages, bt_stride, max_blocks, num_seqs, min_pages, by_cta;
};

__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap* map, int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(0), "r"(page), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t cvt_e4m3x2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(two));
  return r;
}

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

constexpr uint32_t kMagic = 0x64646464u;   // bytes of 1024 in fp16
constexpr uint32_t kOffset = 0x64806480u;  // 1152 twice

// four consecutive codes -> (0, 1), (2, 3) as fp16 pairs
template <bool kE4m3>
__device__ __forceinline__ void codes_in_order(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (kE4m3) {
    lo = cvt_e4m3x2(w);
    hi = cvt_e4m3x2(w >> 16);
  } else {
    w ^= 0x80808080u;
    lo = sub_f16x2(__byte_perm(w, kMagic, 0x4140), kOffset);
    hi = sub_f16x2(__byte_perm(w, kMagic, 0x4342), kOffset);
  }
}

// bytes (a0, a1, b0, b1) of two tokens a, b and two dims -> (a0, b0), (a1, b1)
template <bool kE4m3>
__device__ __forceinline__ void codes_by_dim(uint32_t w, uint32_t& d0, uint32_t& d1) {
  if (kE4m3) {
    w = __byte_perm(w, 0, 0x3120);
    d0 = cvt_e4m3x2(w);
    d1 = cvt_e4m3x2(w >> 16);
  } else {
    w ^= 0x80808080u;
    d0 = sub_f16x2(__byte_perm(w, kMagic, 0x4240), kOffset);
    d1 = sub_f16x2(__byte_perm(w, kMagic, 0x4341), kOffset);
  }
}

// Pages that sequence s brings to the list: none for an empty or refused one.
__device__ __forceinline__ int pages_of(const Bs8DecodeParams& p, int s, bool& refused) {
  const int n = __ldg(p.seq_lens + s);
  refused = n < 0 || n > (long long)p.max_blocks * PKV_PAGE_TOKENS;
  return refused ? 0 : (int)(((unsigned)n + PKV_PAGE_TOKENS - 1) / PKV_PAGE_TOKENS);
}

struct Smem {
  uint64_t full[kStages], empty[kStages];
  int sum[kThreads / 32];
  int before;  // pages before first_seq, the sequence that the CTA begins in
  int first_seq;
  int bad[kStages];
};

template <bool kE4m3>
struct Head {  // a consumer's state for one segment
  uint32_t qa[4], qb[4];  // q fragments: dims 16 t + 4 i, + 1 and + 2, + 3
  float o[4][4];          // O^T: dims 16 c + 2 g (+ 1), heads 2 t, 2 t + 1 (their second columns for t > 1)
  float m, l;             // running maximum and this lane's sum of head g % 4
  float unit, unit2;      // scale of the scores, in two factors: their product may be too small for a float

  // q of a sequence as this lane will need it: 16 dims of head g % 4
  struct Q {
    uint4 a, b;
  };
  __device__ static Q fetch(const Bs8DecodeParams& p, int seq, int head) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    static_assert(PKV_GROUP == 4, "two columns for each head of a group");
    const uint4* src = reinterpret_cast<const uint4*>(
        p.q + ((size_t)seq * PKV_NUM_Q_HEADS + head * PKV_GROUP + (g & 3)) * PKV_HEAD_DIM + 16 * t);
    return Q{src[0], src[1]};
  }

  __device__ void start(const Bs8DecodeParams& p, const Q& q) {
    float x[16];
    const uint32_t w[8] = {q.a.x, q.a.y, q.a.z, q.a.w, q.b.x, q.b.y, q.b.z, q.b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[2 * e] = bf16lo_to_f32(w[e]);
      x[2 * e + 1] = bf16hi_to_f32(w[e]);
    }
    uint32_t bits = 0;  // of the largest finite |q|: magnitudes order as their bits
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint32_t b = __float_as_uint(x[e]) & 0x7FFFFFFFu;
      bits = max(bits, b < 0x7F800000u ? b : 0u);
    }
    bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, 1));
    bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, 2));
    // 2^up brings it into [2^14, 2^15), unless it is 0; infinities and NaN stay
    // what they are, in their own head.  up lies in [-113, 141]: two factors
    // keep each a normal number.
    const int up = bits ? 14 - ((int)(bits >> 23) - 127) : 0;
    const float f0 = __uint_as_float((uint32_t)(127 + up / 2) << 23);
    const float f1 = __uint_as_float((uint32_t)(127 + up - up / 2) << 23);
    const float d0 = __uint_as_float((uint32_t)(127 - up / 2) << 23);
    const float d1 = __uint_as_float((uint32_t)(127 - (up - up / 2)) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      qa[i] = pack_f16x2(x[4 * i] * f0 * f1, x[4 * i + 1] * f0 * f1);
      qb[i] = pack_f16x2(x[4 * i + 2] * f0 * f1, x[4 * i + 3] * f0 * f1);
    }
    unit = p.scale * 1.4426950408889634f * d0;
    unit2 = d1;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c][e] = 0.f;
    m = -INFINITY;
    l = 0.f;
  }

  // Two probabilities in fp16: rounded (first = 0), or what the rounding leaves (-1).
  __device__ __forceinline__ static uint32_t column(float p0, float p1, float first) {
    const uint32_t near = pack_f16x2(p0, p1);
    const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&near));
    return pack_f16x2(fmaf(r.x, first, p0), fmaf(r.y, first, p1));
  }

  // Two pages in shared memory at `pages`, scales at `scales`; `live` tokens of
  // the 32 are the sequence's.
  __device__ __forceinline__ void step(uint32_t pages, const float* scales, int head, int live) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float x[2][4];
#pragma unroll
    for (int u = 0; u < kStagePages; ++u) {
      const float ks = scales[u * 2 * kHeads + head] * unit * unit2;
#pragma unroll
      for (int tile = 0; tile < 2; ++tile) {
        // K rows of 64 bytes, 16-byte chunks swizzled by (row / 2) % 4
        const int row = 8 * tile + g;
        const uint32_t at = pages + u * kBs8PageBytes + head * kBs8BlockBytes + row * 64 + ((t ^ ((row >> 1) & 3)) << 4);
        uint32_t w[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t b0, b1;
          codes_in_order<kE4m3>(w[i], b0, b1);
          mma_f16(d, qa[i], 0u, qb[i], 0u, b0, b1);
        }
        x[u][2 * tile] = d[0] * ks;
        x[u][2 * tile + 1] = d[1] * ks;
      }
    }
    const bool tail = live < kStagePages * PKV_PAGE_TOKENS;
    if (tail) {
#pragma unroll
      for (int u = 0; u < kStagePages; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (u * PKV_PAGE_TOKENS + (e >> 1) * 8 + 2 * t + (e & 1) >= live) x[u][e] = -INFINITY;
    }
    float top = fmaxf(fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[0][2], x[0][3])),
                      fmaxf(fmaxf(x[1][0], x[1][1]), fmaxf(x[1][2], x[1][3])));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if (__any_sync(0xffffffffu, top > m)) {  // some head's maximum grows: rescale
      const float now = fmaxf(m, top);
      const float keep = m == -INFINITY ? 0.f : exp2_approx(m - now);
      const float k0 = __shfl_sync(0xffffffffu, keep, 8 * t), k1 = __shfl_sync(0xffffffffu, keep, 8 * t + 4);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        o[c][0] *= k0;
        o[c][1] *= k1;
        o[c][2] *= k0;
        o[c][3] *= k1;
      }
      l *= keep;
      m = now;
    }
    const float shift = m - kLift, first = g < PKV_GROUP ? 0.f : -1.f;
#pragma unroll
    for (int u = 0; u < kStagePages; ++u) {
      // a page that the last stage does not have: whatever shared memory holds is no scale
      const float vs = u * PKV_PAGE_TOKENS < live ? scales[u * 2 * kHeads + kHeads + head] : 0.f;
      float pr[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) pr[e] = exp2_approx(x[u][e] - shift);
      l += (pr[0] + pr[1]) + (pr[2] + pr[3]);
      const uint32_t b0 = column(pr[0], pr[1], first), b1 = column(pr[2], pr[3], first);
      // V^T: matrices of 8 tokens x 16 bytes, (chunk, tokens 0..7), (chunk, 8..15), and the next chunk's
      const int row = lane & 15;
      const uint32_t base = pages + u * kBs8PageBytes + (kHeads + head) * kBs8BlockBytes + row * 64;
#pragma unroll
      for (int c2 = 0; c2 < 2; ++c2) {
        const int chunk = 2 * c2 + (lane >> 4);
        uint32_t w[4];
        ldsm_x4_t(base + ((chunk ^ ((row >> 1) & 3)) << 4), w[0], w[1], w[2], w[3]);
        if (tail) {  // codes behind the sequence's end may be anything, NaN among them
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok = u * PKV_PAGE_TOKENS + (e & 1) * 8 + 2 * t;
            if (tok >= live) w[e] = 0u;
            else if (tok + 1 >= live) w[e] &= 0x0000FFFFu;
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a0, a1, a2, a3;
          codes_by_dim<kE4m3>(w[2 * h], a0, a1);
          codes_by_dim<kE4m3>(w[2 * h + 1], a2, a3);
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          mma_f16(d, a0, a1, a2, a3, b0, b1);
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float2 low = mul2(make_float2(d[e], d[e + 1]), make_float2(kLower, kLower));
            o[2 * c2 + h][e] = fmaf(vs, low.x, o[2 * c2 + h][e]);
            o[2 * c2 + h][e + 1] = fmaf(vs, low.y, o[2 * c2 + h][e + 1]);
          }
        }
      }
    }
  }

  // The segment's result: the output rows, or a part for the merge.
  __device__ void finish(const Bs8DecodeParams& p, int seq, int head, bool bad, float* part) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float sum = l + __shfl_xor_sync(0xffffffffu, l, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c][e] += __shfl_xor_sync(0xffffffffu, o[c][e], 2);  // a head's two columns
    if (part) {
      if (g < PKV_GROUP && t == 0)
        *reinterpret_cast<float2*>(part + PKV_NUM_Q_HEADS * PKV_HEAD_DIM + 2 * (head * PKV_GROUP + g)) =
            make_float2(m, bad ? kNothing : sum);
      if (t < 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float* dst = part + (head * PKV_GROUP + 2 * t + h) * PKV_HEAD_DIM + 2 * g;
#pragma unroll
          for (int c = 0; c < 4; ++c) *reinterpret_cast<float2*>(dst + 16 * c) = make_float2(o[c][h], o[c][2 + h]);
        }
      }
      return;
    }
    const float s0 = __shfl_sync(0xffffffffu, sum, 8 * t & 31), s1 = __shfl_sync(0xffffffffu, sum, (8 * t + 4) & 31);
    if (t < 2) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float inv = bad ? 0.f : kRaise * (1.f / (h ? s1 : s0));
        uint16_t* dst = p.out + ((size_t)seq * PKV_NUM_Q_HEADS + head * PKV_GROUP + 2 * t + h) * PKV_HEAD_DIM + 2 * g;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint32_t*>(dst + 16 * c) = bad ? 0u : pack_bf16x2(o[c][h] * inv, o[c][2 + h] * inv);
      }
    }
  }
};

template <bool kE4m3, bool kWhole>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) bs8_decode_kernel(const __grid_constant__ CUtensorMap map,
                                                                          const Bs8DecodeParams p) {
  extern __shared__ uint8_t dyn[];
  __shared__ Smem sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = (smem_u32(dyn) + 1023u) & ~1023u;
  const uint32_t scale_at = ring + kStages * kStageBytes;
  const float* scale_ptr = reinterpret_cast<const float*>(dyn + (scale_at - smem_u32(dyn)));
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), kConsumers);
    }
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();

  // Where this CTA's share of the list of pages (below 2^30 of them) begins: `before` pages and
  // `seq` sequences are in front of the one it begins in.
  int begin, end, seq, page;
  unsigned share;
  const auto shares = [&](int total) {
    share = ((unsigned)total + gridDim.x - 1) / gridDim.x;
    share = max(share + (share & 1u), (unsigned)p.min_pages);
    begin = (int)min((unsigned)total, share * blockIdx.x);
    end = min(total, begin + (int)share);
  };
  const auto nothing = [&](int s, bool refused) {  // the rows of a sequence with nothing to read
    uint4* row = reinterpret_cast<uint4*>(p.out + (size_t)s * PKV_NUM_Q_HEADS * PKV_HEAD_DIM);
    for (int i = 0; i < PKV_NUM_Q_HEADS * PKV_HEAD_DIM / 8; ++i) row[i] = make_uint4(0, 0, 0, 0);
    if (refused) report_error(p.d_err, PKV_ERR_DEVICE_INDEX);
  };
  // Which CTAs share sequence s, whose n pages begin at `at` (unless every CTA says so itself), and
  // the rows of one with nothing to read: written by one CTA for each sequence, while the producer is
  // under way already.
  const auto record = [&](int s, int at, int n, bool refused) {
    if (s % (int)gridDim.x != (int)blockIdx.x) return;
    if (!p.by_cta) {
      const int c0 = (int)((unsigned)at / share), c1 = n ? (int)((unsigned)(at + n - 1) / share) : c0;
      p.span[s] = c0 == c1 ? make_int2(-1, -1) : make_int2(c0, c1);
    }
    if (n == 0) nothing(s, refused);
  };
  const int hop = kWhole ? (int)gridDim.x : 1;  // from one of the CTA's sequences to its next
  if (kWhole) {
    pdl_launch_dependents();
    begin = page = share = 0;
    end = INT_MAX;
    bool refused;
    for (seq = blockIdx.x; seq < p.num_seqs && pages_of(p, seq, refused) == 0;) seq += hop;
    for (int s = blockIdx.x + (int)threadIdx.x * hop; s < p.num_seqs; s += kThreads * hop)
      if (pages_of(p, s, refused) == 0) nothing(s, refused);
    __syncwarp();
  } else if (p.num_seqs <= 32) {  // every warp finds out by itself, without a barrier (0.2 us less)
    bool refused = false;
    const int n = lane < p.num_seqs ? pages_of(p, lane, refused) : 0;
    int run = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += v;
    }
    shares(__shfl_sync(0xffffffffu, run, 31));
    const int before = run - n;
    const uint32_t here = __ballot_sync(0xffffffffu, before <= begin && begin < run);
    seq = here ? __ffs(here) - 1 : 0;
    page = begin - __shfl_sync(0xffffffffu, before, seq);
    pdl_launch_dependents();
    if (warp == 0 && lane < p.num_seqs) record(lane, before, n, refused);
  } else {  // a consumer thread's sequences, then the sums over all
    const int per = (p.num_seqs + kConsumers * 32 - 1) / (kConsumers * 32);
    const int s0 = min(p.num_seqs, (int)threadIdx.x * per), s1 = min(p.num_seqs, s0 + per);
    int mine = 0;
    for (int s = s0; s < s1; ++s) {
      bool refused;
      mine += pages_of(p, s, refused);
    }
    int run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += v;
    }
    if (lane == 31) sh.sum[warp] = run;
    __syncthreads();
    int before = run - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += sh.sum[w];
      total += sh.sum[w];
    }
    shares(total);
    if (before <= begin && begin < before + mine) {
      int at = before;
      for (int s = s0; s < s1; ++s) {
        bool refused;
        const int n = pages_of(p, s, refused);
        if (at <= begin && begin < at + n) {
          sh.first_seq = s;
          sh.before = at;
        }
        at += n;
      }
    }
    __syncthreads();
    seq = sh.first_seq;
    page = begin - sh.before;
    pdl_launch_dependents();
    int at = before;
    for (int s = s0; s < s1; ++s) {
      bool refused;
      const int n = pages_of(p, s, refused);
      record(s, at, n, refused);
      at += n;
    }
  }
  if (kWhole ? seq >= p.num_seqs : begin >= end) {
    if (p.by_cta && threadIdx.x == 0) p.span[blockIdx.x] = make_int2(-1, -1);
    return;
  }

  int at = begin;
  int stage = 0;
  uint32_t phase = 0;

  if (warp == kConsumers) {  // producer
    bool alive = true;
    int filled = 0;
    while ((kWhole ? seq < p.num_seqs : at < end) && alive) {
      bool refused;
      const int pages = pages_of(p, seq, refused);
      const int todo = min(pages - page, end - at);
      const int32_t* table = p.block_tables + (size_t)seq * p.bt_stride + page;
      for (int i = 0; i < todo && alive; i += 32) {
        int id = i + lane < todo ? __ldg(table + i + lane) : 0;
        const bool wrong = id < 0 || id >= p.num_pages;
        if (wrong) id = 0;
        const uint32_t wrongs = __ballot_sync(0xffffffffu, wrong);
        if (wrongs && lane == 0) report_error(p.d_err, PKV_ERR_DEVICE_INDEX);
        for (int k = 0; k < 32 && i + k < todo; k += kStagePages) {
          const int id0 = __shfl_sync(0xffffffffu, id, k), id1 = __shfl_sync(0xffffffffu, id, k + 1);
          if (lane == 0) {
            if (filled >= kStages && !mbar_wait_bounded(smem_u32(&sh.empty[stage]), phase ^ 1u, kWaitUs)) {
              alive = false;
            } else {
              const int n = i + k + 1 < todo ? 2 : 1;
              const uint32_t bar = smem_u32(&sh.full[stage]);
              const uint32_t dst = ring + stage * kStageBytes, sc = scale_at + stage * kStagePages * kScaleBytes;
              sh.bad[stage] = (wrongs >> k) & 3u;
              mbar_arrive_expect_tx(bar, n * (kBs8PageBytes + kScaleBytes));
              tma_load_page(dst, &map, id0, bar);
              bulk_load(sc, p.scales + (size_t)id0 * 2 * kHeads, kScaleBytes, bar);
              if (n == 2) {
                tma_load_page(dst + kBs8PageBytes, &map, id1, bar);
                bulk_load(sc + kScaleBytes, p.scales + (size_t)id1 * 2 * kHeads, kScaleBytes, bar);
              }
            }
          }
          alive = __shfl_sync(0xffffffffu, (int)alive, 0) != 0;
          if (!alive) break;
          ++filled;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      at += todo;
      page = 0;
      seq += hop;
      while (at < end && seq < p.num_seqs && pages_of(p, seq, refused) == 0) seq += hop;
    }
    if (!alive) {  // every copy in flight lands before the CTA's shared memory goes
      if (lane == 0) {
        report_error(p.d_err, PKV_ERR_TIMEOUT);
        for (int i = 0; i < kStages; ++i) {
          const int back = (stage + i) % kStages;
          mbar_wait_bounded(smem_u32(&sh.full[back]), back >= stage ? phase ^ 1u : phase, kWaitUs);
        }
      }
    }
    return;
  }

  const int head = warp;
  Head<kE4m3> st;
  bool alive = true;
  int2 split = make_int2(-1, -1);  // the sequence that begins here and goes on, and the last CTA that has a part of it
  bool refused;
  int pages = pages_of(p, seq, refused);
  auto q = Head<kE4m3>::fetch(p, seq, head);
  while ((kWhole ? seq < p.num_seqs : at < end) && alive) {
    const int len = __ldg(p.seq_lens + seq);
    const int todo = min(pages - page, end - at);
    st.start(p, q);
    // the next sequence, and its q under way while this one is worked on
    int next = seq + hop, next_pages = 0;
    if (at + todo < end) {
      while (next < p.num_seqs && (next_pages = pages_of(p, next, refused)) == 0) next += hop;
      if (next < p.num_seqs) q = Head<kE4m3>::fetch(p, next, head);
    }
    bool bad = false;
    for (int i = 0; i < todo; i += kStagePages) {
      if (!mbar_wait_bounded(smem_u32(&sh.full[stage]), phase, kWaitUs)) {
        alive = false;
        break;
      }
      const int n = min(kStagePages, todo - i);
      bad |= sh.bad[stage] != 0;
      st.step(ring + stage * kStageBytes, scale_ptr + stage * kStagePages * 2 * kHeads, head,
              min(n * PKV_PAGE_TOKENS, len - (page + i) * PKV_PAGE_TOKENS));
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.empty[stage]));
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (!alive) break;
    const bool whole = todo == pages;
    // a part: of a sequence that began in an earlier CTA (slot 0) or begins here (slot 1)
    float* part = whole ? nullptr : p.parts + ((size_t)blockIdx.x * 2 + (page > 0 ? 0 : 1)) * kPartFloats;
    st.finish(p, seq, head, bad, part);
    if (!whole && page == 0) split = make_int2(seq, (int)((unsigned)(at + pages - 1) / share));
    at += todo;
    page = 0;
    seq = next;
    pages = next_pages;
  }
  if (p.by_cta && threadIdx.x == 0) p.span[blockIdx.x] = split;
  if (!alive && lane == 0) report_error(p.d_err, PKV_ERR_TIMEOUT);
}

// Merge of the parts of split sequences.  A CTA of 512 threads takes `heads`
// query heads of one sequence; 16 lanes -- four dims each -- add up every
// (32 / heads)-th part of a head, weighted by 2^(m - M) / L, with everything a
// thread needs loaded at once: this kernel is latency (the end of the decode
// kernel seen, the record, the parts), about 3 us behind it.  The order is
// fixed, so the result does not depend on timing.  Many sequences have few parts
// each: 8 or 16 heads per CTA, and the 16 lanes find M and L themselves from all
// parts' (m, l), so that nothing is exchanged before the sums.  Few sequences
// have up to two parts per SM: one head per CTA, whose threads fetch one (m, l)
// each and exchange M, L and the weights (16 warps that each fetch all of 304
// cost 5 us).
constexpr int kMergeThreads = 512;
constexpr int kMergeBatch = 8;  // parts in flight per thread
constexpr int kKept = 4;        // of all parts' (m, l): those that a lane has in flight and keeps

// kPerSm: 1 has the registers for everything in flight (90), where one wave is
// enough; else two at a time matter more.
template <bool kOneHead, int kPerSm>
__global__ void __launch_bounds__(kMergeThreads, kPerSm) bs8_merge_kernel(const float* parts, const int2* span,
                                                                  uint16_t* out, int heads, int by_cta) {
  extern __shared__ float weights[];  // one head: of all parts
  __shared__ float4 sums[kMergeThreads / 32][16];
  __shared__ float tops[kMergeThreads / 32], dens[kMergeThreads / 32];
  if (kOneHead) heads = 1;
  const int ctas = PKV_NUM_Q_HEADS / heads;
  const int item = blockIdx.x / ctas;
  const int per = kMergeThreads / heads;  // threads of a head
  const int head = (blockIdx.x % ctas) * heads + threadIdx.x / per;
  const int group = (threadIdx.x % per) >> 4, groups = per >> 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & 15;
  const int dims = head * PKV_HEAD_DIM + 4 * sub, ml = PKV_NUM_Q_HEADS * PKV_HEAD_DIM + 2 * head;
  pdl_wait();
  pdl_launch_dependents();
  int2 c = span[item];
  if (c.x < 0) return;
  const int seq = by_cta ? c.x : item;
  if (by_cta) c.x = item;
  const int n = c.y - c.x + 1;
  // the sequence begins in its first CTA (slot 1) and continues in the others (slot 0)
  const float* base = parts + (size_t)c.x * 2 * kPartFloats;
  const auto part = [&](int i) { return base + ((size_t)i * 2 + (i == 0 ? 1 : 0)) * kPartFloats; };
  const auto ml_of = [&](int i) { return *reinterpret_cast<const float2*>(part(i) + ml); };

  float2 all[kKept];
  const int all0 = kOneHead ? threadIdx.x : sub, step = kOneHead ? kMergeThreads : 16;
#pragma unroll
  for (int u = 0; u < (kOneHead ? 1 : kKept); ++u)
    all[u] = all0 + step * u < n ? ml_of(all0 + step * u) : make_float2(-INFINITY, 0.f);
  float4 v[kMergeBatch];
  float mine[kMergeBatch];
#pragma unroll
  for (int u = 0; u < kMergeBatch; ++u) {
    const int i = group + u * groups;
    mine[u] = -INFINITY;
    v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < n) {
      if (!kOneHead) mine[u] = ml_of(i).x;
      v[u] = *reinterpret_cast<const float4*>(part(i) + dims);
    }
  }
  float m = all[0].x, sum = 0.f;
  bool bad = false;
  if (kOneHead) {
    for (int i = all0 + step; i < n; i += step) m = fmaxf(m, ml_of(i).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) tops[warp] = m;
    __syncthreads();
    for (int w = 0; w < kMergeThreads / 32; ++w) m = fmaxf(m, tops[w]);
    for (int i = all0; i < n; i += step) {
      const float2 e = i == all0 ? all[0] : ml_of(i);
      weights[i] = exp2_approx(e.x - m);
      sum = fmaf(e.y, weights[i], sum);
      bad |= e.y == kNothing;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) dens[warp] = sum;
    bad = __syncthreads_or(bad);
    sum = 0.f;
    for (int w = 0; w < kMergeThreads / 32; ++w) sum += dens[w];
  } else {
#pragma unroll
    for (int u = 1; u < kKept; ++u) m = fmaxf(m, all[u].x);
#pragma unroll 4
    for (int i = all0 + step * kKept; i < n; i += step) m = fmaxf(m, ml_of(i).x);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
    for (int u = 0; u < kKept; ++u) {
      if (all0 + step * u < n) sum = fmaf(all[u].y, exp2_approx(all[u].x - m), sum);
      bad |= all[u].y == kNothing;
    }
#pragma unroll 4
    for (int i = all0 + step * kKept; i < n; i += step) {
      const float2 e = ml_of(i);
      sum = fmaf(e.y, exp2_approx(e.x - m), sum);
      bad |= e.y == kNothing;
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    bad = (__ballot_sync(0xffffffffu, bad) >> (lane & 16) & 0xFFFFu) != 0;
  }

  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = group;; i0 += kMergeBatch * groups) {
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      if (i0 + u * groups >= n) continue;
      const float w = kOneHead ? weights[i0 + u * groups] : exp2_approx(mine[u] - m);
      acc.x = fmaf(w, v[u].x, acc.x);
      acc.y = fmaf(w, v[u].y, acc.y);
      acc.z = fmaf(w, v[u].z, acc.z);
      acc.w = fmaf(w, v[u].w, acc.w);
    }
    if (i0 + kMergeBatch * groups >= n) break;
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      const int i = i0 + (kMergeBatch + u) * groups;
      if (i < n) {
        if (!kOneHead) mine[u] = ml_of(i).x;
        v[u] = *reinterpret_cast<const float4*>(part(i) + dims);
      }
    }
  }
  __syncwarp();
  acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 16);
  acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 16);
  acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 16);
  acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 16);
  const int team = per >> 5;  // warps of a head
  if (team > 1) {
    if (lane < 16) sums[warp][lane] = acc;
    __syncthreads();
  }
  if (warp % team || lane >= 16) return;
  for (int w = warp + 1; w < warp + team; ++w) {
    const float4 e = sums[w][lane];
    acc.x += e.x;
    acc.y += e.y;
    acc.z += e.z;
    acc.w += e.w;
  }
  const float inv = kRaise * (1.f / sum);
  *reinterpret_cast<uint2*>(out + (size_t)seq * PKV_NUM_Q_HEADS * PKV_HEAD_DIM + dims) =
      bad ? make_uint2(0, 0)
          : make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

size_t parts_bytes(int sms) { return (size_t)sms * kCtasPerSm * 2 * kPartFloats * sizeof(float); }

size_t span_bytes(int sms, int num_seqs) {
  return sizeof(int2) * (size_t)(num_seqs > kBySequence ? sms * kCtasPerSm : num_seqs > 0 ? num_seqs : 1);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" size_t paged_gqa_decode_bs8_workspace_bytes(int num_seqs) {
  if (num_seqs < 0 || num_seqs > kMaxSeqsBs8) return 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  const int sms = sm_count(dev);
  if (sms <= 0) return 0;
  return parts_bytes(sms) + span_bytes(sms, num_seqs);
}

extern "C" int paged_gqa_decode_bs8(const void* q, const void* kv_pool, const float* kv_scales, int num_pages,
                                    int code_type, const int32_t* block_tables, int bt_row_stride,
                                    int max_blocks, const int32_t* seq_lens, int num_seqs, int max_seq_len,
                                    void* out, float scale, void* workspace, size_t workspace_bytes,
                                    int* d_err, void* stream) {
  if (num_seqs < 0 || num_pages < 1 || max_blocks < 1 || bt_row_stride < max_blocks || max_seq_len < 0 ||
      (code_type != PKV_BS8_INT8 && code_type != PKV_BS8_E4M3) || !isfinite(scale))
    return PKV_ERR_INVALID_ARGUMENT;
  if (num_seqs == 0) return PKV_OK;
  if (!q || !kv_pool || !kv_scales || !block_tables || !seq_lens || !out || !workspace)
    return PKV_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(kv_pool) || !aligned16(kv_scales) || !aligned16(out) || !aligned16(workspace) ||
      ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(seq_lens) |
        reinterpret_cast<uintptr_t>(d_err)) & 3u))
    return PKV_ERR_MISALIGNED;
  if (num_seqs > kMaxSeqsBs8 || (long long)max_blocks * num_seqs >= (1ll << 30)) return PKV_ERR_UNSUPPORTED_SHAPE;
  int dev = 0;
  int rc = bind_stream_device(stream, &dev);
  if (rc != PKV_OK) return rc;
  const int sms = sm_count(dev);
  if (sms <= 0) return cuda_status(cudaErrorInvalidDevice, "sm_count");
  if (workspace_bytes < parts_bytes(sms) + span_bytes(sms, num_seqs)) return PKV_ERR_WORKSPACE_TOO_SMALL;

  Bs8DecodeParams p;
  p.q = static_cast<const uint16_t*>(q);
  p.scales = kv_scales;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.out = static_cast<uint16_t*>(out);
  p.parts = static_cast<float*>(workspace);
  p.span = reinterpret_cast<int2*>(static_cast<uint8_t*>(workspace) + parts_bytes(sms));
  p.d_err = d_err;
  p.scale = scale;
  p.num_pages = num_pages;
  p.bt_stride = bt_row_stride;
  p.max_blocks = max_blocks;
  p.num_seqs = num_seqs;
  p.min_pages = kMinPages;

  CUtensorMap map;
  rc = make_bs8_map(&map, kv_pool, num_pages);
  if (rc != PKV_OK) return rc;
  const bool e4m3 = code_type == PKV_BS8_E4M3;
  // no more CTAs than the length bound can give work to (the shares follow the actual lengths)
  const long long longest = max_seq_len > 0 ? max_seq_len : (long long)max_blocks * PKV_PAGE_TOKENS;
  const long long most_pages = (longest + PKV_PAGE_TOKENS - 1) / PKV_PAGE_TOKENS;
  const bool whole = most_pages <= (num_seqs < 8 * (kWholePagesMost - kWholePages) ? kWholePages + num_seqs / 8 : kWholePagesMost);
  p.by_cta = !whole && num_seqs > kBySequence;
  long long ctas = whole ? num_seqs : (most_pages * num_seqs + kMinPages - 1) / kMinPages;
  if (ctas > (long long)sms * kCtasPerSm) ctas = (long long)sms * kCtasPerSm;
  if (ctas < 1) ctas = 1;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto* decode = e4m3 ? (whole ? bs8_decode_kernel<true, true> : bs8_decode_kernel<true, false>)
                      : (whole ? bs8_decode_kernel<false, true> : bs8_decode_kernel<false, false>);
  rc = cuda_status(cudaFuncSetAttribute(decode, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes),
                   "cudaFuncSetAttribute(decode bs8)");
  if (rc != PKV_OK) return rc;
  rc = cuda_status(cudaLaunchKernelEx(&cfg, decode, map, p), "cudaLaunchKernelEx(decode bs8)");
  if (rc != PKV_OK || ctas == 1 || whole) return rc;  // one CTA splits nothing
  // Heads per CTA of the merge.  1, 8 and 16 of them (us): 1 sequence of 131071 tokens 32.5,
  // 42.7, 48.4; 8 of 16384 29.8, 30.9, 32.0; 16 of 2048 15.6, 13.7, 13.7; 32 of 8192 55.5,
  // 50.3, 50.2; 39 of 2048 29.7, 24.3, 22.5; 256 of 2048 144, 105, 97.  Two CTAs per SM from
  // more CTAs than SMs on: 76 of 2048 (152 CTAs) 33.9, two per SM 35.5; 77 35.6 and 35.9;
  // 128 53.2 and 52.8; 256 of 1024 56.6 and 56.2.
  const int heads = num_seqs <= 8 ? 1 : num_seqs * 4 <= sms ? 8 : 16;
  const long long items = p.by_cta ? ctas - 1 : num_seqs;  // nothing goes on behind the last CTA
  cfg.gridDim = dim3((unsigned)(items * (PKV_NUM_Q_HEADS / heads)));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = heads == 1 ? (size_t)ctas * sizeof(float) : 0;
  const float* parts = p.parts;
  const int2* span = p.span;
  auto* merge = heads == 1 ? bs8_merge_kernel<true, 2>
                : (int)cfg.gridDim.x > sms ? bs8_merge_kernel<false, 2> : bs8_merge_kernel<false, 1>;
  return cuda_status(cudaLaunchKernelEx(&cfg, merge, parts, span, p.out, heads, p.by_cta), "cudaLaunchKernelEx(merge bs8)");
}
