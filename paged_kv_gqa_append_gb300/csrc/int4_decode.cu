// One decode step of grouped-query attention over pages of 4-bit codes with a scale
// and a minimum for every row, sm_103a.
//
// For sequence s with n tokens, KV head g and its query heads h (one pass with a
// running reference instead of the maximum, exponentials in base 2):
//   x_j = scale log2(e) (ks_j (q_h . ck_j) + kl_j sum q_h),   p_j = 2^(x_j - R)
//   out_h = (sum_j (p_j vs_j) cv_j + sum_j p_j vl_j) / sum_j p_j
// so scales and minima touch scores and probabilities only, and the codes 0..15
// themselves enter the MMAs.  A code is the fp16 number of the same bits, c 2^-24, or
// c 2^-20 where it stands 4 bits higher: two bit masks and one shift turn 32 bits into
// the eight codes as four registers of operands, and the factors cost nothing -- those
// of K go into q, those of V into the end.
//
// Tiles: a page is the 16 rows of m16n8k16.  S^T = K q^T has the four query heads twice
// in its eight columns, side by side, so a lane holds its score once for each copy: it
// computes one probability and puts the rounding to fp16 into one column and what that
// left into the other (22 bits in all), which the product O^T = V^T P^T has room for.
// The accumulators' layout is turned into the B operand's by movmatrix.  The order of a
// block (int4.cuh) gives each lane its 16 codes of K, 16 of V and scales as three
// 16-byte words.  Products of one page are added to the output's sums outside the tensor
// core, which would round them towards zero: with codes that are never negative that
// would add up.
//
// References: R is the next whole number over the largest score, set again only when four probabilities
// relative to it pass 8.  The weights p vs and p vl are multiplied by a power of two, `lift`, that brings the
// largest of p vs and p vl / 16 to 2^12 or more, below 2^13, set again only when four p vs pass 2^16 or four p vl
// 2^60 (int4_lift.cuh, with what makes both seldom): a head's sums are near that, whatever V's size.  So the usual
// step -- two pages -- has one vote, on sums that it needs anyway, and no reduction.
// What is merged are means, which neither overflow nor vanish for any V that bf16 holds, and their weights as R
// and a sum relative to 2^R: a sum of the two, or a logarithm, would lose the latter beside a large R.
//
// Work (three ways, chosen on the host by the caller's bound): a CTA for each sequence, a warp per KV head;
// a cluster for each sequence and KV head, the warps taking pairs of pages in turn and putting together what
// they found in shared memory; or equal shares of the list of all pages, with a merge behind them.  Blocks
// come to shared memory by asynchronous copies, each warp its own, two steps ahead; no barrier in the loop.
//
// Bound: the arithmetic pipes and memory alike.  A step is 16 HMMAs (8 cycles of an SM quarter each, during
// which it issues no FP32 operation either), some 80 FP32 and 120 integer operations (2 cycles), 80 of these
// for the unpacking: with 16 warps an SM takes 100 cycles for it (pages in the L2), as long as its share of
// the measured copy rate takes for the 2304 bytes; more warps do not help (24: the same).  300 sequences of
// 2048 tokens run at 78 % of the copy rate (67 us); 32 of 2048 tokens take 12.5 us (5.6 us of bytes), 97 ragged
// ones to 8191 54 us (33.5), one of 131071 24.4 us (11.1), one of 37 3.0 us; with near-equal scores and rows of one
// size the same to 0.4 us.  In shares 3.5 us go by before the first copy and 4 to 6 us in the merge; of 32
// sequences' 256 CTAs 104 SMs have two and 48 one.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "int4.cuh"
#include "int4_lift.cuh"
#include "internal.h"
#include "pkv.h"
#include "ptx.cuh"
#include "split_merge.cuh"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kHeads = PKV_NUM_KV_HEADS;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kPages = 2;                // of a stage: what a step takes
constexpr int kRing = 3;                 // stages on their way to a warp, and the one that it works on
constexpr int kStageBytes = kPages * kI4BlockBytes;
constexpr int kCtasPerSm = 2;
constexpr int kMaxSeqsInt4 = 4096;
constexpr int kMinPages = 4;             // least share of a CTA
constexpr int kList = 1024;              // page ids of a share held at a time (even)
constexpr int kMostCluster = 8;
constexpr float kStart = -FLT_MAX;       // R before the first score
constexpr float kMostLift = 0x1p126f;
// Means are merged 2^10 times smaller than they are, so that roundings beside bf16's largest do not overflow.
constexpr float kMeanDown = 0x1p-10f, kMeanUp = 0x1p10f;

struct Int4DecodeParams {
  const uint16_t* q;
  const uint8_t* pool;
  const int32_t *block_tables, *seq_lens;
  uint16_t* out;
  float* parts;
  int2* span;  // by sequence: first and last CTA of a split one; by CTA: the split sequence that begins
               // there and its last CTA; else (-1, -1)
  int* d_err;
  float scale;
  int num_pages, bt_stride, max_blocks, num_seqs, min_pages, by_cta, own;  // own: a CTA for each sequence
};

template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}

__device__ __forceinline__ void mma_add(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the product alone: zeros that need no registers
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// movmatrix_trans (ptx.cuh), free to move
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Pages of sequence s: none for an empty or refused one.
__device__ __forceinline__ int pages_of(const Int4DecodeParams& p, int s, bool& refused) {
  const int n = __ldg(p.seq_lens + s);
  refused = n < 0 || n > (long long)p.max_blocks * PKV_PAGE_TOKENS;
  return refused ? 0 : (int)(((unsigned)n + PKV_PAGE_TOKENS - 1) / PKV_PAGE_TOKENS);
}

// A warp's state for the four query heads of one KV head over some pages.  Lane (g, t) = 4 g + t
// has the scores of head t with slots g and g + 8, and dims 8 g .. 8 g + 7 of its output.
struct Group {
  uint32_t q[8];       // B operands of the four k-steps
  float fa, fb, fl;    // x = (S fa ks) fb + kl fl
  bool apart;          // some head's fa is not 1
  float ref, lift;
  float l, low;        // this lane's sum of p, of p vl lift
  float o[4][4];       // tile w: dims 8 g + 2 w (two columns), 8 g + 2 w + 1 (16 times too large), lifted

  // q of head g / 2, dims 16 t .. 16 t + 15
  __device__ static void fetch(const Int4DecodeParams& p, int seq, int head, uint4 (&raw)[2]) {
    static_assert(PKV_GROUP == 4, "two columns for each head of a group");
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint4* src = reinterpret_cast<const uint4*>(
        p.q + ((size_t)seq * PKV_NUM_Q_HEADS + head * PKV_GROUP + (g >> 1)) * PKV_HEAD_DIM + 16 * t);
    raw[0] = src[0];
    raw[1] = src[1];
  }

  __device__ void start(const uint4 (&raw)[2], float scale) {
    const int t = threadIdx.x & 3;
    float x[16];
    const uint32_t w[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
    uint32_t bits = 0;  // of the largest finite |q|: magnitudes order as their bits
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[2 * e] = bf16lo_to_f32(w[e]);
      x[2 * e + 1] = bf16hi_to_f32(w[e]);
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint32_t b = __float_as_uint(x[e]) & 0x7FFFFFFFu;
      bits = max(bits, b < 0x7F800000u ? b : 0u);
    }
    bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, 1));
    bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, 2));
    // 2^up brings it into [2^14, 2^15), unless it is 0; infinities and NaN stay what they are, in
    // their own head.  up lies in [-113, 141]: two factors keep each a normal number.
    const int up = bits ? 14 - ((int)(bits >> 23) - 127) : 0;
    const int u0 = up / 2, u1 = up - u0;
    const float f0 = __uint_as_float((uint32_t)(127 + u0) << 23), f1 = __uint_as_float((uint32_t)(127 + u1) << 23);
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      x[e] = x[e] * f0 * f1;
      sum += x[e];
    }
    // word i of K has dims 16 t + 8 i + (0..7), four bits each: those 4 apart share a register, and
    // every second pair is 16 times too large
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float* y = x + 8 * i + 2 * j;
        q[4 * i + 2 * j] = pack_f16x2(y[0], y[4]);
        q[4 * i + 2 * j + 1] = pack_f16x2(y[1] * 0.0625f, y[5] * 0.0625f);
      }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    const float c = scale * 1.4426950408889634f;
    const float d0 = __uint_as_float((uint32_t)(127 - u0) << 23), d1 = __uint_as_float((uint32_t)(127 - u1) << 23);
    // from the head of the q that this lane has to that of its scores
    // S is below 2, 2^-10 or more times the largest q of a code of 1: S ks overflows for no scale that bf16
    // holds, and where it loses bits (scales below 2^-116) the score is nothing unless d0 d1 c 2^24 is beyond
    // 2^90 -- then S is multiplied by a part of that first.
    const float both = d0 * 0x1p24f * (d1 * c);
    const bool far = !(fabsf(both) < 0x1p90f);
    fa = __shfl_sync(0xffffffffu, far ? d0 * 0x1p24f : 1.f, 8 * t);
    fb = __shfl_sync(0xffffffffu, far ? d1 * c : both, 8 * t);
    apart = __any_sync(0xffffffffu, far);
    fl = __shfl_sync(0xffffffffu, (sum * d0) * (d1 * c), 8 * t);
    ref = kStart;
    l = low = 0.f;
    lift = kMostLift;
#pragma unroll
    for (int w4 = 0; w4 < 4; ++w4)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[w4][e] = 0.f;
  }

  static constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u;
  static constexpr int kSlots = 2 * kPages;  // of a lane: g and g + 8 of either page

  // Two pages whose blocks are in shared memory, at this lane's first bytes; `live` of their 32 slots
  // are the sequence's.  A score is rounded before the reference is taken from it, so that equal ones
  // have equal probabilities whatever their size and whatever references they meet.
  __device__ __forceinline__ void step(uint32_t blocks, int live) {
    const int lane = threadIdx.x & 31, g = lane >> 2;
    const uint32_t words = blocks - 16 * (lane - g) + kI4Scales;
    float x[kSlots], p[kSlots], vs[kSlots], vl[kSlots];
#pragma unroll
    for (int u = 0; u < kPages; ++u) {
      const uint4 k = lds128(blocks + u * kI4BlockBytes);
      const uint4 sc = lds128(words + u * kI4BlockBytes);
      float s[4];
      mma_first(s, k.x & kLow, k.z & kLow, k.x & kHigh, k.z & kHigh, q[0], q[1]);
      mma_add(s, k.y & kLow, k.w & kLow, k.y & kHigh, k.w & kHigh, q[4], q[5]);
      const uint32_t a = k.x >> 8, b = k.z >> 8, c = k.y >> 8, d = k.w >> 8;
      mma_add(s, a & kLow, b & kLow, a & kHigh, b & kHigh, q[2], q[3]);
      mma_add(s, c & kLow, d & kLow, c & kHigh, d & kHigh, q[6], q[7]);
      if (apart) {
        s[0] *= fa;
        s[2] *= fa;
      }
      x[2 * u] = fmaf(s[0] * bf16lo_to_f32(sc.x), fb, bf16hi_to_f32(sc.x) * fl);
      x[2 * u + 1] = fmaf(s[2] * bf16lo_to_f32(sc.y), fb, bf16hi_to_f32(sc.y) * fl);
      p[2 * u] = exp2_approx(x[2 * u] - ref);
      p[2 * u + 1] = exp2_approx(x[2 * u + 1] - ref);
      vs[2 * u] = bf16lo_to_f32(sc.z);
      vl[2 * u] = bf16hi_to_f32(sc.z);
      vs[2 * u + 1] = bf16lo_to_f32(sc.w);
      vl[2 * u + 1] = bf16hi_to_f32(sc.w);
    }
    if (live < kPages * PKV_PAGE_TOKENS) {  // what lies behind the sequence's end may be anything
#pragma unroll
      for (int i = 0; i < kSlots; ++i)
        if (g + 8 * i >= live) {
          x[i] = -INFINITY;
          p[i] = vs[i] = vl[i] = 0.f;
        }
    }
    float y[kSlots], z[kSlots];
    const auto sum_of = [](const float (&v)[kSlots]) { return (v[0] + v[1]) + (v[2] + v[3]); };
    const auto weigh = [&]() {
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        const float lifted = p[i] * lift;
        y[i] = lifted * vs[i];
        z[i] = lifted * vl[i];
      }
    };
    weigh();
    float psum = sum_of(p), zsum = sum_of(z);
    if (__any_sync(0xffffffffu, i4_votes(psum, sum_of(y), zsum))) {
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) top = fmaxf(top, x[i]);
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float now = i4_reference(ref, top);
      const float keep = exp2_approx(ref - now);  // (a head whose reference stays: 1)
      l *= keep;
      // the lifted sums stay as they are, unless that lifts them too far
      const float more = fminf(lift * exp2_approx(now - ref), kMostLift);
      lower(more * keep / lift);
      lift = more;
      ref = now;
      float most = 0.f;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        p[i] = exp2_approx(x[i] - ref);
        most = fmaxf(most, p[i] * fmaxf(fabsf(vs[i]), 0.0625f * fabsf(vl[i])));
      }
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
      const float to = i4_lift(lift, most);
      if (to != lift) {  // (the same for all lanes of a head)
        lower(to / lift);
        lift = to;
      }
      weigh();
      psum = sum_of(p);
      zsum = sum_of(z);
      __syncwarp();
    }
    l += psum;
    low += zsum;
    uint32_t b0[kPages], b1[kPages];
    uint4 v[kPages];
#pragma unroll
    for (int u = 0; u < kPages; ++u) {
      // rounded to fp16, and what that leaves
      const uint32_t near = pack_f16x2(y[2 * u], y[2 * u + 1]);
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&near));
      const uint32_t rest = pack_f16x2(y[2 * u] - h.x, y[2 * u + 1] - h.y);
      b0[u] = transposed(__byte_perm(near, rest, 0x5410));
      b1[u] = transposed(__byte_perm(near, rest, 0x7632));
      v[u] = lds128(blocks + u * kI4BlockBytes + kI4V);  // slots 2 t, 2 t + 1 (x, y), and 8 more (z, w)
    }
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float d[4];
#pragma unroll
        for (int u = 0; u < kPages; ++u) {
          const uint32_t even = w ? v[u].y : v[u].x, odd = w ? v[u].w : v[u].z;
          const uint32_t a = j ? even >> 8 : even, b = j ? odd >> 8 : odd;
          if (u == 0) mma_first(d, a & kLow, a & kHigh, b & kLow, b & kHigh, b0[u], b1[u]);
          else mma_add(d, a & kLow, a & kHigh, b & kLow, b & kHigh, b0[u], b1[u]);
        }
        float* to = o[2 * w + j];
        const float2 f = add2(make_float2(to[0], to[1]), make_float2(d[0], d[1]));
        const float2 h = add2(make_float2(to[2], to[3]), make_float2(d[2], d[3]));
        to[0] = f.x;
        to[1] = f.y;
        to[2] = h.x;
        to[3] = h.y;
      }
  }

  __device__ __forceinline__ void lower(float by) {
    low *= by;
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[w][e] *= by;
  }

  // The means of dims 8 g .. 8 g + 7 of head t, times `unit`, and their weight: (R, the sum of the
  // probabilities relative to 2^R), (kStart, 0) and means of 0 where there were no pages.
  __device__ __forceinline__ float2 finish(float (&x)[8], float unit) {
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, d);
      low += __shfl_xor_sync(0xffffffffu, low, d);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l, down = unit / lift;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      x[2 * w] = fmaf(o[w][0] + o[w][1], 0x1p24f, low) * inv * down;
      x[2 * w + 1] = fmaf(o[w][2] + o[w][3], 0x1p20f, low) * inv * down;
    }
    return make_float2(ref, l);
  }
};

__device__ __forceinline__ void write_row(uint16_t* out, int seq, int head, const float (&x)[8], bool bad) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (!bad)
    v = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  *reinterpret_cast<uint4*>(out + ((size_t)seq * PKV_NUM_Q_HEADS + head * PKV_GROUP + t) * PKV_HEAD_DIM + 8 * g) = v;
}

// A warp's ring of stages, filled by its own asynchronous copies.
struct Ring {
  uint32_t base;        // this lane's first bytes of it
  const uint8_t* from;  // of the head's block of page 0
  int slot, next;       // worked on, and written next
  bool some;            // the lanes that a block's last 128 bytes go to
  __device__ __forceinline__ Ring(uint32_t at, const uint8_t* pool, int head)
      : base(at + 16 * (threadIdx.x & 31)),
        from(pool + (size_t)head * kI4BlockBytes + 16 * (threadIdx.x & 31)),
        slot(0),
        next(0),
        some((threadIdx.x & 31) < 8) {}
  __device__ __forceinline__ void copy(int u, int page) {
    const uint32_t dst = base + next + u * kI4BlockBytes;
    const uint8_t* src = from + (size_t)(uint32_t)page * kI4PageBytes;
    asm volatile(
        "cp.async.cg.shared.global [%0], [%1], 16;\n\t"
        "cp.async.cg.shared.global [%0 + 512], [%1 + 512], 16;" ::"r"(dst), "l"(src)
        : "memory");
    if (some) asm volatile("cp.async.cg.shared.global [%0 + 1024], [%1 + 1024], 16;" ::"r"(dst), "l"(src) : "memory");
  }
  __device__ __forceinline__ void commit() {
    cp_async_commit();
    next = next == (kRing - 1) * kStageBytes ? 0 : next + kStageBytes;
  }
  // the oldest stage has landed, for all lanes, and the one before it is no longer read; where this
  // lane's bytes of it are
  __device__ __forceinline__ uint32_t wait() {
    cp_async_wait<kRing - 2>();
    __syncwarp();
    const uint32_t here = base + slot;
    slot = slot == (kRing - 1) * kStageBytes ? 0 : slot + kStageBytes;
    return here;
  }
  __device__ __forceinline__ void restart() {
    cp_async_wait<0>();
    __syncwarp();
    slot = next = 0;
  }
};

struct alignas(16) Held {  // what a warp of the kernel for whole sequences has found: means and their weight (Group::finish)
  float o[PKV_GROUP][PKV_HEAD_DIM];
  float2 weight[PKV_GROUP];
  int bad;
};

// One sequence and KV head for each cluster of CTAs (of one or more): every warp takes every
// (warps)-th pair of pages, and what they find is put together in shared memory, over the cluster's CTAs
// too.  Nothing goes through global memory.
__global__ void __launch_bounds__(kThreads, kCtasPerSm) int4_whole_kernel(const Int4DecodeParams p) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ Held sum;
  const cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)gridDim.x, rank = (int)blockIdx.x;
  const int head = blockIdx.y, seq = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  bool refused;
  const int pages = pages_of(p, seq, refused), len = __ldg(p.seq_lens + seq);
  uint16_t* out = p.out + ((size_t)seq * PKV_NUM_Q_HEADS + head * PKV_GROUP) * PKV_HEAD_DIM;
  if (pages == 0) {
    if (rank == 0 && warp == 0) reinterpret_cast<uint4*>(out)[lane] = make_uint4(0, 0, 0, 0);
    if (refused && rank == 0 && threadIdx.x == 0) report_error(p.d_err, PKV_ERR_DEVICE_INDEX);
    return;
  }
  // pairs of pages: this warp's first one, and the distance to the next
  const int first = rank * kWarps + warp, stride = ctas * kWarps, pairs = (pages + 1) / kPages;
  const int count = first < pairs ? (pairs - first + stride - 1) / stride : 0;
  const int32_t* table = p.block_tables + (size_t)seq * p.bt_stride;
  bool bad = false;
  // ids of 16 pairs, and of the 16 behind them under way
  const auto ids = [&](int i) {
    const int at = (first + (i + (lane >> 1)) * stride) * kPages + (lane & 1);
    if (i + (lane >> 1) >= count || at >= pages) return 0;
    const int id = __ldg(table + at);
    const bool ok = id >= 0 && id < p.num_pages;
    bad |= !ok;
    return ok ? id : 0;
  };
  int id = ids(0), coming = count > 16 ? ids(16) : 0;
  uint4 raw[2];
  Group::fetch(p, seq, head, raw);
  Ring ring(smem_u32(dyn) + warp * (kRing * kStageBytes), p.pool, head);
  const auto issue = [&](int i) {
    if (i < count) {
      if (i && (i & 15) == 0) {
        id = coming;
        coming = ids(i + 16);
      }
#pragma unroll
      for (int u = 0; u < kPages; ++u) ring.copy(u, __shfl_sync(0xffffffffu, id, (2 * i + u) & 31));
    }
    ring.commit();
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) issue(i);
  Group st;
  st.start(raw, p.scale);
  for (int i = 0; i < count; ++i) {
    const uint32_t blocks = ring.wait();
    st.step(blocks, len - (first + i * stride) * (kPages * PKV_PAGE_TOKENS));
    issue(i + kRing - 1);
  }
  float x[8];
  const float2 weight = st.finish(x, kMeanDown);
  // into the warp's own ring, which nothing is on its way to any more
  static_assert(sizeof(Held) <= kRing * kStageBytes && kI4BlockBytes % 16 == 0, "room for what a warp found");
  cp_async_wait<0>();
  __syncwarp();
  Held* mine = reinterpret_cast<Held*>(dyn + warp * (kRing * kStageBytes));
  {
    const int g = lane >> 2, t = lane & 3;
    float4* to = reinterpret_cast<float4*>(mine->o[t] + 8 * g);
    to[0] = make_float4(x[0], x[1], x[2], x[3]);
    to[1] = make_float4(x[4], x[5], x[6], x[7]);
    if (g == 0) mine->weight[t] = weight;
  }
  bad = __syncthreads_or(bad);
  if (bad && threadIdx.x == 0) report_error(p.d_err, PKV_ERR_DEVICE_INDEX);
  const int h = threadIdx.x / PKV_HEAD_DIM, d = threadIdx.x % PKV_HEAD_DIM;
  static_assert(kThreads == PKV_GROUP * PKV_HEAD_DIM, "a thread for each output");
  const auto of = [&](int w) { return reinterpret_cast<const Held*>(dyn + w * (kRing * kStageBytes)); };
  float ref = kStart, o = 0.f, total = 0.f, scaled[kWarps];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) ref = fmaxf(ref, of(w)->weight[h].x);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += scaled[w] = exp2_approx(of(w)->weight[h].x - ref) * of(w)->weight[h].y;
  const float inv = total == 0.f ? 0.f : 1.f / total;  // (a CTA that no pages are left for: 0)
#pragma unroll
  for (int w = 0; w < kWarps; ++w) o = fmaf(scaled[w] * inv, of(w)->o[h][d], o);
  if (ctas == 1) {
    const float y = bad ? 0.f : o * kMeanUp, z = __shfl_down_sync(0xffffffffu, y, 1);
    if (d % 2 == 0) *reinterpret_cast<uint32_t*>(out + threadIdx.x) = pack_bf16x2(y, z);
    return;
  }
  sum.o[h][d] = o;
  if (d == 0) sum.weight[h] = make_float2(ref, total);
  if (threadIdx.x == 0) sum.bad = bad;
  cluster.sync();
  // each CTA an equal part of the 256 outputs, a thread two of them
  const int at = rank * (kThreads / ctas) + 2 * (int)threadIdx.x;
  if (2 * (int)threadIdx.x < kThreads / ctas) {
    const int hh = at / PKV_HEAD_DIM, dd = at % PKV_HEAD_DIM;
    ref = kStart;
    total = 0.f;
    bad = false;
    float2 weights[kMostCluster], means[kMostCluster], y = make_float2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < kMostCluster; ++c) {
      const Held* other = cluster.map_shared_rank(&sum, c < ctas ? c : 0);
      weights[c] = c < ctas ? other->weight[hh] : make_float2(kStart, 0.f);
      means[c] = c < ctas ? *reinterpret_cast<const float2*>(other->o[hh] + dd) : make_float2(0.f, 0.f);
      if (c < ctas) bad |= other->bad != 0;
    }
#pragma unroll
    for (int c = 0; c < kMostCluster; ++c) ref = fmaxf(ref, weights[c].x);
#pragma unroll
    for (int c = 0; c < kMostCluster; ++c) {
      weights[c].x = exp2_approx(weights[c].x - ref) * weights[c].y;
      total += weights[c].x;
    }
    const float inv = 1.f / total;
#pragma unroll
    for (int c = 0; c < kMostCluster; ++c) {
      const float scaled = weights[c].x * inv;
      y.x = fmaf(scaled, means[c].x, y.x);
      y.y = fmaf(scaled, means[c].y, y.y);
    }
    *reinterpret_cast<uint32_t*>(out + at) = bad ? 0u : pack_bf16x2(y.x * kMeanUp, y.y * kMeanUp);
  }
  cluster.sync();  // nobody's shared memory goes while it is read
}

struct ShareSmem {
  int sum[kWarps];
  int first_seq, before;  // the sequence that the CTA's share begins in, and the pages before that
  int bad;                // ids among the listed ones that cannot be one
  alignas(8) int list[kList];  // page ids in pairs of one sequence; 0 for one that cannot be and behind an odd one
  uint32_t wrong[kList / 32];   // those that cannot be
};

// The pages of all sequences are one long list; every CTA takes an equal share of it, whatever the
// lengths, one KV head per warp.  Parts of split sequences go to the workspace (split_merge.cuh).
__global__ void __launch_bounds__(kThreads, kCtasPerSm) int4_share_kernel(const Int4DecodeParams p) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ ShareSmem sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();

  // Where this CTA's share of the list of pages (below 2^30 of them) begins.
  int begin, end, seq, page;
  unsigned share;
  const auto shares = [&](int total) {
    share = max(((unsigned)total + gridDim.x - 1) / gridDim.x, (unsigned)p.min_pages);
    begin = (int)min((unsigned)total, share * blockIdx.x);
    end = min(total, begin + (int)share);
  };
  const auto record = [&](int s, int at, int n, bool refused) {
    if (s % (int)gridDim.x != (int)blockIdx.x) return;
    if (!p.by_cta) {
      const int c0 = (int)((unsigned)at / share), c1 = n ? (int)((unsigned)(at + n - 1) / share) : c0;
      p.span[s] = c0 == c1 ? make_int2(-1, -1) : make_int2(c0, c1);
    }
    if (n == 0) {
      uint4* row = reinterpret_cast<uint4*>(p.out + (size_t)s * PKV_NUM_Q_HEADS * PKV_HEAD_DIM);
      for (int i = 0; i < PKV_NUM_Q_HEADS * PKV_HEAD_DIM / 8; ++i) row[i] = make_uint4(0, 0, 0, 0);
      if (refused) report_error(p.d_err, PKV_ERR_DEVICE_INDEX);
    }
  };
  if (p.own) {
    bool refused;
    pdl_launch_dependents();
    seq = blockIdx.x;
    begin = page = 0;
    end = pages_of(p, seq, refused);
    share = max(end, 1);
    if (end == 0 && warp == 0) {
      uint4* row = reinterpret_cast<uint4*>(p.out + (size_t)seq * PKV_NUM_Q_HEADS * PKV_HEAD_DIM);
      for (int i = lane; i < PKV_NUM_Q_HEADS * PKV_HEAD_DIM / 8; i += 32) row[i] = make_uint4(0, 0, 0, 0);
      if (refused && lane == 0) report_error(p.d_err, PKV_ERR_DEVICE_INDEX);
    }
  } else if (p.num_seqs <= 32) {  // every warp finds out by itself
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
  } else {  // a thread's sequences, then the sums over all
    const int per = (p.num_seqs + kThreads - 1) / kThreads;
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
    for (int w = 0; w < kWarps; ++w) {
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
  if (begin >= end) {
    if (p.by_cta && threadIdx.x == 0) p.span[blockIdx.x] = make_int2(-1, -1);
    return;
  }

  const int head = warp;
  Ring ring(smem_u32(dyn) + warp * (kRing * kStageBytes), p.pool, head);
  int2 split = make_int2(-1, -1);  // the sequence that begins here and goes on, and its last CTA
  bool refused, bad = false;
  int pages = pages_of(p, seq, refused), from = page;
  int left = __ldg(p.seq_lens + seq) - page * PKV_PAGE_TOKENS;  // tokens from the next page on
  int list_seq = seq, list_page = page, list_at = begin;
  uint4 raw[2];
  Group::fetch(p, seq, head, raw);
  Group st;
  st.start(raw, p.scale);
  for (int at = begin; at < end;) {
    if (at > begin) __syncthreads();  // the last ids are no longer read
    if (threadIdx.x == 0) sh.bad = 0;
    if (threadIdx.x < kList / 32) sh.wrong[threadIdx.x] = 0;
    __syncthreads();
    int items = 0;
    while (list_at < end && items < kList) {  // the ids of the next pages, sequence by sequence
      const int n = pages_of(p, list_seq, refused), some = min(min(n - list_page, end - list_at), kList - items);
      const int32_t* table = p.block_tables + (size_t)list_seq * p.bt_stride + list_page;
      for (int j = threadIdx.x; j < some + (some & 1); j += kThreads) {
        const int id = j < some ? __ldg(table + j) : 0;
        const bool ok = id >= 0 && id < p.num_pages;
        sh.list[items + j] = ok ? id : 0;
        if (!ok) {
          sh.bad = 1;
          atomicOr(&sh.wrong[(items + j) / 32], 1u << (items + j) % 32);
          report_error(p.d_err, PKV_ERR_DEVICE_INDEX);
        }
      }
      items += some + (some & 1);
      list_at += some;
      list_page += some;
      if (list_page == n) {
        list_page = 0;
        do ++list_seq;
        while (list_seq < p.num_seqs && pages_of(p, list_seq, refused) == 0);
      }
    }
    __syncthreads();
    const bool any_bad = sh.bad != 0;
    const auto issue = [&](int i) {
      if (i < items) {
        const int2 id = *reinterpret_cast<const int2*>(sh.list + i);
        ring.copy(0, id.x);
        ring.copy(1, id.y);
      }
      ring.commit();
    };
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) issue(i * kPages);
    for (int i = 0; i < items; i += kPages) {
      const uint32_t blocks = ring.wait();
      const int n = min(kPages, min(pages - page, end - at));
      if (any_bad) bad |= (sh.wrong[i / 32] >> i % 32 & 3u) != 0;  // (the one behind an odd page is not)
      st.step(blocks, min(n * PKV_PAGE_TOKENS, left));
      issue(i + (kRing - 1) * kPages);
      page += n;
      at += n;
      left -= n * PKV_PAGE_TOKENS;
      if (page < pages && at < end) continue;
      // the end of the sequence, or of the share inside it
      float x[8];
      const bool all = from == 0 && page == pages;
      const float2 weight = st.finish(x, all ? 1.f : kMeanDown);
      if (all) {
        write_row(p.out, seq, head, x, bad);
      } else {
        const int g = lane >> 2, t = lane & 3, hq = head * PKV_GROUP + t;
        float* part = p.parts + ((size_t)blockIdx.x * 2 + (from > 0 ? 0 : 1)) * kPartFloats;
        float4* to = reinterpret_cast<float4*>(part + hq * PKV_HEAD_DIM + 8 * g);
        to[0] = make_float4(x[0], x[1], x[2], x[3]);
        to[1] = make_float4(x[4], x[5], x[6], x[7]);
        if (g == 0)
          *reinterpret_cast<float2*>(part + PKV_NUM_Q_HEADS * PKV_HEAD_DIM + 2 * hq) =
              make_float2(weight.x, bad ? kNothing : weight.y);
        if (from == 0) split = make_int2(seq, (int)((unsigned)(at - page + pages - 1) / share));
      }
      if (at < end) {
        do ++seq;
        while (seq < p.num_seqs && (pages = pages_of(p, seq, refused)) == 0);
        left = __ldg(p.seq_lens + seq);
        page = from = 0;
        bad = false;
        Group::fetch(p, seq, head, raw);
        st.start(raw, p.scale);
      }
    }
    ring.restart();
  }
  if (p.by_cta && threadIdx.x == 0) p.span[blockIdx.x] = split;
}

constexpr int kSmemBytes = kWarps * kRing * kStageBytes;

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" size_t paged_gqa_decode_int4_workspace_bytes(int num_seqs) {
  if (num_seqs < 0 || num_seqs > kMaxSeqsInt4) return 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  const int sms = sm_count(dev);
  if (sms <= 0) return 0;
  return parts_bytes(sms * kCtasPerSm) + span_bytes(sms * kCtasPerSm, num_seqs);
}

extern "C" int paged_gqa_decode_int4(const void* q, const void* kv_pool, int num_pages, const int32_t* block_tables,
                                     int bt_row_stride, int max_blocks, const int32_t* seq_lens, int num_seqs,
                                     int max_seq_len, void* out, float scale, void* workspace,
                                     size_t workspace_bytes, int* d_err, void* stream) {
  if (num_seqs < 0 || num_pages < 1 || max_blocks < 1 || bt_row_stride < max_blocks || max_seq_len < 0 || !isfinite(scale))
    return PKV_ERR_INVALID_ARGUMENT;
  if (num_seqs == 0) return PKV_OK;
  if (!q || !kv_pool || !block_tables || !seq_lens || !out || !workspace) return PKV_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(kv_pool) || !aligned16(out) || !aligned16(workspace) ||
      ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(seq_lens) |
        reinterpret_cast<uintptr_t>(d_err)) & 3u))
    return PKV_ERR_MISALIGNED;
  if (num_seqs > kMaxSeqsInt4 || (long long)max_blocks * num_seqs >= (1ll << 30)) return PKV_ERR_UNSUPPORTED_SHAPE;
  int dev = 0;
  int rc = bind_stream_device(stream, &dev);
  if (rc != PKV_OK) return rc;
  const int sms = sm_count(dev);
  if (sms <= 0) return cuda_status(cudaErrorInvalidDevice, "sm_count");
  const int most = sms * kCtasPerSm;
  if (workspace_bytes < parts_bytes(most) + span_bytes(most, num_seqs)) return PKV_ERR_WORKSPACE_TOO_SMALL;

  Int4DecodeParams p;
  p.q = static_cast<const uint16_t*>(q);
  p.pool = static_cast<const uint8_t*>(kv_pool);
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.out = static_cast<uint16_t*>(out);
  p.parts = static_cast<float*>(workspace);
  p.span = reinterpret_cast<int2*>(static_cast<uint8_t*>(workspace) + parts_bytes(most));
  p.d_err = d_err;
  p.scale = scale;
  p.num_pages = num_pages;
  p.bt_stride = bt_row_stride;
  p.max_blocks = max_blocks;
  p.num_seqs = num_seqs;
  p.min_pages = kMinPages;

  const long long longest = max_seq_len > 0 ? max_seq_len : (long long)max_blocks * PKV_PAGE_TOKENS;
  const long long most_pages = (longest + PKV_PAGE_TOKENS - 1) / PKV_PAGE_TOKENS;
  // How the work is split, by the caller's bound (us: a CTA per sequence / clusters / shares):
  //  - a CTA for each of many sequences, if they are short, or if such CTAs keep the SMs about as busy as
  //    shares would: 80 of 8 pages 7.0 / 9.6 / 11.3, 256 of 16 13.4 / 28.8 / 21.9, 2000 ragged to 4 38 /
  //    - / 48, 300 of 128 66 / - / 79; 100 of 64 23.6 / 22.2 / 23.1, 64 of 32 14.1 / 11.6 / 15.0;
  //  - else a cluster for each sequence and KV head, as many CTAs as two for each SM allow, as long as
  //    these take few pages each: 1 of 128 pages - / 4.5 / 7.7, 4 of 128 - / 5.5 / 8.2, 32 of 128 - / 12.3 /
  //    17.6, 64 of 128 - / 22.4 / 24.7;
  //  - else shares: 1 of 8192 pages - / 39.9 / 24.0, 97 ragged to 512 - / 58 / 54.  (Between the two clusters are
  //    ahead by now, 1 of 1024 - / 9.6 / 10.9, 32 of 512 - / 33.3 / 37.7; the limits are where both were even.)
  const int slots = kCtasPerSm * sms, waves = (num_seqs + slots - 1) / slots;
  const double busy = num_seqs <= sms ? 0.86 * num_seqs / sms : (double)num_seqs / (waves * slots);
  p.own = 2 * num_seqs > sms && (most_pages <= 24 || (most_pages <= 128 && busy >= 0.6));
  int ctas = 1;
  while (ctas < kMostCluster && num_seqs * kHeads * ctas * 2 <= slots && most_pages > ctas * kWarps) ctas *= 2;
  const bool whole = !p.own && most_pages <= 64 * (ctas + 1) && most_pages * num_seqs <= 64 * 128;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  auto* kernel = whole ? int4_whole_kernel : int4_share_kernel;
  rc = cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes),
                   "cudaFuncSetAttribute(decode int4)");
  if (rc != PKV_OK) return rc;
  if (whole) {
    p.by_cta = 0;
    cfg.gridDim = dim3((unsigned)ctas, kHeads, (unsigned)num_seqs);
    cfg.numAttrs = 2;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, p), "cudaLaunchKernelEx(decode int4)");
  }
  p.by_cta = !p.own && num_seqs > kBySequence;
  // no more CTAs than the bound can give work to (the shares follow the actual lengths)
  long long shares = p.own ? num_seqs : (most_pages * num_seqs + kMinPages - 1) / kMinPages;
  if (!p.own && shares > most) shares = most;
  if (shares < 1) shares = 1;
  cfg.gridDim = dim3((unsigned)shares);
  cfg.numAttrs = 1;
  rc = cuda_status(cudaLaunchKernelEx(&cfg, kernel, p), "cudaLaunchKernelEx(decode int4)");
  if (rc != PKV_OK || shares == 1 || p.own) return rc;  // nothing is split
  return launch_merge<true>(cfg, p.parts, p.span, p.out, num_seqs, (int)shares, p.by_cta, sms, kMeanUp, "cudaLaunchKernelEx(merge int4)");
}
