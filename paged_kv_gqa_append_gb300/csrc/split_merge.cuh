// Sequences split over CTAs: the parts that the decode kernels over quantised pages
// (bs8_decode.cu, int4_decode.cu) leave, and their merge.
//
// Every CTA of such a kernel takes an equal share of the list of all pages.  A share
// that begins or ends inside a sequence leaves a part of it: o [64] and (m, l) for each
// of the 32 heads, l the sum of its probabilities relative to 2^m (kNothing: it has a bad
// page).  o is the sum over V, not divided, relative to 2^m (8 bits), or that divided by l
// (4 bits: sums that neither overflow nor vanish whatever V's size).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "pkv.h"
#include "ptx.cuh"

namespace pkv {
namespace {

// Up to this many sequences the merge looks at every sequence; beyond it at every
// CTA, in each of which one split sequence begins at most (8-bit codes, 4096 sequences of
// 64 tokens in shares: 72 us, by sequence 93 us; 1000 ragged ones to 300: 46 and 51 us;
// 256 of 2048: 95.5 us both; 97 ragged ones to 8191: 73.7 and 72.6 us).
constexpr int kBySequence = 128;
constexpr float kNothing = -1.f;  // l of a part with a bad page

// Workspace: per CTA two parts (of a sequence begun in an earlier CTA, and of
// one that goes on in the next) of 32 heads, o [64] then (m, l) pairs; then
// which CTAs a split sequence lies in, by sequence or by CTA.
constexpr int kPartFloats = PKV_NUM_Q_HEADS * (PKV_HEAD_DIM + 2);

inline size_t parts_bytes(int ctas) { return (size_t)ctas * 2 * kPartFloats * sizeof(float); }

inline size_t span_bytes(int ctas, int num_seqs) {
  return sizeof(int2) * (size_t)(num_seqs > kBySequence ? ctas : num_seqs > 0 ? num_seqs : 1);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Merge of the parts of split sequences.  A CTA of 512 threads takes `heads`
// query heads of one sequence; 16 lanes -- four dims each -- add up every
// (32 / heads)-th part of a head, weighted by 2^(m - M) / L, with everything a
// thread needs loaded at once: this kernel is latency (the end of the decode
// kernel seen, the record, the parts), about 3 us behind it.  The order is
// fixed, so the result does not depend on timing.  kMeans: the parts' o are divided by
// their l, which then belongs to their weight.  Many sequences have few parts
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
template <bool kOneHead, int kPerSm, bool kMeans>
__global__ void __launch_bounds__(kMergeThreads, kPerSm) split_merge_kernel(const float* parts, const int2* span,
                                                                   uint16_t* out, int heads, int by_cta, float raise) {
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
      const float w = exp2_approx(e.x - m);
      weights[i] = kMeans ? w * e.y : w;
      sum = fmaf(e.y, w, sum);
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

  const float inv = 1.f / sum;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = group;; i0 += kMergeBatch * groups) {
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      const int i = i0 + u * groups;
      if (i >= n) continue;
      float w = kOneHead ? weights[i] : exp2_approx(mine[u] - m);
      if (kMeans) w *= kOneHead ? inv : ml_of(i).y * inv;  // (l is in the L1 since (m, l) was fetched)
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
  const float by = kMeans ? raise : raise * inv;
  *reinterpret_cast<uint2*>(out + (size_t)seq * PKV_NUM_Q_HEADS * PKV_HEAD_DIM + dims) =
      bad ? make_uint2(0, 0)
          : make_uint2(pack_bf16x2(acc.x * by, acc.y * by), pack_bf16x2(acc.z * by, acc.w * by));
}

// The merge behind a decode of `ctas` CTAs, with the attributes and the stream of `cfg`; `raise`
// multiplies the results.
//
// Heads per CTA of the merge.  1, 8 and 16 of them (us, 8-bit codes): 1 sequence of 131071
// tokens 32.5, 42.7, 48.4; 8 of 16384 29.8, 30.9, 32.0; 16 of 2048 15.6, 13.7, 13.7; 32 of
// 8192 55.5, 50.3, 50.2; 39 of 2048 29.7, 24.3, 22.5; 256 of 2048 144, 105, 97.  Two CTAs per
// SM from more CTAs than SMs on: 76 of 2048 (152 CTAs) 33.9, two per SM 35.5; 77 35.6 and
// 35.9; 128 53.2 and 52.8; 256 of 1024 56.6 and 56.2.
template <bool kMeans>
int launch_merge(cudaLaunchConfig_t cfg, const float* parts, const int2* span, uint16_t* out, int num_seqs,
                 int ctas, int by_cta, int sms, float raise, const char* what) {
  const int heads = num_seqs <= 8 ? 1 : num_seqs * 4 <= sms ? 8 : 16;
  const long long items = by_cta ? ctas - 1 : num_seqs;  // nothing goes on behind the last CTA
  cfg.gridDim = dim3((unsigned)(items * (PKV_NUM_Q_HEADS / heads)));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = heads == 1 ? (size_t)ctas * sizeof(float) : 0;
  auto* merge = heads == 1 ? split_merge_kernel<true, 2, kMeans>
                : (int)cfg.gridDim.x > sms ? split_merge_kernel<false, 2, kMeans> : split_merge_kernel<false, 1, kMeans>;
  return cuda_status(cudaLaunchKernelEx(&cfg, merge, parts, span, out, heads, by_cta, raise), what);
}

}  // namespace
}  // namespace pkv
