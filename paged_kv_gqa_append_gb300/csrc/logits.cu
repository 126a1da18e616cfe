// Penalties, biases and a grammar's mask on next-token logits, and the
// selection of the next token, in one pass over the logits (sm_103a).
//
// Row r, token i, x = logits[r][i] in fp32, every operation rounded to nearest:
//   seen(i): i is in the row's history;  n(i): how often in its generated part
//   1. seen:    x = x > 0 ? x / repetition : x * repetition
//   2. n > 0:   x = x - frequency * n, then x = x - presence
//   3. biased:  x = x + bias        (the last entry of an id counts)
//   4. masked out: x = -inf
// and the id chosen is the first of the largest non-NaN x among the tokens
// that the mask leaves, -1 if there is none.
//
// A cluster of 8 CTAs handles a row, each a contiguous eighth of the
// vocabulary (a multiple of 32 tokens, one mask word).  A CTA keeps one word
// per token of its part in shared memory -- how often it was generated,
// whether it was seen at all, and the last bias entry + 1 -- and fills it from
// the row's whole history and bias list, which it reads from L2: integer
// atomics in its own shared memory, the same words in any order.  (Reading an
// eighth each and adding through distributed shared memory took two cluster
// barriers, and cost more than the reads.)  Then the part is streamed once, 16
// bytes at a time, each thread keeping its best (value, id); warp shuffles,
// shared memory and the cluster's first CTA reduce them under a total order.
// The first loads of the stream are issued before the words are built.
//
// The word is 32 bits: 10 of bias entry, 1 seen, 21 of count, so that a part
// of the 128256-token vocabulary is 64 KiB and three CTAs share an SM.  Longer
// histories or more biases take 64-bit words; parts larger than the table go
// in passes.
//
// Bound: memory, the logits read (and written, when they are kept).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "internal.h"
#include "pkv.h"
#include "ptx.cuh"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kCtas = 8;
constexpr int kTableBytes = 65536;
constexpr int kBatch = 8;  // 16-byte loads in flight per thread

template <typename W>
struct Word;
template <>
struct Word<uint32_t> {
  static constexpr int kEntry = 22;
  static constexpr uint32_t kSeen = 1u << 21;
  static constexpr long long kMostHistory = (1 << 21) - 1, kMostBiases = (1 << 10) - 1;
};
template <>
struct Word<unsigned long long> {
  static constexpr int kEntry = 32;
  static constexpr unsigned long long kSeen = 1ull << 31;
};

struct LogitsParams {
  const void* logits;
  long long stride, out_stride, hist_stride, bias_stride, mask_stride;
  float* out;
  int32_t* ids;
  const int32_t *history, *history_lens, *prompt_lens;
  const float *repetition, *presence, *frequency;
  const int32_t* bias_ids;
  const float* bias_values;
  const uint32_t* mask;
  int vocab, part, table, bias_count;  // tokens per CTA, tokens per pass
};

// 16 bytes of logits in fp32
__device__ __forceinline__ void widen(const uint4& a, float (&v)[4], const float*) {
  v[0] = __uint_as_float(a.x);
  v[1] = __uint_as_float(a.y);
  v[2] = __uint_as_float(a.z);
  v[3] = __uint_as_float(a.w);
}
__device__ __forceinline__ void widen(const uint4& a, float (&v)[8], const __nv_bfloat16*) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = bf16lo_to_f32(w[e]);
    v[2 * e + 1] = bf16hi_to_f32(w[e]);
  }
}
__device__ __forceinline__ void widen(const uint4& a, float (&v)[8], const __half*) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
    v[2 * e] = f.x;
    v[2 * e + 1] = f.y;
  }
}
__device__ __forceinline__ float load1(const float* x) { return __ldcs(x); }
__device__ __forceinline__ float load1(const __nv_bfloat16* x) { return __bfloat162float(*x); }
__device__ __forceinline__ float load1(const __half* x) { return __half2float(*x); }

// (v, i) comes before (bv, bi): larger, or equal and lower; i < 0 is nothing, a NaN never wins
__device__ __forceinline__ void take(float v, int i, float& bv, int& bi) {
  if (i < 0 || v != v) return;
  if (bi < 0 || v > bv || (v == bv && i < bi)) {
    bv = v;
    bi = i;
  }
}

struct Row {
  float rep, pres, freq;
  const float* bias;
};

// steps 1 to 3 for a token whose word is not 0
template <typename W>
__device__ __forceinline__ float change(float x, W word, const Row& r) {
  using L = Word<W>;
  const uint32_t n = (uint32_t)(word & (L::kSeen - 1));
  if (word & (L::kSeen | (L::kSeen - 1))) x = x > 0.f ? __fdiv_rn(x, r.rep) : __fmul_rn(x, r.rep);
  if (n) {
    x = __fsub_rn(x, __fmul_rn(r.freq, (float)n));
    x = __fsub_rn(x, r.pres);
  }
  const uint32_t entry = (uint32_t)(word >> L::kEntry);
  if (entry) x = __fadd_rn(x, __ldg(r.bias + entry - 1));
  return x;
}

template <typename T, typename W>
__global__ void __launch_bounds__(kThreads, 3) logits_kernel(const LogitsParams p) {
  using L = Word<W>;
  constexpr int N = 16 / (int)sizeof(T);  // tokens per 16 bytes
  extern __shared__ __align__(16) uint8_t dyn[];
  W* const table = reinterpret_cast<W*>(dyn);
  __shared__ float best_v[kThreads / 32], part_v[kCtas];
  __shared__ int best_i[kThreads / 32], part_i[kCtas];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int row = blockIdx.x / kCtas;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  cluster.barrier_arrive();  // waited for before the first write into another CTA's shared memory
  pdl_wait();
  pdl_launch_dependents();

  const T* x = static_cast<const T*>(p.logits) + (size_t)row * (size_t)p.stride;
  float* out = p.out ? p.out + (size_t)row * (size_t)p.out_stride : nullptr;
  const uint32_t* mask = p.mask ? p.mask + (size_t)row * (size_t)p.mask_stride : nullptr;
  Row r{1.f, 0.f, 0.f, p.bias_values + (size_t)row * (size_t)p.bias_stride};
  int hist = 0, prompt = 0;
  if (p.history) {
    hist = (int)max(0ll, min((long long)__ldg(p.history_lens + row), p.hist_stride));
    prompt = p.prompt_lens ? __ldg(p.prompt_lens + row) : 0;
    if (p.repetition) r.rep = __ldg(p.repetition + row);
    if (p.presence) r.pres = __ldg(p.presence + row);
    if (p.frequency) r.freq = __ldg(p.frequency + row);
  }
  const bool tables = hist > 0 || p.bias_count > 0;

  float bv = -INFINITY;
  int bi = -1;
  for (int base = 0; base < p.part; base += p.table) {
    const long long first = (long long)rank * p.part + base;
    const int size = min(p.table, p.part - base);  // tokens of this pass
    const int n = (int)max(0ll, min((long long)size, (long long)p.vocab - first));
    const bool wide = ((reinterpret_cast<uintptr_t>(x + first) | (out ? reinterpret_cast<uintptr_t>(out + first) : 0)) & 15u) == 0;
    const int vecs = wide ? n / N : 0;
    const uint4* src = reinterpret_cast<const uint4*>(x + first);
    uint4 raw[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if ((int)threadIdx.x + u * kThreads < vecs) raw[u] = __ldcs(src + threadIdx.x + u * kThreads);

    if (tables) {
      for (int i = threadIdx.x; i < size * (int)sizeof(W) / 16; i += kThreads)
        reinterpret_cast<uint4*>(dyn)[i] = make_uint4(0, 0, 0, 0);
      __syncthreads();
      if (p.bias_count > 0) {
        const int32_t* b = p.bias_ids + (size_t)row * (size_t)p.bias_stride;
        for (int k = threadIdx.x; k < p.bias_count; k += kThreads) {
          const long long at = (long long)__ldg(b + k) - first;
          if (at >= 0 && at < n) atomicMax(table + at, (W)(k + 1) << L::kEntry);
        }
        __syncthreads();  // the maxima stand before counts come under them
      }
      if (hist > 0) {
        const int32_t* h = p.history + (size_t)row * (size_t)p.hist_stride;
        for (int k0 = threadIdx.x; k0 < hist; k0 += kBatch * kThreads) {
          int id[kBatch];
#pragma unroll
          for (int u = 0; u < kBatch; ++u) id[u] = k0 + u * kThreads < hist ? __ldg(h + k0 + u * kThreads) : -1;
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            const long long at = (long long)id[u] - first;
            if (id[u] < 0 || at < 0 || at >= n) continue;
            if (k0 + u * kThreads < prompt)
              atomicOr(table + at, L::kSeen);
            else
              atomicAdd(table + at, (W)1);
          }
        }
        __syncthreads();
      }
    }

    for (int k0 = threadIdx.x; k0 < vecs; k0 += kBatch * kThreads) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int k = k0 + u * kThreads;
        if (k >= vecs) break;
        float v[N];
        widen(raw[u], v, (const T*)nullptr);
        uint32_t allowed = (1u << N) - 1;
        if (mask) allowed &= __ldg(mask + ((first + N * k) >> 5)) >> (N * k & 31);
        if (tables) {
#pragma unroll
          for (int e0 = 0; e0 < N; e0 += 16 / (int)sizeof(W)) {
            const uint4 words = *reinterpret_cast<const uint4*>(table + N * k + e0);
            if (words.x | words.y | words.z | words.w) {
              W w[16 / sizeof(W)];
              memcpy(w, &words, 16);
#pragma unroll
              for (int e = 0; e < 16 / (int)sizeof(W); ++e)
                if (w[e]) v[e0 + e] = change<W>(v[e0 + e], w[e], r);
            }
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          if (!((allowed >> e) & 1u)) v[e] = -INFINITY;
          top = fmaxf(top, v[e]);  // fmaxf drops NaN
        }
        // a larger value came (or there is none yet): the ids of a thread ascend, so the first of it stands
        if (top > bv || (bi < 0 && allowed)) {
#pragma unroll
          for (int e = 0; e < N; ++e)
            if ((allowed >> e) & 1u) take(v[e], (int)first + N * k + e, bv, bi);
        }
        if (out) {
#pragma unroll
          for (int e = 0; e < N; e += 4)
            __stcs(reinterpret_cast<float4*>(out + first + N * k + e), make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]));
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int k = k0 + (kBatch + u) * kThreads;
        if (k < vecs) raw[u] = __ldcs(src + k);
      }
    }
    for (int k = N * vecs + threadIdx.x; k < n; k += kThreads) {
      float v = load1(x + first + k);
      if (tables && table[k]) v = change<W>(v, table[k], r);
      if (mask && !((__ldg(mask + ((first + k) >> 5)) >> (k & 31)) & 1u))
        v = -INFINITY;
      else
        take(v, (int)first + k, bv, bi);
      if (out) __stcs(out + first + k, v);
    }
    if (base + p.table < p.part) __syncthreads();  // the next pass clears the table
  }

#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float ov = __shfl_down_sync(0xffffffffu, bv, o);
    const int oi = __shfl_down_sync(0xffffffffu, bi, o);
    take(ov, oi, bv, bi);
  }
  if (lane == 0) {
    best_v[warp] = bv;
    best_i[warp] = bi;
  }
  __syncthreads();
  cluster.barrier_wait();  // every CTA of the cluster has started
  if (warp == 0) {
    bv = lane < kThreads / 32 ? best_v[lane] : 0.f;
    bi = lane < kThreads / 32 ? best_i[lane] : -1;
#pragma unroll
    for (int o = kThreads / 64; o > 0; o >>= 1) {
      const float ov = __shfl_down_sync(0xffffffffu, bv, o);
      const int oi = __shfl_down_sync(0xffffffffu, bi, o);
      take(ov, oi, bv, bi);
    }
    if (lane == 0) {
      cluster.map_shared_rank(part_v, 0)[rank] = bv;
      cluster.map_shared_rank(part_i, 0)[rank] = bi;
    }
  }
  cluster.sync();
  if (rank == 0 && threadIdx.x == 0 && p.ids) {
    float v = 0.f;
    int i = -1;
    for (int k = 0; k < kCtas; ++k) take(part_v[k], part_i[k], v, i);
    p.ids[row] = i;
  }
}

template <typename T, typename W>
int launch_logits(LogitsParams& p, int rows, bool tables, cudaStream_t stream) {
  size_t smem = 0;
  p.table = p.part;
  if (tables) {
    constexpr int kMost = kTableBytes / (int)sizeof(W);
    if (p.table > kMost) p.table = kMost;
    smem = (size_t)p.table * sizeof(W);
    const int rc = cuda_status(cudaFuncSetAttribute(logits_kernel<T, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                    kTableBytes),
                               "cudaFuncSetAttribute(logits)");
    if (rc != PKV_OK) return rc;
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows * kCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cuda_status(cudaLaunchKernelEx(&cfg, logits_kernel<T, W>, p), "cudaLaunchKernelEx(logits)");
}

template <typename T>
int launch_logits(LogitsParams& p, int rows, cudaStream_t stream) {
  const bool tables = p.history || p.bias_count > 0;
  const bool narrow = p.hist_stride <= Word<uint32_t>::kMostHistory && p.bias_count <= Word<uint32_t>::kMostBiases;
  return narrow ? launch_logits<T, uint32_t>(p, rows, tables, stream)
                : launch_logits<T, unsigned long long>(p, rows, tables, stream);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_process_logits(const void* logits, int dtype, int rows, int vocab, long long row_stride,
                                  float* out, long long out_stride, int32_t* out_ids,
                                  const int32_t* history, long long history_stride,
                                  const int32_t* history_lens, const int32_t* prompt_lens,
                                  const float* repetition, const float* presence, const float* frequency,
                                  const int32_t* bias_ids, const float* bias_values, int bias_count,
                                  const uint32_t* allow_mask, long long mask_stride, void* stream) {
  if (rows < 0 || vocab < 1 || row_stride < vocab || bias_count < 0 ||
      (dtype != PKV_LOGITS_F32 && dtype != PKV_LOGITS_BF16 && dtype != PKV_LOGITS_F16))
    return PKV_ERR_INVALID_ARGUMENT;
  if (out && out_stride < vocab) return PKV_ERR_INVALID_ARGUMENT;
  if (history ? (!history_lens || history_stride < 1) : (history_lens || prompt_lens || repetition || presence || frequency))
    return PKV_ERR_INVALID_ARGUMENT;
  if (bias_count > 0 && (!bias_ids || !bias_values)) return PKV_ERR_INVALID_ARGUMENT;
  if (allow_mask && mask_stride < ((long long)vocab + 31) / 32) return PKV_ERR_INVALID_ARGUMENT;
  if (rows == 0) return PKV_OK;
  if (!logits || (!out && !out_ids)) return PKV_ERR_INVALID_ARGUMENT;
  // in place means the same rows
  if (out == logits && out && (dtype != PKV_LOGITS_F32 || (rows > 1 && out_stride != row_stride)))
    return PKV_ERR_INVALID_ARGUMENT;
  const uintptr_t words = reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(out_ids) |
                          reinterpret_cast<uintptr_t>(history) | reinterpret_cast<uintptr_t>(history_lens) |
                          reinterpret_cast<uintptr_t>(prompt_lens) | reinterpret_cast<uintptr_t>(repetition) |
                          reinterpret_cast<uintptr_t>(presence) | reinterpret_cast<uintptr_t>(frequency) |
                          reinterpret_cast<uintptr_t>(bias_ids) | reinterpret_cast<uintptr_t>(bias_values) |
                          reinterpret_cast<uintptr_t>(allow_mask);
  if ((words & 3u) || (reinterpret_cast<uintptr_t>(logits) & (dtype == PKV_LOGITS_F32 ? 3u : 1u)))
    return PKV_ERR_MISALIGNED;
  if (rows > (1 << 27) || vocab > (1 << 30) || history_stride > (1ll << 30)) return PKV_ERR_UNSUPPORTED_SHAPE;
  int dev = 0;
  const int rc = bind_stream_device(stream, &dev);
  if (rc != PKV_OK) return rc;

  LogitsParams p;
  p.logits = logits;
  p.stride = row_stride;
  p.out_stride = out_stride;
  p.hist_stride = history ? history_stride : 0;
  p.bias_stride = bias_count;
  p.mask_stride = mask_stride;
  p.out = out;
  p.ids = out_ids;
  p.history = history;
  p.history_lens = history_lens;
  p.prompt_lens = prompt_lens;
  p.repetition = repetition;
  p.presence = presence;
  p.frequency = frequency;
  p.bias_ids = bias_ids;
  p.bias_values = bias_values;
  p.mask = allow_mask;
  p.vocab = vocab;
  p.bias_count = bias_count;
  p.part = ((vocab + kCtas - 1) / kCtas + 31) & ~31;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == PKV_LOGITS_F32) return launch_logits<float>(p, rows, st);
  if (dtype == PKV_LOGITS_BF16) return launch_logits<__nv_bfloat16>(p, rows, st);
  return launch_logits<__half>(p, rows, st);
}
