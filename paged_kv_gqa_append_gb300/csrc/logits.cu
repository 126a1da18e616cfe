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
// vocabulary (a multiple of 32 tokens, one mask word).  A CTA keeps one 32-bit
// word per token of its part in shared memory -- bit 31: seen, below it the
// count -- and, with biases, a second one: the last bias entry + 1.  Each CTA
// walks an eighth of the history and adds to the owner's word through
// distributed shared memory, so the history is read once per row; integer
// atomics make the words the same in any order.  Then the part is streamed
// once, 16 bytes at a time, each thread keeping its best (value, id); warp
// shuffles, shared memory and the cluster's first CTA reduce them under a
// total order.  A part larger than the tables goes in passes.
//
// Bound: memory, the logits read (and written, when they are kept).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "pkv.h"
#include "ptx.cuh"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kCtas = 8;
constexpr int kMaxTokens = 16384;  // tokens per table: 64 KiB a table
constexpr uint32_t kSeen = 1u << 31;

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

__device__ __forceinline__ void load4(const float* x, float (&v)[4]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(x));
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* x, float (&v)[4]) {
  const uint2 a = __ldcs(reinterpret_cast<const uint2*>(x));
  v[0] = bf16lo_to_f32(a.x); v[1] = bf16hi_to_f32(a.x);
  v[2] = bf16lo_to_f32(a.y); v[3] = bf16hi_to_f32(a.y);
}
__device__ __forceinline__ void load4(const __half* x, float (&v)[4]) {
  const uint2 a = __ldcs(reinterpret_cast<const uint2*>(x));
  const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&a.x));
  const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&a.y));
  v[0] = lo.x; v[1] = lo.y; v[2] = hi.x; v[3] = hi.y;
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
  bool penalties;
};

// steps 1 and 2 for a token whose word is not 0
__device__ __forceinline__ float penalise(float x, uint32_t word, const Row& r) {
  x = x > 0.f ? __fdiv_rn(x, r.rep) : __fmul_rn(x, r.rep);
  const uint32_t n = word & ~kSeen;
  if (n) {
    x = __fsub_rn(x, __fmul_rn(r.freq, (float)n));
    x = __fsub_rn(x, r.pres);
  }
  return x;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) logits_kernel(const LogitsParams p) {
  extern __shared__ uint32_t table[];  // [p.table] words, then [p.table] bias entries
  __shared__ float best_v[kThreads / 32], part_v[kCtas];
  __shared__ int best_i[kThreads / 32], part_i[kCtas];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int row = blockIdx.x / kCtas;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();

  const long long lo = (long long)rank * p.part;
  const T* x = static_cast<const T*>(p.logits) + (size_t)row * (size_t)p.stride;
  float* out = p.out ? p.out + (size_t)row * (size_t)p.out_stride : nullptr;
  const uint32_t* mask = p.mask ? p.mask + (size_t)row * (size_t)p.mask_stride : nullptr;
  Row r{1.f, 0.f, 0.f, p.history != nullptr};
  if (p.repetition) r.rep = __ldg(p.repetition + row);
  if (p.presence) r.pres = __ldg(p.presence + row);
  if (p.frequency) r.freq = __ldg(p.frequency + row);
  int hist = 0, prompt = 0;
  if (r.penalties) {
    hist = (int)min((long long)__ldg(p.history_lens + row), p.hist_stride);
    prompt = p.prompt_lens ? __ldg(p.prompt_lens + row) : 0;
    r.penalties = hist > 0;
  }
  const bool biased = p.bias_count > 0;
  const bool tables = r.penalties || biased;  // the same for the whole cluster
  uint32_t* entry = table + p.table;
  if (!tables) cluster.sync();  // every CTA runs before one writes into another's shared memory

  float bv = 0.f;
  int bi = -1;
  for (int base = 0; base < p.part; base += p.table) {
    const int size = min(p.table, p.part - base);  // tokens of this pass in every part
    if (tables) {
      const int words = biased ? 2 * p.table : p.table;
      for (int i = threadIdx.x * 4; i < words; i += kThreads * 4)
        *reinterpret_cast<uint4*>(table + i) = make_uint4(0, 0, 0, 0);
      cluster.sync();  // all tables are clear
      if (r.penalties) {
        const int32_t* h = p.history + (size_t)row * (size_t)p.hist_stride;
        for (int k = rank * kThreads + threadIdx.x; k < hist; k += kCtas * kThreads) {
          const int id = __ldg(h + k);
          if (id < 0 || id >= p.vocab) continue;
          const int owner = id / p.part, at = id - owner * p.part - base;
          if (at < 0 || at >= size) continue;
          uint32_t* w = cluster.map_shared_rank(table, owner) + at;
          if (k < prompt)
            atomicOr(w, kSeen);
          else
            atomicAdd(w, 1u);
        }
      }
      if (biased) {
        const int32_t* b = p.bias_ids + (size_t)row * (size_t)p.bias_stride;
        for (int k = rank * kThreads + threadIdx.x; k < p.bias_count; k += kCtas * kThreads) {
          const int id = __ldg(b + k);
          if (id < 0 || id >= p.vocab) continue;
          const int owner = id / p.part, at = id - owner * p.part - base;
          if (at < 0 || at >= size) continue;
          atomicMax(cluster.map_shared_rank(entry, owner) + at, (uint32_t)k + 1u);
        }
      }
      cluster.sync();  // all words are in
    }
    const float* bias = biased ? p.bias_values + (size_t)row * (size_t)p.bias_stride : nullptr;
    const long long first = lo + base;
    const int n = (int)max(0ll, min((long long)size, (long long)p.vocab - first));
    const bool wide = ((reinterpret_cast<uintptr_t>(x + first) & (4 * sizeof(T) - 1)) |
                       (out ? (reinterpret_cast<uintptr_t>(out + first) & 15u) : 0)) == 0;
    const int n4 = wide ? n / 4 : 0;
#pragma unroll 2
    for (int k = threadIdx.x; k < n4; k += kThreads) {
      float v[4];
      load4(x + first + 4 * k, v);
      uint32_t allowed = 0xFu;
      if (mask) allowed = (__ldg(mask + ((first + 4 * k) >> 5)) >> (4 * k & 31)) & 0xFu;
      if (r.penalties) {
        const uint4 w = *reinterpret_cast<const uint4*>(table + 4 * k);
        if (w.x | w.y | w.z | w.w) {
          if (w.x) v[0] = penalise(v[0], w.x, r);
          if (w.y) v[1] = penalise(v[1], w.y, r);
          if (w.z) v[2] = penalise(v[2], w.z, r);
          if (w.w) v[3] = penalise(v[3], w.w, r);
        }
      }
      if (biased) {
        const uint4 w = *reinterpret_cast<const uint4*>(entry + 4 * k);
        if (w.x | w.y | w.z | w.w) {
          if (w.x) v[0] = __fadd_rn(v[0], __ldg(bias + w.x - 1));
          if (w.y) v[1] = __fadd_rn(v[1], __ldg(bias + w.y - 1));
          if (w.z) v[2] = __fadd_rn(v[2], __ldg(bias + w.z - 1));
          if (w.w) v[3] = __fadd_rn(v[3], __ldg(bias + w.w - 1));
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if ((allowed >> e) & 1u)
          take(v[e], (int)first + 4 * k + e, bv, bi);
        else
          v[e] = -INFINITY;
      }
      if (out) __stcs(reinterpret_cast<float4*>(out + first) + k, make_float4(v[0], v[1], v[2], v[3]));
    }
    for (int k = 4 * n4 + threadIdx.x; k < n; k += kThreads) {
      float v = load1(x + first + k);
      if (r.penalties && table[k]) v = penalise(v, table[k], r);
      if (biased && entry[k]) v = __fadd_rn(v, __ldg(bias + entry[k] - 1));
      if (mask && !((__ldg(mask + ((first + k) >> 5)) >> (k & 31)) & 1u))
        v = -INFINITY;
      else
        take(v, (int)first + k, bv, bi);
      if (out) __stcs(out + first + k, v);
    }
    if (base + p.table < p.part) __syncthreads();  // the next pass clears this table
  }

  if (p.ids == nullptr) return;
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
  if (threadIdx.x == 0) {
    for (int k = 1; k < kThreads / 32; ++k) take(best_v[k], best_i[k], bv, bi);
    cluster.map_shared_rank(part_v, 0)[rank] = bv;
    cluster.map_shared_rank(part_i, 0)[rank] = bi;
  }
  cluster.sync();
  if (rank == 0 && threadIdx.x == 0) {
    float v = 0.f;
    int i = -1;
    for (int k = 0; k < kCtas; ++k) take(part_v[k], part_i[k], v, i);
    p.ids[row] = i;
  }
}

template <typename T>
int launch_logits(const LogitsParams& p, int rows, size_t smem, cudaStream_t stream) {
  int rc = PKV_OK;
  if (smem > 48 * 1024) {
    rc = cuda_status(cudaFuncSetAttribute(logits_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          2 * kMaxTokens * 4),
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
  return cuda_status(cudaLaunchKernelEx(&cfg, logits_kernel<T>, p), "cudaLaunchKernelEx(logits)");
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
  p.hist_stride = history_stride;
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
  const bool tables = history || bias_count > 0;
  p.table = tables && p.part > kMaxTokens ? kMaxTokens : p.part;
  const size_t smem = tables ? (size_t)p.table * 4 * (bias_count > 0 ? 2 : 1) : 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == PKV_LOGITS_F32) return launch_logits<float>(p, rows, smem, st);
  if (dtype == PKV_LOGITS_BF16) return launch_logits<__nv_bfloat16>(p, rows, smem, st);
  return launch_logits<__half>(p, rows, smem, st);
}
