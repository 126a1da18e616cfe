// RoPE + append into pages of 4-bit codes with a scale and a minimum for every row
// (token, KV head, K or V), and the pages read back as bf16, for sm_103a.
//
// A row is never written again once it is there -- at 4 bits a second rounding would
// cost as much as the first -- so tokens of one page are independent of each other.
// They are still handled together where a call brings several (append_rows.cuh: a
// warp has its head's K or V rows of up to 16 tokens in registers): the block's
// order puts a token's V codes 2 bytes apart by 64, and a warp that has all 16 rows
// of a page arranges them in shared memory and writes 512 bytes at once.
//
// Bound: memory, 2.6 KiB per token for K and V and 8 KiB for q: 14400 tokens of eight prompts, with q, and
// the 906 pages read back, 39.0 us (29.1 us of bytes); a step of 32 tokens and the read 4.5 us (5.2 on another
// machine), two launches of five dependent loads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "append_rows.cuh"
#include "int4.cuh"
#include "internal.h"
#include "pkv.h"
#include "ptx.cuh"

namespace pkv {
namespace {

struct Int4AppendParams : AppendRows {
  uint8_t* pool;
};

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {  // NaN if either is
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// K (kv = 0) or V rows of one head of a run: slots [slot, slot + n) of the page
// that `entry` of the block table names.  `stage`: 512 bytes of the warp's.
__device__ __forceinline__ void append_run(const Int4AppendParams& p, int t, int pos, int n, const int32_t* entry,
                                           int kv, int head, uint8_t* stage) {
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
  if (kv == 0 && p.cos) {
    float4 c[4], s[4];  // rows beside the run (of zeros) take its first entry
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * i + sub - slot;
      const size_t row = (size_t)(r >= 0 && r < n ? pos + r : pos) * PKV_ROPE_PAIRS + 4 * j;
      c[i] = __ldg(reinterpret_cast<const float4*>(p.cos + row));
      s[i] = __ldg(reinterpret_cast<const float4*>(p.sin + row));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (4 * i + 4 <= slot || 4 * i >= slot + n) continue;  // none of the warp's four rows
      float2 x[4];
      widen8(raw[i], x);
      rotate8(x, c[i], s[i]);
      raw[i] = narrow8(x);
    }
  }
  if (page < 0 || page >= p.num_pages) {
    if (threadIdx.x == 0) report_error(p.d_err, PKV_ERR_DEVICE_INDEX);
    return;
  }
  uint8_t* block = p.pool + ((size_t)page * PKV_NUM_KV_HEADS + head) * kI4BlockBytes;
  const bool whole = n == PKV_PAGE_TOKENS;
  uint8_t* to = whole ? stage - (kv ? kI4V : 0) : block;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * i + sub;
    if (4 * i + 4 <= slot || 4 * i >= slot + n) continue;
    uint32_t hi = max_bf16x2(max_bf16x2(raw[i].x, raw[i].y), max_bf16x2(raw[i].z, raw[i].w));
    uint32_t lo = min_bf16x2(min_bf16x2(raw[i].x, raw[i].y), min_bf16x2(raw[i].z, raw[i].w));
    // the larger of the highs in the upper half, the larger of the negated lows in the lower
    uint32_t m = max_bf16x2(__byte_perm(hi, lo ^ 0x80008000u, 0x1054), __byte_perm(hi, lo ^ 0x80008000u, 0x3276));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
    const I4Row row = i4_row(-bf16lo_to_f32(m), bf16hi_to_f32(m));
    const float a[4] = {bf16lo_to_f32(raw[i].x), bf16hi_to_f32(raw[i].x), bf16lo_to_f32(raw[i].y), bf16hi_to_f32(raw[i].y)};
    const float b[4] = {bf16lo_to_f32(raw[i].z), bf16hi_to_f32(raw[i].z), bf16lo_to_f32(raw[i].w), bf16hi_to_f32(raw[i].w)};
    const uint16_t ca = (uint16_t)i4_codes4(a, row), cb = (uint16_t)i4_codes4(b, row);
    if (r >= slot && r < slot + n) {
      *reinterpret_cast<uint16_t*>(to + (kv ? i4_v_at(r, j) : i4_k_at(r, j))) = ca;
      *reinterpret_cast<uint16_t*>(to + (kv ? i4_v_at(r, j + 8) : i4_k_at(r, j + 8))) = cb;
      if (j == 0) *reinterpret_cast<uint32_t*>(block + i4_scale_at(r, kv)) = row.word;
    }
  }
  if (whole) {
    __syncwarp();
    *reinterpret_cast<uint4*>(block + (kv ? kI4V : 0) + 16 * lane) = *reinterpret_cast<const uint4*>(stage + 16 * lane);
    __syncwarp();
  }
}

__global__ void __launch_bounds__(kAppendWarps * 32, 2) int4_append_kernel(const Int4AppendParams p) {
  __shared__ uint4 stage[kAppendWarps][32];
  pdl_wait();
  pdl_launch_dependents();
  // with q, the two kinds of CTA take turns, so that both kinds are on every SM
  const int kinds = p.q_in ? 2 : 1;
  const int t0 = blockIdx.x / kinds * p.chunk, t1 = min(p.T, t0 + p.chunk);
  uint8_t* mine = reinterpret_cast<uint8_t*>(stage[threadIdx.x >> 5]);
  if (blockIdx.x % kinds == 0)
    append_chunk(p, t0, t1, [&](int t, int pos, int n, const int32_t* entry, int kv, int head) {
      append_run(p, t, pos, n, entry, kv, head, mine);
    });
  else
    rotate_chunk(p, t0, t1);
}

// out[i] = the page page_ids[i] as bf16: lo + code * scale, rounded once.  One CTA per
// page, which it holds in shared memory; bound by the instructions of the conversion
// (half of the issue slots) and the wait for the page, with nothing of the next one
// under way: 906 pages, 5.5 us of bytes (9 KiB read, 32 KiB written a page), take 8.6 us
// with 256 threads and 9.9 us with 1024, 100 pages 2.8 and 2.2 us, so that a grid of one
// CTA per SM at most takes 1024.
template <int kReadThreads>
__global__ void __launch_bounds__(kReadThreads) int4_read_kernel(const uint8_t* __restrict__ pool, int num_pages,
                                                                 const int32_t* __restrict__ page_ids,
                                                                 uint16_t* __restrict__ out, int* d_err) {
  __shared__ uint4 held[kI4PageBytes / 16];
  pdl_wait();
  pdl_launch_dependents();
  const int page = __ldg(page_ids + blockIdx.x);
  const bool ok = page >= 0 && page < num_pages;
  if (!ok && threadIdx.x == 0) report_error(d_err, PKV_ERR_DEVICE_INDEX);
  const uint4* src = reinterpret_cast<const uint4*>(pool + (size_t)(ok ? page : 0) * kI4PageBytes);
  if (ok)
    for (int i = threadIdx.x; i < kI4PageBytes / 16; i += kReadThreads) held[i] = __ldcs(src + i);
  __syncthreads();
  uint4* dst = reinterpret_cast<uint4*>(out + (size_t)blockIdx.x * PKV_PAGE_ELEMS);
#pragma unroll
  for (int i = threadIdx.x; i < PKV_PAGE_ELEMS / 8; i += kReadThreads) {  // eight dims each
    const int c = i & 7, r = (i >> 3) & 15, head = (i >> 7) & 7, kv = i >> 10;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (ok) {
      const uint8_t* block = reinterpret_cast<const uint8_t*>(held) + head * kI4BlockBytes;
      const uint32_t w = kv ? *reinterpret_cast<const uint16_t*>(block + i4_v_at(r, 2 * c)) |
                                  (uint32_t)*reinterpret_cast<const uint16_t*>(block + i4_v_at(r, 2 * c + 1)) << 16
                            : *reinterpret_cast<const uint32_t*>(block + i4_k_at(r, 2 * c));
      const uint32_t row = *reinterpret_cast<const uint32_t*>(block + i4_scale_at(r, kv));
      const float scale = bf16lo_to_f32(row), lo = bf16hi_to_f32(row);
      uint32_t x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[e] = pack_bf16x2(__fmaf_rn((float)(w >> (8 * e) & 15u), scale, lo), __fmaf_rn((float)(w >> (8 * e + 4) & 15u), scale, lo));
      v = make_uint4(x[0], x[1], x[2], x[3]);
    }
    dst[i] = v;
  }
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int kv_append_rope_int4(const void* k, long long k_stride, const void* v, long long v_stride,
                                   const int32_t* cu_new, const int32_t* seq_lens, int T,
                                   const int32_t* block_tables, int num_seqs, int bt_row_stride,
                                   int max_blocks, void* kv_pool, int num_pages, const float* rope_cos,
                                   const float* rope_sin, int max_pos, const void* q_in, long long q_stride,
                                   void* q_out, int* d_err, void* stream) {
  if (T < 0 || num_seqs < 1 || max_blocks < 1 || bt_row_stride < max_blocks || num_pages < 1)
    return PKV_ERR_INVALID_ARGUMENT;
  if ((rope_cos == nullptr) != (rope_sin == nullptr) || (q_in == nullptr) != (q_out == nullptr) ||
      (q_in && !rope_cos) || (rope_cos && max_pos < 1))
    return PKV_ERR_INVALID_ARGUMENT;
  if (T == 0) return PKV_OK;
  if (!k || !v || !cu_new || !seq_lens || !block_tables || !kv_pool) return PKV_ERR_INVALID_ARGUMENT;
  if (k_stride < PKV_NUM_KV_HEADS * PKV_HEAD_DIM || v_stride < PKV_NUM_KV_HEADS * PKV_HEAD_DIM ||
      (q_in && q_stride < PKV_NUM_Q_HEADS * PKV_HEAD_DIM))
    return PKV_ERR_INVALID_ARGUMENT;
  if (!aligned16(k) || !aligned16(v) || !aligned16(kv_pool) || !aligned16(q_in) || !aligned16(q_out) ||
      !aligned16(rope_cos) || !aligned16(rope_sin) || (k_stride & 7) || (v_stride & 7) || (q_in && (q_stride & 7)))
    return PKV_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(cu_new) | reinterpret_cast<uintptr_t>(seq_lens) |
       reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(d_err)) & 3u)
    return PKV_ERR_MISALIGNED;
  if (T > (1 << 29) || num_seqs > (1 << 30) || max_blocks > (1 << 26)) return PKV_ERR_UNSUPPORTED_SHAPE;
  int dev = 0;
  const int rc = bind_stream_device(stream, &dev);
  if (rc != PKV_OK) return rc;

  Int4AppendParams p;
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
  p.d_err = d_err;
  p.T = T;
  p.num_seqs = num_seqs;
  p.bt_stride = bt_row_stride;
  p.most = max_blocks * PKV_PAGE_TOKENS;
  if (rope_cos && max_pos < p.most) p.most = max_pos;
  p.num_pages = num_pages;
  p.chunk = append_chunk_tokens(T, num_seqs, sm_count(dev));

  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)T + p.chunk - 1) / p.chunk) * (q_in ? 2 : 1));
  cfg.blockDim = dim3(kAppendWarps * 32);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, int4_append_kernel, p), "cudaLaunchKernelEx(append int4)");
}

extern "C" int kv_read_int4(const void* kv_pool, int num_pages, const int32_t* page_ids, int count, void* out,
                            int* d_err, void* stream) {
  if (count < 0 || num_pages < 1) return PKV_ERR_INVALID_ARGUMENT;
  if (count == 0) return PKV_OK;
  if (!kv_pool || !page_ids || !out) return PKV_ERR_INVALID_ARGUMENT;
  if (!aligned16(kv_pool) || !aligned16(out) ||
      ((reinterpret_cast<uintptr_t>(page_ids) | reinterpret_cast<uintptr_t>(d_err)) & 3u))
    return PKV_ERR_MISALIGNED;
  int dev = 0;
  const int rc = bind_stream_device(stream, &dev);
  if (rc != PKV_OK) return rc;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)count);
  const bool few = count <= sm_count(dev);
  cfg.blockDim = dim3(few ? 1024 : 256);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, few ? int4_read_kernel<1024> : int4_read_kernel<256>, static_cast<const uint8_t*>(kv_pool), num_pages, page_ids,
                                        static_cast<uint16_t*>(out), d_err),
                     "cudaLaunchKernelEx(read int4)");
}
