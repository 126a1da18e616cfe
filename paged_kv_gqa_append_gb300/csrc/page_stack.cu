// Block tables that grow and shrink on the GPU: pages for every row's new tokens
// popped from the stack of free ones, with the rows' offsets, the tokens'
// positions and their slots in every layer; and the pages of finished rows pushed
// back (sm_103a).
//
// Row s takes L (ceil((n + new) / 16) - ceil(n / 16)) pages.  With the sums of
// that, and of the new tokens, over the rows before it, everything else is
// arithmetic: page i of the call is free[count - 1 - i] and belongs to the row,
// layer and block that i falls into; token t belongs to the row that t falls into,
// and its slot needs the one table entry that the row already had or a page that
// is being popped, whose place in the stack is known, so that nothing waits for
// the tables to be written.
//
// One cluster of CTAs does a call.  Every CTA works out the sums over all rows by
// itself (8 bytes a row, from the L2) and keeps them in shared memory; pages and
// tokens are then shared out over all threads, whatever the rows' lengths, and find
// their row by bisection.  Lengths and the count may be changed in place, since no
// CTA writes them before the cluster's barrier says that all have read them.
//
// Bound: latency.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "pkv.h"
#include "ptx.cuh"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kMostRows = 4096;
constexpr int kMostCtas = 8;
constexpr int kMostThreads = 1024;
constexpr int kRun = 8;  // pages that a thread takes one after another: 32 bytes of the stack

struct StackParams {
  const int32_t *lens, *added, *count;
  const uint8_t* finished;
  int32_t *tables, *free_pages, *lens_out, *count_out, *cu, *positions, *token_seq, *slots, *d_err;
  long long layer_stride;
  int row_stride, max_blocks, layers, num_pages, rows, T;
};

__device__ __forceinline__ int blocks_of(int n) { return (n + PKV_PAGE_TOKENS - 1) / PKV_PAGE_TOKENS; }

struct Sums {
  int tokens[kMostRows + 1];  // new tokens of the rows before (grow)
  int pages[kMostRows + 1];   // pages of the rows before, over all layers
  long long warp_tokens[kMostThreads / 32], warp_pages[kMostThreads / 32];
  int bad;                    // of the cluster's first CTA: a page id that cannot be one
};

// What row s brings: new tokens and pages per layer; false if it cannot be.
template <bool kGrow>
__device__ __forceinline__ bool row_of(const StackParams& p, int s, int& tokens, int& pages) {
  const int n = p.lens[s];
  if (kGrow) {
    tokens = p.added ? p.added[s] : 1;
    pages = 0;
    if (n < 0 || tokens < 0 || (long long)n + tokens > (long long)p.max_blocks * PKV_PAGE_TOKENS) return false;
    pages = blocks_of(n + tokens) - blocks_of(n);
    return true;
  }
  tokens = pages = 0;
  if (!p.finished[s]) return true;
  if (n < 0 || n > (long long)p.max_blocks * PKV_PAGE_TOKENS) return false;
  pages = blocks_of(n);
  return true;
}

// The sums over all rows; true if every row can be.  The totals are right beyond 32
// bits, the single sums only where the totals are within them.
template <bool kGrow>
__device__ bool sum_rows(const StackParams& p, Sums& sh, long long& all_tokens, long long& all_pages) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int per = (p.rows + (int)blockDim.x - 1) / (int)blockDim.x;
  const int s0 = min(p.rows, (int)threadIdx.x * per), s1 = min(p.rows, s0 + per);
  long long t = 0, g = 0;
  bool good = true;
  for (int s = s0; s < s1; ++s) {
    int a, b;
    good &= row_of<kGrow>(p, s, a, b);
    t += a;
    g += (long long)b * p.layers;
  }
  long long rt = t, rg = g;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long vt = __shfl_up_sync(0xffffffffu, rt, o), vg = __shfl_up_sync(0xffffffffu, rg, o);
    if (lane >= o) {
      rt += vt;
      rg += vg;
    }
  }
  if (lane == 31) {
    sh.warp_tokens[warp] = rt;
    sh.warp_pages[warp] = rg;
  }
  good = __syncthreads_and(good);
  long long bt = rt - t, bg = rg - g;
  all_tokens = all_pages = 0;
  for (int w = 0; w < warps; ++w) {
    if (w < warp) {
      bt += sh.warp_tokens[w];
      bg += sh.warp_pages[w];
    }
    all_tokens += sh.warp_tokens[w];
    all_pages += sh.warp_pages[w];
  }
  for (int s = s0; s < s1; ++s) {
    int a, b;
    row_of<kGrow>(p, s, a, b);
    sh.tokens[s] = (int)bt;
    sh.pages[s] = (int)bg;
    bt += a;
    bg += (long long)b * p.layers;
  }
  if (threadIdx.x == 0) {
    sh.tokens[p.rows] = (int)all_tokens;
    sh.pages[p.rows] = (int)all_pages;
  }
  __syncthreads();
  return good;
}

// The row that i falls into: the last s with sums[s] <= i (sums[0] = 0 <= i < sums[rows]).
__device__ __forceinline__ int row_at(const int* sums, int rows, int i) {
  int lo = 0, hi = rows;  // sums[lo] <= i < sums[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// One page of the call after another: row, layer and block.
struct PageAt {
  int row, left, layer, block, first, per;  // left: pages of the row from this one on
  __device__ __forceinline__ void seek(const StackParams& p, const Sums& sh, bool grow, int i) {
    row = row_at(sh.pages, p.rows, i);
    enter(p, sh, grow, i - sh.pages[row]);
  }
  __device__ __forceinline__ void enter(const StackParams& p, const Sums& sh, bool grow, int within) {
    const int need = sh.pages[row + 1] - sh.pages[row];
    per = need / p.layers;
    first = 0;
    if (grow) {  // behind the pages that the row has: the sums say where its new tokens end
      const int n = p.lens[row];
      first = blocks_of(n);
    }
    left = need - within;
    layer = within / per;
    block = first + within % per;
  }
  __device__ __forceinline__ void next(const StackParams& p, const Sums& sh, bool grow) {
    if (--left == 0) {
      do ++row;
      while (row < p.rows && sh.pages[row + 1] == sh.pages[row]);
      if (row < p.rows) enter(p, sh, grow, 0);
    } else if (++block == first + per) {
      block = first;
      ++layer;
    }
  }
  __device__ __forceinline__ long long entry(const StackParams& p) const {
    return layer * p.layer_stride + (long long)row * p.row_stride + block;
  }
};

__global__ void __launch_bounds__(kMostThreads) grow_kernel(const StackParams p) {
  __shared__ Sums sh;
  const cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int threads = (int)blockDim.x * ctas, me = rank * (int)blockDim.x + (int)threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const int count = *p.count;
  long long tokens, pages;
  const bool good = sum_rows<true>(p, sh, tokens, pages);
  const bool listed = p.positions || p.token_seq || p.slots;
  int why = PKV_OK;
  if (!good || count < 0 || count > p.num_pages || (listed && tokens > p.T) || tokens > 0x7FFFFFFF)
    why = PKV_ERR_DEVICE_INDEX;
  else if (pages > count)
    why = PKV_ERR_POOL_EXHAUSTED;
  if (why != PKV_OK && me == 0) report_error(p.d_err, why);
  const int total = why == PKV_OK ? (int)tokens : 0, taken = why == PKV_OK ? (int)pages : 0;

  bool odd = false;  // an id on the stack that cannot be one
  // pages: a few each, or runs of them
  const int run = taken <= threads ? 1 : kRun;
  for (long long i0 = (long long)me * run; i0 < taken; i0 += (long long)threads * run) {
    PageAt at;
    at.seek(p, sh, true, (int)i0);
    const int n = min(run, taken - (int)i0);
    int id[kRun];
#pragma unroll
    for (int u = 0; u < kRun; ++u)
      if (u < n) id[u] = p.free_pages[count - 1 - ((int)i0 + u)];
#pragma unroll
    for (int u = 0; u < kRun; ++u) {
      if (u >= n) break;
      p.tables[at.entry(p)] = id[u];
      odd |= id[u] < 0 || id[u] >= p.num_pages;
      if (u + 1 < n) at.next(p, sh, true);
    }
  }
  // tokens: 32 to a warp; a warp takes all layers of them, or a part where there are few
  const int groups = listed ? (p.T + 31) / 32 : 0, warps = threads / 32, lane = threadIdx.x & 31;
  int split = 1;  // parts of the layers
  while (split < p.layers && (long long)groups * split < warps) split *= 2;
  const int per = (p.layers + split - 1) / split;
  for (long long w = me / 32; w < (long long)groups * split; w += warps) {
    const int part = (int)(w / groups), t = (int)(w % groups) * 32 + lane;
    if (t >= p.T) continue;
    const bool live = t < total;
    int row = -1, pos = -1, n = 0;
    if (live) {
      row = row_at(sh.tokens, p.rows, t);
      n = p.lens[row];
      pos = n + t - sh.tokens[row];
    }
    if (part == 0) {
      if (p.positions) p.positions[t] = pos;
      if (p.token_seq) p.token_seq[t] = row;
    }
    if (!p.slots) continue;
    const int old = blocks_of(n), block = pos / PKV_PAGE_TOKENS;
    const bool held = live && block < old;
    const int more = live ? (sh.pages[row + 1] - sh.pages[row]) / p.layers : 0;
    const int l1 = min(p.layers, (part + 1) * per);
    const int32_t* from = held ? p.tables + (long long)row * p.row_stride + block
                               : p.free_pages + (live ? count - 1 - (sh.pages[row] + block - old) : 0);
    const long long step = held ? p.layer_stride : -(long long)more;
#pragma unroll 4
    for (int l = part * per; l < l1; ++l) {
      int slot = -1;
      if (live) {
        const int id = from[l * step];
        if (id >= 0 && id < p.num_pages)
          slot = id * PKV_PAGE_TOKENS + pos % PKV_PAGE_TOKENS;
        else
          odd = true;
      }
      p.slots[(long long)l * p.T + t] = slot;
    }
  }
  if (odd) report_error(p.d_err, PKV_ERR_DEVICE_INDEX);
  if (me == 0) p.cu[p.rows] = total;
  for (int s = me; s < p.rows; s += threads) p.cu[s] = why == PKV_OK ? sh.tokens[s] : 0;
  // lengths and count last: they may be the ones read, by the other CTAs too
  if (ctas > 1) cluster.sync();
  else __syncthreads();
  for (int s = me; s < p.rows; s += threads) {
    const int n = p.lens[s];
    p.lens_out[s] = why == PKV_OK ? n + (sh.tokens[s + 1] - sh.tokens[s]) : n;
  }
  if (me == 0) *p.count_out = count - taken;
}

__global__ void __launch_bounds__(kMostThreads) release_kernel(const StackParams p) {
  __shared__ Sums sh;
  const cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int threads = (int)blockDim.x * ctas, me = rank * (int)blockDim.x + (int)threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const int count = *p.count;
  long long tokens, pages;
  if (threadIdx.x == 0) sh.bad = 0;
  const bool good = sum_rows<false>(p, sh, tokens, pages);
  const bool fits = good && count >= 0 && count <= p.num_pages && pages <= p.num_pages - count;
  if (ctas > 1) cluster.sync();  // every CTA runs, and has cleared its word
  bool odd = false;
  const int total = fits ? (int)pages : 0;
  const int run = total <= threads ? 1 : kRun;
  for (long long i0 = (long long)me * run; i0 < total; i0 += (long long)threads * run) {
    PageAt at;
    at.seek(p, sh, false, (int)i0);
    const int n = min(run, total - (int)i0);
    int id[kRun];
#pragma unroll
    for (int u = 0; u < kRun; ++u) {
      if (u < n) {
        id[u] = p.tables[at.entry(p)];
        if (u + 1 < n) at.next(p, sh, false);
      }
    }
#pragma unroll
    for (int u = 0; u < kRun; ++u)
      if (u < n) {
        p.free_pages[count + (int)i0 + u] = id[u];  // of no meaning until the count says so
        odd |= id[u] < 0 || id[u] >= p.num_pages;
      }
  }
  if (odd) *cluster.map_shared_rank(&sh.bad, 0) = 1;
  if (ctas > 1) cluster.sync();
  else __syncthreads();
  const bool done = fits && *cluster.map_shared_rank(&sh.bad, 0) == 0;
  if (!done && me == 0) report_error(p.d_err, PKV_ERR_DEVICE_INDEX);
  for (int s = me; s < p.rows; s += threads) {
    const int n = p.lens[s];
    p.lens_out[s] = done && p.finished[s] ? 0 : n;
  }
  if (me == 0) *p.count_out = done ? count + total : count;
  if (ctas > 1) cluster.sync();  // the first CTA's word is read until here
}

// One CTA where little is to be done, else a cluster of eight.
int launch(void (*kernel)(StackParams), const StackParams& p, long long items, void* stream, const char* what) {
  const int ctas = items <= 4096 ? 1 : kMostCtas;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(items <= 1024 ? 512 : 1024);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, p), what);
}

// What both calls refuse on the host.
int check(const StackParams& p) {
  if (p.rows < 0 || p.layers < 1 || p.max_blocks < 1 || p.row_stride < p.max_blocks || p.num_pages < 1 || p.T < 0 ||
      (p.layers > 1 && p.layer_stride < (long long)p.rows * p.row_stride))
    return PKV_ERR_INVALID_ARGUMENT;
  if (!p.free_pages || !p.count || !p.count_out || (p.rows > 0 && (!p.lens || !p.tables || !p.lens_out)))
    return PKV_ERR_INVALID_ARGUMENT;
  if ((reinterpret_cast<uintptr_t>(p.lens) | reinterpret_cast<uintptr_t>(p.added) | reinterpret_cast<uintptr_t>(p.count) |
       reinterpret_cast<uintptr_t>(p.tables) | reinterpret_cast<uintptr_t>(p.free_pages) |
       reinterpret_cast<uintptr_t>(p.lens_out) | reinterpret_cast<uintptr_t>(p.count_out) |
       reinterpret_cast<uintptr_t>(p.cu) | reinterpret_cast<uintptr_t>(p.positions) |
       reinterpret_cast<uintptr_t>(p.token_seq) | reinterpret_cast<uintptr_t>(p.slots) |
       reinterpret_cast<uintptr_t>(p.d_err)) & 3u)
    return PKV_ERR_MISALIGNED;
  if (p.rows > kMostRows || (long long)p.layers * p.max_blocks > (1ll << 30) || p.max_blocks > (1 << 26) ||
      p.num_pages >= (1 << 27) || p.T > (1 << 30))
    return PKV_ERR_UNSUPPORTED_SHAPE;
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_grow_block_tables(const int32_t* seq_lens, const int32_t* new_tokens, int num_seqs,
                                     int32_t* block_tables, int num_layers, long long bt_layer_stride,
                                     int bt_row_stride, int max_blocks, const int32_t* free_pages, int num_pages,
                                     const int32_t* free_count, int32_t* seq_lens_out, int32_t* free_count_out,
                                     int32_t* cu_new, int32_t* positions, int32_t* token_seq, int32_t* slots, int T,
                                     int* d_err, void* stream) {
  StackParams p = {};
  p.lens = seq_lens;
  p.added = new_tokens;
  p.count = free_count;
  p.tables = block_tables;
  p.free_pages = const_cast<int32_t*>(free_pages);  // not written
  p.lens_out = seq_lens_out;
  p.count_out = free_count_out;
  p.cu = cu_new;
  p.positions = positions;
  p.token_seq = token_seq;
  p.slots = slots;
  p.d_err = d_err;
  p.layer_stride = bt_layer_stride;
  p.row_stride = bt_row_stride;
  p.max_blocks = max_blocks;
  p.layers = num_layers;
  p.num_pages = num_pages;
  p.rows = num_seqs;
  p.T = T;
  if (!cu_new) return PKV_ERR_INVALID_ARGUMENT;
  int rc = check(p);
  if (rc != PKV_OK) return rc;
  int dev = 0;
  rc = bind_stream_device(stream, &dev);
  if (rc != PKV_OK) return rc;
  const long long tokens = positions || token_seq || slots ? T : 0;
  return launch(grow_kernel, p, (long long)num_seqs * num_layers + tokens * (slots ? num_layers : 1), stream,
                "cudaLaunchKernelEx(grow)");
}

extern "C" int pkv_release_pages(const int32_t* seq_lens, const uint8_t* finished, int num_seqs,
                                 const int32_t* block_tables, int num_layers, long long bt_layer_stride,
                                 int bt_row_stride, int max_blocks, int32_t* free_pages, int num_pages,
                                 const int32_t* free_count, int32_t* seq_lens_out, int32_t* free_count_out,
                                 int* d_err, void* stream) {
  StackParams p = {};
  p.lens = seq_lens;
  p.finished = finished;
  p.count = free_count;
  p.tables = const_cast<int32_t*>(block_tables);  // not written
  p.free_pages = free_pages;
  p.lens_out = seq_lens_out;
  p.count_out = free_count_out;
  p.d_err = d_err;
  p.layer_stride = bt_layer_stride;
  p.row_stride = bt_row_stride;
  p.max_blocks = max_blocks;
  p.layers = num_layers;
  p.num_pages = num_pages;
  p.rows = num_seqs;
  if (num_seqs > 0 && !finished) return PKV_ERR_INVALID_ARGUMENT;
  int rc = check(p);
  if (rc != PKV_OK) return rc;
  int dev = 0;
  rc = bind_stream_device(stream, &dev);
  if (rc != PKV_OK) return rc;
  return launch(release_kernel, p, (long long)num_seqs * num_layers * 8, stream, "cudaLaunchKernelEx(release)");
}
