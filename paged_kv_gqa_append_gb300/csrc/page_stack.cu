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
// Every CTA works out the sums over all rows by itself (8 bytes a row, from the L2) and keeps them in
// shared memory; pages and tokens are then shared out over all threads, whatever the rows' lengths, and
// find their row by bisection.  A small call is one CTA's.  A large one is two kernels: one fills the
// tables, or copies the pages, and leaves the lengths and the count as they are, since others may still
// read them; the second changes these -- for a release when its cluster has checked what the first has
// copied.  (A large grow into other lengths and another count than it reads needs only the first.)  The
// second kernel's sums are done while the first one runs.
//
// Bound: latency, of five dependent loads and barriers behind a launch: a step of 32 rows and 16 layers
// takes 4.6 us, 61000 tokens of 64 prompts with their slots in 16 layers 9.3 us (0.8 us of bytes), 131000
// pages of 128 finished rows 11.4 us (0.2 us of bytes).
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "page_units.cuh"
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
  int fill, commit;  // which half of a call a kernel does: everything but the lengths and the count, and these
};

__device__ __forceinline__ int blocks_of(int n) { return (n + PKV_PAGE_TOKENS - 1) / PKV_PAGE_TOKENS; }

struct Sums {
  int tokens[kMostRows + 1];  // new tokens of the rows before (grow)
  int pages[kMostRows + 1];   // pages of the rows before, over all layers
  long long warp_tokens[kMostThreads / 32], warp_pages[kMostThreads / 32];
};

// What row s brings: new tokens and pages per layer; false if it cannot be.
template <bool kGrow>
__device__ __forceinline__ bool row_of(const StackParams& p, int s, int& tokens, int& pages) {
  const int n = __ldcg(p.lens + s);
  if (kGrow) {
    tokens = p.added ? __ldcg(p.added + s) : 1;
    pages = 0;
    if (n < 0 || tokens < 0 || (long long)n + tokens > (long long)p.max_blocks * PKV_PAGE_TOKENS) return false;
    pages = blocks_of(n + tokens) - blocks_of(n);
    return true;
  }
  tokens = pages = 0;
  if (!__ldcg(p.finished + s)) return true;
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

// One popped page of the call after another: row, layer and block.
struct PageAt {
  int row, left, layer, block, first, per;  // left: pages of the row from this one on
  __device__ __forceinline__ void seek(const StackParams& p, const Sums& sh, int i) {
    row = row_at(sh.pages, p.rows, i);
    enter(p, sh, i - sh.pages[row]);
  }
  __device__ __forceinline__ void enter(const StackParams& p, const Sums& sh, int within) {
    const int need = sh.pages[row + 1] - sh.pages[row];
    per = need / p.layers;
    first = blocks_of(p.lens[row]);  // behind the pages that the row has
    left = need - within;
    layer = within / per;
    block = first + within % per;
  }
  __device__ __forceinline__ void next(const StackParams& p, const Sums& sh) {
    if (--left == 0) {
      do ++row;
      while (row < p.rows && sh.pages[row + 1] == sh.pages[row]);
      if (row < p.rows) enter(p, sh, 0);
    } else if (++block == first + per) {
      block = first;
      ++layer;
    }
  }
  __device__ __forceinline__ long long entry(const StackParams& p) const {
    return layer * p.layer_stride + (long long)row * p.row_stride + block;
  }
};

// Table entries, positions, rows and slots: `taken` pages, `total` tokens.
__device__ __forceinline__ void fill_tables(const StackParams& p, const Sums& sh, int me, int threads, int count, int total,
                                            int taken, bool listed) {
  bool odd = false;  // an id on the stack that cannot be one
  // pages: a few each, or runs of them
  const int run = taken <= threads ? 1 : kRun;
  for (long long i0 = (long long)me * run; i0 < taken; i0 += (long long)threads * run) {
    PageAt at;
    at.seek(p, sh, (int)i0);
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
      if (u + 1 < n) at.next(p, sh);
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
}

__global__ void __launch_bounds__(kMostThreads) grow_kernel(const StackParams p) {
  __shared__ Sums sh;
  const int threads = (int)(blockDim.x * gridDim.x), me = (int)(blockIdx.x * blockDim.x + threadIdx.x);
  // (behind a kernel for the other half, which has waited itself, what is read here is long there)
  if (p.fill) {
    pdl_wait();
    pdl_launch_dependents();
  }
  const int count = __ldcg(p.count);
  long long tokens, pages;
  const bool good = sum_rows<true>(p, sh, tokens, pages);
  const bool listed = p.positions || p.token_seq || p.slots;
  int why = PKV_OK;
  if (!good || count < 0 || count > p.num_pages || (listed && tokens > p.T) || tokens > 0x7FFFFFFF)
    why = PKV_ERR_DEVICE_INDEX;
  else if (pages > count)
    why = PKV_ERR_POOL_EXHAUSTED;
  if (why != PKV_OK && me == 0) report_error(p.d_err, why);  // (the first code stays)
  const int total = why == PKV_OK ? (int)tokens : 0, taken = why == PKV_OK ? (int)pages : 0;

  if (p.fill) fill_tables(p, sh, me, threads, count, total, taken, listed);
  if (p.fill) {
    if (me == 0) p.cu[p.rows] = total;
    for (int s = me; s < p.rows; s += threads) p.cu[s] = why == PKV_OK ? sh.tokens[s] : 0;
  }
  if (!p.commit) return;
  if (!p.fill) {
    pdl_wait();
    pdl_launch_dependents();
  }
  __syncthreads();  // they may be the ones read: then this CTA is alone
  for (int s = me; s < p.rows; s += threads) {
    const int n = p.lens[s];
    p.lens_out[s] = why == PKV_OK ? n + (sh.tokens[s + 1] - sh.tokens[s]) : n;
  }
  if (me == 0) *p.count_out = count - taken;
}

// The copy (fill) by any number of CTAs; the check of what has been copied and the lengths (commit) by
// one cluster.
__global__ void __launch_bounds__(kMostThreads) release_kernel(const StackParams p) {
  __shared__ Sums sh;
  __shared__ int bad[kMostCtas];  // of the cluster's CTAs: a page id that cannot be one
  const int threads = (int)(blockDim.x * gridDim.x), me = (int)(blockIdx.x * blockDim.x + threadIdx.x);
  const bool several = p.commit && gridDim.x > 1;
  if (several) cg::this_cluster().barrier_arrive();
  // (behind a kernel for the other half, which has waited itself, what is read here is long there)
  if (p.fill) {
    pdl_wait();
    pdl_launch_dependents();
  }
  const int count = __ldcg(p.count);
  long long tokens, pages;
  const bool good = sum_rows<false>(p, sh, tokens, pages);
  const bool fits = good && count >= 0 && count <= p.num_pages && pages <= p.num_pages - count;
  const int total = fits ? (int)pages : 0;
  int32_t* to = p.free_pages + (fits ? count : 0);  // of no meaning until the count says so
  if (p.fill) {
    // a warp for each row and layer: its pages lie side by side in the table and on the stack
    const int rows = fits ? p.rows : 0, lane = threadIdx.x & 31;
    for (UnitWalk u(me / 32, threads / 32, p.layers); u.row < rows; u.next()) {
      const int need = sh.pages[u.row + 1] - sh.pages[u.row];
      if (need == 0) continue;
      const int n = need / p.layers;
      const int32_t* from = p.tables + u.layer * p.layer_stride + (long long)u.row * p.row_stride;
      int32_t* here = to + sh.pages[u.row] + u.layer * n;
#pragma unroll 4
      for (int i = lane; i < n; i += 32) here[i] = from[i];
    }
  }
  if (!p.commit) return;
  if (!p.fill) {
    pdl_wait();
    pdl_launch_dependents();
  }
  __syncthreads();
  bool odd = false;
#pragma unroll 8
  for (int i = me; i < total; i += threads) {
    const int id = __ldcg(to + i);
    odd |= id < 0 || id >= p.num_pages;
  }
  odd = __syncthreads_or(odd);
  if (several) {
    const cg::cluster_group cluster = cg::this_cluster();
    cluster.barrier_wait();  // all of them run
    if (threadIdx.x < gridDim.x) *cluster.map_shared_rank(&bad[blockIdx.x], threadIdx.x) = odd;
    cluster.sync();
    for (int c = 0; c < (int)gridDim.x; ++c) odd |= bad[c] != 0;
  }
  const bool done = fits && !odd;
  if (!done && me == 0) report_error(p.d_err, PKV_ERR_DEVICE_INDEX);
  for (int s = me; s < p.rows; s += threads) {
    const int n = p.lens[s];
    p.lens_out[s] = done && p.finished[s] ? 0 : n;
  }
  if (me == 0) *p.count_out = done ? count + total : count;
}

// One kernel of a call: `ctas` CTAs, one cluster if `cluster`.
int launch(void (*kernel)(StackParams), StackParams p, int fill, int commit, int ctas, int threads, bool cluster,
           void* stream, const char* what) {
  p.fill = fill;
  p.commit = commit;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster ? ctas : 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, p), what);
}

// Up to kAlone items of a grow (rows over all layers, and slots) and kAloneRows rows over all layers of a
// release one CTA does a call (a step of 32 rows and 16 layers 4.6 us); with more, as many CTAs as have
// kShare items each, or a warp for each row and layer (release of 64 rows of 16 layers and up to 125
// pages: 6.8 us, by one CTA 28.8 us; of 8 such rows 5.9 and 8.4 us; of 4 6.0 us by either).  How many pages a
// grow takes the host does not know: 64 prompts to 1920 tokens in 16 layers, without lists, are taken for a step
// and cost one CTA 40 us; with their lists, in place, they are many CTAs' and take 9.5 us.
constexpr long long kAlone = 1024;
constexpr int kAloneRows = 64;
constexpr int kShare = 2048, kFillThreads = 512;
int fill_ctas(long long items, int sms) {
  const long long n = (items + kShare - 1) / kShare;
  return (int)(n < 2 * sms ? n : 2 * sms);
}

bool overlaps(const int32_t* a, const int32_t* b, int n) { return a < b + n && b < a + n; }

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
  const int sms = sm_count(dev);
  if (sms <= 0) return cuda_status(cudaErrorInvalidDevice, "sm_count");
  const long long tokens = positions || token_seq || slots ? T : 0;
  const long long items = (long long)num_seqs * num_layers + tokens * (slots ? num_layers : 1);
  const char* what = "cudaLaunchKernelEx(grow)";
  if (items <= kAlone) return launch(grow_kernel, p, 1, 1, 1, 512, false, stream, what);
  // lengths and count that are read change behind all that read them, in a kernel of their own
  const bool in_place = overlaps(seq_lens_out, seq_lens, num_seqs) || free_count_out == free_count;
  rc = launch(grow_kernel, p, 1, !in_place, fill_ctas(items, sms), kFillThreads, false, stream, what);
  if (rc != PKV_OK || !in_place) return rc;
  return launch(grow_kernel, p, 0, 1, 1, 1024, false, stream, what);
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
  const int sms = sm_count(dev);
  if (sms <= 0) return cuda_status(cudaErrorInvalidDevice, "sm_count");
  const long long rows = (long long)num_seqs * num_layers;  // of the tables, of a few pages each
  const char* what = "cudaLaunchKernelEx(release)";
  if (rows <= kAloneRows) return launch(release_kernel, p, 1, 1, 1, 1024, false, stream, what);
  rc = launch(release_kernel, p, 1, 0, fill_ctas(rows * (kShare * 32 / kFillThreads), sms), kFillThreads, false, stream, what);
  if (rc != PKV_OK) return rc;
  return launch(release_kernel, p, 0, 1, kMostCtas, 1024, true, stream, what);
}
