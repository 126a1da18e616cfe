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
// A cluster of up to 8 CTAs handles a row, each a contiguous part of the
// vocabulary (a multiple of 32 tokens, one mask word).  The tokens that steps 1
// to 3 change are few, so they are worked out first: a CTA reads the row's whole
// history and bias list (from L2) and keeps those of its part in a hash table in
// shared memory -- open addressing, 2048 slots, at most about half of them used
// -- with how often a token was generated, whether it was seen at all, and its
// last bias entry.  All warps first queue the ids that are in the part and take their tokens out of the bitmap of those that the
// stream is to handle, which starts as the mask.  Then half of the warps enter
// the queue into the table, 32 ids at a time, and finish the tokens, while the
// other half streams already (256 rows of 128256 fp32 with penalties, 300 biases and
// the logits kept 55.9 us; all warps first at the table, then at the stream 1.5 us
// more, a quarter of them 2.7 us).
// Integer atomics give the same numbers in any order, wherever a token's slot
// is.  Whoever enters a token lists its slot, and the listed ones are finished
// one thread each.
// A part with more than 1024 such tokens is done in passes over smaller ranges,
// halved until one fits (a range of 1024 tokens always does).
//
// The stream over the part (16 bytes per load, from the first 16-byte boundary on:
// 160 rows of 68906 bf16 20 us, by single values 36 us; units of a few loads per
// warp, claimed by whoever is free) tests a few bits per load and treats what is
// not its own as -inf; the finished tokens are written over that, and compete, behind
// it (looking them up from the stream made it five times as long: some lane of a
// warp nearly always has one).  Logits changed in place are read for the table
// before the stream starts.  The table is small on purpose: what shared memory
// takes from the L1 is missing as room for loads in flight (a word per token of
// the part, 64 KiB a CTA, took 85 us for 256 rows of 128256 with penalties and
// biases).  The ids and a warp's first unit are loaded ahead, so that memory is
// busy while the ids are queued.  A thread keeps its largest value and its id; warp
// shuffles and shared memory reduce them under a total order, and every CTA sends
// its best to the cluster's first one, which alone waits for them (a closing
// cluster barrier kept all 8 until the last had drained its stores).
//
// Bound: memory, the logits read (and written, when they are kept): 256 rows of
// 128256 fp32 logits take 26.0 us for the ids alone (74 % of the measured copy
// rate), 42.2 us with the logits written, 55.9 us with penalties and biases.  One
// row is latency: 3.5 us, 5.8 us with penalties and a mask.  Lists that hold much of
// the vocabulary cost a pass for every 1024 tokens, each over the whole lists: 1.1 ms
// for a bias of every token.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "logits_table.cuh"
#include "pkv.h"
#include "ptx.cuh"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kCtas = 8;
constexpr int kMostTokens = 16384;  // of a pass: the bitmaps
constexpr uint32_t kSeen = 1u << 31;
constexpr uint32_t kAllowed = 1u << 15;                            // of a listed slot: the mask leaves it
constexpr uint32_t kBias = 1u << 14, kPrompt = 2u << 14, kWhat = 3u << 14;  // of a queued id; else generated
constexpr int kEnterShare = 2;  // 1 of so many warps enters tokens while the others stream
// Where more wait in the queue, all warps enter them first: the stream would be over
// before (184 rows of 15603 with 1200 ids 15.2 us, 17.3 us apart).
constexpr int kEnterApart = 256;
constexpr uint32_t kMaskedBits = 0xFFFFDEADu;  // a NaN that stands for "masked out" in the table
constexpr uint32_t kWaitUs = 2000000;  // limit of the wait for the cluster's other CTAs
// The CTAs of a row finish together but for those whose part has many listed tokens: up
// to a pass for every 1024 tokens instead of every 16384, each over both lists.  Up to
// this product of a part's tokens and the lists' ids that is 2^20 ids more, half a
// millisecond, far within kWaitUs; beyond it the cluster closes with a barrier, which
// does not show beside such lists.
constexpr long long kLongLists = 1ll << 30;
constexpr int kExchangeFailed = -2;    // id of a row whose CTAs did not hear from each other

// How a CTA works.  Many rows: four small CTAs per SM, so that one's table is
// filled while others stream (256 x 128256 fp32 with penalties, biases and
// output 55.9 us, with 2 x 512 threads 20 us more).  When all CTAs fit on the GPU at
// once there is nothing else to overlap with, and more threads shorten both
// parts (32 x 128256 bf16 11.5 us, with 256 threads 3 us more).
struct Many {
  static constexpr int kThreads = 256, kResident = 4;
  static constexpr int kBatch = 4;  // 16-byte loads in flight per thread
  static constexpr int kIds = 4;    // ids in flight per thread
};
struct Few {
  static constexpr int kThreads = 512, kResident = 2;
  static constexpr int kBatch = 2;
  static constexpr int kIds = 4;
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
  int vocab, ctas, part, bias_count;  // ctas: per row; part: tokens per CTA
  int long_lists;
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

// Logits as whole numbers in the same order, -0 equal to 0, above 0 = none.
__device__ __forceinline__ uint32_t order_of(float v, int i) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return i < 0 ? 0u : b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The warp's largest, and the lowest id among its equals (0xFFFFFFFF: none).
__device__ __forceinline__ void best_of_warp(uint32_t& top, uint32_t& id) {
  const uint32_t most = __reduce_max_sync(0xffffffffu, top);
  id = __reduce_min_sync(0xffffffffu, top == most ? id : 0xFFFFFFFFu);
  top = most;
}

// 8 bytes into the shared memory of the cluster's first CTA, counted on its
// barrier; both addresses as they are in this CTA's own window.
__device__ __forceinline__ void send8(uint32_t dst, uint32_t bar, uint64_t value) {
  asm volatile(
      "{\n\t.reg .b32 a, b;\n\t"
      "mapa.shared::cluster.u32 a, %0, 0;\n\tmapa.shared::cluster.u32 b, %1, 0;\n\t"
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [a], %2, [b];\n\t}" ::"r"(dst),
      "r"(bar), "l"(value)
      : "memory");
}

// Phase 0 of `bar`, whose bytes come from other CTAs of the cluster; false after kWaitUs.
__device__ __forceinline__ bool wait_cluster(uint32_t bar) {
  const uint64_t t0 = global_timer_ns();
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar)
        : "memory");
    if (ok) return true;
    if (global_timer_ns() - t0 > (uint64_t)kWaitUs * 1000ull) return false;
  }
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The first CTA's last warp after a wait that ran out: the others may still send into its
// shared memory, so it stays until they have exited (a barrier counts exited threads as
// arrived).  Then all of it is there.
__device__ __noinline__ bool wait_for_exit(uint32_t bar, bool closed) {
  if (!closed) cluster_barrier();
  return __all_sync(0xffffffffu, wait_cluster(bar));
}

struct Row {
  float rep, pres, freq;
  const float* bias;
};

// steps 1 to 3 for a token of the table: its count (with kSeen) and bias entry + 1
__device__ __forceinline__ float change(float x, uint32_t count, uint32_t entry, const Row& r) {
  if (count) x = x > 0.f ? __fdiv_rn(x, r.rep) : __fmul_rn(x, r.rep);
  count &= ~kSeen;
  if (count) {
    x = __fsub_rn(x, __fmul_rn(r.freq, (float)count));
    x = __fsub_rn(x, r.pres);
  }
  if (entry) x = __fadd_rn(x, __ldg(r.bias + entry - 1));
  return x;
}

// The table in shared memory (logits_table.cuh).
struct SharedTable {
  uint32_t* keys;
  int* listed;
  __device__ __forceinline__ uint32_t key(uint32_t i) const { return *(volatile uint32_t*)(keys + i); }
  __device__ __forceinline__ uint32_t claim(uint32_t i, uint32_t at) const { return atomicCAS(keys + i, kEmpty, at); }
  __device__ __forceinline__ bool full() const { return *(volatile int*)listed >= kList; }
};

// A thread's share of a list of ids, kIds at a time (-1: none).
template <int kThreads, int kIds>
__device__ __forceinline__ void load_ids(const int32_t* ids, int k0, int count, int (&id)[kIds]) {
#pragma unroll
  for (int u = 0; u < kIds; ++u) id[u] = k0 + u * kThreads < count ? __ldg(ids + k0 + u * kThreads) : -1;
}

template <typename T, bool kAligned, int kThreads, int kResident, int kBatch, int kIds>
__global__ void __launch_bounds__(kThreads, kResident) logits_kernel(const LogitsParams p) {
  constexpr int N = 16 / (int)sizeof(T);  // tokens per 16 bytes
  constexpr int kWarps = kThreads / 32, kEnterWarps = kWarps / kEnterShare;
  constexpr int kRound = kIds * kThreads;          // ids at a time
  constexpr int kQueue = kRound + (kRound > 1024 ? 512 : kRound);  // ids of the part that wait for the table (48 KB in all)
  static_assert(kList + kThreads <= kSlots * 3 / 4, "the table never fills up");
  static_assert(kMostTokens <= 1 << 14 && 65536 % kRound == 0, "the bits of the queue");
  // the table: token of the pass, its count (then its finished logit), its bias entry + 1
  __shared__ __align__(16) uint32_t key[kSlots], count[kSlots], entry[kSlots];
  __shared__ uint2 best[kWarps];
  __shared__ uint64_t best_of[kCtas], arrived;  // of the cluster's first CTA: (id, order) of all
  __shared__ uint32_t allow[kMostTokens / 32 + 1];  // the stream's tokens, a bit per token of the pass
  __shared__ uint16_t list[kList];              // slot, and kAllowed
  __shared__ float list_x[kList];
  __shared__ uint32_t queue[kQueue];  // token of the pass, what it is (kBias and so on), low 16 bits of the bias entry
  __shared__ int listed, queued, next_unit;
  const int rank = (int)cg::this_cluster().block_rank();
  const int row = blockIdx.x / p.ctas;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (rank == 0 && threadIdx.x == 0) {
    mbar_init(smem_u32(&arrived), 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(smem_u32(&arrived), p.ctas * 8);
  }
  __syncwarp();
  // waited for before the first write into another CTA's shared memory
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();
  pdl_launch_dependents();

  const T* x = static_cast<const T*>(p.logits) + (size_t)row * (size_t)p.stride;
  float* out = p.out ? p.out + (size_t)row * (size_t)p.out_stride : nullptr;
  const uint32_t* mask = p.mask ? p.mask + (size_t)row * (size_t)p.mask_stride : nullptr;
  const int32_t* history = p.history + (size_t)row * (size_t)p.hist_stride;
  const int32_t* bias_ids = p.bias_ids + (size_t)row * (size_t)p.bias_stride;

  float bv = -INFINITY;  // the largest value above -inf, and its id
  int bi = -1;
  bool nothing_yet = true;
  int span = min(p.part, kMostTokens);
  for (int base = 0; base < p.part;) {
    const int first = min(p.vocab, (int)min((long long)rank * p.part + base, (long long)p.vocab));
    const int n = min(min(span, p.part - base), p.vocab - first);  // tokens of this pass
    // the stream begins behind `skip` tokens, on a 16-byte boundary
    const int skip = kAligned ? 0 : min(n, (int)((16u - (uint32_t)(reinterpret_cast<uintptr_t>(x + first) & 15u)) % 16u / sizeof(T)));
    const int vecs = (n - skip) / N;
    const uint4* src = reinterpret_cast<const uint4*>(x + first + skip);
    const bool out_wide = kAligned || (reinterpret_cast<uintptr_t>(out + first + skip) & 15u) == 0;
    int hist = 0, prompt = 0;
    int hist_id[kIds], bias_id[kIds];  // the first of both lists
    load_ids<kThreads>(history, threadIdx.x, (int)p.hist_stride, hist_id);
    load_ids<kThreads>(bias_ids, threadIdx.x, p.bias_count, bias_id);
    if (p.history) {
      hist = (int)max(0ll, min((long long)__ldg(p.history_lens + row), p.hist_stride));
      if (p.prompt_lens) prompt = __ldg(p.prompt_lens + row);
    }
    const bool bits = mask || p.history || p.bias_count > 0;
    if (bits)
      for (int i = threadIdx.x; i < (n + 31) / 32; i += kThreads) allow[i] = mask ? __ldg(mask + (first >> 5) + i) : 0xFFFFFFFFu;
    // a unit of the stream: kBatch loads of a warp; the first is its own in any case
    int unit = warp;
    const auto vec_of = [&](int which, int u) { return (which * kBatch + u) * 32 + lane; };
    uint4 raw[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (vec_of(unit, u) < vecs) raw[u] = __ldcs(src + vec_of(unit, u));

    const bool tables = hist > 0 || p.bias_count > 0;
    if (tables) {
      const SharedTable table{key, &listed};
      const bool may_overflow = n > kList;
      // the first `total` of the queue into the table, by the first `threads` threads; `high`: of the bias entries
      const auto enter = [&](int threads, int total, uint32_t high) {
        for (int i0 = threadIdx.x & ~31; i0 < total; i0 += threads) {
          bool entered = false;
          int slot = -1;
          float v = 0.f;
          uint32_t word = 0xFFFFFFFFu;
          if (i0 + lane < total) {
            const uint32_t e = queue[i0 + lane];
            const int at = (int)(e & 0x3FFFu);
            v = load1(x + first + at);  // needed if the token is new; under way meanwhile
            if (mask) word = __ldg(mask + ((first + at) >> 5)) >> (at & 31);
            slot = slot_of(table, at, may_overflow, entered);
            if (slot >= 0) {
              const uint32_t what = e & kWhat;
              if (what == kBias)
                atomicMax(entry + slot, (high | e >> 16) + 1u);
              else if (what == kPrompt)
                atomicOr(count + slot, kSeen);
              else
                atomicAdd(count + slot, 1u);
            }
          }
          const uint32_t fresh = __ballot_sync(0xffffffffu, entered);
          if (fresh) {
            int where = 0;
            if (lane == 0) where = atomicAdd(&listed, __popc(fresh));
            where = __shfl_sync(0xffffffffu, where, 0) + __popc(fresh & ((1u << lane) - 1));
            if (entered && where < kList) {
              list[where] = (uint16_t)(slot | (word & 1u ? kAllowed : 0u));
              list_x[where] = v;
            }
          }
        }
      };
      int room = kQueue, done = 0;  // ids that still fit in any case; those that are in the table
      uint32_t high = 0;
      // ids of the part into the queue, their tokens out of the stream's hands
      const auto collect = [&](const int32_t* ids, int total, const int (&head)[kIds], bool biases) {
        for (int k0 = 0; k0 < total; k0 += kRound) {
          const bool turn = biases && (uint32_t)k0 >> 16 << 16 != high;
          const int most = min(kRound, total - k0);
          if (turn || room < most) {
            __syncthreads();
            const int waiting = queued;
            __syncthreads();
            room = kQueue - waiting;
            if (turn || room < most) {
              enter(kThreads, waiting, high);
              done += waiting;
              room = kQueue;
              if (threadIdx.x == 0) queued = 0;
              __syncthreads();
            }
            if (biases) high = (uint32_t)k0 >> 16 << 16;
          }
          room -= most;
          int id[kIds], packed = 0;
          if (k0 == 0) {
#pragma unroll
            for (int u = 0; u < kIds; ++u) id[u] = (int)threadIdx.x + u * kThreads < total ? head[u] : -1;
          } else {
            load_ids<kThreads>(ids, k0 + threadIdx.x, total, id);
          }
          // padding (negative, or behind the vocabulary) is in no part
          uint32_t in[kIds];
#pragma unroll
          for (int u = 0; u < kIds; ++u) {
            in[u] = __ballot_sync(0xffffffffu, id[u] >= 0 && (unsigned)(id[u] - first) < (unsigned)n);
            packed += __popc(in[u]);
          }
          if (packed == 0) continue;
          int where = 0;
          if (lane == 0) where = atomicAdd(&queued, packed);
          where = __shfl_sync(0xffffffffu, where, 0);
#pragma unroll
          for (int u = 0; u < kIds; ++u) {
            if (in[u] >> lane & 1u) {
              const int at = id[u] - first, k = k0 + (int)threadIdx.x + u * kThreads;
              queue[where + __popc(in[u] & ((1u << lane) - 1))] =
                  (uint32_t)at | (biases ? kBias | (uint32_t)k << 16 : k < prompt ? kPrompt : 0u);
              atomicAnd(allow + (at >> 5), ~(1u << (at & 31)));
            }
            where += __popc(in[u]);
          }
        }
      };
      Row r{1.f, 0.f, 0.f, p.bias_values + (size_t)row * (size_t)p.bias_stride};
      if (p.repetition) r.rep = __ldg(p.repetition + row);
      if (p.presence) r.pres = __ldg(p.presence + row);
      if (p.frequency) r.freq = __ldg(p.frequency + row);
      for (int i = threadIdx.x; i < kSlots / 4; i += kThreads) {
        reinterpret_cast<uint4*>(key)[i] = make_uint4(kEmpty, kEmpty, kEmpty, kEmpty);
        reinterpret_cast<uint4*>(count)[i] = make_uint4(0, 0, 0, 0);
        reinterpret_cast<uint4*>(entry)[i] = make_uint4(0, 0, 0, 0);
      }
      if (threadIdx.x == 0) {
        listed = queued = 0;
        next_unit = kWarps;
      }
      __syncthreads();
      if (p.bias_count > 0) collect(bias_ids, p.bias_count, bias_id, true);
      collect(history, hist, hist_id, false);
      __syncthreads();
      const int waiting = queued;
      // Some warps do the rest while the others stream -- unless the list may overflow, which has to
      // be known first, or the stream writes over the logits that are needed here.
      const bool apart = done + waiting <= kList && static_cast<const void*>(out) != static_cast<const void*>(x);
      const int threads = apart && waiting <= kEnterApart ? kEnterWarps * 32 : kThreads;
      if ((int)threadIdx.x < threads) {
        enter(threads, waiting, high);
        __syncwarp();
        asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
        if (listed >= kList && may_overflow && !apart) {  // it may be incomplete: a smaller range
          span = max(kList, ((n + 1) / 2 + 31) & ~31);
          __syncthreads();
          continue;
        }
        for (int i = threadIdx.x; i < listed; i += threads) {
          const uint32_t e = list[i], slot = e & (kSlots - 1);
          const float v = change(list_x[i], count[slot], entry[slot], r);
          count[slot] = !(e & kAllowed) ? kMaskedBits : v != v ? 0x7FFFFFFFu : __float_as_uint(v);
        }
      }
    } else if (bits) {
      __syncthreads();
    }

    // Whole units have no branch inside, so that their tests and loads overlap; a thread's ids
    // ascend, so of equal values the first stands.
    while (unit * (kBatch * 32) < vecs) {
      int next = unit + kWarps;
      if (tables) {  // not all warps began at the same time
        if (lane == 0) next = atomicAdd(&next_unit, 1);
        next = __shfl_sync(0xffffffffu, next, 0);
      }
      uint32_t allowed[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int k = vec_of(unit, u);
        allowed[u] = 0;
        if (k < vecs) {
          const int at = skip + N * k;
          uint32_t w = 0xFFu;
          if (bits) w = skip % N ? __funnelshift_r(allow[at >> 5], allow[(at >> 5) + 1], at & 31) : allow[at >> 5] >> (at & 31);
          allowed[u] = w & ((1u << N) - 1);
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int k = vec_of(unit, u);
        float v[N];
        widen(raw[u], v, (const T*)nullptr);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = (allowed[u] >> e) & 1u ? v[e] : -INFINITY;
        float top = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));  // fmaxf drops NaN
        if (N == 8) top = fmaxf(top, fmaxf(fmaxf(v[N - 4], v[N - 3]), fmaxf(v[N - 2], v[N - 1])));
        int at = N - 1;
#pragma unroll
        for (int e = N - 2; e >= 0; --e) at = v[e] == top ? e : at;
        const bool better = top > bv;
        bv = better ? top : bv;
        bi = better ? first + skip + N * k + at : bi;
        if (out && k < vecs) {
          float* to = out + first + skip + N * k;
          if (out_wide) {
#pragma unroll
            for (int e = 0; e < N; e += 4)
              __stcs(reinterpret_cast<float4*>(to + e), make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]));
          } else {
#pragma unroll
            for (int e = 0; e < N; ++e) __stcs(to + e, v[e]);
          }
        }
        if (vec_of(next, u) < vecs) raw[u] = __ldcs(src + vec_of(next, u));
      }
      unit = next;
    }
    const auto single = [&](int k, bool& can) {
      can = !bits || ((allow[k >> 5] >> (k & 31)) & 1u);
      return can ? load1(x + first + k) : -INFINITY;
    };
    for (int i = threadIdx.x; i < n - N * vecs; i += kThreads) {  // in front of the stream and behind it
      const int k = i < skip ? i : i + N * vecs;
      bool can;
      const float v = single(k, can);
      if (can && (v > bv || (v == bv && first + k < bi))) {
        bv = v;
        bi = first + k;
      }
      if (out) __stcs(out + first + k, v);
    }
    if (tables) {
      __syncthreads();  // the stream has written its -inf
      for (int i = threadIdx.x; i < listed; i += kThreads) {
        const int slot = list[i] & (kSlots - 1), id = first + (int)key[slot];
        const uint32_t value = count[slot];
        if (value != kMaskedBits) take(__uint_as_float(value), id, bv, bi);
        if (out) out[id] = value != kMaskedBits ? __uint_as_float(value) : -INFINITY;
      }
    }
    // Nothing above -inf in the part so far: the first -inf that is allowed counts (rare).
    if (nothing_yet) {
      nothing_yet = !__syncthreads_or(bv > -INFINITY);
      if (nothing_yet) {
        for (int k = threadIdx.x; k < n; k += kThreads) {
          bool can;
          const float v = single(k, can);
          if (can) take(v, first + k, bv, bi);
        }
      }
    }
    base += min(span, p.part - base);
    if (base < p.part) __syncthreads();  // the next pass uses the table again
  }

  uint32_t top = order_of(bv, bi), id = (uint32_t)bi;
  best_of_warp(top, id);
  if (lane == 0) best[warp] = make_uint2(top, id);
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA of the cluster has started
  if (!p.ids) return;
  if (warp != 0) {
    if (p.long_lists) cluster_barrier();
  } else {
    const uint2 w = lane < kThreads / 32 ? best[lane] : make_uint2(0u, 0xFFFFFFFFu);
    top = w.x;
    id = w.y;
    best_of_warp(top, id);
    if (lane == 0) send8(smem_u32(&best_of[rank]), smem_u32(&arrived), (uint64_t)id << 32 | top);
    __syncwarp();
    if (p.long_lists) cluster_barrier();
    if (rank == 0) {
      bool all = __all_sync(0xffffffffu, wait_cluster(smem_u32(&arrived)));
      if (!all) all = wait_for_exit(smem_u32(&arrived), p.long_lists);
      const uint64_t e = lane < p.ctas ? best_of[lane] : 0xFFFFFFFFull << 32;
      top = (uint32_t)e;
      id = (uint32_t)(e >> 32);
      best_of_warp(top, id);
      if (lane == 0) p.ids[row] = all ? (int)id : kExchangeFailed;
    }
  }
}

template <typename T, typename Shape>
int launch_logits(LogitsParams& p, int rows, int ctas, cudaStream_t stream) {
  p.ctas = ctas;
  p.part = ((p.vocab + ctas - 1) / ctas + 31) & ~31;
  p.long_lists = (p.hist_stride + p.bias_count) > kLongLists / p.part;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows * ctas);
  cfg.blockDim = dim3(Shape::kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // every row on a 16-byte boundary, read and written
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.logits) | reinterpret_cast<uintptr_t>(p.out) |
                       (rows > 1 ? (uintptr_t)p.stride * sizeof(T) | (p.out ? (uintptr_t)p.out_stride * 4 : 0) : 0);
  auto* kernel = (at & 15u) == 0
                     ? logits_kernel<T, true, Shape::kThreads, Shape::kResident, Shape::kBatch, Shape::kIds>
                     : logits_kernel<T, false, Shape::kThreads, Shape::kResident, Shape::kBatch, Shape::kIds>;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, p), "cudaLaunchKernelEx(logits)");
}

template <typename T>
int launch_logits(LogitsParams& p, int rows, int sms, cudaStream_t stream) {
  if ((long long)rows * kCtas <= (long long)sms * Few::kResident) return launch_logits<T, Few>(p, rows, kCtas, stream);
  // As many CTAs per row as run at once, but parts that one pass holds, and lists that leave a
  // part's tokens few.  1, 2, 4 and 8 CTAs per row (us, the rule's first): 40 rows of 15603
  // bf16 8: 6.2 (6.5, 5.4, 5.5); 184 with 100 ids 2: 8.4 (7.9, 11.3, 15.9), with 1231 ids 4:
  // 15.6 (27.6, 14.5, 19.5); 150 of 32000 fp32 with 1024 ids 4: 14.0 (20.6, 13.7, 16.6); 64 of
  // 128256 fp32 8: 15.7 (56, 31, 20); 256 of 50000 fp32 4: 17.5 (24.5, 17.9, 22.8); 1000 of
  // 32000 bf16 with 1000 ids 2: 43.2 (43.4, 52.5, 81.8); where it is off, by 20 % at most but
  // for 200 of 4000 with 3000 ids, 8: 22.0 (50.8, 29.6, 16.3).
  int ctas = 1;
  while (ctas < kCtas && ((long long)rows * ctas * 2 <= (long long)sms * Many::kResident || (p.vocab + ctas - 1) / ctas > kMostTokens ||
                          (p.hist_stride + p.bias_count) / ctas > kList / 2))
    ctas *= 2;
  return launch_logits<T, Many>(p, rows, ctas, stream);
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
  if (rows > (1 << 27) || vocab > (1 << 30) || history_stride > (1ll << 30) || bias_count > (1 << 30))
    return PKV_ERR_UNSUPPORTED_SHAPE;
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
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == PKV_LOGITS_F32) return launch_logits<float>(p, rows, sm_count(dev), st);
  if (dtype == PKV_LOGITS_BF16) return launch_logits<__nv_bfloat16>(p, rows, sm_count(dev), st);
  return launch_logits<__half>(p, rows, sm_count(dev), st);
}
