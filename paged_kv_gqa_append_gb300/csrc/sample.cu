// The next token of each row, drawn from softmax(logits / temperature) restricted by
// top-k, top-p and min-p, from given exponential variates (sm_103a).
//
// With w_i = 2^(c (x_i - max x)), c = log2(e) / T, the token drawn is the kept one with
// the largest w_i / e_i: the race of independent exponentials, which follows the kept
// tokens' distribution.  Which tokens are kept needs no sorting.  The kept ones are the
// first so many by rank, so
//   - the winner of the race among all candidates is the answer if it is kept: the
//     tokens ranked before it are fewer than k, their w sum to less than p Z, and its own
//     w reaches the floor -- one pass of counting and adding;
//   - else nothing behind it is kept either, and the race goes on among the tokens ranked
//     before it.
// A rejected winner is a random token of what is left, so a few rounds are enough; noise
// that is made to take many is met by bisecting for the last kept token after kRounds.
//
// Candidates: k tokens are at least as large as the smallest of the warps' q-th largest thread maxima
// when there are k / q warps; min-p bounds the logits by max x; for top-p the same bound is tried, and
// holds if the tokens from it on have p of the sum.  So there are usually a few hundred candidates in a
// row, listed in shared memory warp by warp in order, and only their noise is read; the row's first CTA
// gets all lists and settles the row alone.  Where the lists overflow, or without limits, the passes go
// over all logits, and the CTAs agree behind a cluster barrier after each.
//
// A cluster of CTAs has a row, each a part of it in shared memory (bulk copies, read from the GPU's memory
// once).  The first pass takes an operation, an exponential and an addition per logit: the exponent's
// reference is c times a logit, rounded, and the sum is moved to the exact one at the end (logits that are
// not finite, or so large that this rounding shows, are summed again one by one).  Sums are over fixed
// positions in a fixed order; ties of a race go to the lowest id.
//
// Bound: the steps of a row, one after another -- its parts' copies, the first sums, the bound, the lists,
// the first CTA's rounds, with two cluster barriers -- in as many rows at once as shared memory holds (57 of
// 128256 fp32 logits).  One such row with top-k and top-p takes 10.4 us, 32 bf16 rows with top-p and min-p
// 18 us, 256 fp32 rows with all limits 61.5 us (the logits, nearly all that such rows read, are 19.3 us of bytes
// at the measured copy rate); 256 rows without limits 88 us (logits and noise: 38.7 us), with a top-p that most
// of a flat row is in 146 to 175 us.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "pkv.h"
#include "ptx.cuh"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kMostCtas = 8;
constexpr int kLeast = 4096;         // tokens of a CTA that make another one worth its barrier
constexpr int kMostHeld = 100 << 10;  // bytes of logits in a CTA's shared memory
constexpr int kChunk = 1024;          // 16-byte vectors of a copy there
constexpr int kChunks = (kMostHeld / 16 + kChunk - 1) / kChunk;
constexpr uint32_t kWaitUs = 2000000;  // limit of the waits for the copies
constexpr int kList = 64;            // candidates of a warp
constexpr int kMostQ = 16;
constexpr int kTryQ = 4;             // of the bound tried for top-p
constexpr int kCandidates = 2048;  // of a row, at most, in lists
constexpr int kRounds = 12;

struct SampleParams {
  const void* logits;
  const float* noise;
  long long stride, noise_stride;
  const float *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* ids;
  float* log_probs;
  int vocab, ctas;
};

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float log2_approx(float x) {  // of a normal number
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <class T>
struct Wide;
template <>
struct Wide<float> {
  static constexpr int kN = 4;
  __device__ static void widen(const uint4& a, float (&x)[4]) {
    x[0] = __uint_as_float(a.x);
    x[1] = __uint_as_float(a.y);
    x[2] = __uint_as_float(a.z);
    x[3] = __uint_as_float(a.w);
  }
  __device__ static float one(float x) { return x; }
};
template <>
struct Wide<__nv_bfloat16> {
  static constexpr int kN = 8;
  __device__ static void widen(const uint4& a, float (&x)[8]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = bf16lo_to_f32(w[e]);
      x[2 * e + 1] = bf16hi_to_f32(w[e]);
    }
  }
  __device__ static float one(__nv_bfloat16 x) { return __bfloat162float(x); }
};
template <>
struct Wide<__half> {
  static constexpr int kN = 8;
  __device__ static void widen(const uint4& a, float (&x)[8]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
    }
  }
  __device__ static float one(__half x) { return __half2float(x); }
};

// NaN as -inf, +inf as the largest number: differences are never NaN where one is finite.
__device__ __forceinline__ float tame(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }
__device__ __forceinline__ float tame_noise(float e) { return fminf(fmaxf(e, 0x1p-126f), FLT_MAX); }

// Floats in order as unsigned numbers, and back.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// What a thread, a warp, a CTA and a row have found: in the first pass
struct First {
  float max, sum, bound;  // largest logit, sum of w under that maximum, the bound
};
// and in the others.
struct Found {
  float race, x;     // the race: its best, and that token's logit
  int id;
  float mass;        // the sum of w of the tokens asked about
  int count, flags;  // how many they are; whether a list overflowed
};
struct Tally {  // of the lists
  float mass;
  int count, overflow;
};
__device__ __forceinline__ bool better(float r, int i, float than, int id) { return r > than || (r == than && i < id); }
__device__ __forceinline__ void combine(First& a, const First& b, float c) {
  const float m = fmaxf(a.max, b.max);
  // (rounded one by one: the same whichever of the two is whose)
  a.sum = __fadd_rn(__fmul_rn(a.sum, exp2_approx((a.max - m) * c)), __fmul_rn(b.sum, exp2_approx((b.max - m) * c)));
  a.max = m;
  a.bound = fminf(a.bound, b.bound);
}
__device__ __forceinline__ void combine(Found& a, const Found& b) {
  if (better(b.race, b.id, a.race, a.id)) {
    a.race = b.race;
    a.x = b.x;
    a.id = b.id;
  }
  a.mass += b.mass;
  a.count += b.count;
  a.flags |= b.flags;
}
// over groups of n lanes; all lanes get the result
__device__ __forceinline__ void over_lanes(First& f, int n, float c) {
  for (int o = n / 2; o > 0; o >>= 1) {
    First g;
    g.max = __shfl_xor_sync(0xffffffffu, f.max, o);
    g.sum = __shfl_xor_sync(0xffffffffu, f.sum, o);
    g.bound = __shfl_xor_sync(0xffffffffu, f.bound, o);
    combine(f, g, c);
  }
}
__device__ __forceinline__ void over_lanes(Tally& f, int n) {
  for (int o = n / 2; o > 0; o >>= 1) {
    f.mass += __shfl_xor_sync(0xffffffffu, f.mass, o);
    f.count += __shfl_xor_sync(0xffffffffu, f.count, o);
    f.overflow |= __shfl_xor_sync(0xffffffffu, f.overflow, o);
  }
}
__device__ __forceinline__ void over_lanes(Found& f, int n) {
  for (int o = n / 2; o > 0; o >>= 1) {
    Found g;
    g.race = __shfl_xor_sync(0xffffffffu, f.race, o);
    g.x = __shfl_xor_sync(0xffffffffu, f.x, o);
    g.id = __shfl_xor_sync(0xffffffffu, f.id, o);
    g.mass = __shfl_xor_sync(0xffffffffu, f.mass, o);
    g.count = __shfl_xor_sync(0xffffffffu, f.count, o);
    g.flags = __shfl_xor_sync(0xffffffffu, f.flags, o);
    combine(f, g);
  }
}

struct Pivot {
  float x;
  int id;
  __device__ __forceinline__ bool before(float y, int i) const { return y > x || (y == x && i < id); }
};

template <int kWarps>
struct SmemOf {
  First firsts[kWarps], first_rows[kMostCtas];
  Tally tallies[kWarps], tally_rows[kMostCtas];
  Found warps[2][kWarps], rows[2][kMostCtas];  // two of each: one is read while the next is written
  float x[kWarps][kList];
  int id[kWarps][kList], here[kWarps];
  uint64_t landed[kChunks];
};

template <class T, bool kHeld, int kCtaThreads>
struct Row {
  static constexpr int kThreads = kCtaThreads, kWarps = kThreads / 32;
  using Smem = SmemOf<kWarps>;
  static constexpr int kN = Wide<T>::kN;
  static constexpr int kBatch = 4;  // 16-byte loads in flight per thread, where they are not held
  const SampleParams& p;
  Smem& sh;
  uint4* held;               // the part's logits, if they are held
  const T* logits;
  const float* noise;
  int head, vectors, v0, v1;  // tokens before the first 16-byte boundary; whole vectors, and this CTA's
  int rank, turn;
  bool wide_noise;

  __device__ Row(const SampleParams& q, Smem& s, uint4* h) : p(q), sh(s), held(h), turn(0) {
    const int r = blockIdx.x / p.ctas;
    rank = blockIdx.x % p.ctas;
    logits = static_cast<const T*>(p.logits) + (long long)r * p.stride;
    noise = p.noise ? p.noise + (long long)r * p.noise_stride : nullptr;
    head = min(p.vocab, (int)((16 - (reinterpret_cast<uintptr_t>(logits) & 15)) % 16 / sizeof(T)));
    vectors = (p.vocab - head) / kN;
    const int per = (vectors + p.ctas - 1) / p.ctas;
    v0 = min(vectors, rank * per);
    v1 = min(vectors, v0 + per);
    wide_noise = (reinterpret_cast<uintptr_t>(noise + head) & 15) == 0;
  }
  // the tokens beside the vectors: one each for the first threads of the first CTA
  __device__ __forceinline__ int extra() const {
    const int loose = head + (p.vocab - head - vectors * kN);
    if (rank != 0 || (int)threadIdx.x >= loose) return -1;
    return (int)threadIdx.x < head ? (int)threadIdx.x : (int)threadIdx.x + vectors * kN;
  }
  __device__ __forceinline__ void raw(int v, float (&x)[kN]) const {
    Wide<T>::widen(kHeld ? held[v - v0] : __ldg(reinterpret_cast<const uint4*>(logits + head) + v), x);
  }
  __device__ __forceinline__ void vector(int v, float (&x)[kN]) const {
    raw(v, x);
#pragma unroll
    for (int e = 0; e < kN; ++e) x[e] = tame(x[e]);
  }
  // f(x, id) for every logit of this thread, always in the same order
  template <class F>
  __device__ __forceinline__ void every(const F& f) const {
    const int i = extra();
    if (i >= 0) f(tame(Wide<T>::one(logits[i])), i);
    for (int v = v0 + threadIdx.x; v < v1; v += kThreads) {
      float x[kN];
      vector(v, x);
#pragma unroll
      for (int e = 0; e < kN; ++e) f(x[e], head + v * kN + e);
    }
  }

  // the same, but for some of those below x
  template <class F>
  __device__ __forceinline__ void every_from(float from, const F& f) const {
    const int i = extra();
    if (i >= 0) f(tame(Wide<T>::one(logits[i])), i);
#pragma unroll 2
    for (int v = v0 + threadIdx.x; v < v1; v += kThreads) {
      float x[kN];
      vector(v, x);
      float m = x[0];
#pragma unroll
      for (int e = 1; e < kN; ++e) m = fmaxf(m, x[e]);
      if (m < from) continue;
#pragma unroll
      for (int e = 0; e < kN; ++e) f(x[e], head + v * kN + e);
    }
  }

  // The CTA's, of all threads; every thread gets it.
  __device__ __forceinline__ Found of_cta(Found f) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    over_lanes(f, 32);
    if (lane == 0) sh.warps[turn][warp] = f;
    __syncthreads();
    f = sh.warps[turn][lane % kWarps];
    over_lanes(f, kWarps);
    turn ^= 1;
    return f;
  }
  // The row's: sent to every CTA of the cluster.
  __device__ __forceinline__ Found of_row(Found f) {
    f = of_cta(f);
    if (p.ctas == 1) return f;
    const cg::cluster_group cluster = cg::this_cluster();
    Found* to = &sh.rows[turn][rank];
    if ((int)threadIdx.x < p.ctas) *cluster.map_shared_rank(to, threadIdx.x) = f;
    cluster.sync();
    f = sh.rows[turn][threadIdx.x & (p.ctas - 1)];
    over_lanes(f, p.ctas);
    return f;
  }
  // (once, after the one of First)
  __device__ __forceinline__ Tally of_row(Tally f) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    over_lanes(f, 32);
    if (lane == 0) sh.tallies[warp] = f;
    __syncthreads();
    f = sh.tallies[lane % kWarps];
    over_lanes(f, kWarps);
    if (p.ctas == 1) return f;
    const cg::cluster_group cluster = cg::this_cluster();
    Tally* to = &sh.tally_rows[rank];
    if ((int)threadIdx.x < p.ctas) *cluster.map_shared_rank(to, threadIdx.x) = f;
    cluster.sync();
    f = sh.tally_rows[threadIdx.x & (p.ctas - 1)];
    over_lanes(f, p.ctas);
    return f;
  }
  __device__ __forceinline__ First of_row(First f, float c) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    over_lanes(f, 32, c);
    if (lane == 0) sh.firsts[warp] = f;
    __syncthreads();
    f = sh.firsts[lane % kWarps];
    over_lanes(f, kWarps, c);
    if (p.ctas == 1) return f;
    const cg::cluster_group cluster = cg::this_cluster();
    cluster.barrier_wait();  // all of them run
    First* to = &sh.first_rows[rank];
    if ((int)threadIdx.x < p.ctas) *cluster.map_shared_rank(to, threadIdx.x) = f;
    cluster.sync();
    f = sh.first_rows[threadIdx.x & (p.ctas - 1)];
    over_lanes(f, p.ctas, c);
    return f;
  }
};

// Everything before the place returned is kept, and nothing else, where `out` is not: the last kept place
// by bisection, first the logit, then the id.  check(place) says what lies before a place.
template <class Kept, class Check>
__device__ Pivot last_kept(const Pivot& out, float most, int vocab, const Kept& kept, const Check& check) {
  uint32_t lo = key_of(out.x) - 1, hi = key_of(most);  // (hi, 0) is kept, (lo, 0), behind `out`, is not
  while (hi - lo > 1) {
    const uint32_t mid = lo + (hi - lo) / 2;
    const Found f = check(Pivot{of_key(mid), 0});
    if (kept(of_key(mid), f.count, f.mass))
      hi = mid;
    else
      lo = mid;
  }
  int in = 0, behind = vocab;  // the place (hi, in) is kept, (hi, behind) is not or there is none
  while (behind - in > 1) {
    const int mid = in + (behind - in) / 2;
    const Found f = check(Pivot{of_key(hi), mid});
    if (kept(of_key(hi), f.count, f.mass))
      in = mid;
    else
      behind = mid;
  }
  return Pivot{of_key(hi), in + 1};
}

struct Candidates {
  float x[kCandidates], noise[kCandidates];
  int id[kCandidates];
};

// The candidates of all CTAs' lists, brought to the first one, which settles the row.  noise: of this
// lane's entries of its warp's list.  The logits held in shared memory make room for them.
template <class R, class Kept, class Finish>
__device__ __forceinline__ void resolve(R& row, const float (&noise)[kList / 32], int total, float c, float most,
                                        const Kept& kept, const Finish& finish) {
  constexpr int kThreads = R::kThreads, kEach = kCandidates / kThreads;
  const SampleParams& p = row.p;
  typename R::Smem& sh = row.sh;
  const cg::cluster_group cluster = cg::this_cluster();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Candidates* mine = reinterpret_cast<Candidates*>(row.held);
  {
    Candidates* to = p.ctas == 1 ? mine : cluster.map_shared_rank(mine, 0);
    int at = 0;  // of the warp's list among all
    if (p.ctas > 1)
      for (int i = 0; i < row.rank; ++i) at += sh.tally_rows[i].count;
    for (int w = 0; w < warp; ++w) at += sh.here[w];
#pragma unroll
    for (int e = 0; e < kList / 32; ++e) {
      const int j = lane + 32 * e;
      if (j >= sh.here[warp]) break;
      to->x[at + j] = sh.x[warp][j];
      to->id[at + j] = sh.id[warp][j];
      to->noise[at + j] = noise[e];
    }
  }
  if (p.ctas > 1) cluster.sync();
  else __syncthreads();
  if (row.rank != 0) return;
  float x[kEach], r[kEach], w[kEach];
  int id[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = threadIdx.x + e * kThreads;
    x[e] = i < total ? mine->x[i] : -INFINITY;
    id[e] = i < total ? mine->id[i] : INT_MAX;
    r[e] = i < total ? mine->noise[i] : 1.f;
    w[e] = 0.f;
  }
#pragma unroll
  for (int e = 0; e < kEach; ++e)
    if (id[e] != INT_MAX) {
      const float y = (x[e] - most) * c;
      r[e] = y - log2f(r[e]);
      w[e] = exp2_approx(y);
    }
  // what lies before a place, and the best race there
  const auto look = [&](const Pivot& at) {
    Found f{-INFINITY, -INFINITY, INT_MAX, 0.f, 0, 0};
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (id[e] != INT_MAX && at.before(x[e], id[e])) combine(f, Found{r[e], x[e], id[e], w[e], 1, 0});
    return row.of_cta(f);
  };
  Found now = look(Pivot{-INFINITY, INT_MAX});
  Pivot at{now.x, now.id};
  bool done = false;
  for (int round = 0; round < kRounds && !done; ++round) {
    at = Pivot{now.x, now.id};
    const Found f = look(at);
    done = kept(at.x, f.count, f.mass);
    if (!done) now = f;
  }
  if (!done) now = look(last_kept(at, most, p.vocab, kept, look));
  finish(now);
}

// kCtaThreads: with 512 a row is done sooner; with 256 a CTA spends less on its reductions, and three of
// them share an SM, so that many rows with limits are done sooner (256 fp32 rows of 128256 61.5 us, with 512
// threads, two CTAs per SM 85 us, three, which spill, 73 us; without limits 98 us, with 512 threads 88 us; 32
// bf16 rows 23.7 and 18.0 us).  The host sees which limits are given, not their values: many rows whose limits are
// all off cost the 98 us.
template <class T, bool kHeld, int kCtaThreads, int kPerSm>
__global__ void __launch_bounds__(kCtaThreads, kPerSm) sample_kernel(const SampleParams p) {
  extern __shared__ uint4 held[];
  using R = Row<T, kHeld, kCtaThreads>;
  constexpr int kN = R::kN, kThreads = R::kThreads, kWarps = R::kWarps;
  __shared__ typename R::Smem sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row_id = blockIdx.x / p.ctas;
  if (kHeld) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < kChunks; ++i) mbar_init(smem_u32(&sh.landed[i]), 1);
      fence_mbar_init();
    }
    __syncthreads();
  }
  // no CTA writes into another's shared memory before that one runs
  if (p.ctas > 1) cg::this_cluster().barrier_arrive();
  pdl_wait();
  pdl_launch_dependents();
  R row(p, sh, held);
  if (kHeld && threadIdx.x == 0) {
    for (int i = 0, v = row.v0; v < row.v1; ++i, v += kChunk) {
      const uint32_t bytes = min(kChunk, row.v1 - v) * 16;
      mbar_arrive_expect_tx(smem_u32(&sh.landed[i]), bytes);
      bulk_load(smem_u32(held + (v - row.v0)), row.logits + row.head + (size_t)v * kN, bytes, smem_u32(&sh.landed[i]));
    }
  }
  // a copy in flight needs its CTA's shared memory
  const auto all_landed = [&]() {
    bool good = true;
    if (kHeld)
      for (int i = 0, v = row.v0; v < row.v1; ++i, v += kChunk) good &= mbar_wait_bounded(smem_u32(&sh.landed[i]), 0, kWaitUs);
    return good;
  };
  const float temp = p.temperature ? p.temperature[row_id] : 1.f;
  const float top_p = p.top_p ? p.top_p[row_id] : 1.f, floor = p.min_p ? p.min_p[row_id] : 0.f;
  const int want_k = p.top_k ? p.top_k[row_id] : 0;
  const bool greedy = temp == 0.f;
  const auto answer = [&](int id, float lp) {
    if (row.rank == 0 && threadIdx.x == 0) {
      p.ids[row_id] = id;
      if (p.log_probs) p.log_probs[row_id] = lp;
    }
  };
  if (!(temp >= 0.f && temp < INFINITY) || top_p != top_p || floor != floor || (!greedy && !p.noise)) {
    answer(-1, NAN);
    all_landed();
    if (p.ctas > 1) cg::this_cluster().barrier_wait();
    return;
  }
  const float c = greedy ? 1.4426950408889634f : fminf(1.4426950408889634f / temp, FLT_MAX);
  const int limit = want_k > 0 && want_k < p.vocab ? want_k : INT_MAX;

  // First pass: the largest logit and the sum of w, first as if all logits were finite or -inf: the sum
  // of 2^(c x - at), one operation before the exponential, `at` near c times the largest one so far.
  float top = -FLT_MAX, at = -FLT_MAX, sum = 0.f;
  const auto take = [&](const float (&x)[kN]) {
    float m = x[0];
#pragma unroll
    for (int e = 1; e < kN; ++e) m = fmaxf(m, x[e]);
    if (m > top) {
      const float now = __fmul_rn(m, c);
      sum *= exp2_approx(at - now);
      at = now;
      top = m;
    }
    float part = 0.f;
#pragma unroll
    for (int e = 0; e < kN; ++e) part += exp2_approx(fmaf(x[e], c, -at));
    sum += part;
  };
  bool good = true;  // the logits have arrived
  if (kHeld) {
#pragma unroll 2
    for (int v = row.v0 + threadIdx.x, i = 0; v < row.v1; v += kThreads, ++i) {
      if (i % (kChunk / kThreads) == 0) good &= mbar_wait_bounded(smem_u32(&sh.landed[i / (kChunk / kThreads)]), 0, kWaitUs);
      float x[kN];
      Wide<T>::widen(held[v - row.v0], x);
      take(x);
    }
  } else {
    const uint4* src = reinterpret_cast<const uint4*>(row.logits + row.head);
    for (int v = row.v0 + threadIdx.x; v < row.v1; v += R::kBatch * kThreads) {
      uint4 raw[R::kBatch];
#pragma unroll
      for (int u = 0; u < R::kBatch; ++u)
        if (v + u * kThreads < row.v1) raw[u] = __ldg(src + v + u * kThreads);
#pragma unroll
      for (int u = 0; u < R::kBatch; ++u) {
        if (v + u * kThreads >= row.v1) break;
        float x[kN];
        Wide<T>::widen(raw[u], x);
        take(x);
      }
    }
  }
  // Not so, or c x so large that its rounding shows, or one token more: again, one by one.  (No logit at
  // all leaves `at` where it was.)
  if (!(sum < INFINITY) || !(fabsf(at) < 0x1p20f) || row.extra() >= 0) {
    top = -FLT_MAX;
    sum = 0.f;
    row.every([&](float x, int) {
      if (x > top) {
        sum *= exp2_approx((top - x) * c);
        top = x;
      }
      sum += exp2_approx((x - top) * c);
    });
  } else {
    sum *= exp2_approx(-fmaf(top, c, -at));  // from the rounded place to the exact one
  }
  if (!good) sum = NAN;  // every CTA of the row will see it
  // the q-th largest of the warp's thread maxima: with that many in every warp, at least `limit`
  const int teams = kWarps * p.ctas;
  const bool by_k = limit != INT_MAX && (limit + teams - 1) / teams <= kMostQ;
  const bool by_p = top_p < 1.f;
  const int q = greedy ? 0 : by_k ? (limit + teams - 1) / teams : by_p ? kTryQ : 0;
  float bound = -INFINITY;
  {
    uint32_t key = key_of(top);
    for (int i = 0; i < q; ++i) {
      const uint32_t most = __reduce_max_sync(0xffffffffu, key);
      bound = of_key(most);
      const uint32_t who = __ballot_sync(0xffffffffu, key == most);
      if (lane == __ffs(who) - 1) key = 0;
    }
  }
  const First whole = row.of_row(First{top, sum, bound}, c);
  const float most = whole.max, z = whole.sum;
  bound = whole.bound;
  if (!(z > 0.f)) {  // nothing above -inf, or (NaN) logits that did not arrive
    if (z != z) {
      all_landed();
      answer(-2, NAN);
      return;
    }
    answer(-1, NAN);
    return;
  }
  const auto finish = [&](const Found& f) {
    answer(f.id, (greedy ? f.x - most : (f.x - most) / temp) - logf(z));
  };

  if (greedy) {
    int first = INT_MAX;
    row.every([&](float x, int i) {
      if (x == most) first = min(first, i);
    });
    finish(row.of_row(Found{first == INT_MAX ? -INFINITY : 0.f, most, first, 0.f, 0, 0}));
    return;
  }

  // Second pass: candidates from `bound` on, listed, and their race.
  const bool by_floor = floor > 0.f;
  if (!by_k && !by_p) bound = -INFINITY;
  const bool tried = by_p && !by_k;  // holds only if the tokens from the bound on have the mass
  float sure = by_k ? bound : -INFINITY;
  if (by_floor) {  // a little below what the floor's comparison of w decides
    const float y = (log2f(fminf(floor, 1.f)) - 0x1p-12f) / c;
    sure = fmaxf(sure, most + (y - fabsf(most) * 0x1p-20f));
    bound = fmaxf(bound, sure);
  }
  // The race over all logits from `least` on that are ranked before the pivot (`all`: the pivot is behind
  // everything).  A thread looks for its best with the fast logarithm, then computes that one's again.
  float race = -INFINITY, best_x = -INFINITY;
  int best = INT_MAX;
  const auto race_all = [&](float least, const Pivot& at, bool all) {
    race = -INFINITY;
    best = INT_MAX;
    constexpr int kSteps = kN == 4 ? 2 : 1;
    for (int v = row.v0 + threadIdx.x; v < row.v1; v += kSteps * kThreads) {
      float e[kSteps][kN], x[kSteps][kN];
      bool any[kSteps];
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        const int vu = v + u * kThreads;
        any[u] = false;
        if (vu >= row.v1) break;
        row.vector(vu, x[u]);
        float m = x[u][0];
#pragma unroll
        for (int j = 1; j < kN; ++j) m = fmaxf(m, x[u][j]);
        any[u] = m >= least && m >= at.x;
        if (!any[u]) continue;
        const int id = row.head + vu * kN;
        if (row.wide_noise) {
#pragma unroll
          for (int j = 0; j < kN; j += 4) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(row.noise + id + j));
            e[u][j] = f.x;
            e[u][j + 1] = f.y;
            e[u][j + 2] = f.z;
            e[u][j + 3] = f.w;
          }
        } else {
#pragma unroll
          for (int j = 0; j < kN; ++j) e[u][j] = __ldg(row.noise + id + j);
        }
      }
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        if (!any[u]) continue;
        const int id = row.head + (v + u * kThreads) * kN;
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          const float r = (x[u][j] - most) * c - log2_approx(tame_noise(e[u][j]));
          // (ids ascend: the first of equals stays)
          if (r > race && (all || (x[u][j] >= least && at.before(x[u][j], id + j)))) {
            race = r;
            best = id + j;
          }
        }
      }
    }
    const auto exactly = [&](int i) {
      best_x = tame(Wide<T>::one(row.logits[i]));
      return (best_x - most) * c - log2f(tame_noise(row.noise[i]));
    };
    best_x = -INFINITY;
    race = best == INT_MAX ? -INFINITY : exactly(best);
    const int i = row.extra();
    if (i >= 0) {
      const float x = best_x, x2 = tame(Wide<T>::one(row.logits[i]));
      if (x2 >= least && at.before(x2, i)) {
        const float r = exactly(i);
        if (better(r, i, race, best)) {
          race = r;
          best = i;
        } else {
          best_x = x;
        }
      }
    }
  };
  const auto raced = [&]() { return Found{race, best_x, best, 0.f, 0, 0}; };
  // A token with `count` tokens before it, whose w sum to `mass`: is it kept?
  const auto kept = [&](float x, int count, float mass) {
    return count == 0 || (count < limit && (!by_p || mass < top_p * z) && (!by_floor || exp2_approx((x - most) * c) >= floor));
  };
  const bool limits = limit != INT_MAX || by_p || by_floor;
  bool listed = bound > -INFINITY;
  if (listed) {
    int here = 0;  // candidates of this warp
    float mass = 0.f;
    const auto list = [&](bool hit, float x, int i) {
      const uint32_t hits = __ballot_sync(0xffffffffu, hit);
      const int at = here + __popc(hits & ((1u << lane) - 1u));
      if (hit && at < kList) {
        mass += exp2_approx((x - most) * c);
        sh.x[warp][at] = x;
        sh.id[warp][at] = i;
      }
      here += __popc(hits);
    };
    const int i = row.extra();
    const float loose = i >= 0 ? tame(Wide<T>::one(row.logits[i])) : -INFINITY;
    list(i >= 0 && loose >= bound, loose, i);
    for (int v = row.v0 + threadIdx.x; v - lane < row.v1 && here <= kList; v += kThreads) {
      float x[kN];
      bool any = false;
      if (v < row.v1) {
        row.raw(v, x);
        float m = x[0];
#pragma unroll
        for (int j = 1; j < kN; ++j) m = fmaxf(m, x[j]);
        any = m >= bound;
      }
      if (!__any_sync(0xffffffffu, any)) continue;
#pragma unroll
      for (int j = 0; j < kN; ++j) list(any && x[j] >= bound, any ? tame(x[j]) : 0.f, row.head + v * kN + j);
    }
    const bool overflow = here > kList;
    here = min(here, kList);
    if (lane == 0) sh.here[warp] = here;
    __syncwarp();
    float chance[kList / 32];  // on its way while the CTAs agree
#pragma unroll
    for (int e = 0; e < kList / 32; ++e)
      chance[e] = lane + 32 * e < here ? tame_noise(__ldg(row.noise + sh.id[warp][lane + 32 * e])) : 1.f;
    const Tally f = row.of_row(Tally{mass, lane == 0 ? here : 0, overflow});
    // (where the sums of w before the bound reach p Z, but for their rounding)
    listed = !f.overflow && f.count <= kCandidates && (!tried || bound == sure || f.mass >= top_p * z * (1.f + 0x1p-18f));
    if (listed) {
      resolve(row, chance, f.count, c, most, kept, finish);
      return;
    }
  }
  race_all(sure, Pivot{-INFINITY, INT_MAX}, sure == -INFINITY);
  Found now = row.of_row(raced());
  if (!limits) {
    finish(now);
    return;
  }

  // Rounds: is the winner kept?  Else the race among those ranked before it.
  const auto check = [&](const Pivot& at) {
    float mass = 0.f;
    int count = 0;
    row.every_from(at.x, [&](float x, int i) {
      const bool front = at.before(x, i);
      mass += front ? exp2_approx((x - most) * c) : 0.f;
      count += front;
    });
    return row.of_row(Found{-INFINITY, 0.f, INT_MAX, mass, count, 0});
  };
  Pivot place{now.x, now.id};
  for (int round = 0; round < kRounds; ++round) {
    place = Pivot{now.x, now.id};
    const Found f = check(place);
    if (kept(place.x, f.count, f.mass)) {
      finish(now);
      return;
    }
    race_all(sure, place, false);
    now = row.of_row(raced());
  }
  race_all(sure, last_kept(place, most, p.vocab, kept, check), false);
  finish(row.of_row(raced()));
}

template <class T>
int launch(const SampleParams& p, cudaLaunchConfig_t cfg, int sms) {
  const size_t part = ((size_t)p.vocab / Wide<T>::kN + p.ctas - 1) / p.ctas * 16;
  const bool held = part <= kMostHeld, many = (int)cfg.gridDim.x > 2 * sms;
  const bool limits = p.top_k || p.top_p || p.min_p;
  cfg.dynamicSmemBytes = held && part > sizeof(Candidates) ? part : sizeof(Candidates);
  cfg.blockDim = dim3(held && many && limits ? 256 : 512);
  auto* kernel = !held ? sample_kernel<T, false, 512, 2>
                 : !many ? sample_kernel<T, true, 512, 2>
                         : limits ? sample_kernel<T, true, 256, 3> : sample_kernel<T, true, 512, 3>;
  const int rc = cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostHeld),
                             "cudaFuncSetAttribute(sample)");
  if (rc != PKV_OK) return rc;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, p), "cudaLaunchKernelEx(sample)");
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_sample_logits(const void* logits, int dtype, int rows, int vocab, long long row_stride,
                                 const float* noise, long long noise_stride, const float* temperature,
                                 const int32_t* top_k, const float* top_p, const float* min_p, int32_t* out_ids,
                                 float* log_probs, void* stream) {
  if (rows < 0 || vocab < 1 || row_stride < vocab || (noise && noise_stride < vocab) || dtype < PKV_LOGITS_F32 ||
      dtype > PKV_LOGITS_F16)
    return PKV_ERR_INVALID_ARGUMENT;
  if (rows == 0) return PKV_OK;
  if (!logits || !out_ids || (!noise && !temperature)) return PKV_ERR_INVALID_ARGUMENT;
  if ((reinterpret_cast<uintptr_t>(logits) & (dtype == PKV_LOGITS_F32 ? 3u : 1u)) ||
      ((reinterpret_cast<uintptr_t>(noise) | reinterpret_cast<uintptr_t>(temperature) |
        reinterpret_cast<uintptr_t>(top_k) | reinterpret_cast<uintptr_t>(top_p) | reinterpret_cast<uintptr_t>(min_p) |
        reinterpret_cast<uintptr_t>(out_ids) | reinterpret_cast<uintptr_t>(log_probs)) & 3u))
    return PKV_ERR_MISALIGNED;
  if (vocab > (1 << 30) || rows > (1 << 27)) return PKV_ERR_UNSUPPORTED_SHAPE;
  int dev = 0;
  const int rc = bind_stream_device(stream, &dev);
  if (rc != PKV_OK) return rc;

  const int sms = sm_count(dev);
  if (sms <= 0) return cuda_status(cudaErrorInvalidDevice, "sm_count");
  SampleParams p;
  p.logits = logits;
  p.noise = noise;
  p.stride = row_stride;
  p.noise_stride = noise_stride;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.ids = out_ids;
  p.log_probs = log_probs;
  p.vocab = vocab;
  p.ctas = 1;
  while (p.ctas < kMostCtas && vocab > p.ctas * kLeast) p.ctas *= 2;

  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows * p.ctas);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (dtype == PKV_LOGITS_F32) return launch<float>(p, cfg, sms);
  if (dtype == PKV_LOGITS_BF16) return launch<__nv_bfloat16>(p, cfg, sms);
  return launch<__half>(p, cfg, sms);
}
