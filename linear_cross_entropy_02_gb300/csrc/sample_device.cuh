// Kernels of sampling (sample.cu), which also find what the filters keep of a row for
// the verification of drafted tokens (verify.cu).
//
// The row is never sorted. In rank order (falling logit, ties by index) every
// filter keeps a prefix, so only its end has to be found. Weights are whole
// multiples of 2^-40 of the largest one and are added as 64-bit integers, so
// that no sum depends on the order or on how many CTAs share a row: the token is
// a function of the logits, the settings and u alone.
//
// A row takes two passes. The first reads it from HBM, keeps the maximum and
// counts logits in 4096 bins of (x - anchor) / T, the anchor being the maximum
// of the row's first part (of the row, if that part holds nothing finite). Then:
//   top_k that some bins cover with at most kListKeys logits: the second pass
//     collects those logits in shared memory, where all three filters cut them
//     and the token is drawn.
//   top_p: the counts times the weights of the bins' middles (exact float sums
//     for the few largest) say in which bins the end of the prefix should lie;
//     the second pass adds up all weights exactly, those above these bins by
//     segments of the vocabulary, and collects the logits in the bins. The exact
//     sums then confirm that the end lies among the collected logits.
//   neither: the second pass adds up the weights by segments.
// The segment that holds the answer is walked once more by a warp. Rows for
// which this does not work out (more than kListKeys logits in the way, as when
// most are equal, or an estimate that the exact sums refute) go through the
// general selection: a histogram of exact weights, then splitting the bin that
// holds the answer by the logits' bits until it is small enough or all equal.
//
// One CTA per row, or two rows to an SM, where there are rows for every SM: all
// exchange is within the CTA, and the second pass finds the row in shared memory or,
// if it is too long, in the L2. Few rows are spread over a cluster of up to eight
// CTAs each, with maxima, counts and sums exchanged through distributed shared memory.
//
// One row of 129280 bf16 with top-k 50 takes 16.6 us, nearly all of it a chain of
// barriers; 77 rows of 50257 with top-k 100 23 us; 512 rows of 129280 fp32 with top-p
// 180 us (1.5 TB/s): some 70 issue slots a logit over both passes take 58% of that,
// SMs without a row, in the second of 1.7 rounds of two rows each, 14%, and waiting
// for operands, loads, barriers and counts in shared memory the rest; HBM is at 29%.
#pragma once

#include <math.h>

#include <atomic>
#include <type_traits>

#include "flce_device.cuh"
#include "head_device.cuh"
#include "head_internal.h"
#include "model_internal.h"

namespace flce {

namespace {

constexpr int kMostWarps = 32;
constexpr int kMaxCluster = 8;
constexpr int kListKeys = 8192;
constexpr int kFew = 64;       // entries that are compared each with each
constexpr int kShort = 256;    // the same for a list of candidates
constexpr float kRange = 28.f;  // exp(-28) 2^40 < 1
constexpr float kFixed = 1099511627776.f;  // 2^40
constexpr float kLeast = 1.4e-45f;  // the smallest positive number

// General selection.
constexpr int kBins = 1024;
constexpr float kBinsPerUnit = (kBins - 1) / kRange;
// Counts of the first pass: 4096 bins from 8 above the anchor to 28 below it;
// the last one holds what is further below, whose weights are zero.
constexpr int kCountBins = 4096;
constexpr float kAbove = 8.f;
constexpr float kPlaces = kAbove + kRange;  // a place of 0 to 1 is this many units of t
constexpr float kUnitsPerBin = kPlaces / (kCountBins - 1);
// Logits above 4 below the anchor are weighed one by one for the estimate: a
// bin's middle is up to 0.4% off for one logit, which only matters where a few
// logits carry the row. (All of a normal row's logits would slow the pass:
// 4 below the maximum there are some per cent of them.)
constexpr int kWeighedBins = static_cast<int>((kAbove + 4.f) / kUnitsPerBin);
// How far around the estimated end logits are collected, of the whole weight:
// the first margin if the list holds what lies in it, else the second.
constexpr float kMargin = 0.0005f, kSmallMargin = 0.0001f;
// Segments of a slice whose weights are kept apart, at most.
constexpr int kSegments = 256;
constexpr int kFirstVectors = 4;  // per thread: the part of the row that sets the anchor
constexpr int kAnswerBins = 2048;   // segments of the vocabulary for a list of kept tokens
constexpr int kMostShared = 227 * 1024;
constexpr int kMostVocab = 1 << 22;

struct Hist {
  uint32_t count[kBins];
  uint32_t lo[kBins];  // 64-bit weights in halves: shared memory adds 32 bits at a time
  uint32_t hi[kBins];
};
struct Counts {
  uint32_t count[kCountBins];
  float weight[kWeighedBins];
};
struct Answer {
  uint32_t lo[kAnswerBins], hi[kAnswerBins];
};

// CUTS: no token is drawn; what the filters keep of each row goes to p.cuts.
template <bool CUTS>
using ParamsOf = std::conditional_t<CUTS, VerifyParams, SampleParams>;

// Shared memory of a CTA in front of its slice of the row; the same place in
// every CTA of the cluster.
struct Shared {
  uint64_t list[kListKeys];
  union {
    Hist hist[2];
    Counts counts;
    Answer answer;
  };
  uint64_t seg_weight[kSegments];
  uint32_t seg_ties[kMostWarps];
  uint64_t scan[kMostWarps + 1];
  uint64_t sum_total, sum_above;  // of this slice, in the second pass
  uint64_t found_above, found_value, goal;
  uint32_t found_bin, found_count;
  float tops[kMaxCluster];  // of all CTAs
  uint32_t bads[kMaxCluster];
  uint32_t first;      // lowest index of the largest logit in this slice
  uint32_t key_lo, key_hi;
  uint32_t listed[4];  // lengths of the lists of a row, one counter per use
  uint64_t few[kFew];
  uint32_t few_count;
  uint32_t result_key, result_count;
  unsigned long long cut_lo[2], cut_hi[2];  // first and last bin to collect; low words: logits before and up to them
  uint32_t general;         // CTA 0: the row needs the general selection
  uint32_t red[kMostWarps], red2[kMostWarps];
  float fscan[kMostWarps];
  float cut_x[2];
  uint32_t told[3];  // by CTA 0: where the prefix ends
};

__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 and +0 are the same logit
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
// Rank order of a list: falling logit, then rising index.
__device__ __forceinline__ uint64_t list_entry(float x, uint32_t index) {
  return static_cast<uint64_t>(~order_key(x)) << 32 | index;
}
__device__ __forceinline__ float entry_value(uint64_t e) { return key_value(~static_cast<uint32_t>(e >> 32)); }

// ---------------------------------------------------------------- the row's CTAs
// MULTI: the row is shared by a cluster; else by one CTA, and these are plain
// barriers and accesses.
// The cluster's barrier is not the aligned form: threads come here from code
// that only some of them run.
template <bool MULTI>
__device__ __forceinline__ void row_barrier() {
  if constexpr (MULTI)
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  else
    __syncthreads();
}

template <bool MULTI>
__device__ __forceinline__ uint32_t remote(const uint32_t* mine, uint32_t rank) {
  if constexpr (!MULTI) return *mine;
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(mine), rank)) : "memory");
  return v;
}
template <bool MULTI>
__device__ __forceinline__ float remote(const float* mine, uint32_t rank) {
  return __uint_as_float(remote<MULTI>(reinterpret_cast<const uint32_t*>(mine), rank));
}
template <bool MULTI>
__device__ __forceinline__ uint64_t remote(const uint64_t* mine, uint32_t rank) {
  if constexpr (!MULTI) return *mine;
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(mapa_shared(smem_u32(mine), rank)) : "memory");
  return v;
}

// Adds to a word of CTA `rank`.
__device__ __forceinline__ void remote_add(uint32_t* mine, uint32_t rank, uint32_t v) {
  asm volatile("red.shared::cluster.add.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(mine), rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void remote_add(float* mine, uint32_t rank, float v) {
  asm volatile("red.shared::cluster.add.f32 [%0], %1;" ::"r"(mapa_shared(smem_u32(mine), rank)), "f"(v) : "memory");
}

__device__ __forceinline__ void remote_store(uint32_t* mine, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(mine), rank)), "r"(v) : "memory");
}

// Appends to CTA 0's list; what does not fit is only counted. (One addition to
// the length for a warp's entries together, by votes or a scan, measured slower.)
template <bool MULTI>
__device__ __forceinline__ void append(Shared& s, uint32_t* listed, uint64_t entry) {
  if constexpr (!MULTI) {
    const uint32_t at = atomicAdd(listed, 1u);
    if (at < static_cast<uint32_t>(kListKeys)) s.list[at] = entry;
  } else {
    uint32_t at;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], 1;"
                 : "=r"(at)
                 : "r"(mapa_shared(smem_u32(listed), 0))
                 : "memory");
    if (at < static_cast<uint32_t>(kListKeys))
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa_shared(smem_u32(&s.list[at]), 0)), "l"(entry)
                   : "memory");
  }
}

// ---------------------------------------------------------------- sums in a CTA
__device__ __forceinline__ uint64_t warp_inclusive(uint64_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  return v;
}
__device__ __forceinline__ uint64_t warp_total(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Exclusive prefix sum over the CTA's threads; *total gets the whole. Begins
// with a barrier, so `scan` may be used again at once.
template <int kThreads>
__device__ uint64_t block_exclusive(uint64_t v, uint64_t* scan, uint64_t* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t inc = warp_inclusive(v);
  __syncthreads();
  if (lane == 31) scan[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const uint64_t w = lane < kThreads / 32 ? scan[lane] : 0;
    const uint64_t wi = warp_inclusive(w);
    __syncwarp();
    scan[lane] = wi - w;
    if (lane == 31) scan[kMostWarps] = wi;
  }
  __syncthreads();
  *total = scan[kMostWarps];
  return scan[warp] + inc - v;
}

// The same of a count and an estimated weight at once.
template <int kThreads>
__device__ __forceinline__ void block_exclusive(Shared& s, uint32_t n, float w, uint32_t* n_before, float* w_before,
                                                float* w_total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t ni = n;
  float wi = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, ni, o);
    const float b = __shfl_up_sync(0xffffffffu, wi, o);
    if (lane >= o) {
      ni += a;
      wi += b;
    }
  }
  __syncthreads();
  if (lane == 31) {
    s.red[warp] = ni;
    s.fscan[warp] = wi;
  }
  __syncthreads();
  // every warp adds up the warps before it, in one order
  uint32_t a = lane < kThreads / 32 ? s.red[lane] : 0;
  float b = lane < kThreads / 32 ? s.fscan[lane] : 0.f;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t c = __shfl_up_sync(0xffffffffu, a, o);
    const float d = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += c;
      b += d;
    }
  }
  *w_total = __shfl_sync(0xffffffffu, b, 31);
  const uint32_t pn = __shfl_sync(0xffffffffu, a, warp == 0 ? 0 : warp - 1);
  const float pw = __shfl_sync(0xffffffffu, b, warp == 0 ? 0 : warp - 1);
  *n_before = (warp == 0 ? 0u : pn) + ni - n;
  *w_before = (warp == 0 ? 0.f : pw) + wi - w;
}

// Adds a 64-bit weight to a bin, in halves with the carry.
__device__ __forceinline__ void add_weight(uint32_t* lo, uint32_t* hi, uint64_t w) {
  const uint32_t low = static_cast<uint32_t>(w);
  uint32_t high = static_cast<uint32_t>(w >> 32);
  const uint32_t old = atomicAdd(lo, low);
  if (old > ~low) ++high;
  if (high) atomicAdd(hi, high);
}

// The smallest whole number b with (double)b >= bound: what lies before a kept
// token is less than that.
__device__ __forceinline__ uint64_t reach(double bound) {
  if (!(bound > 0.0)) return 0;
  int64_t b = static_cast<int64_t>(ceil(bound));
  while (b > 1 && __ll2double_rn(b - 1) >= bound) --b;
  return static_cast<uint64_t>(b);
}
__device__ __forceinline__ uint64_t top_p_goal(float top_p, uint64_t whole) {
  return reach(__dmul_rn(static_cast<double>(top_p), __ll2double_rn(static_cast<int64_t>(whole))));
}
// u times the kept weight, below it.
__device__ __forceinline__ uint64_t answer_goal(float u, uint64_t whole) {
  const int64_t n = static_cast<int64_t>(whole);
  const int64_t g = static_cast<int64_t>(__dmul_rn(static_cast<double>(u), __ll2double_rn(n)));
  return static_cast<uint64_t>(g < 0 ? 0 : g < n ? g : n - 1);
}
// f() of one thread for all of the CTA: goals take double precision, which 1024
// threads would queue for.
template <typename F>
__device__ __forceinline__ uint64_t by_one(Shared& s, F f) {
  if (threadIdx.x == 0) s.goal = f();
  __syncthreads();
  return s.goal;
}

// floor(e 2^40) for e in [0, 1] as hi 2^20 + lo. Adding to 2^23 with rounding
// towards zero leaves the whole part in the mantissa; what it left is exact.
// (The 64-bit conversion instruction runs at the rate of double precision,
// which this chip has little of: with it the second pass took three times as long.)
struct Halves {
  uint32_t hi, lo;
};
__device__ __forceinline__ Halves halves(float e) {
  const float a = __fmaf_rz(e, 1048576.f, 8388608.f);
  const float rest = __fmaf_rn(e, 1048576.f, 8388608.f - a);
  const float b = __fmaf_rz(rest, 1048576.f, 8388608.f);
  return {__float_as_uint(a) - 0x4B000000u, __float_as_uint(b) - 0x4B000000u};
}

// Sums of weights of up to 4096 logits, in halves that do not overflow.
struct Sum {
  uint32_t hi = 0, lo = 0;
  __device__ __forceinline__ void add(Halves h) {
    hi += h.hi;
    lo += h.lo;
  }
  // over the warp's lanes
  __device__ __forceinline__ uint64_t total() const {
    const uint64_t h = __reduce_add_sync(0xffffffffu, hi & 0xFFFFu) +
                       (static_cast<uint64_t>(__reduce_add_sync(0xffffffffu, hi >> 16)) << 16);
    const uint64_t l = __reduce_add_sync(0xffffffffu, lo & 0xFFFFu) +
                       (static_cast<uint64_t>(__reduce_add_sync(0xffffffffu, lo >> 16)) << 16);
    return (h << 20) + l;
  }
};

// ---------------------------------------------------------------- a row
// The part of a row that a CTA works on, and the row's settings.
template <typename T, int kThreads>
struct Row {
  static constexpr int E = 16 / sizeof(T);
  const T* data;  // in shared memory (padded with -infinity to whole vectors) or in global memory
  bool padded;    // shared memory
  bool aligned;   // data is on a vector boundary
  int n, vecs;
  int c0;         // vocabulary index of the first logit
  float top, inv; // largest logit of the row, 1 / temperature
  float anchor, per_place;  // places: (anchor - x) per_place + kAbove / kPlaces, kept in [0, 1]
  float min_p;
  uint32_t rank, ctas;

  __device__ __forceinline__ Raw<T, E> get(int v) const {
    if (aligned && (padded || (v + 1) * E <= n)) return load_raw<T, E>(data + v * E);
    float x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = v * E + e < n ? to_float<T>(data[v * E + e]) : -INFINITY;
    return pack<T, E>(x);
  }
  __device__ __forceinline__ float scaled(float x) const { return __fmul_rn(x - top, inv); }
  __device__ __forceinline__ float exponential(float x) const { return expf(scaled(x)); }
  __device__ __forceinline__ static uint64_t fixed(float e) {
    const Halves h = halves(e);
    return (static_cast<uint64_t>(h.hi) << 20) + h.lo;
  }
  __device__ __forceinline__ uint64_t weight(float x) const { return fixed(exponential(x)); }
  // Bin of the general selection, and place among the counting bins.
  __device__ __forceinline__ int bin(float x) const {
    return min(kBins - 1, __float2int_rz(scaled(x) * -kBinsPerUnit));
  }
  // Counting bin: two multiply-adds, the second rounding towards zero into the
  // mantissa of 2^23. Falls as x rises.
  __device__ __forceinline__ int count_bin(float x) const {
    const float u = __saturatef(__fmaf_rn(__fsub_rn(anchor, x), per_place, kAbove / kPlaces));
    return static_cast<int>(__float_as_uint(__fmaf_rz(u, static_cast<float>(kCountBins - 1), 8388608.f)) - 0x4B000000u);
  }
  // The smallest logit in a counting bin before `cut`, infinity if there is none.
  // For a whole warp: each step tries 32 points of the range of keys that is left,
  // at first the neighbourhood of the inverse of count_bin, if it holds the answer.
  __device__ __forceinline__ float first_before(int cut) const {
    const uint32_t lane = threadIdx.x & 31;
    const float guess = anchor - (static_cast<float>(cut) * (1.f / (kCountBins - 1)) - kAbove / kPlaces) / per_place;
    const float off = 1e-6f * (fabsf(anchor) + fabsf(guess));
    uint32_t lo = order_key(-INFINITY), hi = order_key(INFINITY);  // hi: known to be before, or infinity
    const float below = guess - off, above = guess + off;
    if (fabsf(below) < INFINITY && count_bin(below) >= cut) lo = order_key(below);
    if (fabsf(above) < INFINITY && count_bin(above) < cut) hi = order_key(above);
    while (lo < hi) {
      const uint32_t step = (hi - lo + 31) / 32;
      const uint32_t k = lo + lane * step;
      const uint32_t yes = __ballot_sync(0xffffffffu, k >= hi || count_bin(key_value(k)) < cut);
      const uint32_t at = yes ? __ffs(yes) - 1 : 32;  // the first point that is before
      const uint32_t l = lo;
      if (at < 32) hi = min(hi, l + at * step);
      if (at > 0) lo = l + (at - 1) * step + 1;
    }
    return key_value(hi);
  }
  // Vectors per segment: whole rounds of a warp.
  __device__ __forceinline__ static int segment_vecs(int vecs) {
    return max(32, (vecs + 32 * kSegments - 1) / (32 * kSegments) * 32);
  }

  // f(x, index) for this thread's logits, four vectors' loads in flight.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (int v = threadIdx.x; v < vecs; v += 4 * kThreads) {
      Raw<T, E> raw[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (v + j * kThreads < vecs) raw[j] = get(v + j * kThreads);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (v + j * kThreads >= vecs) break;
        float x[E];
        unpack<T, E>(raw[j], x);
#pragma unroll
        for (int e = 0; e < E; ++e) f(x[e], static_cast<uint32_t>(c0 + (v + j * kThreads) * E + e));
      }
    }
  }
};

template <int kThreads>
__device__ void clear(Hist& h) {
  for (int i = threadIdx.x; i < kBins; i += kThreads) h.count[i] = h.lo[i] = h.hi[i] = 0;
  __syncthreads();
}

__device__ __forceinline__ float reciprocal(uint64_t whole) {
  return __double2float_rn(__drcp_rn(__ll2double_rn(static_cast<int64_t>(whole))));
}

// The row's kept set (CUTS), by one thread: all logits up to `last` in rank order, of at
// least min_p.
template <typename T, int kThreads>
__device__ __forceinline__ void write_cut(const Row<T, kThreads>& row, const VerifyParams& p, int64_t r, uint64_t last, uint64_t whole) {
  p.cuts[r] = {last, whole, row.top, row.inv, row.min_p, reciprocal(whole)};
}

template <typename T, int kThreads>
__device__ __forceinline__ void write_answer(const Row<T, kThreads>& row, const SampleParams& p, int64_t r, uint32_t index, float x,
                                             uint64_t whole) {
  p.tokens[r] = index;
  if (p.logprobs) p.logprobs[r] = row.scaled(x) - logf(__ll2float_rn(static_cast<int64_t>(whole)) * (1.f / kFixed));
}

// Over the CTA, in every thread.
template <int kThreads>
__device__ __forceinline__ uint64_t block_total(Shared& s, uint64_t v) {
  v = warp_total(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.scan[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_total((threadIdx.x & 31) < kThreads / 32 ? s.scan[threadIdx.x & 31] : 0);
}

// The entry of the CTA's list of n at which the running sum in rank order,
// `start` before the first, reaches the goal (start < goal); ~0 if it does not.
// All entries lie in [lo, hi]. WEIGHT: sums of weights, else counts. A histogram
// over the range of entries (they are whole numbers in rank order, all
// different), again over the bin that holds the goal, until that has at most
// kFew. Uses the first histogram.
template <typename T, int kThreads, bool WEIGHT>
__device__ uint64_t list_reach(const Row<T, kThreads>& row, Shared& s, int n, uint64_t lo, uint64_t hi, uint64_t start,
                               uint64_t goal) {
  Hist& h = s.hist[0];
  __syncthreads();  // the list is complete, the histogram's place free
  while (true) {
    const int bits = 64 - __clzll(static_cast<long long>(hi - lo));
    const int shift = bits > 10 ? bits - 10 : 0;
    static_assert(kBins == 1 << 10, "a range of 10 + shift bits");
    clear<kThreads>(h);
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const uint64_t e = s.list[i];
      if (e >= lo && e <= hi) {
        const int b = static_cast<int>((e - lo) >> shift);
        atomicAdd(&h.count[b], 1u);
        if (WEIGHT) add_weight(&h.lo[b], &h.hi[b], row.weight(entry_value(e)));
      }
    }
    __syncthreads();
    constexpr int B = kBins / kThreads;  // bins of a thread
    uint64_t v[B], sum = 0, total;
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const int b = B * threadIdx.x + j;
      v[j] = WEIGHT ? h.lo[b] + (static_cast<uint64_t>(h.hi[b]) << 32) : h.count[b];
      sum += v[j];
    }
    uint64_t before = start + block_exclusive<kThreads>(sum, s.scan, &total);
    if (start + total < goal) return ~0ull;
#pragma unroll
    for (int j = 0; j < B; ++j) {
      if (before < goal && goal <= before + v[j]) {
        s.found_bin = B * threadIdx.x + j;
        s.found_above = before;
        s.found_count = h.count[B * threadIdx.x + j];
        s.few_count = 0;
      }
      before += v[j];
    }
    __syncthreads();
    start = s.found_above;
    lo += static_cast<uint64_t>(s.found_bin) << shift;
    hi = min(hi, lo + ((uint64_t{1} << shift) - 1));
    if (s.found_count <= static_cast<uint32_t>(kFew)) break;
    __syncthreads();
  }
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t e = s.list[i];
    if (e >= lo && e <= hi) s.few[atomicAdd(&s.few_count, 1u)] = e;
  }
  __syncthreads();
  const int few = static_cast<int>(s.found_count);
  if (threadIdx.x < few) {
    const uint64_t e = s.few[threadIdx.x];
    uint64_t before = start;
    for (int i = 0; i < few; ++i)
      if (s.few[i] < e) before += WEIGHT ? row.weight(entry_value(s.few[i])) : 1;
    if (before < goal && goal <= before + (WEIGHT ? row.weight(entry_value(e)) : 1)) s.found_value = e;
  }
  __syncthreads();
  return s.found_value;
}

// ---------------------------------------------------------------- general selection
// Sums the row's histograms. want(total) gives the goal; the
// bin whose running sum first reaches it goes to found_* (found_bin = kBins if
// none does). WEIGHT: sums of weights, else counts.
template <int kThreads, bool MULTI, bool WEIGHT, typename F>
__device__ uint64_t find_bin(Shared& s, const Hist& h, uint32_t ctas, F want, uint64_t* total) {
  constexpr int B = kBins / kThreads;  // bins of a thread
  uint64_t v[B], sum = 0;
  uint32_t n[B];
#pragma unroll
  for (int j = 0; j < B; ++j) {
    const int b = B * threadIdx.x + j;
    v[j] = n[j] = 0;
    for (uint32_t r = 0; r < ctas; ++r) {
      n[j] += remote<MULTI>(&h.count[b], r);
      if (WEIGHT) v[j] += remote<MULTI>(&h.lo[b], r) + (static_cast<uint64_t>(remote<MULTI>(&h.hi[b], r)) << 32);
    }
    if (!WEIGHT) v[j] = n[j];
    sum += v[j];
  }
  if (threadIdx.x == 0) s.found_bin = kBins;
  uint64_t before = block_exclusive<kThreads>(sum, s.scan, total);
  const uint64_t goal = by_one(s, [&] { return want(*total); });
#pragma unroll
  for (int j = 0; j < B; ++j) {
    if (before < goal && goal <= before + v[j]) {
      s.found_bin = B * threadIdx.x + j;
      s.found_above = before;
      s.found_count = n[j];
    }
    before += v[j];
  }
  __syncthreads();
  return goal;
}

// Finds the logit (as a key) and the number of logits equal to it at which the
// running sum over the ranked logits above `limit` (a key) first reaches the
// goal, which want(total) gives. Returns false if the sum never does: nothing is
// cut off. *total_out and *goal_out: the whole sum and the goal.
template <typename T, int kThreads, bool MULTI, bool WEIGHT, typename F>
__device__ bool select(const Row<T, kThreads>& row, Shared& s, int& buf, uint32_t* listed, uint32_t limit, F want,
                       uint32_t* key_out, uint32_t* count_out, uint64_t* total_out, uint64_t* goal_out) {
  Hist* h = &s.hist[buf];
  buf ^= 1;
  clear<kThreads>(*h);
  row.each([&](float x, uint32_t) {
    const int b = row.bin(x);
    if (b < kBins - 1 && order_key(x) > limit) {  // the last bin's weights are zero
      atomicAdd(&h->count[b], 1u);
      if (WEIGHT) add_weight(&h->lo[b], &h->hi[b], row.weight(x));
    }
  });
  row_barrier<MULTI>();
  uint64_t goal = 0;
  uint64_t total = 0;
  goal = find_bin<kThreads, MULTI, WEIGHT>(s, *h, row.ctas, want, &total);
  *total_out = total;
  *goal_out = goal;
  if (s.found_bin == kBins) return false;
  const int bin = static_cast<int>(s.found_bin);
  uint64_t above = s.found_above;
  uint32_t count = s.found_count, key_lo = 0, key_hi = 0xFFFFFFFFu;
  bool by_key = false;
  auto inside = [&](float x) {
    const uint32_t k = order_key(x);
    return by_key ? k >= key_lo && k <= key_hi : k > limit && row.bin(x) == bin;
  };
  while (count > static_cast<uint32_t>(kListKeys)) {
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
    row.each([&](float x, uint32_t) {
      if (inside(x)) {
        lo = min(lo, order_key(x));
        hi = max(hi, order_key(x));
      }
    });
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
      s.red[threadIdx.x >> 5] = lo;
      s.red2[threadIdx.x >> 5] = hi;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kThreads / 32; ++w) {
        lo = min(lo, s.red[w]);
        hi = max(hi, s.red2[w]);
      }
      s.key_lo = lo;
      s.key_hi = hi;
    }
    row_barrier<MULTI>();
    key_lo = 0xFFFFFFFFu;
    key_hi = 0;
    for (uint32_t r = 0; r < row.ctas; ++r) {
      key_lo = min(key_lo, remote<MULTI>(&s.key_lo, r));
      key_hi = max(key_hi, remote<MULTI>(&s.key_hi, r));
    }
    by_key = true;
    if (key_lo == key_hi) {
      const uint64_t w = WEIGHT ? row.weight(key_value(key_lo)) : 1;
      *key_out = key_lo;
      *count_out = static_cast<uint32_t>((goal - above + w - 1) / w);
      return true;
    }
    // bins by the distance from the highest key
    int shift = 0;
    while (((key_hi - key_lo) >> shift) >= static_cast<uint32_t>(kBins)) ++shift;
    h = &s.hist[buf];
    buf ^= 1;
    clear<kThreads>(*h);
    row.each([&](float x, uint32_t) {
      const uint32_t k = order_key(x);
      if (k >= key_lo && k <= key_hi) {
        const int b = static_cast<int>((key_hi - k) >> shift);
        atomicAdd(&h->count[b], 1u);
        if (WEIGHT) add_weight(&h->lo[b], &h->hi[b], row.weight(x));
      }
    });
    row_barrier<MULTI>();
    uint64_t inside_total;
    find_bin<kThreads, MULTI, WEIGHT>(s, *h, row.ctas, [&](uint64_t) { return goal - above; }, &inside_total);
    const uint32_t b = s.found_bin;
    above += s.found_above;
    count = s.found_count;
    const uint32_t top = key_hi - (b << shift);
    const uint32_t width = (1u << shift) - 1;
    key_lo = top - key_lo > width ? top - width : key_lo;
    key_hi = top;
  }
  // few enough: CTA 0 looks through them
  row.each([&](float x, uint32_t i) {
    if (inside(x)) append<MULTI>(s, listed, list_entry(x, i));
  });
  row_barrier<MULTI>();
  if (row.rank == 0) {
    const uint64_t e = list_reach<T, kThreads, WEIGHT>(row, s, static_cast<int>(count), list_entry(row.top, 0), list_entry(-INFINITY, ~0u),
                                             above, goal);
    uint32_t ties = 0;  // of the same logit, up to that entry
    for (int i = threadIdx.x; i < static_cast<int>(count); i += kThreads)
      ties += s.list[i] >> 32 == e >> 32 && s.list[i] <= e;
    ties = __reduce_add_sync(0xffffffffu, ties);
    if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = ties;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kThreads / 32; ++w) ties += s.red[w];
      s.result_key = ~static_cast<uint32_t>(e >> 32);
      s.result_count = ties;
    }
  }
  row_barrier<MULTI>();
  *key_out = remote<MULTI>(&s.result_key, 0);
  *count_out = remote<MULTI>(&s.result_count, 0);
  return true;
}

// The token by the general selection.
template <typename T, int kThreads, bool MULTI, bool CUTS>
__device__ void general_answer(const Row<T, kThreads>& row, Shared& s, const ParamsOf<CUTS>& p, int64_t r, int64_t top_k,
                               float top_p, float u) {
  constexpr int E = Row<T, kThreads>::E, kWarps = kThreads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int buf = 0;
  // the kept set: logits above `key`, and the first `ties` of those equal to it
  uint32_t key = 0, ties = 0;
  uint64_t over, goal_p;
  if (top_k > 0 && top_k < p.vocab)
    if (!select<T, kThreads, MULTI, false>(row, s, buf, &s.listed[1], 0u, [&](uint64_t) { return static_cast<uint64_t>(top_k); },
                                 &key, &ties, &over, &goal_p))
      key = ties = 0;
  if (top_p < 1.f) {
    const uint64_t w = ties ? row.weight(key_value(key)) : 0;
    uint32_t k2, t2;
    const bool cut = select<T, kThreads, MULTI, true>(
        row, s, buf, &s.listed[2], key, [&](uint64_t total) { return top_p_goal(top_p, total + ties * w); }, &k2, &t2,
        &over, &goal_p);
    if (cut) {
      key = k2;
      ties = t2;
    } else if (ties) {
      const uint64_t need = (goal_p - over + w - 1) / (w ? w : 1);
      ties = need < ties ? static_cast<uint32_t>(need) : ties;
    }
  }

  // running sums in index order: a warp per segment of the slice
  const float e_tie = ties ? row.exponential(key_value(key)) : 0.f;
  const uint64_t w_tie = e_tie >= row.min_p ? Row<T, kThreads>::fixed(e_tie) : 0;
  const int seg = (row.vecs + kWarps - 1) / kWarps;
  const int v0 = warp * seg, v1 = min(v0 + seg, row.vecs);
  auto kept_weight = [&](float f) -> uint64_t {
    if (order_key(f) <= key) return 0;
    const float e = row.exponential(f);
    return e >= row.min_p ? Row<T, kThreads>::fixed(e) : 0;
  };
  uint64_t sum = 0;
  uint32_t equal = 0;
  for (int v = v0 + lane; v < v1; v += 32) {
    float f[E];
    unpack<T, E>(row.get(v), f);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      sum += kept_weight(f[e]);
      if (ties) equal += order_key(f[e]) == key;
    }
  }
  sum = warp_total(sum);
  equal = __reduce_add_sync(0xffffffffu, equal);
  __syncthreads();
  if (lane == 0) {
    s.seg_weight[warp] = sum;
    s.seg_ties[warp] = equal;
  }
  row_barrier<MULTI>();
  // every warp finds the segment of the answer; it goes on if that is its own
  const int segs = static_cast<int>(row.ctas) * kWarps;
  uint64_t total = 0, my_before = 0, my_weight = 0;
  uint32_t tie_total = 0, my_tie_before = 0;
  const int mine = static_cast<int>(row.rank) * kWarps + warp;
  for (int base = 0; base < segs; base += 32) {
    const int i = base + lane;
    uint64_t w = i < segs ? remote<MULTI>(&s.seg_weight[i % kWarps], i / kWarps) : 0;
    const uint32_t t = i < segs ? remote<MULTI>(&s.seg_ties[i % kWarps], i / kWarps) : 0;
    const uint32_t t_inc = static_cast<uint32_t>(warp_inclusive(t));
    const uint32_t t_before = tie_total + t_inc - t;
    const uint32_t t_kept = t_before < ties ? min(t, ties - t_before) : 0;
    w += t_kept * w_tie;
    const uint64_t w_inc = warp_inclusive(w);
    const int src = mine - base;
    if (src >= 0 && src < 32) {
      my_before = total + __shfl_sync(0xffffffffu, w_inc - w, src);
      my_weight = __shfl_sync(0xffffffffu, w, src);
      my_tie_before = __shfl_sync(0xffffffffu, t_before, src);
    }
    total += __shfl_sync(0xffffffffu, w_inc, 31);
    tie_total += __shfl_sync(0xffffffffu, t_inc, 31);
  }
  if constexpr (CUTS) {
    // (a member that only the warp with the last tie writes, if there are ties)
    if (row.rank == 0 && threadIdx.x == 0) {
      RowCut& cut = p.cuts[r];
      cut.whole = total;
      cut.top = row.top;
      cut.inv = row.inv;
      cut.min_p = row.min_p;
      cut.over = reciprocal(total);
      if (ties == 0) cut.last = key == 0 ? ~0ull : (static_cast<uint64_t>(~key) << 32) - 1;
    }
    if (ties > 0 && my_tie_before < ties && ties <= my_tie_before + equal) {
      uint32_t tie_before = my_tie_before;
      for (int b = v0; b < v1; b += 32) {
        const int v = b + lane;
        float f[E];
        uint32_t eq = 0;
        if (v < v1) {
          unpack<T, E>(row.get(v), f);
#pragma unroll
          for (int e = 0; e < E; ++e) eq += order_key(f[e]) == key;
        }
        const uint32_t eq_inc = static_cast<uint32_t>(warp_inclusive(eq));
        uint32_t tb = tie_before + eq_inc - eq;
        if (v < v1) {
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (order_key(f[e]) == key && ++tb == ties) p.cuts[r].last = list_entry(f[e], static_cast<uint32_t>(row.c0 + v * E + e));
        }
        tie_before += __shfl_sync(0xffffffffu, eq_inc, 31);
      }
    }
    row_barrier<MULTI>();  // the segments' sums have been read by all
    return;
  }
  const uint64_t goal = by_one(s, [&] { return answer_goal(u, total); });
  if (my_before <= goal && goal < my_before + my_weight) {
    uint64_t before = my_before;
    uint32_t tie_before = my_tie_before;
    for (int b = v0; b < v1; b += 32) {
      const int v = b + lane;
      float f[E];
      uint32_t eq = 0;
      uint64_t w = 0;
      if (v < v1) {
        unpack<T, E>(row.get(v), f);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          w += kept_weight(f[e]);
          if (ties) eq += order_key(f[e]) == key;
        }
      }
      const uint32_t eq_inc = static_cast<uint32_t>(warp_inclusive(eq));
      uint32_t tb = tie_before + eq_inc - eq;
      w += (tb < ties ? min(eq, ties - tb) : 0) * w_tie;
      const uint64_t inc = warp_inclusive(w);
      uint64_t mb = before + inc - w;
      if (v < v1 && mb <= goal && goal < mb + w) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          uint64_t we = kept_weight(f[e]);
          if (ties && order_key(f[e]) == key) we = tb++ < ties ? w_tie : 0;
          if (mb <= goal && goal < mb + we) {
            write_answer(row, p, r, static_cast<uint32_t>(row.c0 + v * E + e), f[e], total);
          }
          mb += we;
        }
      }
      before += __shfl_sync(0xffffffffu, inc, 31);
      tie_before += __shfl_sync(0xffffffffu, eq_inc, 31);
    }
  }
  row_barrier<MULTI>();  // the segments' sums have been read by all
}

// ---------------------------------------------------------------- answers from a list
// The token from a list of n <= kShort candidates, at least the first top_k by
// rank. An entry's rank and what lies before it come from comparing it with all
// the others, in rank order and again in index order: few barriers, no sort.
template <typename T, int kThreads, bool CUTS>
__device__ void short_list_answer(const Row<T, kThreads>& row, Shared& s, const ParamsOf<CUTS>& p, int64_t r, int n, int64_t top_k,
                                  float top_p, float u) {
  uint64_t* weights = reinterpret_cast<uint64_t*>(&s.hist[0]);
  static_assert(sizeof(s.hist) >= kShort * sizeof(uint64_t), "weights in the histograms' place");
  constexpr int P = kThreads / kShort;  // lanes that share an entry's comparisons
  const int i = threadIdx.x / P, part = threadIdx.x % P;
  uint64_t mine = ~0ull, w = 0, before = 0;
  float e = 0.f;
  int rank = 0;
  // over an entry's lanes
  auto joined = [](uint64_t v) {
#pragma unroll
    for (int o = 1; o < P; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  __syncthreads();
  if (i < n) {
    mine = s.list[i];
    e = row.exponential(entry_value(mine));
    w = Row<T, kThreads>::fixed(e);
    if (part == 0) weights[i] = w;
  }
  __syncthreads();
  if (i < n) {
#pragma unroll 4
    for (int k = part; k < n; k += P) {
      const bool first = s.list[k] < mine;
      rank += first;
      before += first ? weights[k] : 0;
    }
  }
  rank = static_cast<int>(joined(static_cast<uint64_t>(rank)));
  before = joined(before);
  bool keep = i < n && (top_k <= 0 || rank < top_k);
  if (top_p < 1.f) {
    const uint64_t whole = block_total<kThreads>(s, keep && part == 0 ? w : 0);
    const uint64_t far = by_one(s, [&] { return top_p_goal(top_p, whole); });
    keep = keep && (rank == 0 || before < far);
  }
  keep = keep && (rank == 0 || e >= row.min_p);
  if (CUTS && threadIdx.x == 0) s.found_value = 0;  // (block_total's barriers on either side)
  const uint64_t whole = block_total<kThreads>(s, keep && part == 0 ? w : 0);
  if constexpr (CUTS) {
    if (keep && part == 0) atomicMax(reinterpret_cast<unsigned long long*>(&s.found_value), static_cast<unsigned long long>(mine));
    __syncthreads();
    if (threadIdx.x == 0) write_cut(row, p, r, s.found_value, whole);
    return;
  }
  if (i < n && part == 0) weights[i] = keep ? w : 0;
  const uint64_t goal = by_one(s, [&] { return answer_goal(u, whole); });
  const uint32_t index = static_cast<uint32_t>(mine);
  before = 0;
  if (keep) {
#pragma unroll 4
    for (int k = part; k < n; k += P) before += static_cast<uint32_t>(s.list[k]) < index ? weights[k] : 0;
  }
  before = joined(before);
  if (keep && part == 0 && before <= goal && goal < before + w) write_answer(row, p, r, index, entry_value(mine), whole);
}

// The segment that holds the answer, of those in s.answer: to found_bin, and what
// lies before it to found_above. Returns the goal.
template <int kThreads>
__device__ uint64_t answer_bin(Shared& s, float u, uint64_t* whole) {
  constexpr int A = kAnswerBins / kThreads;
  const Answer& a = s.answer;
  uint64_t w[A], sum = 0;
#pragma unroll
  for (int j = 0; j < A; ++j) {
    const int b = A * threadIdx.x + j;
    w[j] = a.lo[b] + (static_cast<uint64_t>(a.hi[b]) << 32);
    sum += w[j];
  }
  uint64_t before = block_exclusive<kThreads>(sum, s.scan, whole);
  const uint64_t total = *whole, goal = by_one(s, [&] { return answer_goal(u, total); });
#pragma unroll
  for (int j = 0; j < A; ++j) {
    if (before <= goal && goal < before + w[j]) {
      s.found_bin = A * threadIdx.x + j;
      s.found_above = before;
    }
    before += w[j];
  }
  __syncthreads();
  return goal;
}

// The same for a long list.
template <typename T, int kThreads, bool CUTS>
__device__ void list_answer(const Row<T, kThreads>& row, Shared& s, const ParamsOf<CUTS>& p, int64_t r, int n, int64_t top_k,
                            float top_p, float u, float x_hi) {
  const uint64_t lo = list_entry(row.top, 0), hi = list_entry(x_hi, ~0u);
  uint64_t last = ~0ull;  // last entry that the filters by rank keep
  if (top_k > 0 && n > top_k) last = list_reach<T, kThreads, false>(row, s, n, lo, hi, 0, static_cast<uint64_t>(top_k));
  if (top_p < 1.f) {
    uint64_t sum = 0;
    for (int i = threadIdx.x; i < n; i += kThreads)
      if (s.list[i] <= last) sum += row.weight(entry_value(s.list[i]));
    const uint64_t whole = block_total<kThreads>(s, sum);
    const uint64_t goal = by_one(s, [&] { return top_p_goal(top_p, whole); });
    last = min(last, list_reach<T, kThreads, true>(row, s, n, lo, hi, 0, goal));
  }
  // kept weights by segments of the vocabulary, A of them per thread
  Answer& a = s.answer;
  constexpr int A = kAnswerBins / kThreads;
  static_assert(kMostVocab / kAnswerBins * sizeof(uint32_t) + sizeof(Answer) <= sizeof(s.hist),
                "segments, and the places of the tokens in one");
  const uint32_t width = static_cast<uint32_t>((p.vocab + kAnswerBins - 1) / kAnswerBins);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < A; ++j) a.lo[A * threadIdx.x + j] = a.hi[A * threadIdx.x + j] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t entry = s.list[i];
    const float e = row.exponential(entry_value(entry));
    if (entry <= last && e >= row.min_p) {
      const uint32_t b = static_cast<uint32_t>(entry) / width;
      add_weight(&a.lo[b], &a.hi[b], Row<T, kThreads>::fixed(e));
    }
  }
  __syncthreads();
  uint64_t whole;
  const uint64_t goal = answer_bin<kThreads>(s, u, &whole);
  if constexpr (CUTS) {
    // (a list that is kept whole: nothing beside it is)
    if (threadIdx.x == 0) write_cut(row, p, r, min(last, hi), whole);
    return;
  }
  // the tokens of that segment (at most `width`): each one's running sum is that of those before it
  uint32_t* place = reinterpret_cast<uint32_t*>(&a + 1);
  const uint32_t bin = s.found_bin;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t entry = s.list[i];
    if (entry <= last && static_cast<uint32_t>(entry) / width == bin && row.exponential(entry_value(entry)) >= row.min_p)
      place[atomicAdd(&s.listed[3], 1u)] = i;
  }
  __syncthreads();
  const int here = static_cast<int>(s.listed[3]);
  for (int i = threadIdx.x; i < here; i += kThreads) {
    const uint64_t mine = s.list[place[i]];
    const uint32_t index = static_cast<uint32_t>(mine);
    uint64_t b = s.found_above;
    for (int k = 0; k < here; ++k) {
      const uint64_t other = s.list[place[k]];
      if (static_cast<uint32_t>(other) < index) b += row.weight(entry_value(other));
    }
    if (b <= goal && goal < b + row.weight(entry_value(mine)))
      write_answer(row, p, r, index, entry_value(mine), whole);
  }
}

// ---------------------------------------------------------------- second pass
// One vector's logits: their weights to `all` and, from x_lo on (and at least
// min_p), to `acc`; logits from x_hi to x_lo to CTA 0's list. Without CUT every
// logit counts as above. MIN_P: the row has that filter, and `above` gets what
// is above without it.
template <typename T, int kThreads, bool MULTI, bool CUT, bool MIN_P>
__device__ __forceinline__ void sum_vector(const Row<T, kThreads>& row, Shared& s, const Raw<T, Row<T, kThreads>::E>& raw, int v, float x_lo,
                                           float x_hi, Sum& acc, Sum& all, Sum& above) {
  constexpr int E = Row<T, kThreads>::E;
  float x[E];
  unpack<T, E>(raw, x);
  bool some = false;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float ex = row.exponential(x[e]);
    const Halves w = halves(ex), none = {0u, 0u};
    const bool enough = !MIN_P || ex >= row.min_p;
    if (CUT) {
      const bool over = x[e] >= x_lo;
      all.add(w);
      if (MIN_P) above.add(over ? w : none);
      acc.add(over && enough ? w : none);
      some |= !over && x[e] >= x_hi;
    } else {
      acc.add(enough ? w : none);
    }
  }
  // (asked once for a vector: a branch at each logit cost a third of the pass)
  if (CUT && some) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (x[e] >= x_hi && !(x[e] >= x_lo))
        append<MULTI>(s, &s.listed[0], list_entry(x[e], static_cast<uint32_t>(row.c0 + v * E + e)));
  }
}

// Adds up this slice's weights: sum_total all of them, sum_above those from x_lo
// on, seg_weight[] the latter (at least min_p) by segments. The warps take the
// segments in turn, each a few rounds of 32 vectors; four vectors' loads per lane
// are in flight.
template <typename T, int kThreads, bool MULTI, bool CUT, bool MIN_P>
__device__ void sum_segments(const Row<T, kThreads>& row, Shared& s, float x_lo, float x_hi) {
  constexpr int E = Row<T, kThreads>::E, kWarps = kThreads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = Row<T, kThreads>::segment_vecs(row.vecs);  // vectors per segment
  const int segs = (row.vecs + per - 1) / per;
  for (int i = threadIdx.x; i < kSegments; i += kThreads)
    if (i >= segs) s.seg_weight[i] = 0;
  Sum all, above;
  uint64_t total = 0, over = 0;
  for (int seg = warp; seg < segs; seg += kWarps) {
    Sum acc;
    const int v0 = seg * per, v1 = min(v0 + per, row.vecs);
    int base = v0;
    if (row.aligned) {
      const T* q = row.data + (v0 + lane) * E;
      for (; base + 128 <= v1 && (row.padded || (base + 128) * E <= row.n); base += 128, q += 128 * E) {
        Raw<T, E> raw[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) raw[j] = load_raw<T, E>(q + j * 32 * E);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          sum_vector<T, kThreads, MULTI, CUT, MIN_P>(row, s, raw[j], base + j * 32 + lane, x_lo, x_hi, acc, all, above);
      }
    }
#pragma unroll 2
    for (int v = base + lane; v < v1; v += 32)
      sum_vector<T, kThreads, MULTI, CUT, MIN_P>(row, s, row.get(v), v, x_lo, x_hi, acc, all, above);
    const uint64_t w = acc.total();
    if (lane == 0) s.seg_weight[seg] = w;
    if (!MIN_P) over += w;
    if (CUT && (per >= 1024 || seg + kWarps >= segs)) {  // a long row's sums would overflow their halves
      total += all.total();
      if (MIN_P) over += above.total();
      all = above = Sum();
    }
  }
  if (CUT) {
    if (lane == 0) {
      atomicAdd(reinterpret_cast<unsigned long long*>(&s.sum_total), static_cast<unsigned long long>(total));
      atomicAdd(reinterpret_cast<unsigned long long*>(&s.sum_above), static_cast<unsigned long long>(over));
    }
  }
}

// The answer from the second pass's sums, by CTA 0: joins the kept part of the
// list (n entries) with the segments and walks the segment of the answer.
// Returns false if the exact sums do not confirm that the prefix ends in the list.
template <typename T, int kThreads, bool MULTI, bool CUTS>
__device__ bool segment_answer(const Row<T, kThreads>& row, Shared& s, const ParamsOf<CUTS>& p, int64_t r, int slice, float top_p,
                               float u, bool cut, float x_lo, float x_hi) {
  constexpr int E = Row<T, kThreads>::E;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int vocab = static_cast<int>(p.vocab);
  uint64_t cut_entry = ~0ull;  // last kept entry of the list
  int n = 0;
  if (cut) {
    uint64_t total = 0, above = 0;
    for (uint32_t c = 0; c < row.ctas; ++c) {
      total += remote<MULTI>(&s.sum_total, c);
      above += remote<MULTI>(&s.sum_above, c);
    }
    n = static_cast<int>(min(s.listed[0], static_cast<uint32_t>(kListKeys)));
    const uint64_t goal = by_one(s, [&] { return top_p_goal(top_p, total); });
    if (s.listed[0] > static_cast<uint32_t>(kListKeys) || above >= goal) return false;
    // entries of the list lie from x_hi to below x_lo
    cut_entry = list_reach<T, kThreads, true>(row, s, n, static_cast<uint64_t>(~(order_key(x_lo) - 1u)) << 32,
                                    static_cast<uint64_t>(~order_key(x_hi)) << 32 | 0xFFFFFFFFu, above, goal);
    if (cut_entry == ~0ull) return false;
    __syncthreads();  // the histogram's place is used again
  }
  // the segments of all slices
  Answer& a = s.answer;
  constexpr int A = kAnswerBins / kThreads;
  static_assert(kAnswerBins == kMaxCluster * kSegments, "a bin per segment of the largest cluster");
#pragma unroll
  for (int j = 0; j < A; ++j) {
    const int b = A * threadIdx.x + j;
    const uint64_t w = b < static_cast<int>(row.ctas) * kSegments ? remote<MULTI>(&s.seg_weight[b % kSegments], b / kSegments) : 0;
    a.lo[b] = static_cast<uint32_t>(w);
    a.hi[b] = static_cast<uint32_t>(w >> 32);
  }
  __syncthreads();
  if (cut) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
      if (s.list[i] > cut_entry) continue;
      const float e = row.exponential(entry_value(s.list[i]));
      if (e >= row.min_p) {
        const int index = static_cast<int>(static_cast<uint32_t>(s.list[i]));
        const int c = index / slice;
        const int vecs = (min(slice, vocab - c * slice) + E - 1) / E;
        const int b = c * kSegments + (index - c * slice) / E / Row<T, kThreads>::segment_vecs(vecs);
        add_weight(&a.lo[b], &a.hi[b], Row<T, kThreads>::fixed(e));
      }
    }
    __syncthreads();
  }
  uint64_t whole;
  const uint64_t goal = answer_bin<kThreads>(s, u, &whole);
  if constexpr (CUTS) {
    if (threadIdx.x == 0) write_cut(row, p, r, cut_entry, whole);
    return true;
  }
  if (warp != 0) return true;
  // one warp walks the segment, from global memory if it is another CTA's
  const int c = static_cast<int>(s.found_bin) / kSegments, seg = static_cast<int>(s.found_bin) % kSegments;
  Row<T, kThreads> part = row;
  if (c != static_cast<int>(row.rank)) {
    part.data = static_cast<const T*>(p.x) + r * p.ld + static_cast<int64_t>(c) * slice;
    part.padded = false;
    part.aligned = reinterpret_cast<uintptr_t>(part.data) % 16 == 0;
    part.c0 = c * slice;
    part.n = min(slice, vocab - part.c0);
    part.vecs = (part.n + E - 1) / E;
  }
  const int sub = Row<T, kThreads>::segment_vecs(part.vecs);
  const int v1 = min((seg + 1) * sub, part.vecs);
  uint64_t run = s.found_above;
  Raw<T, E> ahead[4];
  for (int base = seg * sub, k = 0; base < v1; base += 32, ++k) {
    const int v = base + lane;
    if ((k & 3) == 0) {  // four rounds' loads at once
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (v + 32 * j < v1) ahead[j] = part.get(v + 32 * j);
    }
    float x[E];
    uint64_t w[E], sum = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = 0;
    if (v < v1) {
      unpack<T, E>((k & 3) == 0 ? ahead[0] : (k & 3) == 1 ? ahead[1] : (k & 3) == 2 ? ahead[2] : ahead[3], x);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float ex = part.exponential(x[e]);
        bool keep = ex >= part.min_p;
        if (cut)
          keep = keep && x[e] >= x_hi &&
                 (x[e] >= x_lo || list_entry(x[e], static_cast<uint32_t>(part.c0 + v * E + e)) <= cut_entry);
        w[e] = keep ? Row<T, kThreads>::fixed(ex) : 0;
        sum += w[e];
      }
    }
    const uint64_t inc = warp_inclusive(sum);
    uint64_t b = run + inc - sum;
    if (b <= goal && goal < b + sum) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (b <= goal && goal < b + w[e]) {
          write_answer(part, p, r, static_cast<uint32_t>(part.c0 + v * E + e), x[e], whole);
        }
        b += w[e];
      }
    }
    run += __shfl_sync(0xffffffffu, inc, 31);
  }
  return true;
}

// Verification: row r's first logit, its request, whose settings it has, and its place; rows of the
// target come first, then those of the draft. False if it lies behind the request's last draft. Called by whole
// warps, which look at 32 drafts at a time.
template <typename T>
__device__ __forceinline__ bool verify_row(const VerifyParams& p, uint32_t r, const T** start, int64_t* request, int* at_place) {
  const uint32_t target_rows = static_cast<uint32_t>(p.target_rows);
  const bool target = r < target_rows;
  const uint32_t at = target ? r : r - target_rows, per = static_cast<uint32_t>(p.drafts) + (target ? 1 : 0);
  const int place = static_cast<int>(at % per);
  *request = at / per;
  *at_place = place;
  *start = target ? static_cast<const T*>(p.x) + *request * p.batch_ld + place * p.ld
                  : static_cast<const T*>(p.draft) + *request * p.draft_batch_ld + place * p.draft_ld;
  bool none = false;
  const int64_t* tokens = p.draft_tokens + *request * p.drafts;
  for (int i = static_cast<int>(threadIdx.x) & 31; i < place + (target ? 0 : 1); i += 32) {
    const int64_t token = __ldg(tokens + i);
    none = none || token < 0 || token >= p.vocab;
  }
  return !__any_sync(0xffffffffu, none);
}

// ---------------------------------------------------------------- the kernel
template <typename T, int kThreads, bool MULTI, bool CUTS>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) sample_kernel(const ParamsOf<CUTS> p, const int slice, const int in_smem) {
  extern __shared__ __align__(16) uint8_t dyn[];
  Shared& s = *reinterpret_cast<Shared*>(dyn);
  T* kept = reinterpret_cast<T*>(dyn + (sizeof(Shared) + 15) / 16 * 16);
  constexpr int E = Row<T, kThreads>::E, kWarps = kThreads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Row<T, kThreads> row;
  row.rank = 0;
  row.ctas = 1;
  if constexpr (MULTI) {
    row.rank = cluster_ctarank();
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(row.ctas));
    // waited for before the first write into another CTA: it has to be running
    asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  }
  const int64_t r = blockIdx.x / row.ctas;
  const int vocab = static_cast<int>(p.vocab);
  int64_t request = 0;
  const T* start = nullptr;
  if constexpr (CUTS) {
    int place;
    // rows behind a request's last draft are not looked at
    if (!verify_row(p, static_cast<uint32_t>(r), &start, &request, &place)) {
      if constexpr (MULTI) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
      return;
    }
  }
  row.c0 = static_cast<int>(row.rank) * slice;
  row.n = max(0, min(slice, vocab - row.c0));
  row.vecs = (row.n + E - 1) / E;
  if constexpr (CUTS)
    row.data = start + row.c0;
  else
    row.data = static_cast<const T*>(p.x) + r * p.ld + row.c0;
  row.padded = false;
  row.aligned = reinterpret_cast<uintptr_t>(row.data) % 16 == 0;

  const int64_t own = CUTS ? request : r;  // whose settings
  const float temperature = p.temperatures ? p.temperatures[own] : p.temperature;
  const int64_t top_k = p.top_ks ? p.top_ks[own] : p.top_k;
  const float top_p = p.top_ps ? p.top_ps[own] : p.top_p;
  const float u = CUTS ? 0.f : p.u[r];
  row.min_p = p.min_ps ? p.min_ps[own] : p.min_p;
  // (a reciprocal of zero would make NaN of a logit of -infinity)
  row.inv = fmaxf(1.f / temperature, kLeast);
  row.per_place = fmaxf(fminf(row.inv * (1.f / kPlaces), 3e38f), kLeast);
  bool bad = temperature != temperature || top_p != top_p || row.min_p != row.min_p || u != u;
  const bool greedy = !(temperature > 0.f) || row.inv == INFINITY || top_k == 1 || top_p <= 0.f || row.min_p > 1.f;
  const bool need_k = top_k > 0 && top_k < p.vocab;
  const bool need_counts = !greedy && !bad && (need_k || top_p < 1.f);

  if (need_counts) {
    for (int i = threadIdx.x; i < kCountBins; i += kThreads) s.counts.count[i] = 0;
    for (int i = threadIdx.x; i < kWeighedBins; i += kThreads) s.counts.weight[i] = 0.f;
  }
  if (threadIdx.x < 4) s.listed[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    s.sum_total = s.sum_above = 0;
    s.general = 0;
  }
  if (threadIdx.x < 2) {
    s.cut_lo[threadIdx.x] = s.cut_hi[threadIdx.x] = ~0ull;
  }

  // ---- first pass: largest logit, counts
  float top = -INFINITY;
  int top_vec = -1;
  auto count = [&](const Raw<T, E>& raw) {
    float x[E];
    unpack<T, E>(raw, x);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int b = row.count_bin(x[e]);
      if (b < kCountBins - 1) atomicAdd(&s.counts.count[b], 1u);  // the last bin's are not needed
      if (b < kWeighedBins) atomicAdd(&s.counts.weight[b], expf(fminf((x[e] - row.anchor) * row.inv, 60.f)));
    }
  };
  // vectors [from, to), four per thread in flight
  auto sweep = [&](int from, int to, bool counting) {
    for (int v = from + threadIdx.x; v < to; v += 4 * kThreads) {
      Raw<T, E> raw[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (v + j * kThreads < to) raw[j] = row.get(v + j * kThreads);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int w = v + j * kThreads;
        if (w >= to) break;
        if (in_smem) store_raw<T, E>(kept + w * E, raw[j]);
        float x[E];
        unpack<T, E>(raw[j], x);
        float m = x[0];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          m = fmaxf(m, x[e]);
          bad |= x[e] != x[e];
        }
        if (m > top) {
          top = m;
          top_vec = w;
        }
        if (counting) count(raw[j]);
      }
    }
  };
  // the largest of the CTA's `top`s so far
  auto block_top = [&]() {
    const uint32_t k = __reduce_max_sync(0xffffffffu, order_key(top));
    __syncthreads();
    if (lane == 0) s.red[warp] = k;
    __syncthreads();
    return key_value(__reduce_max_sync(0xffffffffu, lane < kWarps ? s.red[lane] : 0u));
  };
  // without a cluster the first part of the row sets the anchor, and the counts
  // of all but that part come with the only read from HBM; a cluster's slices
  // are short and are looked through again with the row's maximum as the anchor,
  // and so is a row whose first part holds nothing finite. (The anchor must not lie
  // above the maximum: logits in the last bin are left out as weighing nothing.)
  const int first = MULTI ? row.vecs : min(row.vecs, kFirstVectors * kThreads);
  sweep(0, first, false);
  bool anchored = false;
  if (!MULTI && need_counts) {
    row.anchor = block_top();
    anchored = fabsf(row.anchor) < INFINITY;
    if (anchored)
      for (int v = threadIdx.x; v < first; v += kThreads) count(row.get(v));
  }
  sweep(first, row.vecs, anchored);
  if (in_smem) {
    row.data = kept;
    row.padded = row.aligned = true;
  }
  const float slice_top = block_top();
  bad = __syncthreads_or(bad);
  row.top = slice_top;
  if constexpr (MULTI) {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    // told to all before the barrier: reading the others' after it takes 1200 cycles more
    if (threadIdx.x < row.ctas) {
      remote_store(reinterpret_cast<uint32_t*>(&s.tops[row.rank]), threadIdx.x, __float_as_uint(slice_top));
      remote_store(&s.bads[row.rank], threadIdx.x, bad);
    }
    row_barrier<MULTI>();
    for (uint32_t c = 0; c < row.ctas; ++c) {
      row.top = fmaxf(row.top, s.tops[c]);
      bad |= s.bads[c] != 0;
    }
  }
  bad |= !(fabsf(row.top) < INFINITY);  // no finite logit, or +infinity

  if (bad || greedy) {
    uint32_t at = 0xFFFFFFFFu;
    if (!bad && top == row.top) {  // the thread's first vector with it
      float x[E];
      unpack<T, E>(row.get(top_vec), x);
#pragma unroll
      for (int e = E - 1; e >= 0; --e)
        if (x[e] == top) at = static_cast<uint32_t>(row.c0 + top_vec * E + e);
    }
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0) s.red2[warp] = at;
    __syncthreads();
    at = __reduce_min_sync(0xffffffffu, lane < kWarps ? s.red2[lane] : 0xFFFFFFFFu);
    if constexpr (MULTI) {
      if (threadIdx.x == 0) s.first = at;
      row_barrier<MULTI>();
      for (uint32_t c = 0; c < row.ctas; ++c) at = min(at, remote<MULTI>(&s.first, c));
      row_barrier<MULTI>();  // all have read it
    }
    if constexpr (CUTS) {
      // the one token that is kept, with a weight of 1
      if (row.rank == 0 && threadIdx.x == 0) p.cuts[r] = {bad ? 0 : list_entry(row.top, at), bad ? 0 : uint64_t{1} << 40, row.top, 1.f, 0.f, 1.f / kFixed};
      return;
    }
    if (row.rank == 0 && threadIdx.x == 0) {
      p.tokens[r] = bad ? -1 : static_cast<int64_t>(at);
      if (p.logprobs) p.logprobs[r] = bad ? __uint_as_float(0x7FC00000u) : 0.f;
    }
    return;
  }

  // ---- where the prefix ends, by the counts
  bool general = false, listing = false;
  int cut_lo = 0, cut_hi = 0;  // bins to collect: from cut_lo on, before cut_hi
  if (need_counts) {
    if (!anchored) {
      row.anchor = row.top;
      row.each([&](float x, uint32_t) {
        const int b = row.count_bin(x);
        if (b < kCountBins - 1) atomicAdd(&s.counts.count[b], 1u);
        if (b < kWeighedBins) atomicAdd(&s.counts.weight[b], expf((x - row.anchor) * row.inv));
      });
      __syncthreads();
    }
    if constexpr (MULTI) {
      // to CTA 0, which looks for the end and tells the others
      if (row.rank != 0) {
        for (int b = threadIdx.x; b < kCountBins; b += kThreads) {
          const uint32_t c = s.counts.count[b];
          if (c) remote_add(&s.counts.count[b], 0, c);
          if (b < kWeighedBins && c) remote_add(&s.counts.weight[b], 0, s.counts.weight[b]);
        }
      }
      row_barrier<MULTI>();
    }
    if (row.rank == 0) {
      constexpr int kBinsPerThread = kCountBins / kThreads;
      uint32_t n[kBinsPerThread], n_sum = 0;
      float w[kBinsPerThread], w_sum = 0.f;
#pragma unroll
      for (int j = 0; j < kBinsPerThread; ++j) {
        const int b = kBinsPerThread * threadIdx.x + j;
        n[j] = s.counts.count[b];
        w[j] = b < kWeighedBins ? s.counts.weight[b] : n[j] ? n[j] * expf(kAbove - (b + 0.5f) * kUnitsPerBin) : 0.f;
        n_sum += n[j];
        w_sum += w[j];
      }
      uint32_t count_before;
      float weight_before, whole;
      block_exclusive<kThreads>(s, n_sum, w_sum, &count_before, &weight_before, &whole);
#pragma unroll
      for (int j = 0; j < kBinsPerThread; ++j) {
        const uint32_t b = kBinsPerThread * threadIdx.x + j;
        const uint32_t upto = count_before + n[j];
        const unsigned long long bin = static_cast<unsigned long long>(b) << 32;
        if (b == kCountBins - 1) {
          s.found_count = count_before;  // logits in all bins but the last, which is not counted
        } else if (need_k) {
          const uint64_t k = static_cast<uint64_t>(top_k);
          if (count_before < k && k <= upto) s.cut_hi[0] = bin | upto;
        } else if (n[j]) {
          // (rounding may let two neighbouring bins seem to hold a bound, or none: the
          // exact sums decide)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float margin = i == 0 ? kMargin : kSmallMargin;
            const float lo = (top_p - margin) * whole, hi = (top_p + margin) * whole;
            if (weight_before <= lo && lo < weight_before + w[j]) atomicMin(&s.cut_lo[i], bin | count_before);
            if (weight_before <= hi && hi < weight_before + w[j]) atomicMin(&s.cut_hi[i], bin | upto);
          }
        }
        count_before += n[j];
        weight_before += w[j];
      }
      __syncthreads();
      // from the first bin if none holds the lower bound; to the last but one, as the
      // last bin's weights are zero, if none holds the upper
      uint64_t from = 0, to = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        from = need_k || s.cut_lo[i] == ~0ull ? 0 : s.cut_lo[i];
        to = s.cut_hi[i] != ~0ull ? s.cut_hi[i] : static_cast<uint64_t>(kCountBins - 2) << 32 | s.found_count;
        general = static_cast<uint32_t>(to) - static_cast<uint32_t>(from) > static_cast<uint32_t>(kListKeys);
        if (need_k || !general) break;
      }
      general |= !(whole < INFINITY);
      cut_lo = static_cast<int>(from >> 32);
      cut_hi = static_cast<int>(to >> 32) + 1;
      if (MULTI && threadIdx.x < row.ctas) {
        remote_store(&s.told[0], threadIdx.x, static_cast<uint32_t>(cut_lo));
        remote_store(&s.told[1], threadIdx.x, static_cast<uint32_t>(cut_hi));
        remote_store(&s.told[2], threadIdx.x, general);
      }
    }
    if constexpr (MULTI) {
      row_barrier<MULTI>();
      cut_lo = static_cast<int>(s.told[0]);
      cut_hi = static_cast<int>(s.told[1]);
      general = s.told[2] != 0;
    }
    listing = need_k && !general;
  }
  // the same as logits: above the collected bins from x_lo on, in them from x_hi on
  float x_lo = INFINITY, x_hi = INFINITY;
  if (need_counts && !general) {
    if (warp < 2) {
      const float x = (warp == 0 ? cut_lo : cut_hi) > 0 ? row.first_before(warp == 0 ? cut_lo : cut_hi) : INFINITY;
      if (lane == 0) s.cut_x[warp] = x;
    }
    __syncthreads();
    x_lo = s.cut_x[0];
    x_hi = s.cut_x[1];
  }

  // ---- second pass
  if (listing) {
    row.each([&](float x, uint32_t i) {
      if (x >= x_hi) append<MULTI>(s, &s.listed[0], list_entry(x, i));
    });
    row_barrier<MULTI>();
    if (row.rank == 0) {
      const int n = static_cast<int>(s.listed[0]);
      if (n <= kShort)
        short_list_answer<T, kThreads, CUTS>(row, s, p, r, n, top_k, top_p, u);
      else
        list_answer<T, kThreads, CUTS>(row, s, p, r, n, top_k, top_p, u, x_hi);
    }
    return;  // nothing of the other CTAs is read any more
  }
  if (!general) {
    const bool cut = need_counts, min_p = row.min_p > 0.f;
    if (cut && min_p)
      sum_segments<T, kThreads, MULTI, true, true>(row, s, x_lo, x_hi);
    else if (cut)
      sum_segments<T, kThreads, MULTI, true, false>(row, s, x_lo, x_hi);
    else if (min_p)
      sum_segments<T, kThreads, MULTI, false, true>(row, s, x_lo, x_hi);
    else
      sum_segments<T, kThreads, MULTI, false, false>(row, s, x_lo, x_hi);
    row_barrier<MULTI>();
    if (row.rank == 0 && !segment_answer<T, kThreads, MULTI, CUTS>(row, s, p, r, slice, top_p, u, cut, x_lo, x_hi) &&
        threadIdx.x == 0)
      s.general = 1;
    row_barrier<MULTI>();
    general = remote<MULTI>(&s.general, 0) != 0;
    if constexpr (MULTI) row_barrier<MULTI>();  // CTA 0 stays until all have read it
  }
  if (general) general_answer<T, kThreads, MULTI, CUTS>(row, s, p, r, top_k, top_p, u);
}

template <typename T, int kThreads, bool MULTI, bool CUTS>
cudaError_t run(const ParamsOf<CUTS>& p, int ctas, cudaStream_t s) {
  constexpr size_t shared = (sizeof(Shared) + 15) / 16 * 16, most = kMostShared / (1024 / kThreads) / 1024 * 1024;
  static_assert(shared <= most, "two CTAs of half the threads share an SM");
  const int slice = static_cast<int>(((p.vocab + ctas - 1) / ctas + 63) / 64 * 64);
  const size_t kept = static_cast<size_t>(slice) * sizeof(T);
  const bool in_smem = shared + kept <= most;
  auto kernel = sample_kernel<T, kThreads, MULTI, CUTS>;
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  if (!(done.load() >> (dev & 63) & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
    if (e != cudaSuccess) return e;
    done.fetch_or(1ull << (dev & 63));
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = shared + (in_smem ? kept : 0);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(ctas);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, slice, in_smem ? 1 : 0);
}

template <typename T, bool CUTS>
cudaError_t run_typed(const ParamsOf<CUTS>& p, int sms, cudaStream_t s) {
  // One CTA per row where that occupies half of the SMs or more; fewer rows
  // are spread over clusters, down to 4096 logits per CTA. More rows than SMs
  // run two to an SM, so that one row's short phases, which wait on barriers, run
  // under the other's passes: 1024 x 2683 fp32 take 51 us so and 82 one to an SM,
  // 512 x 129280 182 and 187.
  if (p.rows > sms) return run<T, 512, false, CUTS>(p, 1, s);
  int ctas = 1;
  while (ctas < kMaxCluster && p.rows * ctas * 2 <= sms && p.vocab / ctas > 4096) ctas *= 2;
  return ctas > 1 ? run<T, 1024, true, CUTS>(p, ctas, s) : run<T, 1024, false, CUTS>(p, 1, s);
}

}  // namespace

}  // namespace flce
