// One token per row of logits: temperature, top-k, top-p, min-p, and the inverse
// of the kept tokens' distribution function at a given random number.
//
// Nothing is sorted. In rank order (falling logit, ties by index) every filter
// keeps a prefix, so the kept set is described by one logit t and a number c:
// all logits above t, and the first c of those equal to t. top-k needs t at a
// count, top-p at a weight; both come from a histogram of 1024 bins followed by
// an exact look at the bin that holds the answer. Weights are whole multiples
// of 2^-40 of the largest one and are added as 64-bit integers, so that no sum
// depends on the order or on how many CTAs share a row: the token is a function
// of the logits, the settings and u alone.
//
// Bound by memory: a row is read from HBM once, into the shared memory of a
// cluster of up to eight CTAs, which exchange maxima, histograms and sums
// through distributed shared memory. The steps, with a cluster barrier after
// each: load and maximum; histogram; look into the bin; running sums and the
// answer. top_k of up to kListKeys / 2 takes a shorter way: the k-th largest of
// the threads' own maxima bounds the k-th logit from below, the few logits
// above the bound are collected in one CTA and sorted there, and the rest of
// the cluster is done.
//
// The histogram's bins are equal steps of the scaled distance from the maximum,
// t = (x - m) / T in (-28, 0]; beyond that a weight rounds to zero. If the bin
// that holds the answer has too many logits to list (bf16 logits repeat), it is
// split by the bits of their order-preserving integers until it has few
// enough or all are equal.
#include <math.h>

#include <atomic>

#include "flce_device.cuh"
#include "head_device.cuh"
#include "head_internal.h"

namespace flce {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 1024;
constexpr int kListKeys = 2048;
constexpr float kRange = 28.f;  // exp(-28) 2^40 < 1
constexpr float kBinsPerUnit = (kBins - 1) / kRange;
constexpr float kFixed = 1099511627776.f;  // 2^40
constexpr int kMaxSlice = FLCE_SAMPLE_MAX_ROW_BYTES / kMaxCluster;

struct Hist {
  uint32_t count[kBins];
  uint32_t lo[kBins];  // 64-bit weights in halves: shared memory adds 32 bits at a time
  uint32_t hi[kBins];
};

// Shared memory of a CTA in front of its slice of the row; the same place in
// every CTA of the cluster.
struct Shared {
  Hist hist[2];
  uint64_t list[kListKeys];
  uint64_t seg_weight[kWarps];
  uint32_t seg_ties[kWarps];
  uint64_t scan[kWarps + 1];
  uint64_t found_above;
  uint32_t found_bin, found_count;
  float top;
  uint32_t bad;
  uint32_t first;      // lowest index of the largest logit in this slice
  uint32_t key_lo, key_hi;
  uint32_t listed[3];  // lengths of the lists of a row, one counter per use
  uint32_t result_key, result_count;
  uint32_t red[kWarps], red2[kWarps];
};

__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 and +0 are the same logit
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// Barrier of the cluster's threads. Not the aligned form: threads come here
// from code that only some of them run.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Addresses and accesses in the shared memory of CTA `rank` of the cluster.
template <typename V>
__device__ __forceinline__ V remote(const V* mine, uint32_t rank) {
  const uint32_t a = mapa_shared(smem_u32(mine), rank);
  if constexpr (sizeof(V) == 8) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return static_cast<V>(v);
  } else {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    if constexpr (sizeof(V) == 4 && static_cast<V>(0.5f) != static_cast<V>(0))
      return __uint_as_float(v);
    else
      return static_cast<V>(v);
  }
}
__device__ __forceinline__ uint32_t remote_add(uint32_t* mine, uint32_t rank, uint32_t v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;"
               : "=r"(old)
               : "r"(mapa_shared(smem_u32(mine), rank)), "r"(v)
               : "memory");
  return old;
}
__device__ __forceinline__ void remote_store(uint64_t* mine, uint32_t rank, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa_shared(smem_u32(mine), rank)), "l"(v) : "memory");
}

__device__ __forceinline__ uint64_t warp_inclusive(uint64_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  return v;
}

// Exclusive prefix sum over the CTA's threads; *total gets the whole. Begins and
// ends with a barrier, so `scan` may be used again at once.
__device__ uint64_t block_exclusive(uint64_t v, uint64_t* scan, uint64_t* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t inc = warp_inclusive(v);
  __syncthreads();
  if (lane == 31) scan[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const uint64_t w = lane < kWarps ? scan[lane] : 0;
    const uint64_t wi = warp_inclusive(w);
    __syncwarp();
    if (lane < kWarps) scan[lane] = wi - w;
    if (lane == kWarps - 1) scan[kWarps] = wi;
  }
  __syncthreads();
  *total = scan[kWarps];
  return scan[warp] + inc - v;
}

// Adds a 64-bit weight to a bin, in halves with the carry.
__device__ __forceinline__ void add_weight(Hist& h, int b, uint64_t w) {
  const uint32_t lo = static_cast<uint32_t>(w);
  uint32_t hi = static_cast<uint32_t>(w >> 32);
  const uint32_t old = atomicAdd(&h.lo[b], lo);
  if (old > ~lo) ++hi;
  if (hi) atomicAdd(&h.hi[b], hi);
}

// The smallest whole number b with (double)b >= bound: what lies before a kept
// token is less than that.
__device__ __forceinline__ uint64_t reach(double bound) {
  if (!(bound > 0.0)) return 0;
  int64_t b = static_cast<int64_t>(ceil(bound));
  while (b > 1 && __ll2double_rn(b - 1) >= bound) --b;
  return static_cast<uint64_t>(b);
}

// Sorts `n` keys (padded to a power of two by the caller's size m) in place, rising.
__device__ void sort_list(uint64_t* a, int m) {
  for (int size = 2; size <= m; size <<= 1) {
    for (int gap = size >> 1; gap > 0; gap >>= 1) {
      __syncthreads();
      for (int i = threadIdx.x; i < m / 2; i += kThreads) {
        const int l = 2 * i - (i & (gap - 1));
        const uint64_t u = a[l], v = a[l + gap];
        if ((u > v) == ((l & size) == 0)) {
          a[l] = v;
          a[l + gap] = u;
        }
      }
    }
  }
  __syncthreads();
}

__device__ __forceinline__ int pow2_at_least(int n) {
  int m = 2;
  while (m < n) m <<= 1;
  return m;
}

// The row as one CTA sees it.
template <typename T>
struct Row {
  static constexpr int E = 16 / sizeof(T);
  const T* data;  // slice in shared memory, padded with -infinity to whole vectors
  int vecs;
  int c0;         // vocabulary index of the slice's first logit
  float top, inv; // largest logit of the row, 1 / temperature
  float min_p;
  uint32_t rank, ctas;

  __device__ __forceinline__ float scaled(float x) const { return __fmul_rn(x - top, inv); }
  __device__ __forceinline__ int bin(float x) const {
    return min(kBins - 1, __float2int_rz(scaled(x) * -kBinsPerUnit));
  }
  __device__ __forceinline__ uint64_t weight(float x) const { return __float2ull_rz(expf(scaled(x)) * kFixed); }

  // f(x, index) for this thread's logits.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (int v = threadIdx.x; v < vecs; v += kThreads) {
      float x[E];
      unpack<T, E>(load_raw<T, E>(data + v * E), x);
#pragma unroll
      for (int e = 0; e < E; ++e) f(x[e], static_cast<uint32_t>(c0 + v * E + e));
    }
  }
};

__device__ void clear(Hist& h) {
  for (int i = threadIdx.x; i < kBins; i += kThreads) h.count[i] = h.lo[i] = h.hi[i] = 0;
  __syncthreads();
}

// Sums the cluster's histograms, bins 2 t and 2 t + 1 in thread t. want(total)
// gives the goal; the bin whose running sum first reaches it goes to found_*
// (found_bin = kBins if none does). WEIGHT: sums of weights, else counts.
template <bool WEIGHT, typename F>
__device__ void find_bin(Shared& s, const Hist& h, uint32_t ctas, F want) {
  uint64_t v[2];
  uint32_t n[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int b = 2 * threadIdx.x + j;
    v[j] = 0;
    n[j] = 0;
    for (uint32_t r = 0; r < ctas; ++r) {
      n[j] += remote(&h.count[b], r);
      if (WEIGHT) v[j] += remote(&h.lo[b], r) + (static_cast<uint64_t>(remote(&h.hi[b], r)) << 32);
    }
    if (!WEIGHT) v[j] = n[j];
  }
  if (threadIdx.x == 0) s.found_bin = kBins;
  uint64_t total;
  uint64_t before = block_exclusive(v[0] + v[1], s.scan, &total);
  const uint64_t goal = want(total);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (before < goal && goal <= before + v[j]) {
      s.found_bin = 2 * threadIdx.x + j;
      s.found_above = before;
      s.found_count = n[j];
    }
    before += v[j];
  }
  __syncthreads();
}

// Finds the logit (as a key) and the number of logits equal to it at which the
// running sum over the ranked logits above `limit` (a key) first reaches the
// goal. Returns false if the sum never does: nothing is cut off.
template <typename T, bool WEIGHT, typename F>
__device__ bool select(const Row<T>& row, Shared& s, int& buf, uint32_t* listed, uint32_t limit, F want,
                       uint32_t* key_out, uint32_t* count_out) {
  Hist* h = &s.hist[buf];
  buf ^= 1;
  clear(*h);
  row.each([&](float x, uint32_t) {
    const int b = row.bin(x);
    if (b < kBins - 1 && order_key(x) > limit) {
      atomicAdd(&h->count[b], 1u);
      if (WEIGHT) add_weight(*h, b, row.weight(x));
    }
  });
  cluster_barrier();
  uint64_t goal = 0;
  find_bin<WEIGHT>(s, *h, row.ctas, [&](uint64_t total) { return goal = want(total); });
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
      for (int w = 1; w < kWarps; ++w) {
        lo = min(lo, s.red[w]);
        hi = max(hi, s.red2[w]);
      }
      s.key_lo = lo;
      s.key_hi = hi;
    }
    cluster_barrier();
    key_lo = 0xFFFFFFFFu;
    key_hi = 0;
    for (uint32_t r = 0; r < row.ctas; ++r) {
      key_lo = min(key_lo, remote(&s.key_lo, r));
      key_hi = max(key_hi, remote(&s.key_hi, r));
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
    clear(*h);
    row.each([&](float x, uint32_t) {
      const uint32_t k = order_key(x);
      if (k >= key_lo && k <= key_hi) {
        const int b = static_cast<int>((key_hi - k) >> shift);
        atomicAdd(&h->count[b], 1u);
        if (WEIGHT) add_weight(*h, b, row.weight(x));
      }
    });
    cluster_barrier();
    find_bin<WEIGHT>(s, *h, row.ctas, [&](uint64_t) { return goal - above; });
    const uint32_t b = s.found_bin;
    above += s.found_above;
    count = s.found_count;
    const uint32_t top = key_hi - (b << shift);
    const uint32_t width = (1u << shift) - 1;
    key_lo = top - key_lo > width ? top - width : key_lo;
    key_hi = top;
  }
  // few enough: CTA 0 sorts them
  row.each([&](float x, uint32_t i) {
    if (inside(x)) {
      const uint32_t at = remote_add(listed, 0, 1u);
      if (at < static_cast<uint32_t>(kListKeys))
        remote_store(&s.list[at], 0, static_cast<uint64_t>(~order_key(x)) << 32 | i);
    }
  });
  cluster_barrier();
  if (row.rank == 0) {
    const int n = static_cast<int>(count), m = pow2_at_least(n);
    for (int i = n + threadIdx.x; i < m; i += kThreads) s.list[i] = ~0ull;
    sort_list(s.list, m);
    constexpr int per = kListKeys / kThreads;
    uint64_t w[per], sum = 0, total;
#pragma unroll
    for (int j = 0; j < per; ++j) {
      const int i = threadIdx.x * per + j;
      w[j] = i < n ? (WEIGHT ? row.weight(key_value(~static_cast<uint32_t>(s.list[i] >> 32))) : 1) : 0;
      sum += w[j];
    }
    uint64_t before = above + block_exclusive(sum, s.scan, &total);
#pragma unroll
    for (int j = 0; j < per; ++j) {
      const int i = threadIdx.x * per + j;
      if (i < n && before < goal && goal <= before + w[j]) {
        const uint32_t nk = static_cast<uint32_t>(s.list[i] >> 32);
        int f = i;
        while (f > 0 && static_cast<uint32_t>(s.list[f - 1] >> 32) == nk) --f;
        s.result_key = ~nk;
        s.result_count = static_cast<uint32_t>(i - f + 1);
      }
      before += w[j];
    }
  }
  cluster_barrier();
  *key_out = remote(&s.result_key, 0);
  *count_out = remote(&s.result_count, 0);
  return true;
}

// Everything after the selection of few candidates, by one CTA: `n` of them in
// s.list as (inverted key, index), at least the first top_k by rank.
template <typename T>
__device__ void finish_list(const Row<T>& row, Shared& s, int n, int64_t top_k, float top_p, float u, int64_t* token,
                            float* logprob) {
  constexpr int per = kListKeys / kThreads;
  const int m = pow2_at_least(n);
  for (int i = n + threadIdx.x; i < m; i += kThreads) s.list[i] = ~0ull;
  sort_list(s.list, m);
  if (top_k > 0 && n > top_k) n = static_cast<int>(top_k);
  uint64_t* weights = reinterpret_cast<uint64_t*>(&s.hist[0]);  // of kListKeys tokens
  static_assert(sizeof(s.hist) >= sizeof(uint64_t) * kListKeys, "weights of a list in the histograms' place");
  uint64_t w[per], sum = 0, whole;
  bool pass[per];
#pragma unroll
  for (int j = 0; j < per; ++j) {
    const int i = threadIdx.x * per + j;
    w[j] = 0;
    pass[j] = false;
    if (i < n) {
      const float e = expf(row.scaled(key_value(~static_cast<uint32_t>(s.list[i] >> 32))));
      w[j] = __float2ull_rz(e * kFixed);
      pass[j] = i == 0 || e >= row.min_p;
    }
    sum += w[j];
  }
  uint64_t before = block_exclusive(sum, s.scan, &whole);
  const uint64_t far = top_p < 1.f ? reach(__dmul_rn(static_cast<double>(top_p), __ll2double_rn(static_cast<int64_t>(whole))))
                                   : ~0ull;
  if (threadIdx.x == 0) s.first = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < per; ++j) {
    const int i = threadIdx.x * per + j;
    const bool keep = i < n && pass[j] && (i == 0 || before < far);
    if (i < n) weights[i] = keep ? w[j] : 0;
    if (keep) atomicMax(&s.first, static_cast<uint32_t>(i + 1));
    before += w[j];
  }
  __syncthreads();
  const int k = static_cast<int>(s.first), mk = pow2_at_least(k);  // nothing is kept from rank k on
  // by index: (index, rank)
  uint64_t entry[per];
#pragma unroll
  for (int j = 0; j < per; ++j) {
    const int i = threadIdx.x + j * kThreads;
    entry[j] = i < k ? (s.list[i] << 32) | static_cast<uint32_t>(i) : ~0ull;
  }
  uint32_t* keys = reinterpret_cast<uint32_t*>(weights + kListKeys);  // inverted keys by rank
  static_assert(sizeof(s.hist) >= (sizeof(uint64_t) + sizeof(uint32_t)) * kListKeys, "weights and keys of a list");
#pragma unroll
  for (int j = 0; j < per; ++j) {
    const int i = threadIdx.x + j * kThreads;
    if (i < k) keys[i] = static_cast<uint32_t>(s.list[i] >> 32);
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < per; ++j) {
    const int i = threadIdx.x + j * kThreads;
    if (i < mk) s.list[i] = entry[j];
  }
  sort_list(s.list, mk);
  sum = 0;
#pragma unroll
  for (int j = 0; j < per; ++j) {
    const int i = threadIdx.x * per + j;
    w[j] = i < k ? weights[static_cast<uint32_t>(s.list[i])] : 0;
    sum += w[j];
  }
  before = block_exclusive(sum, s.scan, &whole);
  const int64_t total = static_cast<int64_t>(whole);
  int64_t goal = static_cast<int64_t>(__dmul_rn(static_cast<double>(u), __ll2double_rn(total)));
  goal = goal < 0 ? 0 : goal < total ? goal : total - 1;
#pragma unroll
  for (int j = 0; j < per; ++j) {
    const int i = threadIdx.x * per + j;
    const uint64_t g = static_cast<uint64_t>(goal);
    if (i < k && before <= g && g < before + w[j]) {
      *token = static_cast<int64_t>(s.list[i] >> 32);
      if (logprob) {
        const float x = key_value(~keys[static_cast<uint32_t>(s.list[i])]);
        *logprob = row.scaled(x) - logf(__ll2float_rn(total) * (1.f / kFixed));
      }
    }
    before += w[j];
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleParams p, const int slice) {
  extern __shared__ __align__(16) uint8_t dyn[];
  Shared& s = *reinterpret_cast<Shared*>(dyn);
  T* data = reinterpret_cast<T*>(dyn + (sizeof(Shared) + 15) / 16 * 16);
  constexpr int E = Row<T>::E;
  Row<T> row;
  row.rank = cluster_ctarank();
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(row.ctas));
  const int64_t r = blockIdx.x / row.ctas;
  row.data = data;
  row.c0 = static_cast<int>(row.rank) * slice;
  const int vocab = static_cast<int>(p.vocab);
  const int n = max(0, min(slice, vocab - row.c0));
  row.vecs = (n + E - 1) / E;
  const T* x = static_cast<const T*>(p.x) + r * p.ld + row.c0;
  const bool vec_ok = reinterpret_cast<uintptr_t>(x) % 16 == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const float temperature = p.temperatures ? p.temperatures[r] : p.temperature;
  const int64_t top_k = p.top_ks ? p.top_ks[r] : p.top_k;
  const float top_p = p.top_ps ? p.top_ps[r] : p.top_p;
  const float u = p.u[r];
  row.min_p = p.min_ps ? p.min_ps[r] : p.min_p;

  // ---- load, largest logit
  float top = -INFINITY;
  bool bad = false;
#pragma unroll 4
  for (int v = threadIdx.x; v < row.vecs; v += kThreads) {
    float f[E];
    Raw<T, E> raw;
    if (vec_ok && (v + 1) * E <= n) {
      raw = load_raw<T, E>(x + v * E);
      unpack<T, E>(raw, f);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = v * E + e < n ? to_float<T>(x[v * E + e]) : -INFINITY;
      raw = pack<T, E>(f);
    }
    store_raw<T, E>(data + v * E, raw);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      top = fmaxf(top, f[e]);
      bad |= f[e] != f[e];
    }
  }
  const float my_top = top;
  {
    const uint32_t k = __reduce_max_sync(0xffffffffu, order_key(top));
    const bool any = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      s.red[warp] = k;
      s.red2[warp] = any;
    }
    if (threadIdx.x < 3) s.listed[threadIdx.x] = 0;
    __syncthreads();
    if (warp == 0) {
      const uint32_t k2 = __reduce_max_sync(0xffffffffu, lane < kWarps ? s.red[lane] : 0u);
      const bool any2 = __any_sync(0xffffffffu, lane < kWarps && s.red2[lane]);
      if (lane == 0) {
        s.top = key_value(k2);
        s.bad = any2;
      }
    }
  }
  cluster_barrier();
  row.top = -INFINITY;
  bad = false;
  for (uint32_t c = 0; c < row.ctas; ++c) {
    row.top = fmaxf(row.top, remote(&s.top, c));
    bad |= remote(&s.bad, c) != 0;
  }
  bad |= !(fabsf(row.top) < INFINITY);  // no finite logit, or +infinity
  bad |= temperature != temperature || top_p != top_p || row.min_p != row.min_p || u != u;
  row.inv = 1.f / temperature;
  const bool greedy = !(temperature > 0.f) || row.inv == INFINITY || top_k == 1 || top_p <= 0.f || row.min_p > 1.f;

  if (bad || greedy) {
    uint32_t first = 0xFFFFFFFFu;
    if (!bad) row.each([&](float v, uint32_t i) {
      if (v == row.top) first = min(first, i);
    });
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) s.red[warp] = first;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kWarps; ++w) first = min(first, s.red[w]);
      s.first = first;
    }
    cluster_barrier();
    if (row.rank == 0 && threadIdx.x == 0) {
      for (uint32_t c = 1; c < row.ctas; ++c) first = min(first, remote(&s.first, c));
      p.tokens[r] = bad ? -1 : static_cast<int64_t>(first);
      if (p.logprobs) p.logprobs[r] = bad ? __uint_as_float(0x7FC00000u) : 0.f;
    }
    cluster_barrier();  // CTA 0 has read the others' shared memory
    return;
  }

  const bool need_k = top_k > 0 && top_k < p.vocab;
  int buf = 0;
  if (need_k && top_k <= kListKeys / 2) {
    Hist& h = s.hist[buf];
    buf ^= 1;
    clear(h);
    if (threadIdx.x < row.vecs) atomicAdd(&h.count[row.bin(my_top)], 1u);
    cluster_barrier();
    find_bin<false>(s, h, row.ctas, [&](uint64_t) { return static_cast<uint64_t>(top_k); });
    const int cut = min(static_cast<int>(s.found_bin), kBins - 2);  // the last bin's weights are zero
    row.each([&](float v, uint32_t i) {
      if (row.bin(v) <= cut) {
        const uint32_t at = remote_add(&s.listed[0], 0, 1u);
        if (at < static_cast<uint32_t>(kListKeys))
          remote_store(&s.list[at], 0, static_cast<uint64_t>(~order_key(v)) << 32 | i);
      }
    });
    cluster_barrier();
    const uint32_t listed = remote(&s.listed[0], 0);
    if (listed <= static_cast<uint32_t>(kListKeys)) {
      if (row.rank == 0)
        finish_list(row, s, static_cast<int>(listed), top_k, top_p, u, p.tokens + r,
                    p.logprobs ? p.logprobs + r : nullptr);
      cluster_barrier();  // CTA 0's counter has been read by all
      return;
    }
  }

  // ---- the kept set: logits above `key`, and the first `ties` of those equal to it
  uint32_t key = 0, ties = 0;
  if (need_k)
    if (!select<T, false>(row, s, buf, &s.listed[1], 0u, [&](uint64_t) { return static_cast<uint64_t>(top_k); }, &key,
                          &ties))
      key = ties = 0;
  if (top_p < 1.f) {
    const uint64_t w = ties ? row.weight(key_value(key)) : 0;
    uint64_t goal = 0, over = 0;
    uint32_t k2, t2;
    const bool cut = select<T, true>(
        row, s, buf, &s.listed[2], key,
        [&](uint64_t total) {
          over = total;
          const int64_t whole = static_cast<int64_t>(total + ties * w);
          goal = reach(__dmul_rn(static_cast<double>(top_p), __ll2double_rn(whole)));
          return goal;
        },
        &k2, &t2);
    if (cut) {
      key = k2;
      ties = t2;
    } else if (ties) {
      const uint64_t need = (goal - over + w - 1) / (w ? w : 1);
      ties = need < ties ? static_cast<uint32_t>(need) : ties;
    }
  }

  // ---- running sums in index order: a warp per segment of the slice
  const float e_tie = ties ? expf(row.scaled(key_value(key))) : 0.f;
  const uint64_t w_tie = e_tie >= row.min_p ? __float2ull_rz(e_tie * kFixed) : 0;
  const int seg = (row.vecs + kWarps - 1) / kWarps;
  const int v0 = warp * seg, v1 = min(v0 + seg, row.vecs);
  auto kept_weight = [&](float f) -> uint64_t {
    if (order_key(f) <= key) return 0;
    const float e = expf(row.scaled(f));
    return e >= row.min_p ? __float2ull_rz(e * kFixed) : 0;
  };
  uint64_t sum = 0;
  uint32_t equal = 0;
  for (int v = v0 + lane; v < v1; v += 32) {
    float f[E];
    unpack<T, E>(load_raw<T, E>(data + v * E), f);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      sum += kept_weight(f[e]);
      if (ties) equal += order_key(f[e]) == key;
    }
  }
  sum = warp_inclusive(sum);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 31) {
    s.seg_weight[warp] = sum;
    s.seg_ties[warp] = equal;
  }
  cluster_barrier();
  // every warp finds the segment of the answer; it goes on if that is its own
  const int segs = static_cast<int>(row.ctas) * kWarps;
  uint64_t total = 0, my_before = 0, my_weight = 0;
  uint32_t tie_total = 0, my_tie_before = 0;
  const int mine = static_cast<int>(row.rank) * kWarps + warp;
  for (int base = 0; base < segs; base += 32) {
    const int i = base + lane;
    uint64_t w = 0;
    uint32_t t = 0;
    if (i < segs) {
      w = remote(&s.seg_weight[i % kWarps], i / kWarps);
      t = remote(&s.seg_ties[i % kWarps], i / kWarps);
    }
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
  const int64_t whole = static_cast<int64_t>(total);
  int64_t g = static_cast<int64_t>(__dmul_rn(static_cast<double>(u), __ll2double_rn(whole)));
  g = g < 0 ? 0 : g < whole ? g : whole - 1;
  const uint64_t goal = static_cast<uint64_t>(g);
  if (my_before <= goal && goal < my_before + my_weight) {
    uint64_t before = my_before;
    uint32_t tie_before = my_tie_before;
    for (int b = v0; b < v1; b += 32) {
      const int v = b + lane;
      float f[E];
      uint32_t eq = 0;
      uint64_t w = 0;
      if (v < v1) {
        unpack<T, E>(load_raw<T, E>(data + v * E), f);
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
            p.tokens[r] = row.c0 + v * E + e;
            if (p.logprobs) p.logprobs[r] = row.scaled(f[e]) - logf(__ll2float_rn(whole) * (1.f / kFixed));
          }
          mb += we;
        }
      }
      before += __shfl_sync(0xffffffffu, inc, 31);
      tie_before += __shfl_sync(0xffffffffu, eq_inc, 31);
    }
  }
  cluster_barrier();  // the segments' sums have been read by all
}

}  // namespace

cudaError_t launch_sample(const SampleParams& p, int sms, cudaStream_t s) {
  const bool f32 = p.dtype == FLCE_DTYPE_F32;
  const int64_t es = f32 ? 4 : 2;
  // Slices of at most 64 KB let three CTAs share an SM, which hides one's
  // barriers behind another's work; few rows are spread over more CTAs, down
  // to 4096 logits each.
  int ctas = 1;
  while (ctas < kMaxCluster && (p.vocab * es + ctas - 1) / ctas > 64 * 1024) ctas *= 2;
  while (ctas < kMaxCluster && p.rows * ctas * 2 <= sms && p.vocab / ctas > 4096) ctas *= 2;
  const int slice = static_cast<int>(((p.vocab + ctas - 1) / ctas + 63) / 64 * 64);
  const size_t smem = (sizeof(Shared) + 15) / 16 * 16 + static_cast<size_t>(slice) * es;
  auto kernel = f32 ? sample_kernel<float> : sample_kernel<uint16_t>;
  static_assert((sizeof(Shared) + 15) / 16 * 16 + kMaxSlice + 256 <= 227 * 1024, "a slice fits beside the rest");
  static std::atomic<uint64_t> done[2];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  if (!(done[f32].load() >> (dev & 63) & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    done[f32].fetch_or(1ull << (dev & 63));
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(ctas);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, slice);
}

}  // namespace flce
