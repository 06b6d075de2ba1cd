// Embeddings: rows of W looked up by token and scaled, and the gradient, which adds
// rows up by token.
//
// The lookup is a copy, bound by memory: a warp takes a piece of a row with several
// vectors per lane in flight.
//
// The gradient sorts (token, position) pairs and then adds up runs of one token, so
// that every row of grad_W is written once, by one thread per column, and added up in an
// order that the tokens alone decide: no atomics do, and the result is the same in every run.
// Pieces of kChunk tokens are sorted by a CTA each; a key's place among all of them
// is its place in its piece plus what the others hold before it, found by binary search.
// The sorted rows are then cut into tiles of kEmbeddingTile: a tile's CTA walks its rows
// with the sum in registers and writes it where the token changes. Frequent tokens (in
// text the first takes a tenth of all places) fill many tiles; what a tile sums of a
// run that does not begin and end in it goes to the workspace, and a last kernel joins these sums
// in order. 32768 x 4096 bf16 into 128256 rows of fp32 take 355 us, 6.7 TB/s. Where the gradient is not added to what grad_W holds, the rows of absent
// tokens are zeroed by CTAs of the same launch: nothing is written twice.
#include <atomic>

#include "flce_host.h"
#include "head_device.cuh"
#include "model_internal.h"

namespace flce {

namespace {

constexpr int kThreads = 256;
template <int E>
constexpr int kVectors = E == 1 ? 16 : 4;  // per lane of the lookup
constexpr int kChunk = 1024;       // keys sorted by a CTA
constexpr int kMostShared = 48;    // chunks that shared memory holds
constexpr int kSharedGroup = 32;   // of more than that
constexpr int kSharedThreads = 1024;
constexpr int kGradThreads = 128;
constexpr int kJoinWarps = 8;
constexpr int kJoinCtas = 1216;    // for short runs, at least: eight per SM
constexpr int kLongRuns = 8;       // at a time
constexpr int kShortRun = 16;      // tiles
constexpr int kTile = kEmbeddingTile;
constexpr int kBatch = 8;          // rows of a tile in flight
constexpr int kZeroFloats = 65536; // of absent rows per CTA, about

// ------------------------------------------------------------------ forward
template <typename T, int E>
__device__ __forceinline__ void store_floats(T* to, const float (&v)[E]) {
  if constexpr (E == 1) {
    to[0] = from_float<T>(v[0]);
  } else if constexpr (sizeof(T) * E == 8) {
    *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  } else if constexpr (sizeof(T) == 2) {
    store_raw<T, E>(to, pack<T, E>(v));
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 4) *reinterpret_cast<float4*>(to + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
  }
}

template <typename TI, typename TO, int E>
__global__ void __launch_bounds__(kThreads) embedding_kernel(const EmbeddingParams p, const int64_t chunks) {
  constexpr int kUnroll = kVectors<E>;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
  if (unit >= p.rows * chunks) return;
  const int64_t row = unit / chunks, vecs = p.hidden / E;
  const int64_t first = (unit - row * chunks) * (32 * kUnroll) + (threadIdx.x & 31);
  const int64_t token = __ldg(p.tokens + row);
  const bool real = token >= 0 && token < p.vocab;
  const TI* w = static_cast<const TI*>(p.in) + (real ? token : 0) * p.ld;
  TO* out = static_cast<TO*>(p.out) + row * p.hidden;
  Raw<TI, E> raw[kUnroll];
#pragma unroll
  for (int j = 0; j < kUnroll; ++j)
    if (real && first + j * 32 < vecs) raw[j] = load_raw<TI, E>(w + (first + j * 32) * E);
  // no token gives zeros, one behind the vocabulary NaN
  const float other = token < 0 ? 0.f : __uint_as_float(0x7FC00000u);
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    const int64_t v = first + j * 32;
    if (v < vecs) {
      float f[E];
      if (real) {
        unpack<TI, E>(raw[j], f);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] *= p.scale;
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = other;
      }
      store_floats<TO, E>(out + v * E, f);
    }
  }
}

// ------------------------------------------------------------------ sort
// Sorts kChunk (token, position) keys of the CTA's piece, one in each thread; tokens outside
// of the vocabulary count as `vocab` and come last. (A bitonic sort; most of its exchanges are within
// a warp. With two keys per thread, all of them through shared memory, it took 10 us, so 6.)
// Also empties the lists of runs to join.
__global__ void __launch_bounds__(kChunk) embedding_chunk_kernel(const int64_t* tokens, const int64_t rows, const int64_t vocab,
                                                               uint32_t* sorted, uint32_t* places, uint32_t* joins) {
  __shared__ uint64_t other[kChunk];
  const int t = threadIdx.x;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kChunk + t;
  uint64_t key = ~0ull;  // behind the last row
  if (i < rows) {
    const int64_t token = __ldg(tokens + i);
    key = static_cast<uint64_t>(token >= 0 && token < vocab ? token : vocab) << 32 | static_cast<uint32_t>(i);
  }
  if (i < 2) joins[i] = 0;
  // runs of `run` are merged into runs of twice that, up and down in turn
  for (int run = 2; run <= kChunk; run *= 2) {
    for (int step = run / 2; step > 0; step /= 2) {
      uint64_t o;
      if (step >= 32) {
        other[t] = key;
        __syncthreads();
        o = other[t ^ step];
        __syncthreads();
      } else {
        o = __shfl_xor_sync(0xffffffffu, key, step);
      }
      const bool low = ((t & step) == 0) == ((t & run) == 0);
      key = low == (o < key) ? o : key;
    }
  }
  if (i < rows) {
    sorted[i] = static_cast<uint32_t>(key >> 32);
    places[i] = static_cast<uint32_t>(key);
  }
}

// Keys of a[0, n) that come before t: less than t, or (UPTO) equal to it.
template <bool UPTO>
__device__ __forceinline__ uint32_t keys_before(const uint32_t* a, uint32_t n, uint32_t t) {
  uint32_t lo = 0, hi = n;
  while (lo < hi) {
    const uint32_t mid = (lo + hi) / 2;
    const uint32_t k = __ldg(a + mid);
    if (UPTO ? k <= t : k < t)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

// Joins `group` sorted runs of `run` keys each: a key moves to the number of keys before
// it. Of equal tokens the earlier run's come first, as their positions do.
__global__ void __launch_bounds__(kThreads) embedding_merge_kernel(const uint32_t* sorted, const uint32_t* places, uint32_t* to_sorted,
                                                                 uint32_t* to_places, const int64_t rows, const int64_t run,
                                                                 const int group) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= rows) return;
  const uint32_t t = __ldg(sorted + i), place = __ldg(places + i);
  const int64_t mine = i / run, first = mine / group * group;
  int64_t at = first * run + (i - mine * run);
  for (int64_t r = first; r < first + group && r * run < rows; ++r) {
    const uint32_t n = static_cast<uint32_t>(min(run, rows - r * run));
    if (r < mine)
      at += keys_before<true>(sorted + r * run, n, t);
    else if (r > mine)
      at += keys_before<false>(sorted + r * run, n, t);
  }
  to_sorted[at] = t;
  to_places[at] = place;
}

// The same for groups of `group` runs of kChunk keys, up to kMostShared, blockIdx.y-th group in shared
// memory: the keys' loads would otherwise wait for the L2 some ten times for each run. Four
// searches go side by side. All threads load, few of them search: it takes a CTA on every SM. (Sorting 32768
// tokens takes 14 us so, 60 with the kernel above.)
__global__ void __launch_bounds__(kSharedThreads) embedding_merge_shared_kernel(const uint32_t* sorted, const uint32_t* places,
                                                                              uint32_t* to_sorted, uint32_t* to_places,
                                                                              const int64_t all_rows, const int group) {
  const int64_t first = static_cast<int64_t>(blockIdx.y) * group * kChunk;
  const int rows = static_cast<int>(min(static_cast<int64_t>(group) * kChunk, all_rows - first)), runs = (rows + kChunk - 1) / kChunk;
  sorted += first;
  places += first;
  to_sorted += first;
  to_places += first;
  extern __shared__ __align__(16) uint32_t keys[];  // [runs][kChunk], behind the last key the highest number
  const int n4 = rows / 4;
#pragma unroll 8
  for (int i = threadIdx.x; i < n4; i += kSharedThreads) reinterpret_cast<uint4*>(keys)[i] = __ldg(reinterpret_cast<const uint4*>(sorted) + i);
  for (int i = n4 * 4 + threadIdx.x; i < runs * kChunk; i += kSharedThreads) keys[i] = i < rows ? __ldg(sorted + i) : 0xFFFFFFFFu;
  __syncthreads();
  const int each = (rows + gridDim.x - 1) / gridDim.x, from = blockIdx.x * each, to = min(from + each, rows);  // of the CTA
  for (int i = from + threadIdx.x; i < to; i += kSharedThreads) {
    const uint32_t t = keys[i], place = __ldg(places + i);
    const int mine = i / kChunk;
    int at = i % kChunk;
    for (int r0 = 0; r0 < runs; r0 += 4) {
      // the number of keys below `t` of a later run, up to it of an earlier one: below t + 1
      int lo[4];
      uint32_t bound[4];
      const uint32_t* run[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = min(r0 + j, runs - 1);
        lo[j] = 0;
        bound[j] = t + (r < mine ? 1 : 0);
        run[j] = keys + r * kChunk;
      }
#pragma unroll
      for (int step = kChunk / 2; step > 0; step /= 2) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (run[j][lo[j] + step - 1] < bound[j]) lo[j] += step;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        lo[j] += run[j][lo[j]] < bound[j];
        if (r0 + j < runs && r0 + j != mine) at += lo[j];
      }
    }
    to_sorted[at] = t;
    to_places[at] = place;
  }
}

// ------------------------------------------------------------------ gradient
// Writes or adds E columns of a row. (The addition is the only one to its elements in the launch, and by the memory system, so
// that no thread waits for what the row holds: 30000 uniform tokens of 1337 bf16 columns 91 us, 162 by loading and
// storing; 8192 of 1024 columns 40 and 51, but 32768 of 4096 257 and 224. It takes numbers below 2^-126 as zero.)
template <int E>
__device__ __forceinline__ void put(float* to, const float (&v)[E], float scale, bool add) {
  if constexpr (E == 1) {
    if (add)
      atomicAdd(to, v[0] * scale);
    else
      *to = v[0] * scale;
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 4) {
      const float4 f = make_float4(v[e] * scale, v[e + 1] * scale, v[e + 2] * scale, v[e + 3] * scale);
      if (add)
        atomicAdd(reinterpret_cast<float4*>(to + e), f);
      else
        *reinterpret_cast<float4*>(to + e) = f;
    }
  }
}

// CTAs from `tiles` * `slices` on zero rows of absent tokens. A thread's columns: C vectors of E, kGradThreads apart.
template <typename T, int E, int C>
__global__ void __launch_bounds__(kGradThreads) embedding_grad_kernel(const EmbeddingParams p, const int64_t tiles, const int slices,
                                                                    const int zero_rows) {
  constexpr int kColumns = kGradThreads * E * C;
  const int64_t work = tiles * slices;
  float* grad_W = static_cast<float*>(p.out);
  if (blockIdx.x >= work) {
    __shared__ bool present[kGradThreads];
    const int64_t r0 = (blockIdx.x - work) * zero_rows;
    const int n = static_cast<int>(min(static_cast<int64_t>(zero_rows), p.vocab - r0));
    if (threadIdx.x < n) {
      const uint32_t t = static_cast<uint32_t>(r0 + threadIdx.x);
      const uint32_t at = keys_before<false>(p.sorted, static_cast<uint32_t>(p.rows), t);
      present[threadIdx.x] = at < p.rows && p.sorted[at] == t;
    }
    __syncthreads();
    for (int r = 0; r < n; ++r) {
      if (present[r]) continue;
      float* row = grad_W + (r0 + r) * p.hidden;
      if constexpr (E > 1) {
        for (int64_t i = threadIdx.x * 4; i < p.hidden; i += kGradThreads * 4) *reinterpret_cast<float4*>(row + i) = make_float4(0, 0, 0, 0);
      } else {
        for (int64_t i = threadIdx.x; i < p.hidden; i += kGradThreads) row[i] = 0.f;
      }
    }
    return;
  }
  // tokens of the tile with one on either side; none is vocab + 1
  __shared__ uint32_t token[kTile + 2], place[kTile];
  const int64_t tile = blockIdx.x / slices, r0 = tile * kTile;
  const int slice = static_cast<int>(blockIdx.x - tile * slices);
  const uint32_t none = static_cast<uint32_t>(p.vocab) + 1, skipped = static_cast<uint32_t>(p.vocab);
  if (threadIdx.x < kTile + 2) {
    const int64_t i = r0 + static_cast<int>(threadIdx.x) - 1;
    token[threadIdx.x] = i >= 0 && i < p.rows ? p.sorted[i] : none;
    if (threadIdx.x >= 1 && threadIdx.x <= kTile) place[threadIdx.x - 1] = i < p.rows ? p.places[i] : 0;
  }
  __syncthreads();
  const int64_t col = static_cast<int64_t>(slice) * kColumns + threadIdx.x * E;
  float acc[C][E];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < E; ++e) acc[c][e] = 0.f;
  bool leading = token[1] == token[0];  // the run began before this tile
  for (int b = 0; b < kTile; b += kBatch) {
    Raw<T, E> raw[kBatch][C];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const uint32_t t = token[b + j + 1];
      if (t < skipped) {
        const T* row = static_cast<const T*>(p.in) + place[b + j] * p.ld + col;
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (col + c * kGradThreads * E < p.hidden) raw[j][c] = load_raw<T, E>(row + c * kGradThreads * E);
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const uint32_t t = token[b + j + 1];
      if (t >= skipped) return;  // nothing of the vocabulary comes behind
      const bool ends = token[b + j + 2] != t, last = b + j == kTile - 1;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (col + c * kGradThreads * E < p.hidden) {
          float v[E];
          unpack<T, E>(raw[j][c], v);
#pragma unroll
          for (int e = 0; e < E; ++e) acc[c][e] += v[e];
          if (ends || last) {
            const int64_t at = col + c * kGradThreads * E;
            if (leading)
              put<E>(p.head + tile * p.hidden + at, acc[c], 1.f, false);
            else if (!ends)  // it begins here and goes on
              put<E>(p.tail + tile * p.hidden + at, acc[c], 1.f, false);
            else
              put<E>(grad_W + t * p.hidden + at, acc[c], p.scale, p.accumulate != 0);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[c][e] = 0.f;
          }
        }
      }
      if (last && !ends && !leading && slice == 0 && threadIdx.x == 0) {
        const int64_t far = (tile + kShortRun) * kTile;
        if (far < p.rows && p.sorted[far] == t)
          p.joins[1 + tiles - atomicAdd(p.joins + 1, 1u)] = static_cast<uint32_t>(tile);
        else
          p.joins[2 + atomicAdd(p.joins, 1u)] = static_cast<uint32_t>(tile);
      }
      if (ends) leading = false;
    }
  }
}

// Joins the sums of runs that cross tiles, from two lists, whose order means nothing. The first `shorts`
// CTAs take those that reach into less than kShortRun tiles more: E columns of a run for each thread. The others
// take long ones, of which there are few (a text's most frequent tokens): 32 E columns of a run for each CTA,
// every kJoinWarps-th tile for a warp, whose sums are added in order. What this costs is loads that wait for
// loads. (32768 tokens of a text's frequencies, 4096 columns: 39 us with a CTA for each tile and 512 columns
// and a binary search for the run's end, 11 us so.)
template <int E>
__global__ void __launch_bounds__(32 * kJoinWarps) embedding_join_kernel(const EmbeddingParams p, const int shorts, const int64_t tiles) {
  __shared__ float sums[kJoinWarps][32 * E];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto add = [&](const float* from, float (&v)[E]) {
    if constexpr (E == 1) {
      v[0] += *from;
    } else {
      const float4 f = *reinterpret_cast<const float4*>(from);
      v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
    }
  };
  float* out = static_cast<float*>(p.out);
  if (static_cast<int>(blockIdx.x) < shorts) {
    const int blocks = static_cast<int>((p.hidden + 32 * kJoinWarps * E - 1) / (32 * kJoinWarps * E));
    const int64_t col = (static_cast<int64_t>(blockIdx.x % blocks) * (32 * kJoinWarps) + threadIdx.x) * E;
    const uint32_t runs = p.joins[0];
    for (uint32_t k = blockIdx.x / blocks; k < runs; k += shorts / blocks) {
      const int64_t tile = p.joins[2 + k];
      const uint32_t t = p.sorted[(tile + 1) * kTile - 1];
      // tiles that begin in the run, less than kShortRun
      const int64_t first = (tile + 1 + lane) * kTile;
      const int n = __popc(__ballot_sync(0xffffffffu, lane < kShortRun && first < p.rows && p.sorted[first] == t));
      if (col < p.hidden) {
        float acc[E] = {};
        add(p.tail + tile * p.hidden + col, acc);
#pragma unroll 8
        for (int i = 0; i < n; ++i) add(p.head + (tile + 1 + i) * p.hidden + col, acc);
        put<E>(out + t * p.hidden + col, acc, p.scale, p.accumulate != 0);
      }
    }
    return;
  }
  const int longs = static_cast<int>(gridDim.x) - shorts, mine = static_cast<int>(blockIdx.x) - shorts;
  const int blocks = static_cast<int>((p.hidden + 32 * E - 1) / (32 * E));
  const int64_t col = (static_cast<int64_t>(mine % blocks) * 32 + lane) * E;
  const uint32_t runs = p.joins[1];
  for (uint32_t k = mine / blocks; k < runs; k += longs / blocks) {
    const int64_t tile = p.joins[1 + tiles - k];
    const uint32_t t = p.sorted[(tile + 1) * kTile - 1];
    int64_t n = 0;
    while (true) {
      const int64_t first = (tile + 1 + n + threadIdx.x) * kTile;
      const int more = __syncthreads_count(first < p.rows && p.sorted[first] == t);
      n += more;
      if (more < 32 * kJoinWarps) break;
    }
    float acc[E] = {};
    if (col < p.hidden) {
      if (warp == 0) add(p.tail + tile * p.hidden + col, acc);
#pragma unroll 8
      for (int64_t i = warp; i < n; i += kJoinWarps) add(p.head + (tile + 1 + i) * p.hidden + col, acc);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sums[warp][e * 32 + lane] = acc[e];
    __syncthreads();
    if (warp == 0 && col < p.hidden) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        for (int w = 1; w < kJoinWarps; ++w) acc[e] += sums[w][e * 32 + lane];
      put<E>(out + t * p.hidden + col, acc, p.scale, p.accumulate != 0);
    }
    __syncthreads();
  }
}

inline bool on_vectors(const void* p, int64_t ld, size_t es, int E) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % E == 0 && es * E == 16;
}

template <typename TI, typename TO>
cudaError_t run_forward(const EmbeddingParams& p, cudaStream_t s) {
  constexpr int E = 16 / sizeof(TI);
  const bool vectors = p.hidden % E == 0 && on_vectors(p.in, p.ld, sizeof(TI), E) && reinterpret_cast<uintptr_t>(p.out) % 16 == 0;
  const int64_t per = 32LL * (vectors ? kVectors<E> * E : kVectors<1>);
  const int64_t chunks = (p.hidden + per - 1) / per, ctas = (p.rows * chunks + kThreads / 32 - 1) / (kThreads / 32);
  if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  if (vectors)
    embedding_kernel<TI, TO, E><<<static_cast<unsigned>(ctas), kThreads, 0, s>>>(p, chunks);
  else
    embedding_kernel<TI, TO, 1><<<static_cast<unsigned>(ctas), kThreads, 0, s>>>(p, chunks);
  return cudaGetLastError();
}

cudaError_t launch_merge_shared(const EmbeddingParams& p, int64_t runs, int group, int sms, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  if (!(done.load() >> (dev & 63) & 1)) {
    const cudaError_t e =
        cudaFuncSetAttribute(embedding_merge_shared_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared * kChunk * 4);
    if (e != cudaSuccess) return e;
    done.fetch_or(1ull << (dev & 63));
  }
  // one round of CTAs, each with a warp's keys at least
  const int64_t groups = (runs + group - 1) / group, each = sms / groups > 0 ? sms / groups : 1, most = static_cast<int64_t>(group) * kChunk / 32;
  const dim3 grid(static_cast<unsigned>(each < most ? each : most), static_cast<unsigned>(groups));
  embedding_merge_shared_kernel<<<grid, kSharedThreads, static_cast<size_t>(group) * kChunk * 4, s>>>(p.sorted, p.places, p.sorted2, p.places2, p.rows, group);
  return cudaGetLastError();
}

template <typename T, int E, int C>
int run_grad(const EmbeddingParams& p, cudaStream_t stream) {
  const int64_t tiles = (p.rows + kTile - 1) / kTile;
  constexpr int64_t columns = static_cast<int64_t>(kGradThreads) * E * C;
  const int64_t slices = (p.hidden + columns - 1) / columns;
  int zero_rows = 0;
  int64_t ctas = tiles * slices;
  if (!p.accumulate) {
    int64_t z = kZeroFloats / p.hidden;
    zero_rows = static_cast<int>(z < 1 ? 1 : z > kGradThreads ? kGradThreads : z);
    ctas += (p.vocab + zero_rows - 1) / zero_rows;
  }
  if (ctas == 0) return FLCE_OK;
  FLCE_LAUNCH(K_EMBEDDING_GRAD, (embedding_grad_kernel<T, E, C><<<static_cast<unsigned>(ctas), kGradThreads, 0, stream>>>(
                                     p, tiles, static_cast<int>(slices), zero_rows),
                                 cudaGetLastError()));
  if (tiles > 1) {
    constexpr int JE = E > 1 ? 4 : 1;
    // whole rounds of a run's blocks of columns in either part
    const int64_t short_blocks = (p.hidden + 32 * kJoinWarps * JE - 1) / (32 * kJoinWarps * JE), long_blocks = (p.hidden + 32 * JE - 1) / (32 * JE);
    int64_t at_once = kJoinCtas / short_blocks + 1;
    if (at_once > tiles - 1) at_once = tiles - 1;
    const int64_t shorts = at_once * short_blocks, longs = tiles > kShortRun ? kLongRuns * long_blocks : 0;
    FLCE_LAUNCH(K_EMBEDDING_GRAD, (embedding_join_kernel<JE><<<static_cast<unsigned>(shorts + longs), 32 * kJoinWarps, 0, stream>>>(
                                       p, static_cast<int>(shorts), tiles),
                                   cudaGetLastError()));
  }
  return FLCE_OK;
}

template <typename T>
int run_grad_typed(const EmbeddingParams& p, cudaStream_t s) {
  constexpr int E = 16 / sizeof(T);
  if (p.hidden % E == 0 && on_vectors(p.in, p.ld, sizeof(T), E) && reinterpret_cast<uintptr_t>(p.out) % 16 == 0)
    return run_grad<T, E, 1>(p, s);
  return run_grad<T, 1, 4>(p, s);
}

}  // namespace

cudaError_t launch_embedding(const EmbeddingParams& p, cudaStream_t s) {
  if (p.dtype == FLCE_DTYPE_F32)
    return p.out_dtype == FLCE_DTYPE_F32 ? run_forward<float, float>(p, s) : run_forward<float, uint16_t>(p, s);
  return p.out_dtype == FLCE_DTYPE_F32 ? run_forward<uint16_t, float>(p, s) : run_forward<uint16_t, uint16_t>(p, s);
}

int launch_embedding_sort(EmbeddingParams* p, int sms, cudaStream_t stream) {
  const int64_t chunks = (p->rows + kChunk - 1) / kChunk;
  FLCE_LAUNCH(K_EMBEDDING_SORT, (embedding_chunk_kernel<<<static_cast<unsigned>(chunks), kChunk, 0, stream>>>(
                                     p->tokens, p->rows, p->vocab, p->sorted, p->places, p->joins),
                                 cudaGetLastError()));
  for (int64_t run = kChunk; run < p->rows;) {
    const int64_t runs = (p->rows + run - 1) / run;
    const bool shared = run == kChunk;
    const int group = static_cast<int>(shared ? (runs <= kMostShared ? runs : kSharedGroup) : runs < 8 ? runs : 8);
    if (shared)
      FLCE_LAUNCH(K_EMBEDDING_SORT, launch_merge_shared(*p, runs, group, sms, stream));
    else
      FLCE_LAUNCH(K_EMBEDDING_SORT,
                (embedding_merge_kernel<<<static_cast<unsigned>((p->rows + kThreads - 1) / kThreads), kThreads, 0, stream>>>(
                     p->sorted, p->places, p->sorted2, p->places2, p->rows, run, group),
                 cudaGetLastError()));
    uint32_t* t = p->sorted;
    p->sorted = p->sorted2;
    p->sorted2 = t;
    t = p->places;
    p->places = p->places2;
    p->places2 = t;
    run *= group;
  }
  return FLCE_OK;
}

int launch_embedding_grad(const EmbeddingParams& p, cudaStream_t s) {
  return p.dtype == FLCE_DTYPE_F32 ? run_grad_typed<float>(p, s) : run_grad_typed<uint16_t>(p, s);
}

}  // namespace flce
