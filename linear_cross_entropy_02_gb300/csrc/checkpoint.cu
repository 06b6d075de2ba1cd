// 8-bit checkpoints of activations: store and read back (checkpoint_device.cuh has the
// format). Both are copies with little arithmetic, bound by memory.
//
// A warp takes several vectors per lane, so that that many loads are in flight. Rows
// of a multiple of 32 elements without gaps are one long row, whose blocks do not know
// where a row ends. Other rows are stored in chunks of a warp each, or several short rows by
// a warp, and read back in whole vectors all the same, as codes and values of all rows lie end to
// end: a vector takes the scales of the blocks that it has part in.
#include "checkpoint_device.cuh"
#include "model_internal.h"

namespace flce {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

// `chunks` warps per row, each of kUnroll vectors per lane.
template <typename T, int E>
__global__ void __launch_bounds__(kThreads) checkpoint_store_kernel(const CheckpointParams p, const int64_t chunks) {
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
  if (unit >= p.rows * chunks) return;
  const int64_t row = unit / chunks, first = (unit - row * chunks) * (32 * kUnroll) + (threadIdx.x & 31), vecs = p.hidden / E;
  const T* x = static_cast<const T*>(p.x) + row * p.ld;
  Raw<T, E> raw[kUnroll];
#pragma unroll
  for (int j = 0; j < kUnroll; ++j)
    if (first + j * 32 < vecs) raw[j] = load_raw<T, E>(x + (first + j * 32) * E);
#pragma unroll
  for (int j = 0; j < kUnroll; ++j)
    keep_vector<T, E>(raw[j], first + j * 32, first + j * 32 < vecs, 32, p.codes, p.scales, row, p.hidden);
}

// Rows of up to 16 vectors: a row per group of `lanes` lanes, kUnroll groups' worth of rows a warp.
template <typename T, int E>
__global__ void __launch_bounds__(kThreads) checkpoint_store_short_kernel(const CheckpointParams p, const int lanes) {
  const int per = 32 / lanes, lane = threadIdx.x & 31, vec = lane & (lanes - 1);
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32) * (per * kUnroll) + lane / lanes;
  const int vecs = static_cast<int>(p.hidden) / E;
  Raw<T, E> raw[kUnroll];
#pragma unroll
  for (int j = 0; j < kUnroll; ++j)
    if (first + j * per < p.rows && vec < vecs) raw[j] = load_raw<T, E>(static_cast<const T*>(p.x) + (first + j * per) * p.ld + vec * E);
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    const int64_t row = first + j * per;
    keep_vector<T, E>(raw[j], vec, row < p.rows && vec < vecs, lanes, p.codes, p.scales, row, p.hidden);
  }
}

// Vectors of the whole matrix, whatever rows and blocks they reach into. I: 32 bits where they hold an element's index.
template <typename T, int E, typename I>
__global__ void __launch_bounds__(kThreads) checkpoint_load_flat_kernel(const CheckpointParams p) {
  const int64_t all = p.rows * p.hidden;
  const int64_t base = ((static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32) * (32 * kUnroll) + (threadIdx.x & 31)) * E;
  const int hidden = static_cast<int>(p.hidden);
  const int64_t blocks = checkpoint_blocks(p.hidden);
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    const int64_t at = base + j * 32 * E;
    if (at >= all) return;
    uint32_t words[E == 8 ? 2 : 1] = {};
    const int n = at + E <= all ? E : static_cast<int>(all - at);
    if (n == E) {
      if constexpr (E == 8) {
        const uint2 w = *reinterpret_cast<const uint2*>(p.codes + at);
        words[0] = w.x;
        words[1] = w.y;
      } else {
        words[0] = *reinterpret_cast<const uint32_t*>(p.codes + at);
      }
    } else {
      for (int e = 0; e < n; ++e) words[e / 4] |= static_cast<uint32_t>(p.codes[at + e]) << (e % 4 * 8);
    }
    const I row = static_cast<I>(at) / static_cast<I>(hidden);
    int col = static_cast<int>(static_cast<I>(at) - row * static_cast<I>(hidden));
    const uint8_t* byte = p.scales + static_cast<int64_t>(row) * blocks + col / kCheckpointBlock;  // (the next block's is the next byte)
    float scale = scale_value(*byte), f[E];
    read_codes<E>(words, 1.f, f);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      f[e] *= scale;
      ++col;
      if (e + 1 < n && (col % kCheckpointBlock == 0 || col == hidden)) {
        if (col == hidden) col = 0;
        scale = scale_value(*++byte);
      }
    }
    T* out = static_cast<T*>(p.out) + at;
    if (n == E) {
      store_raw<T, E>(out, pack<T, E>(f));
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (e < n) out[e] = from_float<T>(f[e]);
    }
  }
}

template <typename T, int E>
__global__ void __launch_bounds__(kThreads) checkpoint_load_kernel(const CheckpointParams p, const int64_t chunks) {
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
  if (unit >= p.rows * chunks) return;
  const int64_t row = unit / chunks, first = (unit - row * chunks) * (32 * kUnroll) + (threadIdx.x & 31), vecs = p.hidden / E;
  const uint8_t* codes = p.codes + row * p.hidden;
  const uint8_t* scales = p.scales + row * checkpoint_blocks(p.hidden);
  uint32_t words[kUnroll][E == 8 ? 2 : 1];
  uint32_t byte[kUnroll];
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    const int64_t v = first + j * 32;
    if (v < vecs) {
      if constexpr (E == 8) {
        const uint2 w = *reinterpret_cast<const uint2*>(codes + v * E);
        words[j][0] = w.x;
        words[j][1] = w.y;
      } else if constexpr (E == 4) {
        words[j][0] = *reinterpret_cast<const uint32_t*>(codes + v * E);
      } else {
        words[j][0] = codes[v];
      }
      byte[j] = scales[v * E / kCheckpointBlock];
    }
  }
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    const int64_t v = first + j * 32;
    if (v < vecs) {
      float f[E];
      read_codes<E>(words[j], scale_value(byte[j]), f);
      store_raw<T, E>(static_cast<T*>(p.out) + row * p.hidden + v * E, pack<T, E>(f));
    }
  }
}

template <typename T, int E, bool STORE>
cudaError_t run(CheckpointParams p, cudaStream_t s) {
  if (p.hidden % kCheckpointBlock == 0 && (!STORE || p.ld == p.hidden || p.rows == 1)) {
    p.hidden *= p.rows;
    p.rows = 1;
  }
  const int64_t vecs = p.hidden / E;
  if constexpr (STORE) {
    if (vecs <= 16 && p.rows > 1) {
      int lanes = 1;
      while (lanes < vecs) lanes *= 2;
      const int64_t per = static_cast<int64_t>(kThreads / lanes) * kUnroll;
      checkpoint_store_short_kernel<T, E><<<static_cast<unsigned>((p.rows + per - 1) / per), kThreads, 0, s>>>(p, lanes);
      return cudaGetLastError();
    }
  } else if constexpr (E > 1) {
    // (both ways, stored and read back: 20000 x 1337 bf16 76 us so, 94 by single elements; 100000 x 72 23, 45 with a
    // warp for each row; but 30000 x 1000 43, 33 by rows)
    if (p.rows > 1 && (p.hidden % E != 0 || vecs <= 64)) {
      const int64_t all = p.rows * p.hidden, per = static_cast<int64_t>(kThreads) * kUnroll * E, ctas = (all + per - 1) / per;
      if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
      if (all < (int64_t{1} << 31))
        checkpoint_load_flat_kernel<T, E, uint32_t><<<static_cast<unsigned>(ctas), kThreads, 0, s>>>(p);
      else
        checkpoint_load_flat_kernel<T, E, uint64_t><<<static_cast<unsigned>(ctas), kThreads, 0, s>>>(p);
      return cudaGetLastError();
    }
  }
  const int64_t chunks = (vecs + 32 * kUnroll - 1) / (32 * kUnroll);
  const int64_t ctas = (p.rows * chunks + kThreads / 32 - 1) / (kThreads / 32);
  if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  if constexpr (STORE)
    checkpoint_store_kernel<T, E><<<static_cast<unsigned>(ctas), kThreads, 0, s>>>(p, chunks);
  else
    checkpoint_load_kernel<T, E><<<static_cast<unsigned>(ctas), kThreads, 0, s>>>(p, chunks);
  return cudaGetLastError();
}

template <typename T, bool STORE>
cudaError_t run_typed(const CheckpointParams& p, cudaStream_t s) {
  constexpr int E = 16 / sizeof(T);
  const uintptr_t at = reinterpret_cast<uintptr_t>(STORE ? p.x : p.out);
  // (what is read back lies end to end whatever the rows' length)
  const bool vectors = (p.hidden % E == 0 || (!STORE && p.rows > 1)) && at % 16 == 0 && (!STORE || p.ld % E == 0 || p.rows == 1) && reinterpret_cast<uintptr_t>(p.codes) % E == 0;
  return vectors ? run<T, E, STORE>(p, s) : run<T, 1, STORE>(p, s);
}

}  // namespace

cudaError_t launch_checkpoint_store(const CheckpointParams& p, cudaStream_t s) {
  return p.dtype == FLCE_DTYPE_F32 ? run_typed<float, true>(p, s) : run_typed<uint16_t, true>(p, s);
}

cudaError_t launch_checkpoint_load(const CheckpointParams& p, cudaStream_t s) {
  return p.dtype == FLCE_DTYPE_F32 ? run_typed<float, false>(p, s) : run_typed<uint16_t, false>(p, s);
}

}  // namespace flce
