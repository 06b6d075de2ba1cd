// 8-bit checkpoints of activations: store and read back (checkpoint_device.cuh has the
// format). Both are copies with little arithmetic, bound by memory.
//
// A warp takes several vectors per lane, so that that many loads are in flight. Rows
// of a multiple of 32 elements without gaps are one long row, whose blocks do not know
// where a row ends; other rows are cut into chunks of a warp each.
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
  const int64_t chunks = (p.hidden / E + 32 * kUnroll - 1) / (32 * kUnroll);
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
  const bool vectors = p.hidden % E == 0 && at % 16 == 0 && (!STORE || p.ld % E == 0 || p.rows == 1) && reinterpret_cast<uintptr_t>(p.codes) % E == 0;
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
