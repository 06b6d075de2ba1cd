// Layer norm and RMS norm in front of the head, forward and backward.
//
// Both directions are bound by memory: the forward reads and writes N H
// elements, the backward reads 2 N H and writes N H, with about ten operations
// for each. A row stays on chip between the pass that takes its statistics and
// the pass that uses them, so that HBM sees each element once:
//   rows of up to 128 16-byte vectors   one warp per row, no block barrier
//   longer rows                         one CTA per row, C vectors per thread
//   rows beyond that (or 8192 unaligned elements)   three passes through the L2
// A CTA keeps taking rows (grid = what the SMs hold at once): the next row's
// vectors are on their way while the current row's sums go through the
// barrier, and the backward adds up its columns of the weight's gradient in
// registers over all its rows. Those per-CTA sums go to the workspace once and
// a second kernel adds them in a fixed order; no atomics, so the gradient is
// the same in every run.
//
// The variance is the mean of the squared distances from the mean, from
// registers, not mean(x^2) - mean^2, which cancels for rows with an offset. The
// same sums carry the mean of those distances, which is what rounding the mean
// has left, and take it out again: rows whose deviation is small beside their
// offset keep their digits.
#include <math.h>

#include <atomic>

#include "head_device.cuh"
#include "head_internal.h"

namespace flce {

namespace {

// Vectors per thread and threads per CTA of the three kinds of rows.
// E = 8: bf16 vectors, E = 4: fp32 vectors, E = 1: elements.
constexpr int cta_vecs(int E) { return E == 8 ? 2 : E == 4 ? 4 : 8; }
constexpr int warp_vecs(int E) { return E == 8 ? 4 : 8; }
constexpr int kWarpRowThreads = 256;  // eight rows per CTA
constexpr int kMaxThreads = 1024;

// Sums of a and b over the CTA, in every thread. `slot` alternates between 0
// and 1 from call to call: the barrier of the call between keeps a slot's
// readers ahead of its next writers.
__device__ __forceinline__ void block_sum2(float& a, float& b, float2* smem, int& slot) {
  a = warp_sum(a);
  b = warp_sum(b);
  float2* s = smem + slot * 32;
  slot ^= 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) s[warp] = make_float2(a, b);
  __syncthreads();
  const int warps = blockDim.x >> 5;
  const float2 v = lane < warps ? s[lane] : make_float2(0.f, 0.f);
  a = warp_sum(v.x);
  b = warp_sum(v.y);
}

template <bool WARP>
__device__ __forceinline__ void row_sum2(float& a, float& b, float2* smem, int& slot) {
  if (WARP) {
    a = warp_sum(a);
    b = warp_sum(b);
  } else {
    block_sum2(a, b, smem, slot);
  }
}

template <typename T, int E, int C, bool WARP>
__global__ void __launch_bounds__(WARP ? kWarpRowThreads : kMaxThreads) norm_kernel(const NormParams p) {
  __shared__ float2 sums[64];
  int slot = 0;
  const int H = static_cast<int>(p.hidden);
  const int vecs = H / E;
  const int tpr = WARP ? 32 : blockDim.x;
  const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int per = WARP ? kWarpRowThreads / 32 : 1;
  const int64_t step = static_cast<int64_t>(gridDim.x) * per;
  const T* x = static_cast<const T*>(p.x);
  T* y = static_cast<T*>(p.out);
  const float inv_h = 1.f / static_cast<float>(H);
  Raw<T, E> next[C];
  int64_t row = static_cast<int64_t>(blockIdx.x) * per + (WARP ? threadIdx.x >> 5 : 0);
  if (row < p.rows) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (t + c * tpr < vecs) next[c] = load_raw<T, E>(x + row * p.ld_x + (t + c * tpr) * E);
  }
  for (; row < p.rows; row += step) {
    Raw<T, E> cur[C];
#pragma unroll
    for (int c = 0; c < C; ++c) cur[c] = next[c];
    if (row + step < p.rows) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (t + c * tpr < vecs) next[c] = load_raw<T, E>(x + (row + step) * p.ld_x + (t + c * tpr) * E);
    }
    float mean = 0.f, none = 0.f;
    if (!p.rms) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (t + c * tpr < vecs) {
          float v[E];
          unpack<T, E>(cur[c], v);
#pragma unroll
          for (int e = 0; e < E; ++e) mean += v[e];
        }
      }
      row_sum2<WARP>(mean, none, sums, slot);
      mean *= inv_h;
    }
    float sq = 0.f, rest = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (t + c * tpr < vecs) {
        float v[E];
        unpack<T, E>(cur[c], v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float d = v[e] - mean;
          rest += d;
          sq += d * d;
        }
      }
    }
    row_sum2<WARP>(sq, rest, sums, slot);
    rest = p.rms ? 0.f : rest * inv_h;
    const float rstd = 1.f / sqrtf(fmaxf(sq * inv_h - rest * rest, 0.f) + p.eps);
    if (t == 0) {
      if (p.mean && !p.rms) p.mean[row] = mean + rest;
      if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = (t + c * tpr) * E;
      if (t + c * tpr < vecs) {
        float v[E], w[E];
        unpack<T, E>(cur[c], v);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = (v[e] - mean - rest) * rstd;
        if (p.weight) {
          load_weight<E>(p.weight, p.w_f32 != 0, i, w);
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] *= w[e];
        }
        if (p.bias) {
          load_weight<E>(p.bias, p.w_f32 != 0, i, w);
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] += w[e];
        }
        store_raw<T, E>(y + row * p.hidden + i, pack<T, E>(v));
      }
    }
  }
}

// Rows that no register file holds: a CTA per row, which is read three times.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) norm_long_kernel(const NormParams p) {
  __shared__ float2 sums[64];
  int slot = 0;
  const int H = static_cast<int>(p.hidden);
  const float inv_h = 1.f / static_cast<float>(H);
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.ld_x;
    T* y = static_cast<T*>(p.out) + row * p.hidden;
    float mean = 0.f, none = 0.f;
    if (!p.rms) {
      for (int i = threadIdx.x; i < H; i += blockDim.x) mean += to_float<T>(x[i]);
      block_sum2(mean, none, sums, slot);
      mean *= inv_h;
    }
    float sq = 0.f, rest = 0.f;
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
      const float d = to_float<T>(x[i]) - mean;
      rest += d;
      sq += d * d;
    }
    block_sum2(sq, rest, sums, slot);
    rest = p.rms ? 0.f : rest * inv_h;
    const float rstd = 1.f / sqrtf(fmaxf(sq * inv_h - rest * rest, 0.f) + p.eps);
    if (threadIdx.x == 0) {
      if (p.mean && !p.rms) p.mean[row] = mean + rest;
      if (p.rstd) p.rstd[row] = rstd;
    }
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
      float v[1] = {(to_float<T>(x[i]) - mean - rest) * rstd}, w[1];
      if (p.weight) {
        load_weight<1>(p.weight, p.w_f32 != 0, i, w);
        v[0] *= w[0];
      }
      if (p.bias) {
        load_weight<1>(p.bias, p.w_f32 != 0, i, w);
        v[0] += w[0];
      }
      y[i] = from_float<T>(v[0]);
    }
  }
}

// ------------------------------------------------------------------ backward
// A ring of `stages` rows of x and grad_y in shared memory, filled by copies
// that each thread issues for its own vectors and reads back itself: they keep
// two rows beyond the current one in flight without holding registers and
// without a barrier. Single bf16 elements are too small for such a copy and are
// loaded directly (stages is not used).
template <typename T, int E, int C, bool WARP, int NB>
__global__ void __launch_bounds__(WARP ? kWarpRowThreads : kMaxThreads)
    norm_bwd_kernel(const NormParams p, const int stages) {
  constexpr bool RING = sizeof(T) * E >= 4;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ float2 sums[64];
  int slot = 0;
  Raw<T, E>* ring = reinterpret_cast<Raw<T, E>*>(dyn);
  const int H = static_cast<int>(p.hidden);
  const int vecs = H / E;
  const int tpr = WARP ? 32 : blockDim.x;
  const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int per = WARP ? kWarpRowThreads / 32 : 1;
  const int64_t step = static_cast<int64_t>(gridDim.x) * per;
  const T* x = static_cast<const T*>(p.x);
  const T* gy = static_cast<const T*>(p.gy);
  T* gx = static_cast<T*>(p.out);
  const float inv_h = 1.f / static_cast<float>(H);
  float acc_w[C][E], acc_b[C][E];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < E; ++e) acc_w[c][e] = acc_b[c][e] = 0.f;

  auto at = [&](int stage, int which, int c) { return ((stage * 2 + which) * C + c) * blockDim.x + threadIdx.x; };
  auto fetch = [&](int64_t r, int stage) {
    if (RING && r < p.rows) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (t + c * tpr < vecs) {
          copy_async<RING ? static_cast<int>(sizeof(T) * E) : 4>(&ring[at(stage, 0, c)],
                                                                 x + r * p.ld_x + (t + c * tpr) * E);
          copy_async<RING ? static_cast<int>(sizeof(T) * E) : 4>(&ring[at(stage, 1, c)],
                                                                 gy + r * p.ld_gy + (t + c * tpr) * E);
        }
      }
    }
    if (RING) copies_commit();
  };

  int64_t row = static_cast<int64_t>(blockIdx.x) * per + (WARP ? threadIdx.x >> 5 : 0);
  for (int i = 0; i < stages - 1; ++i) fetch(row + i * step, i);
  int stage = 0, fill = stages - 1;
  for (; row < p.rows; row += step) {
    Raw<T, E> rx[C], rg[C];
    const float mean = p.rms ? 0.f : __ldg(p.mean + row);
    const float rstd = __ldg(p.rstd + row);
    if (RING) {
      fetch(row + (stages - 1) * step, fill);
      if (stages == 3)
        copies_wait<2>();
      else if (stages == 2)
        copies_wait<1>();
      else
        copies_wait<0>();
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (t + c * tpr < vecs) {
          rx[c] = ring[at(stage, 0, c)];
          rg[c] = ring[at(stage, 1, c)];
        }
      }
      if (++stage == stages) stage = 0;
      if (++fill == stages) fill = 0;
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (t + c * tpr < vecs) {
          rx[c] = load_raw<T, E>(x + row * p.ld_x + (t + c * tpr) * E);
          rg[c] = load_raw<T, E>(gy + row * p.ld_gy + (t + c * tpr) * E);
        }
      }
    }
    float sg = 0.f, sgx = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (t + c * tpr < vecs) {
        float xv[E], gv[E], w[E];
        unpack<T, E>(rx[c], xv);
        unpack<T, E>(rg[c], gv);
        if (p.weight) load_weight<E>(p.weight, p.w_f32 != 0, (t + c * tpr) * E, w);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float xhat = (xv[e] - mean) * rstd;
          const float g = p.weight ? gv[e] * w[e] : gv[e];
          sg += g;
          sgx += g * xhat;
          acc_w[c][e] += gv[e] * xhat;
          if (NB == 2) acc_b[c][e] += gv[e];
        }
      }
    }
    if (gx == nullptr) continue;  // uniform over the grid
    row_sum2<WARP>(sg, sgx, sums, slot);
    sg = p.rms ? 0.f : sg * inv_h;
    sgx *= inv_h;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (t + c * tpr < vecs) {
        float xv[E], gv[E], w[E];
        unpack<T, E>(rx[c], xv);
        unpack<T, E>(rg[c], gv);
        if (p.weight) load_weight<E>(p.weight, p.w_f32 != 0, (t + c * tpr) * E, w);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float xhat = (xv[e] - mean) * rstd;
          const float g = p.weight ? gv[e] * w[e] : gv[e];
          xv[e] = rstd * (g - sg - xhat * sgx);
        }
        store_raw<T, E>(gx + row * p.hidden + (t + c * tpr) * E, pack<T, E>(xv));
      }
    }
  }
  if (RING) copies_wait<0>();

  // This CTA's sums of its columns. Eight warps with rows of their own add up
  // through shared memory first, in the order of the warps.
#pragma unroll
  for (int which = 0; which < NB; ++which) {
    float* part = which == 0 ? p.part_w : p.part_b;
    if (part == nullptr) continue;
    part += static_cast<int64_t>(blockIdx.x) * p.hidden;
    float* comb = reinterpret_cast<float*>(dyn);
    if (WARP) __syncthreads();
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (t + c * tpr < vecs) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float v = which == 0 ? acc_w[c][e] : acc_b[c][e];
          const int i = (t + c * tpr) * E + e;
          if (WARP)
            comb[(threadIdx.x >> 5) * H + i] = v;
          else
            part[i] = v;
        }
      }
    }
    if (WARP) {
      __syncthreads();
      for (int i = threadIdx.x; i < H; i += blockDim.x) {
        float v = 0.f;
        for (int w = 0; w < per; ++w) v += comb[w * H + i];
        part[i] = v;
      }
    }
  }
}

// Long rows: grad_x by a CTA per row in two passes through the L2.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_long_kernel(const NormParams p) {
  __shared__ float2 sums[64];
  int slot = 0;
  const int H = static_cast<int>(p.hidden);
  const float inv_h = 1.f / static_cast<float>(H);
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.ld_x;
    const T* gy = static_cast<const T*>(p.gy) + row * p.ld_gy;
    T* gx = static_cast<T*>(p.out) + row * p.hidden;
    const float mean = p.rms ? 0.f : p.mean[row], rstd = p.rstd[row];
    float sg = 0.f, sgx = 0.f, w[1] = {1.f};
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
      if (p.weight) load_weight<1>(p.weight, p.w_f32 != 0, i, w);
      const float g = to_float<T>(gy[i]) * w[0];
      sg += g;
      sgx += g * ((to_float<T>(x[i]) - mean) * rstd);
    }
    block_sum2(sg, sgx, sums, slot);
    sg = p.rms ? 0.f : sg * inv_h;
    sgx *= inv_h;
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
      if (p.weight) load_weight<1>(p.weight, p.w_f32 != 0, i, w);
      const float g = to_float<T>(gy[i]) * w[0];
      gx[i] = from_float<T>(rstd * (g - sg - (to_float<T>(x[i]) - mean) * rstd * sgx));
    }
  }
}

// Long rows: the partial sums of row group blockIdx.y, a thread per column.
template <typename T>
__global__ void __launch_bounds__(256) norm_bwd_long_cols_kernel(const NormParams p, const int64_t group) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= p.hidden) return;
  const T* x = static_cast<const T*>(p.x);
  const T* gy = static_cast<const T*>(p.gy);
  const int64_t r0 = blockIdx.y * group, r1 = min(r0 + group, p.rows);
  float w = 0.f, b = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const float g = to_float<T>(gy[r * p.ld_gy + i]);
    w += g * ((to_float<T>(x[r * p.ld_x + i]) - (p.rms ? 0.f : __ldg(p.mean + r))) * __ldg(p.rstd + r));
    b += g;
  }
  if (p.part_w) p.part_w[blockIdx.y * p.hidden + i] = w;
  if (p.part_b) p.part_b[blockIdx.y * p.hidden + i] = b;
}

// 32 columns per CTA, 32 threads on each: thread k takes partial rows k, k + 32, ...
// and the 32 sums are added in order.
__global__ void __launch_bounds__(1024) norm_wgrad_kernel(const float* part_w, const float* part_b, int partials,
                                                          int64_t hidden, float* grad_w, float* grad_b,
                                                          int accumulate, int32_t* status) {
  __shared__ float s[32][33];
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && threadIdx.y == 0) *status = 0;
  const float* part = blockIdx.y == 0 ? part_w : part_b;
  float* grad = blockIdx.y == 0 ? grad_w : grad_b;
  if (grad == nullptr) return;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
  float v = 0.f;
  if (col < hidden) {
#pragma unroll 4
    for (int i = threadIdx.y; i < partials; i += 32) v += part[i * hidden + col];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && col < hidden) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) a += s[i][threadIdx.x];
    grad[col] = accumulate ? grad[col] + a : a;
  }
}

inline bool aligned(const void* p, int64_t ld, size_t es) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * static_cast<int64_t>(es)) % 16 == 0);
}

enum RowKind { ROW_WARP, ROW_CTA, ROW_LONG };

struct Shape {
  bool vec;
  int E;
  RowKind kind;
  int threads;  // of a ROW_CTA
};

Shape shape_of(const NormParams& p) {
  const size_t es = p.dtype == FLCE_DTYPE_F32 ? 4 : 2;
  Shape s;
  s.vec = aligned(p.x, p.ld_x, es) && aligned(p.gy, p.ld_gy, es) && aligned(p.out, p.hidden, es) &&
          p.hidden % (16 / es) == 0 && aligned(p.weight, 0, 1) && aligned(p.bias, 0, 1);
  s.E = s.vec ? static_cast<int>(16 / es) : 1;
  const int64_t vecs = p.hidden / s.E;
  const int C = cta_vecs(s.E);
  s.kind = vecs <= 32 * warp_vecs(s.E) ? ROW_WARP : vecs <= static_cast<int64_t>(kMaxThreads) * C ? ROW_CTA : ROW_LONG;
  s.threads = static_cast<int>(((vecs + C - 1) / C + 31) / 32 * 32);
  return s;
}

constexpr size_t kRingBudget = 96 * 1024;  // two CTAs of an SM keep a ring each

inline unsigned grid_of(int64_t want, int64_t most) { return static_cast<unsigned>(want < most ? want : most); }

template <typename T, int E>
cudaError_t run_fwd(const NormParams& p, const Shape& h, int sms, cudaStream_t s) {
  if (h.kind == ROW_WARP) {
    norm_kernel<T, E, warp_vecs(E), true><<<grid_of((p.rows + 7) / 8, 4LL * sms), kWarpRowThreads, 0, s>>>(p);
  } else {
    norm_kernel<T, E, cta_vecs(E), false>
        <<<grid_of(p.rows, static_cast<int64_t>(sms) * (h.threads > 512 ? 1 : 1024 / h.threads)), h.threads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

template <typename T, int E, bool WARP, int NB>
cudaError_t run_bwd_typed(const NormParams& p, int threads, int stages, size_t smem, int grid, cudaStream_t s) {
  auto k = norm_bwd_kernel<T, E, WARP ? warp_vecs(E) : cta_vecs(E), WARP, NB>;
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  if (smem > 48 * 1024 && !(done.load() >> (dev & 63) & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    if (e != cudaSuccess) return e;
    done.fetch_or(1ull << (dev & 63));
  }
  k<<<grid, threads, smem, s>>>(p, stages);
  return cudaGetLastError();
}

template <typename T, int E>
cudaError_t run_bwd(const NormParams& p, const Shape& h, int sms, int* partials, cudaStream_t s) {
  const bool warp = h.kind == ROW_WARP;
  const int threads = warp ? kWarpRowThreads : h.threads;
  const int C = warp ? warp_vecs(E) : cta_vecs(E);
  const size_t stage = static_cast<size_t>(threads) * C * 2 * sizeof(Raw<T, E>);
  int stages = static_cast<int>(kRingBudget / stage);
  stages = stages > 3 ? 3 : stages < 1 ? 1 : stages;
  size_t smem = stage * stages;
  const size_t comb = warp ? static_cast<size_t>(p.hidden) * (kWarpRowThreads / 32) * sizeof(float) : 0;
  if (comb > smem) smem = comb;
  int grid;
  if (warp)
    grid = static_cast<int>(grid_of((p.rows + 7) / 8, 2LL * sms));
  else
    grid = static_cast<int>(grid_of(p.rows, static_cast<int64_t>(sms) * (h.threads > 512 ? 1 : 2)));
  *partials = grid;
  if (warp)
    return p.part_b ? run_bwd_typed<T, E, true, 2>(p, threads, stages, smem, grid, s)
                    : run_bwd_typed<T, E, true, 1>(p, threads, stages, smem, grid, s);
  return p.part_b ? run_bwd_typed<T, E, false, 2>(p, threads, stages, smem, grid, s)
                  : run_bwd_typed<T, E, false, 1>(p, threads, stages, smem, grid, s);
}

}  // namespace

int norm_partial_rows(int64_t rows, int sms) { return static_cast<int>(rows < 2LL * sms ? rows : 2LL * sms); }

cudaError_t launch_norm(const NormParams& p, int sms, cudaStream_t s) {
  const Shape h = shape_of(p);
  const bool f32 = p.dtype == FLCE_DTYPE_F32;
  if (h.kind == ROW_LONG) {
    const unsigned grid = grid_of(p.rows, 2LL * sms);
    if (f32)
      norm_long_kernel<float><<<grid, kMaxThreads, 0, s>>>(p);
    else
      norm_long_kernel<uint16_t><<<grid, kMaxThreads, 0, s>>>(p);
    return cudaGetLastError();
  }
  if (f32) return h.vec ? run_fwd<float, 4>(p, h, sms, s) : run_fwd<float, 1>(p, h, sms, s);
  return h.vec ? run_fwd<uint16_t, 8>(p, h, sms, s) : run_fwd<uint16_t, 1>(p, h, sms, s);
}

cudaError_t launch_norm_bwd(const NormParams& p, int sms, int* partials, cudaStream_t s) {
  const Shape h = shape_of(p);
  const bool f32 = p.dtype == FLCE_DTYPE_F32;
  if (h.kind == ROW_LONG) {
    if (p.out) {
      const unsigned grid = grid_of(p.rows, 2LL * sms);
      if (f32)
        norm_bwd_long_kernel<float><<<grid, kMaxThreads, 0, s>>>(p);
      else
        norm_bwd_long_kernel<uint16_t><<<grid, kMaxThreads, 0, s>>>(p);
      if (cudaGetLastError() != cudaSuccess) return cudaErrorLaunchFailure;
    }
    const int groups = norm_partial_rows(p.rows, sms);
    const int64_t group = (p.rows + groups - 1) / groups;
    *partials = static_cast<int>((p.rows + group - 1) / group);
    if (!p.part_w && !p.part_b) return cudaSuccess;
    const dim3 grid(static_cast<unsigned>((p.hidden + 255) / 256), static_cast<unsigned>(*partials));
    if (f32)
      norm_bwd_long_cols_kernel<float><<<grid, 256, 0, s>>>(p, group);
    else
      norm_bwd_long_cols_kernel<uint16_t><<<grid, 256, 0, s>>>(p, group);
    return cudaGetLastError();
  }
  if (f32) return h.vec ? run_bwd<float, 4>(p, h, sms, partials, s) : run_bwd<float, 1>(p, h, sms, partials, s);
  return h.vec ? run_bwd<uint16_t, 8>(p, h, sms, partials, s) : run_bwd<uint16_t, 1>(p, h, sms, partials, s);
}

cudaError_t launch_norm_wgrad(const float* part_w, const float* part_b, int partials, int64_t hidden, float* grad_w,
                              float* grad_b, int accumulate, int32_t* status, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((hidden + 31) / 32), grad_b ? 2 : 1);
  norm_wgrad_kernel<<<grid, dim3(32, 32), 0, s>>>(part_w, part_b, partials, hidden, grad_w, grad_b, accumulate, status);
  return cudaGetLastError();
}

}  // namespace flce
