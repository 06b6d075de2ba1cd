// Kernels of layer norm and RMS norm, forward and backward, alone (norm.cu) and behind
// the residual's addition (add_norm.cu, add_norm_8bit.cu).
//
// Both directions are bound by memory: the forward reads and writes N H
// elements, the backward reads 2 N H and writes N H. A row stays in registers
// between the pass that takes its sums and the pass that uses them, so that HBM
// sees each element once.
//
// Forward: a small CTA per row (128 threads where a row has at most eight
// vectors for each), many of them on an SM and none of them staying for a second
// row. On 32768 x 7168 bf16 that is 138 us (6.8 TB/s, a plain copy's rate);
// persistent CTAs of 448 threads that load the next row ahead of time took 172
// to 215, however many barriers were saved. With fp32 weight and bias, 8192 x 6656
// bf16 takes 47 us (4.7 TB/s), bound by instructions and the L1. Rows of up to 128
// vectors take a warp each, or a part of one, without any barrier.
//
// Backward: the weight's gradient is a sum over rows, so here a CTA stays: a
// thread keeps its columns for all of its CTA's rows and adds their terms in
// registers. The rows after the current one are copied ahead of time into a ring
// of shared memory that each thread fills and reads for itself. What bounds it is
// instructions as much as bytes: all but two operations on an element are done in
// one visit before the row's sums are known. (Packed pairs, f32x2, were tried: the
// moves into register pairs cost what the arithmetic saved, 27 to 33 instructions
// an element against 12.) 32768 x 7168 bf16 RMS takes 252 us (5.6 TB/s of 3 N H),
// 10007 x 1337 fp32 with weight and bias 40. Per-CTA sums go to the workspace once
// and a second kernel adds them in a fixed order; no atomics, so the gradient is
// the same in every run.
//
// The variance is the mean of the squared distances from the mean, from
// registers, not mean(x^2) - mean^2, which cancels for rows with an offset. The
// same sums carry the mean of those distances, which is what rounding the mean
// has left, and take it out again: rows whose deviation is small beside their
// offset keep their digits.
#pragma once

#include <math.h>

#include <atomic>
#include <type_traits>

#include "checkpoint_device.cuh"
#include "head_device.cuh"
#include "head_internal.h"
#include "model_internal.h"

namespace flce {

namespace {

// What a kernel does beside the norm. kAdd: the row is x + residual, rounded to x's
// type, and may be written out or kept in 8 bits; backward, a gradient of that sum is
// added to grad_x. kAdd8: the same backward, from the 8-bit checkpoint of the sum.
constexpr int kPlain = 0, kAdd = 1, kAdd8 = 2;
template <int MODE>
using ParamsOf = std::conditional_t<MODE == kPlain, NormParams, AddNormParams>;

constexpr int kMaxVecs = 8;           // vectors per thread of a forward row
constexpr int kWarpRowThreads = 256;  // eight warps per CTA
constexpr int kMaxThreads = 1024;

// Backward: most vectors per thread of a CTA's row. E = 8: bf16 vectors, E = 4: fp32
// vectors, E = 1: elements (tensors whose rows lie differently to vector boundaries).
constexpr int cta_vecs(int E) { return E == 8 ? 2 : E == 4 ? 4 : 8; }

// Sums of two values (or only of the first) over the CTA, in every thread.
// `slot` alternates between 0 and 1 from call to call: the barrier of the call
// between keeps a slot's readers ahead of its next writers. After the barrier
// every thread adds up the warps' sums itself: for up to 16 warps a few wide
// reads are quicker than five more shuffles in a chain.
struct BlockSums {
  float4 v[2][2][8];  // [slot][which value][32 warps]
};
template <bool BOTH>
__device__ __forceinline__ void block_sum(float& a, float& b, BlockSums& smem, int& slot) {
  float4(&s)[2][8] = smem.v[slot];
  slot ^= 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  a = warp_sum(a);
  if (BOTH) b = warp_sum(b);
  if (lane == 0) {
    reinterpret_cast<float*>(s[0])[warp] = a;
    if (BOTH) reinterpret_cast<float*>(s[1])[warp] = b;
    // the rest of the last group of four
    if (warp == warps - 1) {
      for (int i = warps; i & 3; ++i) {
        reinterpret_cast<float*>(s[0])[i] = 0.f;
        if (BOTH) reinterpret_cast<float*>(s[1])[i] = 0.f;
      }
    }
  }
  __syncthreads();
  a = b = 0.f;
  for (int i = 0; i * 4 < warps; ++i) {
    const float4 v = s[0][i];
    a += (v.x + v.y) + (v.z + v.w);
    if (BOTH) {
      const float4 w = s[1][i];
      b += (w.x + w.y) + (w.z + w.w);
    }
  }
}

// Sum over groups of `lanes` (a power of two) lanes.
__device__ __forceinline__ float group_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 1 / sqrt(variance + eps): a variance just below zero is rounding, one that is not a number stays so (fmaxf would
// make zero of it, and numbers of the rest of its row).
__device__ __forceinline__ float inverse_deviation(float variance, float eps) { return 1.f / sqrtf((variance < 0.f ? 0.f : variance) + eps); }

// ------------------------------------------------------------------ forward
// A row held as C vectors per thread, `stride` apart: its statistics and y.
// sum(a, b, Both() or One()) sums a (and b) over the row's threads; vecs is 0 in
// threads without a row.
struct Both {
  static constexpr bool value = true;
};
struct One {
  static constexpr bool value = false;
};
template <typename T, int E, int C, int MODE, typename S>
__device__ __forceinline__ void norm_row(const ParamsOf<MODE>& p, const T* x, T* y, int64_t row, int t, int stride, int vecs,
                                         int lanes, S sum) {
  Raw<T, E> cur[C];
#pragma unroll
  for (int c = 0; c < C; ++c)
    if (t + c * stride < vecs) cur[c] = load_raw<T, E>(x + (t + c * stride) * E);
  if constexpr (MODE != kPlain) {
    // The norm sees the sum as it is kept, rounded once to the residual stream's type:
    // y is that of the norm of the written sum, and the backward pass needs no other.
    if (p.residual) {
      const T* res = static_cast<const T*>(p.residual) + row * p.ld_res;
      Raw<T, E> other[C];
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (t + c * stride < vecs) other[c] = load_raw<T, E>(res + (t + c * stride) * E);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (t + c * stride < vecs) {
          float v[E], r[E];
          unpack<T, E>(cur[c], v);
          unpack<T, E>(other[c], r);
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] += r[e];
          cur[c] = pack<T, E>(v);
        }
      }
    }
    if (p.sum) {
      T* out = static_cast<T*>(p.sum) + row * p.hidden;
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (t + c * stride < vecs) store_raw<T, E>(out + (t + c * stride) * E, cur[c]);
    }
    if (p.codes) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        keep_vector<T, E>(cur[c], t + c * stride, t + c * stride < vecs, lanes, p.codes, p.scales, row, p.hidden);
    }
  }
  // one vector per thread: its weight is on its way before the row's sums
  float w0[E], b0[E];
  if (C == 1 && t < vecs) {
    if (p.weight) load_weight<E>(p.weight, p.w_f32 != 0, t * E, w0);
    if (p.bias) load_weight<E>(p.bias, p.w_f32 != 0, t * E, b0);
  }
  const float inv_h = 1.f / static_cast<float>(static_cast<int>(p.hidden));
  float mean = 0.f, rest = 0.f, sq = 0.f;
  if (!p.rms) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (t + c * stride < vecs) {
        float v[E];
        unpack<T, E>(cur[c], v);
#pragma unroll
        for (int e = 0; e < E; ++e) mean += v[e];
      }
    }
    sum(mean, rest, One());
    mean *= inv_h;
    rest = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (t + c * stride < vecs) {
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
    sum(sq, rest, Both());
    rest *= inv_h;
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (t + c * stride < vecs) {
        float v[E];
        unpack<T, E>(cur[c], v);
#pragma unroll
        for (int e = 0; e < E; ++e) sq += v[e] * v[e];
      }
    }
    sum(sq, rest, One());
    rest = 0.f;
  }
  const float rstd = inverse_deviation(sq * inv_h - rest * rest, p.eps);
  if (t == 0 && vecs > 0) {
    if (p.mean && !p.rms) p.mean[row] = mean + rest;
    if (p.rstd) p.rstd[row] = rstd;
  }
  const float shift = -rest * rstd;
  // (the weights' type is asked once, not for each vector)
  auto finish = [&](auto f32) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = (t + c * stride) * E;
      if (t + c * stride < vecs) {
        float v[E], w[E], b[E];
        unpack<T, E>(cur[c], v);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = fmaf(v[e] - mean, rstd, shift);
        if (p.weight) {
          if (C > 1) load_weight<E>(p.weight, f32.value, i, w);
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] *= C > 1 ? w[e] : w0[e];
        }
        if (p.bias) {
          if (C > 1) load_weight<E>(p.bias, f32.value, i, b);
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] += C > 1 ? b[e] : b0[e];
        }
        store_raw<T, E>(y + i, pack<T, E>(v));
      }
    }
  };
  if (p.w_f32)
    finish(std::true_type());
  else
    finish(std::false_type());
}

// A row per CTA, of THREADS threads if that is not 0.
template <typename T, int E, int C, int THREADS, int MODE>
__global__ void __launch_bounds__(THREADS ? THREADS : kMaxThreads) norm_cta_kernel(const ParamsOf<MODE> p) {
  __shared__ BlockSums sums;
  int slot = 0;
  const int64_t row = blockIdx.x;
  norm_row<T, E, C, MODE>(p, static_cast<const T*>(p.x) + row * p.ld_x, static_cast<T*>(p.out) + row * p.hidden, row, threadIdx.x,
                    THREADS ? THREADS : blockDim.x, static_cast<int>(p.hidden) / E, 32,
                    [&](float& a, float& b, auto both) { block_sum<both.value>(a, b, sums, slot); });
}

// A row per group of `lanes` lanes (32, or fewer if the row has fewer vectors).
template <typename T, int E, int C, int MODE>
__global__ void __launch_bounds__(kWarpRowThreads) norm_warp_kernel(const ParamsOf<MODE> p, const int lanes) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kWarpRowThreads / lanes) + threadIdx.x / lanes;
  const int vecs = row < p.rows ? static_cast<int>(p.hidden) / E : 0;
  norm_row<T, E, C, MODE>(p, static_cast<const T*>(p.x) + row * p.ld_x, static_cast<T*>(p.out) + row * p.hidden, row,
                    threadIdx.x & (lanes - 1), 32, vecs, lanes, [&](float& a, float& b, auto both) {
                      a = group_sum(a, lanes);
                      if (both.value) b = group_sum(b, lanes);
                    });
}

// Rows that no register file holds: a CTA per row, which is read three times.
template <typename T, int MODE>
__global__ void __launch_bounds__(kMaxThreads) norm_long_kernel(const ParamsOf<MODE> p) {
  __shared__ BlockSums sums;
  int slot = 0;
  const int H = static_cast<int>(p.hidden);
  const float inv_h = 1.f / static_cast<float>(H);
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.ld_x;
    T* y = static_cast<T*>(p.out) + row * p.hidden;
    const T* res = nullptr;
    if constexpr (MODE != kPlain) res = p.residual ? static_cast<const T*>(p.residual) + row * p.ld_res : nullptr;
    auto at = [&](int i) {
      if constexpr (MODE == kPlain)
        return to_float<T>(x[i]);
      else
        return res ? to_float<T>(from_float<T>(to_float<T>(x[i]) + to_float<T>(res[i]))) : to_float<T>(x[i]);
    };
    if constexpr (MODE != kPlain) {
      if (p.sum)
        for (int i = threadIdx.x; i < H; i += blockDim.x) static_cast<T*>(p.sum)[row * p.hidden + i] = from_float<T>(at(i));
      if (p.codes) {
        // (whole warps: a block's lanes go through the loop together)
        for (int base = threadIdx.x & ~31; base < H; base += blockDim.x) {
          const int i = base + (threadIdx.x & 31);
          Raw<T, 1> r;
          r.u = from_float<T>(i < H ? at(i) : 0.f);
          keep_vector<T, 1>(r, i, i < H, 32, p.codes, p.scales, row, p.hidden);
        }
      }
    }
    float mean = 0.f, rest = 0.f;
    float s[2] = {0.f, 0.f};
    if (!p.rms) {
      for (int i = threadIdx.x; i < H; i += blockDim.x) s[0] += at(i);
      block_sum<true>(s[0], s[1], sums, slot);
      mean = s[0] * inv_h;
    }
    s[0] = s[1] = 0.f;
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
      const float d = at(i) - mean;
      s[0] += d * d;
      s[1] += d;
    }
    block_sum<true>(s[0], s[1], sums, slot);
    rest = p.rms ? 0.f : s[1] * inv_h;
    const float rstd = inverse_deviation(s[0] * inv_h - rest * rest, p.eps);
    if (threadIdx.x == 0) {
      if (p.mean && !p.rms) p.mean[row] = mean + rest;
      if (p.rstd) p.rstd[row] = rstd;
    }
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
      float v[1] = {(at(i) - mean - rest) * rstd}, w[1];
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
// Where a row's vectors lie. With SHIFT rows need not start on a vector boundary:
// vectors are counted from the boundary before the row, `off` elements earlier, and
// the first and last of them may hold elements that are not the row's. (10007 x 1337
// bf16: 52 us so, 75 by single elements. Aligned rows have kernels without all this,
// which cost them a tenth.)
struct Place {
  int hidden, off, vecs;
  template <int E>
  __device__ __forceinline__ bool inside(int v) const {
    return v * E >= off && (v + 1) * E - off <= hidden;
  }
};
// What x, grad_y and grad_x have in common: the distance of `row` from a boundary.
template <typename T, int E, bool SHIFT, int MODE>
__device__ __forceinline__ Place place_of(const NormParams& p, int64_t row) {
  // (a checkpoint lies as it likes)
  const void* x = MODE == kAdd8 ? p.gy : p.x;
  const int64_t at = static_cast<int64_t>(reinterpret_cast<uintptr_t>(x) / sizeof(T)) + row * (MODE == kAdd8 ? p.ld_gy : p.ld_x);
  const int off = SHIFT ? static_cast<int>(at % E) : 0, hidden = static_cast<int>(p.hidden);
  return {hidden, off, (hidden + off + E - 1) / E};
}
// Whether vector v of the row lies between the first row's first element and the
// last row's last, as its neighbours' elements may be read but nothing else.
template <int E>
__device__ __forceinline__ bool in_matrix(const Place& pl, int64_t row, int64_t ld, int64_t rows, int v) {
  const int64_t start = row * ld + v * E - pl.off;
  return start >= 0 && start + E <= (rows - 1) * ld + pl.hidden;
}
// Vector v of the row (`base`: its element of index 0 of that vector), elements of the row only.
template <typename T, int E>
__device__ __forceinline__ Raw<T, E> load_edge(const T* base, const Place& pl, int v) {
  float f[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = v * E - pl.off + e;
    f[e] = i >= 0 && i < pl.hidden ? to_float<T>(base[e]) : 0.f;
  }
  return pack<T, E>(f);
}
template <typename T, int E>
__device__ __forceinline__ void mask_edge(Raw<T, E>& r, const Place& pl, int v) {
  float f[E];
  unpack<T, E>(r, f);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = v * E - pl.off + e;
    if (i < 0 || i >= pl.hidden) f[e] = 0.f;
  }
  r = pack<T, E>(f);
}

// A thread's weights where they are not on vector boundaries themselves: as fp32 in
// shared memory, in vectors of four `stride` apart; ones if the norm has none,
// zeros beside the row.
template <int E>
struct Weights {
  static constexpr int per = E / 4;
  float4* v;
  int stride;
  __device__ __forceinline__ void fill(const NormParams& p, const Place& pl, int c, int vec) const {
    float w[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = vec * E - pl.off + e;
      float one[1] = {0.f};
      if (i >= 0 && i < pl.hidden) {
        one[0] = 1.f;
        if (p.weight) load_weight<1>(p.weight, p.w_f32 != 0, i, one);
      }
      w[e] = one[0];
    }
#pragma unroll
    for (int k = 0; k < per; ++k)
      v[(c * per + k) * stride] = make_float4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
  }
  __device__ __forceinline__ void get(int c, float (&w)[E]) const {
#pragma unroll
    for (int k = 0; k < per; ++k) {
      const float4 q = v[(c * per + k) * stride];
      w[4 * k] = q.x;
      w[4 * k + 1] = q.y;
      w[4 * k + 2] = q.z;
      w[4 * k + 3] = q.w;
    }
  }
};

// One vector before its row's sums are known: with d = x - mean and
// g = rstd grad_y w, adds grad_y xhat and grad_y to the columns' sums and g and
// g d to the row's, and leaves g for after them.
template <typename T, int E, int NB, bool RMS, typename X>
__device__ __forceinline__ void bwd_visit(const X& rx, const Raw<T, E>& rg, bool weighted, const float (&w)[E],
                                          float mean, float rstd, float (&d)[E], float (&g)[E], float (&acc_w)[E], float (&acc_b)[E],
                                          float& sg, float& sgd) {
  unpack<T, E>(rx, d);
  unpack<T, E>(rg, g);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (!RMS) d[e] -= mean;
    if (NB == 2) acc_b[e] += g[e];
    g[e] *= rstd;
    acc_w[e] += g[e] * d[e];
    if (weighted) g[e] *= w[e];
    if (!RMS) sg += g[e];
    sgd += g[e] * d[e];
  }
}

// grad_x = g + c0 + c2 d, c0 = -mean(g), c2 = -rstd^2 mean(g d); with ADD the gradient
// `more` of the sum that was normalised is added before the one rounding.
template <typename T, int E, bool RMS, bool ADD>
__device__ __forceinline__ void bwd_out(T* o, const float (&d)[E], const float (&g)[E], float c0, float c2, bool inside,
                                        const Place& pl, int vec, const float (&more)[ADD ? E : 1]) {
  float v[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    v[e] = d[e] * c2 + (RMS ? g[e] : g[e] + c0);
    if constexpr (ADD) v[e] += more[e];
  }
  if (inside) {
    store_raw<T, E>(o, pack<T, E>(v));
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = vec * E - pl.off + e;
      if (i >= 0 && i < pl.hidden) o[e] = from_float<T>(v[e]);
    }
  }
}

template <typename T, int E>
constexpr bool kRing = sizeof(T) * E >= 4;  // the smallest asynchronous copy is of 4 bytes
constexpr int ring_arrays(int mode) { return mode == kPlain ? 2 : 3; }

// C vectors per thread of a row, `stride` apart, and the ring of rows ahead: what
// both kernels below share. x - mean stays in registers until the row's sums are
// known (KEEP) only for one vector; else it is made again from the ring, and the
// registers serve for more threads. (32768 x 7168 bf16 RMS: 278 us with, 267
// without, 252 with a ring of two stages instead of three.)
template <typename T, int E, int C, int NB, bool RMS, bool SHIFT, int MODE>
struct BwdRow {
  static_assert(E > 1 || !SHIFT, "single elements are always in place");
  static constexpr bool RING = kRing<T, E>, KEEP = C == 1, ADD = MODE != kPlain, X8 = MODE == kAdd8;
  static constexpr int A = ring_arrays(MODE);  // arrays in the ring: x, grad_y, grad_sum
  // X8: single codes are too short for a copy, and where rows are off the vector boundary codes lie differently.
  static constexpr bool CODES_IN_RING = RING && E >= 4 && !SHIFT;
  // SHIFT: whole words that hold a vector's codes, in registers until they are used
  static constexpr int WINDOW = X8 && SHIFT ? E / 4 + 1 : 1;
  const ParamsOf<MODE>& p;
  Place pl;
  int t, stride, threads;  // first vector, distance between vectors, distance in the ring
  Raw<T, E>* ring;
  Weights<E> weights;  // SHIFT
  uint32_t inside = 0;
  uint32_t bits = 0;  // X8 and SHIFT: of a vector's first code in its word (the same for all rows and vectors of a thread)
  Raw<T, E> next_x[RING ? 1 : C], next_g[RING ? 1 : C], next_s[RING ? 1 : C];
  // X8: the next row's scales, and its codes where the ring does not take them
  uint8_t next_scale[X8 ? C : 1], next_second[X8 && SHIFT ? C : 1], next_code[X8 && !CODES_IN_RING && !SHIFT ? C : 1];
  uint32_t next_window[X8 && SHIFT ? C : 1][WINDOW];
  float acc_w[C][E], acc_b[C][E];

  __device__ __forceinline__ BwdRow(const ParamsOf<MODE>& params, const Place& place, int first, int apart, int ring_apart,
                                    Raw<T, E>* r, const Weights<E>& w, int64_t row)
      : p(params), pl(place), t(first), stride(apart), threads(ring_apart), ring(r), weights(w) {
    if constexpr (X8 && SHIFT) bits = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p.codes) + row * p.hidden - pl.off) % 4 * 8;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if constexpr (SHIFT) {
        if (pl.template inside<E>(t + c * stride)) inside |= 1u << c;
        if (t + c * stride < pl.vecs) weights.fill(p, pl, c, t + c * stride);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) acc_w[c][e] = acc_b[c][e] = 0.f;
    }
  }
  __device__ __forceinline__ bool is_inside(int c) const { return !SHIFT || (inside >> c & 1u); }

  __device__ __forceinline__ void fetch(int64_t row, int stage) {
    if (row < p.rows) {
      const T* xr = X8 ? nullptr : static_cast<const T*>(p.x) + row * p.ld_x + (t * E - pl.off);
      const T* gr = static_cast<const T*>(p.gy) + row * p.ld_gy + (t * E - pl.off);
      const T* sr = nullptr;
      int64_t ld_gs = 0;
      if constexpr (ADD) {
        ld_gs = p.ld_gs;
        if (p.gs) sr = static_cast<const T*>(p.gs) + row * ld_gs + (t * E - pl.off);
      }
      Raw<T, E>* to = ring + stage * A * C * threads;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int v = t + c * stride;
        if (v < pl.vecs) {
          if constexpr (X8 && SHIFT) {
            // from the word boundary before the vector's first code; at the checkpoint's ends byte by byte
            const uint8_t* code = p.codes + row * p.hidden + v * E - pl.off;
            const uintptr_t words = reinterpret_cast<uintptr_t>(code) & ~uintptr_t{3};
            if (words >= reinterpret_cast<uintptr_t>(p.codes) && words + 4 * WINDOW <= reinterpret_cast<uintptr_t>(p.codes) + p.rows * p.hidden) {
#pragma unroll
              for (int i = 0; i < WINDOW; ++i) next_window[c][i] = __ldg(reinterpret_cast<const uint32_t*>(words) + i);
            } else {
#pragma unroll
              for (int i = 0; i < WINDOW; ++i) next_window[c][i] = 0;
#pragma unroll
              for (int i = 0; i < 4 * WINDOW; ++i) {
                const int64_t e = static_cast<int64_t>(words) + i - static_cast<int64_t>(reinterpret_cast<uintptr_t>(code)) + v * E - pl.off;
                if (e >= 0 && e < pl.hidden) next_window[c][i / 4] |= static_cast<uint32_t>(p.codes[row * p.hidden + e]) << (i % 4 * 8);
              }
            }
            const uint8_t* scales = p.scales + row * checkpoint_blocks(p.hidden);
            const int first = max(v * E - pl.off, 0), last = min(v * E - pl.off + E, pl.hidden) - 1;
            next_scale[c] = __ldg(scales + first / kCheckpointBlock);
            next_second[c] = __ldg(scales + last / kCheckpointBlock);
          } else if constexpr (X8) {
            const uint8_t* code = p.codes + row * p.hidden + v * E;
            if constexpr (CODES_IN_RING)
              copy_async<E>(to + c * threads, code);
            else
              next_code[c] = __ldg(code);
            next_scale[c] = __ldg(p.scales + row * checkpoint_blocks(p.hidden) + v * E / kCheckpointBlock);
          }
          if constexpr (RING) {
            if (is_inside(c) || ((X8 || in_matrix<E>(pl, row, p.ld_x, p.rows, v)) && in_matrix<E>(pl, row, p.ld_gy, p.rows, v) &&
                                 (!ADD || !sr || in_matrix<E>(pl, row, ld_gs, p.rows, v)))) {
              if constexpr (!X8) copy_async<sizeof(T) * E>(to + c * threads, xr + c * stride * E);
              copy_async<sizeof(T) * E>(to + (C + c) * threads, gr + c * stride * E);
              if (ADD && sr) copy_async<sizeof(T) * E>(to + (2 * C + c) * threads, sr + c * stride * E);
            } else {
              if constexpr (!X8) to[c * threads] = load_edge<T, E>(xr + c * stride * E, pl, v);
              to[(C + c) * threads] = load_edge<T, E>(gr + c * stride * E, pl, v);
              if (ADD && sr) to[(2 * C + c) * threads] = load_edge<T, E>(sr + c * stride * E, pl, v);
            }
          } else {
            if constexpr (!X8) next_x[c] = load_raw<T, E>(xr + c * stride * E);
            next_g[c] = load_raw<T, E>(gr + c * stride * E);
            if (ADD && sr) next_s[c] = load_raw<T, E>(sr + c * stride * E);
          }
        }
      }
    }
    if constexpr (RING) copies_commit();
  }

  // Vector c of the row in `stage`; `rx` where there is no ring.
  __device__ __forceinline__ Raw<T, E> take(int stage, int which, int c, const Raw<T, E>& held) const {
    if constexpr (RING) {
      Raw<T, E> r = ring[stage * A * C * threads + (which * C + c) * threads];
      if (SHIFT && !is_inside(c)) mask_edge<T, E>(r, pl, t + c * stride);
      return r;
    } else {
      return held;
    }
  }

  // x of vector c of the row in `stage`, as it is held; `code` is a vector's only code, or (SHIFT) its window.
  struct HeldCode {
    uint32_t word[WINDOW];
    uint8_t scale, second;
  };
  using Vector = std::conditional_t<X8, std::conditional_t<SHIFT, ShiftedCodes<E>, CodeVector<E>>, Raw<T, E>>;
  __device__ __forceinline__ Vector take_x(int stage, int c, const Raw<T, E>& held, const HeldCode& code) const {
    if constexpr (!X8) {
      return take(stage, 0, c, held);
    } else if constexpr (SHIFT) {
      ShiftedCodes<E> r;
      const int start = (t + c * stride) * E - pl.off;
#pragma unroll
      for (int i = 0; i < E / 4; ++i) r.words[i] = __funnelshift_r(code.word[i], code.word[i + 1], bits);
      r.scale = scale_value(code.scale);
      r.next = scale_value(code.second);
      r.from = -start;
      r.to = pl.hidden - start;
      // (a vector of at most 8 elements, not of the row but for its blocks, has two at most)
      r.second = (min(start + E, pl.hidden) - 1) / kCheckpointBlock * kCheckpointBlock - start;
      return r;
    } else {
      CodeVector<E> r;
      if constexpr (CODES_IN_RING) {
        const uint32_t* from = reinterpret_cast<const uint32_t*>(ring + stage * A * C * threads + c * threads);
#pragma unroll
        for (int i = 0; i < E / 4; ++i) r.words[i] = from[i];
      } else {
        r.words[0] = code.word[0];
      }
      r.scale = scale_value(code.scale);
      return r;
    }
  }

  // The row in `stage` (vecs: 0 in threads without a row), the row that is `ahead`
  // fetched meanwhile; sum(sgd, sg) adds up over the row's threads.
  template <typename S>
  __device__ __forceinline__ void visit(int64_t row, int vecs, int stage, int64_t ahead, int fill, float mean, float rstd,
                                        int stages, S sum) {
    Raw<T, E> hx[RING ? 1 : C], hg[RING ? 1 : C], hs[RING ? 1 : C];
    HeldCode code[X8 ? C : 1];
    auto hold = [&]() {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if constexpr (!RING) {
          if constexpr (!X8) hx[c] = next_x[c];
          hg[c] = next_g[c];
          if constexpr (ADD) hs[c] = next_s[c];
        }
        if constexpr (X8) {
          code[c].scale = next_scale[c];
          if constexpr (SHIFT) {
            code[c].second = next_second[c];
#pragma unroll
            for (int i = 0; i < WINDOW; ++i) code[c].word[i] = next_window[c][i];
          } else if constexpr (!CODES_IN_RING) {
            code[c].word[0] = next_code[c];
          }
        }
      }
    };
    hold();
    fetch(ahead, fill);
    // (a ring of one stage holds the row that has just been fetched)
    if constexpr (X8)
      if (stages == 1) hold();
    if constexpr (RING) {
      if (stages == 4)
        copies_wait<3>();
      else if (stages == 3)
        copies_wait<2>();
      else if (stages == 2)
        copies_wait<1>();
      else
        copies_wait<0>();
    }
    float d[KEEP ? C : 1][E], g[C][E], sg = 0.f, sgd = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (t + c * stride < vecs) {
        float w[E];
        if constexpr (SHIFT)
          weights.get(c, w);
        else if (p.weight)
          load_weight<E>(p.weight, p.w_f32 != 0, (t + c * stride) * E, w);
        bwd_visit<T, E, NB, RMS>(take_x(stage, c, hx[RING ? 0 : c], code[X8 ? c : 0]),
                                 take(stage, 1, c, hg[RING ? 0 : c]), SHIFT || p.weight != nullptr, w, mean, rstd,
                                 d[KEEP ? c : 0], g[c], acc_w[c], acc_b[c], sg, sgd);
      }
    }
    if (p.out) {
      sum(sgd, sg);
      const float inv_h = 1.f / static_cast<float>(pl.hidden);
      const float c0 = RMS ? 0.f : -sg * inv_h, c2 = -rstd * rstd * (sgd * inv_h);
      T* o = static_cast<T*>(p.out) + row * p.hidden + (t * E - pl.off);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (t + c * stride < vecs) {
          if (!KEEP) {
            unpack<T, E>(take_x(stage, c, hx[RING ? 0 : c], code[X8 ? c : 0]), d[0]);
            if (!RMS) {
#pragma unroll
              for (int e = 0; e < E; ++e) d[0][e] -= mean;
            }
          }
          float more[ADD ? E : 1];
          if constexpr (ADD) {
            if (p.gs) {
              unpack<T, E>(take(stage, 2, c, hs[RING ? 0 : c]), more);
            } else {
#pragma unroll
              for (int e = 0; e < E; ++e) more[e] = 0.f;
            }
          }
          bwd_out<T, E, RMS, ADD>(o + c * stride * E, d[KEEP ? c : 0], g[c], c0, c2, is_inside(c), pl, t + c * stride, more);
        }
      }
    }
  }

  // f(column, c, e) for this thread's columns.
  template <typename F>
  __device__ __forceinline__ void columns(F f) const {
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int i = (t + c * stride) * E - pl.off + e;
        if (SHIFT ? i >= 0 && i < pl.hidden : t + c * stride < pl.vecs) f(i, c, e);
      }
    }
  }
};

// A row per CTA at a time. The ring's vectors are private to the thread that
// copies them, so it needs no barrier of its own. Single bf16 elements are
// loaded a row ahead into registers instead. A CTA's rows are a multiple of eight
// apart, so that they all start at the same distance from a vector boundary and
// its threads keep their columns. REGS: with 72 registers two CTAs of up to 448
// threads share an SM (a row of 7168 bf16 elements).
template <typename T, int E, int C, int NB, int REGS, bool RMS, bool SHIFT, int MODE>
__global__ void __maxnreg__(REGS) norm_bwd_cta_kernel(const ParamsOf<MODE> p, const int stages) {
  constexpr bool RING = kRing<T, E>;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ BlockSums sums;
  int slot = 0;
  const int T_ = blockDim.x;
  float4* w = reinterpret_cast<float4*>(dyn);
  Raw<T, E>* ring = reinterpret_cast<Raw<T, E>*>(w + (SHIFT ? C * Weights<E>::per * T_ : 0)) + threadIdx.x;
  int64_t row = blockIdx.x;
  BwdRow<T, E, C, NB, RMS, SHIFT, MODE> r(p, place_of<T, E, SHIFT, MODE>(p, row), threadIdx.x, T_, T_, ring, {w + threadIdx.x, T_}, row);
  for (int i = 0; i < stages - 1; ++i) r.fetch(row + static_cast<int64_t>(i) * gridDim.x, i);
  float mean = !RMS && row < p.rows ? __ldg(p.mean + row) : 0.f, rstd = row < p.rows ? __ldg(p.rstd + row) : 0.f;
  int stage = 0, fill = stages - 1;
  for (; row < p.rows; row += gridDim.x) {
    // the next row's statistics are on their way too
    const int64_t after = row + gridDim.x;
    const float next_mean = !RMS && after < p.rows ? __ldg(p.mean + after) : 0.f;
    const float next_rstd = after < p.rows ? __ldg(p.rstd + after) : 0.f;
    r.visit(row, r.pl.vecs, stage, row + static_cast<int64_t>(stages - 1) * gridDim.x, fill, mean, rstd, stages,
            [&](float& sgd, float& sg) { block_sum<!RMS>(sgd, sg, sums, slot); });
    mean = next_mean;
    rstd = next_rstd;
    if (++stage == stages) stage = 0;
    if (++fill == stages) fill = 0;
  }
  if constexpr (RING) copies_wait<0>();
  r.columns([&](int i, int c, int e) {
    if (p.part_w) p.part_w[blockIdx.x * p.hidden + i] = r.acc_w[c][e];
    if (NB == 2 && p.part_b) p.part_b[blockIdx.x * p.hidden + i] = r.acc_b[c][e];
  });
}

// Rows on groups of `lanes` lanes (32, or fewer if the row has fewer vectors),
// each with a ring of its own; no barrier until the CTA's groups add up their
// sums, in order. A group's rows are a multiple of eight apart, too.
template <typename T, int E, int NB, bool RMS, bool SHIFT, int MODE>
__global__ void __launch_bounds__(kWarpRowThreads)
    norm_bwd_warp_kernel(const ParamsOf<MODE> p, const int lanes, const int stages) {
  constexpr bool RING = kRing<T, E>;
  constexpr int C = 1;  // vectors per lane
  extern __shared__ __align__(16) uint8_t dyn[];
  float4* w = reinterpret_cast<float4*>(dyn);
  Raw<T, E>* ring = reinterpret_cast<Raw<T, E>*>(w + (SHIFT ? C * Weights<E>::per * kWarpRowThreads : 0)) + threadIdx.x;
  const int H = static_cast<int>(p.hidden);
  const int t = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes, groups = kWarpRowThreads / lanes;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  // whole warps go through the loop together: the groups' sums are shuffles of the warp
  const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + (threadIdx.x >> 5) * (32 / lanes);
  int64_t row = first + (threadIdx.x & 31) / lanes;
  BwdRow<T, E, C, NB, RMS, SHIFT, MODE> r(p, place_of<T, E, SHIFT, MODE>(p, row), t, 32, kWarpRowThreads, ring,
                                    {w + threadIdx.x, kWarpRowThreads}, row);
  for (int i = 0; i < stages - 1; ++i) r.fetch(row + i * step, i);
  float mean = !RMS && row < p.rows ? __ldg(p.mean + row) : 0.f, rstd = row < p.rows ? __ldg(p.rstd + row) : 0.f;
  int stage = 0, fill = stages - 1;
  for (int64_t base = first; base < p.rows; base += step, row += step) {
    const int64_t n = row + step;
    const float next_mean = !RMS && n < p.rows ? __ldg(p.mean + n) : 0.f, next_rstd = n < p.rows ? __ldg(p.rstd + n) : 0.f;
    r.visit(row, row < p.rows ? r.pl.vecs : 0, stage, row + (stages - 1) * step, fill, mean, rstd, stages,
            [&](float& sgd, float& sg) {
              if (!RMS) sg = group_sum(sg, lanes);
              sgd = group_sum(sgd, lanes);
            });
    mean = next_mean;
    rstd = next_rstd;
    if (++stage == stages) stage = 0;
    if (++fill == stages) fill = 0;
  }
  if constexpr (RING) copies_wait<0>();
  float* comb = reinterpret_cast<float*>(dyn);
#pragma unroll
  for (int which = 0; which < NB; ++which) {
    float* part = which == 0 ? p.part_w : p.part_b;
    if (part == nullptr) continue;
    __syncthreads();
    r.columns([&](int i, int c, int e) { comb[group * H + i] = which == 0 ? r.acc_w[c][e] : r.acc_b[c][e]; });
    __syncthreads();
    for (int i = threadIdx.x; i < H; i += kWarpRowThreads) {
      float v = 0.f;
      for (int g = 0; g < groups; ++g) v += comb[g * H + i];
      part[blockIdx.x * p.hidden + i] = v;
    }
  }
}

// Element i of a row's x, from the matrix or from its checkpoint.
template <typename T, int MODE>
__device__ __forceinline__ float bwd_x(const ParamsOf<MODE>& p, int64_t row, int64_t i) {
  if constexpr (MODE != kAdd8) {
    return to_float<T>(static_cast<const T*>(p.x)[row * p.ld_x + i]);
  } else {
    float v[1];
    const uint32_t code[1] = {p.codes[row * p.hidden + i]};
    read_codes<1>(code, scale_value(p.scales[row * checkpoint_blocks(p.hidden) + i / kCheckpointBlock]), v);
    return v[0];
  }
}

// Long rows: grad_x by a CTA per row in two passes through the L2.
template <typename T, int MODE>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_long_kernel(const ParamsOf<MODE> p) {
  __shared__ BlockSums sums;
  int slot = 0;
  const int H = static_cast<int>(p.hidden);
  const float inv_h = 1.f / static_cast<float>(H);
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* gy = static_cast<const T*>(p.gy) + row * p.ld_gy;
    T* gx = static_cast<T*>(p.out) + row * p.hidden;
    const float mean = p.rms ? 0.f : p.mean[row], rstd = p.rstd[row];
    float s[2] = {0.f, 0.f}, w[1] = {1.f};
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
      if (p.weight) load_weight<1>(p.weight, p.w_f32 != 0, i, w);
      const float g = to_float<T>(gy[i]) * w[0];
      s[0] += g;
      s[1] += g * ((bwd_x<T, MODE>(p, row, i) - mean) * rstd);
    }
    block_sum<true>(s[0], s[1], sums, slot);
    const float sg = p.rms ? 0.f : s[0] * inv_h, sgx = s[1] * inv_h;
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
      if (p.weight) load_weight<1>(p.weight, p.w_f32 != 0, i, w);
      const float g = to_float<T>(gy[i]) * w[0];
      float v = rstd * (g - sg - (bwd_x<T, MODE>(p, row, i) - mean) * rstd * sgx);
      if constexpr (MODE != kPlain)
        if (p.gs) v += to_float<T>(static_cast<const T*>(p.gs)[row * p.ld_gs + i]);
      gx[i] = from_float<T>(v);
    }
  }
}

// Long rows: the partial sums of row group blockIdx.y, a thread per column.
template <typename T, int MODE>
__global__ void __launch_bounds__(256) norm_bwd_long_cols_kernel(const ParamsOf<MODE> p, const int64_t group) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= p.hidden) return;
  const T* gy = static_cast<const T*>(p.gy);
  const int64_t r0 = blockIdx.y * group, r1 = min(r0 + group, p.rows);
  float w = 0.f, b = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const float g = to_float<T>(gy[r * p.ld_gy + i]);
    w += g * ((bwd_x<T, MODE>(p, r, i) - (p.rms ? 0.f : __ldg(p.mean + r))) * __ldg(p.rstd + r));
    b += g;
  }
  if (p.part_w) p.part_w[blockIdx.y * p.hidden + i] = w;
  if (p.part_b) p.part_b[blockIdx.y * p.hidden + i] = b;
}

inline bool aligned(const void* p, int64_t ld, size_t es) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * static_cast<int64_t>(es)) % 16 == 0);
}

// Whether rows can be taken as 16-byte vectors.
bool vectors(const NormParams& p) {
  const size_t es = p.dtype == FLCE_DTYPE_F32 ? 4 : 2;
  return aligned(p.x, p.ld_x, es) && aligned(p.gy, p.ld_gy, es) && aligned(p.out, p.hidden, es) &&
         p.hidden % (16 / es) == 0 && aligned(p.weight, 0, 1) && aligned(p.bias, 0, 1);
}
inline bool vectors(const AddNormParams& p) {
  const size_t es = p.dtype == FLCE_DTYPE_F32 ? 4 : 2;
  return vectors(static_cast<const NormParams&>(p)) && aligned(p.residual, p.ld_res, es) && aligned(p.gs, p.ld_gs, es) &&
         aligned(p.sum, p.hidden, es) && reinterpret_cast<uintptr_t>(p.codes) % (16 / es) == 0;
}

// Whether a row starts at the same distance from a 16-byte boundary in x, grad_y
// and grad_x, so that the same vectors serve for all of them.
bool in_step(const NormParams& p) {
  const int64_t es = p.dtype == FLCE_DTYPE_F32 ? 4 : 2, E = 16 / es;
  const uintptr_t x = reinterpret_cast<uintptr_t>(p.x) % 16;
  return p.hidden >= 2 * E && (p.ld_x - p.hidden) % E == 0 && (p.ld_gy - p.hidden) % E == 0 &&
         reinterpret_cast<uintptr_t>(p.gy) % 16 == x && (!p.out || reinterpret_cast<uintptr_t>(p.out) % 16 == x);
}
inline bool in_step(const AddNormParams& p) {
  const int64_t E = p.dtype == FLCE_DTYPE_F32 ? 4 : 8;
  const uintptr_t first = reinterpret_cast<uintptr_t>(p.gy) % 16;
  auto same = [&](const void* q, int64_t ld) { return !q || ((ld - p.hidden) % E == 0 && reinterpret_cast<uintptr_t>(q) % 16 == first); };
  return p.hidden >= 2 * E && same(p.gy, p.ld_gy) && same(p.x, p.ld_x) && same(p.gs, p.ld_gs) && same(p.out, p.hidden);
}

inline unsigned grid_of(int64_t want, int64_t most) { return static_cast<unsigned>(want < most ? want : most); }

// Lanes for a row of `vecs` vectors: a power of two.
inline int lanes_for(int64_t vecs) {
  int l = 1;
  while (l < vecs && l < 32) l *= 2;
  return l;
}

// C vectors for each of THREADS threads (0: `threads`), in steps of STEP.
template <typename T, int E, int THREADS, int STEP, int MOST, int MODE, int C = STEP>
cudaError_t run_fwd_cta(const ParamsOf<MODE>& p, int64_t c, int threads, cudaStream_t s) {
  if constexpr (C < MOST)
    if (c > C) return run_fwd_cta<T, E, THREADS, STEP, MOST, MODE, C + STEP>(p, c, threads, s);
  norm_cta_kernel<T, E, C, THREADS, MODE><<<static_cast<unsigned>(p.rows), threads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int E, int MODE>
cudaError_t run_fwd(const ParamsOf<MODE>& p, int sms, cudaStream_t s) {
  const int64_t vecs = p.hidden / E;
  if (vecs <= 32 * (E == 1 ? 16 : 4)) {
    const int lanes = lanes_for(vecs);
    const int64_t per = kWarpRowThreads / lanes;
    const unsigned grid = static_cast<unsigned>((p.rows + per - 1) / per);
    if (vecs <= 32)
      norm_warp_kernel<T, E, 1, MODE><<<grid, kWarpRowThreads, 0, s>>>(p, lanes);
    else if (vecs <= 32 * 4)
      norm_warp_kernel<T, E, 4, MODE><<<grid, kWarpRowThreads, 0, s>>>(p, lanes);
    else if constexpr (E == 1)
      norm_warp_kernel<T, E, 16, MODE><<<grid, kWarpRowThreads, 0, s>>>(p, lanes);
    return cudaGetLastError();
  }
  // few rows: a thread per vector, for the shortest chain of loads
  const bool few = p.rows < 2LL * sms;
  if constexpr (E == 1) {
    // Single elements: what a thread does once for a row is worth several elements, so
    // that fewer threads take more of them. (10007 x 1337 fp32: 25 us with 128 threads,
    // 31 with 64, 44 with 224; 8000 x 5003 bf16: 66 with 512, 87 with 256.)
    if (!few && vecs <= 128 * 16) return run_fwd_cta<T, E, 128, 4, 16, MODE>(p, (vecs + 127) / 128, 128, s);
    if (!few && vecs <= 256 * 16) return run_fwd_cta<T, E, 256, 4, 16, MODE>(p, (vecs + 255) / 256, 256, s);
    if (!few && vecs <= 512 * 32) return run_fwd_cta<T, E, 512, 4, 32, MODE>(p, (vecs + 511) / 512, 512, s);
    if (vecs <= kMaxThreads * 16) return run_fwd_cta<T, E, kMaxThreads, 4, 16, MODE>(p, (vecs + kMaxThreads - 1) / kMaxThreads, kMaxThreads, s);
  } else if (vecs <= static_cast<int64_t>(kMaxThreads) * kMaxVecs) {
    if (!few && vecs <= 128 * kMaxVecs) return run_fwd_cta<T, E, 128, 1, kMaxVecs, MODE>(p, (vecs + 127) / 128, 128, s);
    int most = few ? kMaxThreads : 128;
    while (most * kMaxVecs < vecs) most *= 2;
    const int64_t c = (vecs + most - 1) / most;
    return run_fwd_cta<T, E, 0, 1, kMaxVecs, MODE>(p, c, static_cast<int>(((vecs + c - 1) / c + 31) / 32 * 32), s);
  }
  norm_long_kernel<T, MODE><<<grid_of(p.rows, 2LL * sms), kMaxThreads, 0, s>>>(p);
  return cudaGetLastError();
}

constexpr size_t kMostShared = 220 * 1024;
constexpr int kCtaStages = 2;  // see BwdRow


// CTAs per SM of the backward: shorter rows take more of them, and each writes
// one partial row, so that the partial sums stay within about a sixth of a
// large batch's bytes.
inline int bwd_ctas(int64_t hidden) {
  const int64_t n = 16384 / hidden;
  return n < 1 ? 1 : n > 8 ? 8 : static_cast<int>(n);
}

// Launches k with dynamic shared memory above the default limit.
template <typename K, typename... A>
cudaError_t launch_large(K k, std::atomic<uint64_t>& done, unsigned grid, int threads, size_t smem, cudaStream_t s, A... args) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  if (smem > 40 * 1024 && !(done.load() >> (dev & 63) & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
    if (e != cudaSuccess) return e;
    done.fetch_or(1ull << (dev & 63));
  }
  k<<<grid, threads, smem, s>>>(args...);
  return cudaGetLastError();
}

// Most vectors of a row.
inline int64_t most_vecs(int64_t hidden, int E, bool shift) { return shift ? (hidden + 2 * E - 2) / E : hidden / E; }

template <typename T, int E, int NB, bool RMS, bool SHIFT, int MODE>
cudaError_t run_bwd_warp(const ParamsOf<MODE>& p, int64_t vecs, int sms, int* partials, cudaStream_t s) {
  const int lanes = lanes_for(vecs);
  const int64_t groups = kWarpRowThreads / lanes;
  // one vector per lane: three rows ahead are few registers and little shared memory
  // (a checkpoint's scales are held for one row ahead)
  const int stages = !kRing<T, E> || MODE == kAdd8 ? 2 : 4;
  const size_t ring = static_cast<size_t>(kWarpRowThreads) * ((kRing<T, E> ? ring_arrays(MODE) * sizeof(Raw<T, E>) * stages : 0) + (SHIFT ? E * sizeof(float) : 0));
  const size_t comb = static_cast<size_t>(groups) * p.hidden * sizeof(float);
  const size_t smem = ring > comb ? ring : comb;
  const unsigned grid = grid_of((p.rows + groups - 1) / groups, static_cast<int64_t>(sms) * 4);
  *partials = static_cast<int>(grid);
  static std::atomic<uint64_t> done{0};
  return launch_large(norm_bwd_warp_kernel<T, E, NB, RMS, SHIFT, MODE>, done, grid, kWarpRowThreads, smem, s, p, lanes, stages);
}

// Shared memory of `vecs` vectors of a row in a CTA: their weights, and their place in one stage of the ring.
template <typename T, int E, bool SHIFT, int MODE>
constexpr size_t weights_bytes(int64_t vecs) { return SHIFT ? static_cast<size_t>(vecs) * E * sizeof(float) : 0; }
template <typename T, int E, bool SHIFT, int MODE>
constexpr size_t stage_bytes(int64_t vecs) { return kRing<T, E> ? static_cast<size_t>(vecs) * ring_arrays(MODE) * sizeof(Raw<T, E>) : 0; }
inline int cta_threads(int64_t vecs, int C) { return static_cast<int>(((vecs + C - 1) / C + 31) / 32 * 32); }

// Whether a CTA takes a row: its threads' registers have to hold it, and its shared memory one stage. (Behind the
// residual's addition, with three arrays in a stage, fp32 rows off the vector boundary do up to 13821 elements.)
template <typename T, int E, bool SHIFT, int MODE>
bool cta_holds(int64_t vecs) {
  constexpr int C = cta_vecs(E);
  if (vecs > static_cast<int64_t>(kMaxThreads) * C) return false;
  const int64_t all = static_cast<int64_t>(cta_threads(vecs, C)) * C;
  return weights_bytes<T, E, SHIFT, MODE>(all) + stage_bytes<T, E, SHIFT, MODE>(all) <= kMostShared;
}

template <typename T, int E, int C, int REGS, int NB, bool RMS, bool SHIFT, int MODE>
cudaError_t run_bwd_cta(const ParamsOf<MODE>& p, int64_t vecs, int sms, int* partials, cudaStream_t s) {
  const int threads = cta_threads(vecs, C);
  int ctas = 65536 / (REGS * threads);
  if (ctas > bwd_ctas(p.hidden)) ctas = bwd_ctas(p.hidden);
  const size_t weights = weights_bytes<T, E, SHIFT, MODE>(static_cast<int64_t>(threads) * C);
  const size_t row = stage_bytes<T, E, SHIFT, MODE>(static_cast<int64_t>(threads) * C);
  int stages = !kRing<T, E> ? 2 : kCtaStages;
  while (stages > 1 && (row * stages + weights) * ctas > kMostShared) --stages;
  // rows that a CTA visits are a multiple of eight apart
  int64_t grid = static_cast<int64_t>(sms) * ctas;
  grid = p.rows <= grid ? p.rows : grid / 8 * 8;
  *partials = static_cast<int>(grid);
  static std::atomic<uint64_t> done{0};
  return launch_large(norm_bwd_cta_kernel<T, E, C, NB, REGS, RMS, SHIFT, MODE>, done, static_cast<unsigned>(grid), threads,
                      row * stages + weights, s, p, stages);
}

template <typename T, int E, int NB, bool RMS, bool SHIFT, int MODE>
cudaError_t run_bwd_row(const ParamsOf<MODE>& p, int sms, int* partials, cudaStream_t s) {
  const int64_t vecs = most_vecs(p.hidden, E, SHIFT);
  if (vecs <= 32) return run_bwd_warp<T, E, NB, RMS, SHIFT, MODE>(p, vecs, sms, partials, s);
  // (Rows of up to four vectors per lane on a warp: 32768 x 1024 bf16 RMS 48 us so, 54
  // by CTAs, but 30000 x 576 with a bias 57 and 48, 20000 x 201 fp32 38 and 27.)
  // Short rows on more threads, for the latency of a row: 10007 x 1337 bf16 46 us with
  // one vector each, 52 with two; fp32 40 with two, 56 with four. Not long ones:
  // 32768 x 4096 bf16 194 us with one, 154 with two; 8192 x 8192 fp32 138 and 133.
  if constexpr (E == 8)
    if (vecs <= 256) return run_bwd_cta<T, E, 1, 64, NB, RMS, SHIFT, MODE>(p, vecs, sms, partials, s);
  if constexpr (E == 4) {
    if (vecs <= 128) return run_bwd_cta<T, E, 1, 64, NB, RMS, SHIFT, MODE>(p, vecs, sms, partials, s);
    if (vecs <= 2 * 448) return run_bwd_cta<T, E, 2, 72, NB, RMS, SHIFT, MODE>(p, vecs, sms, partials, s);
  }
  constexpr int C = cta_vecs(E);
  if (vecs <= 448 * C) return run_bwd_cta<T, E, C, 72, NB, RMS, SHIFT, MODE>(p, vecs, sms, partials, s);
  return run_bwd_cta<T, E, C, 64, NB, RMS, SHIFT, MODE>(p, vecs, sms, partials, s);
}

template <typename T, int E, bool SHIFT, int MODE>
cudaError_t run_bwd(const ParamsOf<MODE>& p, int sms, int* partials, cudaStream_t s) {
  if (cta_holds<T, E, SHIFT, MODE>(most_vecs(p.hidden, E, SHIFT))) {
    if (p.part_b)
      return p.rms ? run_bwd_row<T, E, 2, true, SHIFT, MODE>(p, sms, partials, s) : run_bwd_row<T, E, 2, false, SHIFT, MODE>(p, sms, partials, s);
    return p.rms ? run_bwd_row<T, E, 1, true, SHIFT, MODE>(p, sms, partials, s) : run_bwd_row<T, E, 1, false, SHIFT, MODE>(p, sms, partials, s);
  }
  const int groups = norm_partial_rows(p.rows, p.hidden, sms);
  const int64_t group = (p.rows + groups - 1) / groups;
  *partials = static_cast<int>((p.rows + group - 1) / group);
  if (p.part_w || p.part_b) {  // first, as grad_x may take the place of x or grad_y
    const dim3 grid(static_cast<unsigned>((p.hidden + 255) / 256), static_cast<unsigned>(*partials));
    norm_bwd_long_cols_kernel<T, MODE><<<grid, 256, 0, s>>>(p, group);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (p.out) norm_bwd_long_kernel<T, MODE><<<grid_of(p.rows, 2LL * sms), kMaxThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int E, int MODE>
cudaError_t launch_bwd(const ParamsOf<MODE>& p, int sms, int* partials, cudaStream_t s) {
  if (vectors(p)) return run_bwd<T, E, false, MODE>(p, sms, partials, s);
  if (in_step(p)) return run_bwd<T, E, true, MODE>(p, sms, partials, s);
  return run_bwd<T, 1, false, MODE>(p, sms, partials, s);
}

}  // namespace

}  // namespace flce
