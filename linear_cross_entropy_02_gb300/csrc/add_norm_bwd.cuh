// Backward pass of the norm behind the residual's addition for rows of a multiple of 512
// elements, 2048 to 8192, on vector boundaries: grad_x = grad_sum + the norm's gradient, from
// the sum or from its checkpoint. (Other rows: norm_device.cuh.)
//
// As there, a CTA stays, its threads keep their columns and the weight's gradient for them
// in registers, and rows are copied ahead into a ring that a thread fills and reads for itself.
// What bounds these kernels is instructions and, between a row's two passes, latency: HBM
// would allow 243 us for 32768 x 7168 bf16 RMS from 8 bits. So every thread has the same
// whole number of vectors, and no branch stands between the loads of one and the next
// (394 us with such branches, 316 without); codes stay in registers as halves between the
// passes, and so do weighted gradients unless the bias' sums take their place.
#pragma once

#include <cuda_fp16.h>

#include "norm_device.cuh"

namespace flce {

namespace {

// CTAs on an SM at most: each writes a partial row of the weight's gradient.
constexpr int kMostAddCtas = 4;
constexpr int kLeastWide = 2048, kMostWide = 8192, kWideStep = 512;

// E4M3 codes of a vector as halves (exact).
template <int E>
struct Codes {
  uint32_t h[E / 2];
  __device__ __forceinline__ void read(const uint8_t* from) {
    uint32_t words[E / 4];
    if constexpr (E == 8) {
      const uint2 w = *reinterpret_cast<const uint2*>(from);
      words[0] = w.x;
      words[1] = w.y;
    } else {
      words[0] = *reinterpret_cast<const uint32_t*>(from);
    }
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
          : "=r"(h[2 * i]), "=r"(h[2 * i + 1])
          : "r"(words[i]));
    }
  }
  __device__ __forceinline__ float value(int e) const {
    const __half2 v = *reinterpret_cast<const __half2*>(&h[e / 2]);
    return e & 1 ? __high2float(v) : __low2float(v);
  }
};

// C vectors per thread. HOLD: the weighted gradients stay in registers between the passes.
template <typename T, typename W, int NB, bool RMS, bool X8, bool HOLD, int C, int REGS>
__global__ void __maxnreg__(REGS) add_norm_bwd_kernel(const AddNormParams p, const int stages) {
  constexpr int E = 16 / sizeof(T);
  constexpr int XB = X8 ? E : 16;  // bytes of a vector of x
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ BlockSums sums;
  int slot = 0;
  const int threads = blockDim.x, t = threadIdx.x, vecs = threads * C;
  const int stage_bytes = vecs * (32 + XB);
  const bool more = p.gs != nullptr;
  const float inv_h = 1.f / static_cast<float>(static_cast<int>(p.hidden));
  const int64_t blocks = p.hidden / kCheckpointBlock;
  const W* weight = static_cast<const W*>(p.weight) + t * E;
  float acc_w[C][E], acc_b[NB == 2 ? C : 1][E];
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      acc_w[c][e] = 0.f;
      if (NB == 2) acc_b[NB == 2 ? c : 0][e] = 0.f;
    }
  }
  uint8_t next_scale[X8 ? C : 1];
  auto fetch = [&](int64_t row, int stage) {
    if (row < p.rows) {
      const T* gy = static_cast<const T*>(p.gy) + row * p.ld_gy + t * E;
      const T* gs = static_cast<const T*>(p.gs) + row * p.ld_gs + t * E;
      const uint8_t* x = X8 ? p.codes + row * p.hidden + t * E : reinterpret_cast<const uint8_t*>(static_cast<const T*>(p.x) + row * p.ld_x + t * E);
      const uint8_t* sc = X8 ? p.scales + row * blocks + t * E / kCheckpointBlock : nullptr;
      uint8_t* to = dyn + stage * stage_bytes + t * 16;
      uint8_t* to_x = dyn + stage * stage_bytes + vecs * 32 + t * XB;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        copy_async<16>(to + c * threads * 16, gy + c * threads * E);
        copy_async<XB>(to_x + c * threads * XB, x + c * threads * XB);
        if constexpr (X8) next_scale[c] = __ldg(sc + c * threads * E / kCheckpointBlock);
      }
      if (more) {
#pragma unroll
        for (int c = 0; c < C; ++c) copy_async<16>(to + vecs * 16 + c * threads * 16, gs + c * threads * E);
      }
    }
    copies_commit();
  };
  int64_t row = blockIdx.x;
  if (stages > 1) fetch(row, 0);
  float mean = !RMS && row < p.rows ? __ldg(p.mean + row) : 0.f, rstd = row < p.rows ? __ldg(p.rstd + row) : 0.f;
  int stage = 0;
  for (; row < p.rows; row += gridDim.x) {
    const int64_t after = row + gridDim.x;
    const float next_mean = !RMS && after < p.rows ? __ldg(p.mean + after) : 0.f;
    const float next_rstd = after < p.rows ? __ldg(p.rstd + after) : 0.f;
    float scale[C];
    auto scales = [&]() {
#pragma unroll
      for (int c = 0; c < C; ++c) scale[c] = X8 ? (RMS ? scale_value(next_scale[c]) * rstd : scale_value(next_scale[c])) : rstd;
    };
    scales();
    if (stages > 1) {
      fetch(after, stage ^ 1);
      copies_wait<1>();
    } else {
      fetch(row, 0);
      scales();
      copies_wait<0>();
    }
    const uint8_t* from = dyn + stage * stage_bytes + t * 16;
    const uint8_t* from_x = dyn + stage * stage_bytes + vecs * 32 + t * XB;
    float h[HOLD ? C : 1][E];
    Codes<E> codes[X8 ? C : 1];
    auto xhat = [&](int c, float (&v)[E]) {
      if constexpr (X8) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = RMS ? codes[c].value(e) * scale[c] : fmaf(codes[c].value(e), scale[c], -mean) * rstd;
      } else {
        unpack<T, E>(*reinterpret_cast<const Raw<T, E>*>(from_x + c * threads * XB), v);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = (RMS ? v[e] : v[e] - mean) * rstd;
      }
    };
    auto weighted = [&](int c, const float (&g)[E], float (&v)[E]) {
      if (p.weight) {
        float w[E];
        load_weight<E>(weight + c * threads * E, sizeof(W) == 4, 0, w);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = g[e] * w[e];
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = g[e];
      }
    };
    float sg = 0.f, sgd = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float g[E], x[E];
      float(&k)[E] = h[HOLD ? c : 0];
      unpack<T, E>(*reinterpret_cast<const Raw<T, E>*>(from + c * threads * 16), g);
      if constexpr (X8) codes[c].read(from_x + c * threads * XB);
      xhat(c, x);
      weighted(c, g, k);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (NB == 2) acc_b[NB == 2 ? c : 0][e] += g[e];
        acc_w[c][e] = fmaf(g[e], x[e], acc_w[c][e]);
        if (!RMS) sg += k[e];
        sgd = fmaf(k[e], x[e], sgd);
      }
    }
    if (p.out) {
      block_sum<!RMS>(sgd, sg, sums, slot);
      const float c2 = -rstd * (sgd * inv_h), c0 = RMS ? 0.f : -rstd * (sg * inv_h);
      T* o = static_cast<T*>(p.out) + row * p.hidden + t * E;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float s[E], x[E];
#pragma unroll
        for (int e = 0; e < E; ++e) s[e] = c0;
        if (more) {
          float v[E];
          unpack<T, E>(*reinterpret_cast<const Raw<T, E>*>(from + vecs * 16 + c * threads * 16), v);
#pragma unroll
          for (int e = 0; e < E; ++e) s[e] = RMS ? v[e] : v[e] + c0;
        }
        if constexpr (!HOLD) {
          float g[E];
          unpack<T, E>(*reinterpret_cast<const Raw<T, E>*>(from + c * threads * 16), g);
          weighted(c, g, h[0]);
        }
        xhat(c, x);
#pragma unroll
        for (int e = 0; e < E; ++e) s[e] = fmaf(x[e], c2, fmaf(h[HOLD ? c : 0][e], rstd, s[e]));
        store_raw<T, E>(o + c * threads * E, pack<T, E>(s));
      }
    }
    mean = next_mean;
    rstd = next_rstd;
    if (stages > 1) stage ^= 1;
  }
  copies_wait<0>();
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int64_t at = blockIdx.x * p.hidden + (t + c * threads) * E + e;
      if (p.part_w) p.part_w[at] = acc_w[c][e];
      if (NB == 2 && p.part_b) p.part_b[at] = acc_b[NB == 2 ? c : 0][e];
    }
  }
}

template <typename T, typename W, int NB, bool RMS, bool X8, bool HOLD, int C, int REGS>
cudaError_t run_add_bwd_as(const AddNormParams& p, int sms, int* partials, cudaStream_t s) {
  constexpr int E = 16 / sizeof(T);
  const int vecs = static_cast<int>(p.hidden / E), threads = vecs / C;
  int ctas = 65536 / (REGS * threads);
  if (ctas > kMostAddCtas) ctas = kMostAddCtas;
  const size_t row = static_cast<size_t>(vecs) * (32 + (X8 ? E : 16));
  const int stages = (2 * row + 1024) * ctas <= kMostShared ? 2 : 1;
  const unsigned grid = grid_of(p.rows, static_cast<int64_t>(sms) * ctas);
  *partials = static_cast<int>(grid);
  static std::atomic<uint64_t> done{0};
  return launch_large(add_norm_bwd_kernel<T, W, NB, RMS, X8, HOLD, C, REGS>, done, grid, threads, row * stages, s, p, stages);
}

template <typename T, typename W, bool X8>
cudaError_t run_add_bwd(const AddNormParams& p, int sms, int* partials, cudaStream_t s) {
  constexpr int C = sizeof(T);  // 16 columns per thread
  // (Microseconds for 32768 rows of bf16 from 8 bits: 7168 RMS with 16 columns held 316, not 317, with 32 held
  // 304, and where 144 registers are allowed, 296: ptxas takes 127 or 128 of them all the same, and orders the loads
  // otherwise. 5120 at 128 registers 208, where 144 are counted on, with a CTA less, 246. The one kernel that does take
  // 144, layer norm from the sum with an fp32 weight, leaves room for one CTA of 7168 columns, as a scheduler's 16384
  // registers hold three such warps: 427 us, 330 with 128; with a bf16 weight 326 and 328.
  // With a bias' sums 7168 held 394, not 376; from the sum 353 and 374. 8192 x 7168 fp32 with 32 columns 166,
  // with 16 126.)
  const int64_t hidden = p.hidden;
  if (p.part_b) {
    // (of 8192 columns two CTAs fit with 64 registers only: 16384 rows 249 us, 270 with one)
    if (hidden / 16 * 72 * 2 > 65536)
      return p.rms ? run_add_bwd_as<T, W, 2, true, X8, !X8, C, 64>(p, sms, partials, s)
                   : run_add_bwd_as<T, W, 2, false, X8, !X8, C, 64>(p, sms, partials, s);
    return p.rms ? run_add_bwd_as<T, W, 2, true, X8, !X8, C, 72>(p, sms, partials, s)
                 : run_add_bwd_as<T, W, 2, false, X8, !X8, C, 72>(p, sms, partials, s);
  }
  if constexpr (sizeof(T) == 2) {
    if (hidden > 4096 && hidden % (2 * kWideStep) == 0) {
      if (65536 / (144 * (hidden / 32)) == 65536 / (128 * (hidden / 32))) {
        if (p.rms) return run_add_bwd_as<T, W, 1, true, X8, true, 2 * C, 144>(p, sms, partials, s);
        if constexpr (X8 || sizeof(W) == 2) return run_add_bwd_as<T, W, 1, false, X8, true, 2 * C, 144>(p, sms, partials, s);
      }
      return p.rms ? run_add_bwd_as<T, W, 1, true, X8, true, 2 * C, 128>(p, sms, partials, s)
                   : run_add_bwd_as<T, W, 1, false, X8, true, 2 * C, 128>(p, sms, partials, s);
    }
  }
  if (hidden / 16 * 72 * 2 > 65536)
    return p.rms ? run_add_bwd_as<T, W, 1, true, X8, true, C, 64>(p, sms, partials, s)
                 : run_add_bwd_as<T, W, 1, false, X8, true, C, 64>(p, sms, partials, s);
  return p.rms ? run_add_bwd_as<T, W, 1, true, X8, true, C, 72>(p, sms, partials, s)
               : run_add_bwd_as<T, W, 1, false, X8, true, C, 72>(p, sms, partials, s);
}

// Whether rows are for these kernels. (Shorter ones were slower: 65536 x 1024 RMS from 8 bits 153 us, 112 by
// norm_device.cuh's; 2048 203 and 220.)
inline bool wide_rows(const AddNormParams& p) {
  return p.hidden >= kLeastWide && p.hidden <= kMostWide && p.hidden % kWideStep == 0 && vectors(p);
}

template <typename T, bool X8>
cudaError_t run_wide_bwd(const AddNormParams& p, int sms, int* partials, cudaStream_t s) {
  return p.w_f32 ? run_add_bwd<T, float, X8>(p, sms, partials, s) : run_add_bwd<T, uint16_t, X8>(p, sms, partials, s);
}

}  // namespace

}  // namespace flce
