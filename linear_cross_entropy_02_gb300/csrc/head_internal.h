// Internal interface between the host entries of the operators around the head
// (head_api.cpp) and their kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "flce_head.h"

namespace flce {

enum HeadKernelId {
  K_NORM = FLCE_HEAD_KERNEL_FIRST,
  K_NORM_BWD,
  K_NORM_WGRAD,
  K_MX_QUANT,
  K_MX_DEQUANT,
  K_MX_GEMM,
  K_SAMPLE,
};

// ------------------------------------------------------------ norm
struct NormParams {
  const void* x;
  const void* gy;  // backward: upstream gradient
  int dtype;
  int64_t rows, hidden, ld_x, ld_gy;
  const void* weight;
  const void* bias;
  int w_f32;  // weight and bias are fp32 (else bf16)
  float eps;
  int rms;
  void* out;         // y, or grad_x (nullable)
  float* mean;       // forward: written; backward: read
  float* rstd;
  float* part_w;     // backward: per-CTA partial sums [grid][hidden], or null
  float* part_b;
};
// Most partial rows that launch_norm_bwd writes for a call on this device.
int norm_partial_rows(int64_t rows, int64_t hidden, int sms);
cudaError_t launch_norm(const NormParams& p, int sms, cudaStream_t s);
// Writes grad_x and the partial sums; *partials = rows of part_w / part_b written.
cudaError_t launch_norm_bwd(const NormParams& p, int sms, int* partials, cudaStream_t s);
// grad_w[j] (+)= sum over i of part_w[i][j], in a fixed order (and the same for b).
cudaError_t launch_norm_wgrad(const float* part_w, const float* part_b, int partials, int64_t hidden, float* grad_w,
                              float* grad_b, int accumulate, cudaStream_t s);

// ------------------------------------------------------------ microscaled 4-bit
constexpr int kMxBlock = 32;        // elements per scale
constexpr int kMxTileRows = 128;    // rows per scale tile
constexpr int kMxTileCols = 128;    // elements of K per scale tile (4 blocks)
constexpr int kMxTileBytes = 512;

struct MxQuantParams {
  const void* x;
  int dtype;
  int64_t rows, cols, ld_x;
  uint8_t* codes;
  uint8_t* scales;
};
cudaError_t launch_mx_quantize(const MxQuantParams& p, int sms, cudaStream_t s);
cudaError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out,
                                 int out_dtype, cudaStream_t s);

struct MxGemmParams {
  const void* x;  // tokens that the kernel encodes itself (then a_codes, a_scales are not used), or null
  int x_dtype;
  int64_t ld_x;
  const uint8_t* a_codes;
  const uint8_t* a_scales;
  const uint8_t* w_codes;
  const uint8_t* w_scales;
  int64_t rows, vocab, cols;
  float out_mult, softcap, inv_softcap;
  void* out;
  int out_dtype;
  int64_t ld_out;
  int32_t* status;
  uint64_t timeout_ns;
  int stall;  // FLCE_FLAG_TEST_STALL
};
// Whether launch_mx_gemm takes tokens of this shape as x.
bool mx_gemm_encodes(int64_t rows, int64_t cols);
// FLCE_* code: the tensor maps are encoded here. Sets *status to 0 first.
int launch_mx_gemm(const MxGemmParams& p, int sms, cudaStream_t s);

// ------------------------------------------------------------ sampling
struct SampleParams {
  const void* x;
  int dtype;
  int64_t rows, vocab, ld;
  const float* u;
  const float* temperatures;
  const int32_t* top_ks;
  const float* top_ps;
  const float* min_ps;
  float temperature, top_p, min_p;
  int32_t top_k;
  int64_t* tokens;
  float* logprobs;
};
cudaError_t launch_sample(const SampleParams& p, int sms, cudaStream_t s);

}  // namespace flce
