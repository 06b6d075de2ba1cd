// Host entries of the operators around the head (include/flce_head.h):
// argument checks, workspace carving and launches. No allocation, no host
// synchronisation, errors returned before any launch.
#include <cuda_runtime.h>

#include <cmath>

#include "flce_host.h"
#include "flce_internal.h"
#include "head_internal.h"

using namespace flce;

namespace {

constexpr int64_t kMaxHidden = int64_t{1} << 24;
constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1;
constexpr size_t kHeaderBytes = 256;

inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }
inline bool dtype_ok(int d) { return d == FLCE_DTYPE_BF16 || d == FLCE_DTYPE_F32; }
inline size_t element_size(int d) { return d == FLCE_DTYPE_F32 ? 4 : 2; }
inline bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Whether a result [rows, hidden] at `out` may be written while `in` [rows, ld] is
// read: apart from it, or the same memory row by row.
bool apart_or_same(const void* in, int64_t ld, const void* out, int64_t rows, int64_t hidden, size_t es) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(in), b = reinterpret_cast<uintptr_t>(out);
  const uintptr_t an = (static_cast<uintptr_t>(rows - 1) * ld + hidden) * es, bn = static_cast<uintptr_t>(rows) * hidden * es;
  return a >= b + bn || b >= a + an || (a == b && (ld == hidden || rows == 1));
}

int device_check(int* sms) {
  int cc = 0;
  const int rc = device_info(sms, &cc);
  if (rc != FLCE_OK) return rc;
  return cc == 103 ? FLCE_OK : FLCE_ERR_UNSUPPORTED;
}

// Shapes of a microscaled matrix.
inline bool mx_shape_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && rows <= kMaxRows - kMxTileRows && cols > 0 && cols % kMxBlock == 0 && cols <= kMaxHidden;
}
inline size_t mx_codes(int64_t rows, int64_t cols) { return static_cast<size_t>(rows) * (cols / 2); }
inline size_t mx_scales(int64_t rows, int64_t cols) {
  return static_cast<size_t>((rows + kMxTileRows - 1) / kMxTileRows) * ((cols + kMxTileCols - 1) / kMxTileCols) *
         kMxTileBytes;
}

// A matrix's buffers: given where it has rows, on the boundaries that TMA and word stores need.
int mx_buffers(int64_t rows, const void* codes, const void* scales) {
  if (rows == 0) return FLCE_OK;
  if (!codes || !scales) return FLCE_ERR_ARG;
  return aligned(codes, 16) && aligned(scales, 16) ? FLCE_OK : FLCE_ERR_ALIGN;
}

int check_product(int64_t rows, int64_t vocab, int64_t cols, const void* w_codes, const void* w_scales, float out_mult,
                  float softcap, const void* out, int out_dtype, int64_t* ld_out, const void* workspace) {
  if (!mx_shape_ok(rows, cols) || !mx_shape_ok(vocab, cols) || vocab == 0 || !dtype_ok(out_dtype)) return FLCE_ERR_ARG;
  if (!std::isfinite(out_mult) || !(softcap >= 0.f) || !std::isfinite(softcap)) return FLCE_ERR_ARG;
  if (*ld_out == 0) *ld_out = vocab;
  if (*ld_out < vocab) return FLCE_ERR_ARG;
  if (rows > 0 && (!out || !workspace)) return FLCE_ERR_ARG;
  if (rows > 0 && (!aligned(out, element_size(out_dtype)) || !aligned(workspace, 16))) return FLCE_ERR_ALIGN;
  return mx_buffers(vocab, w_codes, w_scales);
}

MxGemmParams product(int64_t rows, int64_t vocab, int64_t cols, const void* a_codes, const void* a_scales,
                     const void* w_codes, const void* w_scales, float out_mult, float softcap, void* out,
                     int out_dtype, int64_t ld_out, void* workspace) {
  MxGemmParams g = {};
  g.a_codes = static_cast<const uint8_t*>(a_codes);
  g.a_scales = static_cast<const uint8_t*>(a_scales);
  g.w_codes = static_cast<const uint8_t*>(w_codes);
  g.w_scales = static_cast<const uint8_t*>(w_scales);
  g.rows = rows;
  g.vocab = vocab;
  g.cols = cols;
  g.out_mult = out_mult;
  g.softcap = softcap;
  g.inv_softcap = softcap > 0.f ? 1.f / softcap : 0.f;
  g.out = out;
  g.out_dtype = out_dtype;
  g.ld_out = ld_out;
  g.status = &static_cast<Header*>(workspace)->status;
  g.timeout_ns = kDefaultTimeoutNs;
  return g;
}

}  // namespace

extern "C" {

int flce_layer_norm(const void* x, int dtype, int64_t rows, int64_t hidden, int64_t ld_x, const void* weight,
                    const void* bias, int weight_dtype, float eps, int rms, void* y, float* mean, float* rstd,
                    void* stream_handle) {
  if (!dtype_ok(dtype) || !dtype_ok(weight_dtype) || rows < 0 || rows > kMaxRows || hidden <= 0 || hidden > kMaxHidden ||
      ld_x < hidden || !(eps >= 0.f) || !std::isfinite(eps))
    return FLCE_ERR_ARG;
  if (rows == 0) return FLCE_OK;
  if (!x || !y) return FLCE_ERR_ARG;
  const size_t es = element_size(dtype), ws = element_size(weight_dtype);
  if (!aligned(x, es) || !aligned(y, es) || !aligned(weight, ws) || !aligned(bias, ws) || !aligned(mean, 4) ||
      !aligned(rstd, 4))
    return FLCE_ERR_ALIGN;
  if (!apart_or_same(x, ld_x, y, rows, hidden, es)) return FLCE_ERR_ARG;
  int sms = 0;
  const int rc = device_check(&sms);
  if (rc != FLCE_OK) return rc;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  NormParams p = {};
  p.x = x;
  p.dtype = dtype;
  p.rows = rows;
  p.hidden = hidden;
  p.ld_x = ld_x;
  p.weight = weight;
  p.bias = bias;
  p.w_f32 = weight_dtype == FLCE_DTYPE_F32;
  p.eps = eps;
  p.rms = rms != 0;
  p.out = y;
  p.mean = mean;
  p.rstd = rstd;
  FLCE_LAUNCH(K_NORM, launch_norm(p, sms, stream));
  return FLCE_OK;
}

size_t flce_layer_norm_workspace_size(int64_t rows, int64_t hidden) {
  int sms = 0;
  if (rows < 0 || hidden <= 0 || hidden > kMaxHidden || device_check(&sms) != FLCE_OK) return 0;
  const int64_t parts = norm_partial_rows(rows, hidden, sms);
  return kHeaderBytes + 2 * round256(sizeof(float) * static_cast<size_t>(parts > 0 ? parts : 1) * hidden);
}

int flce_layer_norm_backward(const void* grad_y, int64_t ld_grad_y, const void* x, int64_t ld_x, int dtype,
                             int64_t rows, int64_t hidden, const void* weight, int weight_dtype, const float* mean,
                             const float* rstd, int rms, void* grad_x, float* grad_weight, float* grad_bias,
                             int accumulate, void* workspace, size_t workspace_bytes, void* stream_handle) {
  if (!dtype_ok(dtype) || !dtype_ok(weight_dtype) || rows < 0 || rows > kMaxRows || hidden <= 0 || hidden > kMaxHidden ||
      ld_x < hidden || ld_grad_y < hidden)
    return FLCE_ERR_ARG;
  if (!grad_x && !grad_weight && !grad_bias) return FLCE_OK;
  const bool sums = grad_weight || grad_bias;
  if (rows > 0 && (!x || !grad_y || !rstd || (!rms && !mean))) return FLCE_ERR_ARG;
  if (sums && !workspace) return FLCE_ERR_ARG;
  const size_t es = element_size(dtype);
  if (!aligned(x, es) || !aligned(grad_y, es) || !aligned(grad_x, es) ||
      !aligned(weight, element_size(weight_dtype)) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      !aligned(grad_weight, 4) || !aligned(grad_bias, 4) || !aligned(workspace, 16))
    return FLCE_ERR_ALIGN;
  if (rows > 0 && grad_x &&
      (!apart_or_same(x, ld_x, grad_x, rows, hidden, es) || !apart_or_same(grad_y, ld_grad_y, grad_x, rows, hidden, es)))
    return FLCE_ERR_ARG;
  int sms = 0;
  const int rc = device_check(&sms);
  if (rc != FLCE_OK) return rc;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  const size_t half = round256(sizeof(float) * static_cast<size_t>(rows > 0 ? norm_partial_rows(rows, hidden, sms) : 1) * hidden);
  if (sums && workspace_bytes < kHeaderBytes + 2 * half) return FLCE_ERR_WORKSPACE;
  NormParams p = {};
  p.x = x;
  p.gy = grad_y;
  p.dtype = dtype;
  p.rows = rows;
  p.hidden = hidden;
  p.ld_x = ld_x;
  p.ld_gy = ld_grad_y;
  p.weight = weight;
  p.w_f32 = weight_dtype == FLCE_DTYPE_F32;
  p.rms = rms != 0;
  p.out = grad_x;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  char* ws = static_cast<char*>(workspace) + kHeaderBytes;
  p.part_w = grad_weight ? reinterpret_cast<float*>(ws) : nullptr;
  p.part_b = grad_bias ? reinterpret_cast<float*>(ws + half) : nullptr;
  int partials = 0;
  if (rows > 0) FLCE_LAUNCH(K_NORM_BWD, launch_norm_bwd(p, sms, &partials, stream));
  if (sums)
    FLCE_LAUNCH(K_NORM_WGRAD, launch_norm_wgrad(p.part_w, p.part_b, partials, hidden, grad_weight, grad_bias,
                                                accumulate, stream));
  return FLCE_OK;
}

size_t flce_microscale_codes_size(int64_t rows, int64_t cols) {
  return mx_shape_ok(rows, cols) ? mx_codes(rows, cols) : 0;
}

size_t flce_microscale_scales_size(int64_t rows, int64_t cols) {
  return mx_shape_ok(rows, cols) ? mx_scales(rows, cols) : 0;
}

int flce_microscale_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld_x, void* codes,
                             void* scales, void* stream_handle) {
  if (!dtype_ok(dtype) || !mx_shape_ok(rows, cols) || ld_x < cols) return FLCE_ERR_ARG;
  if (rows == 0) return FLCE_OK;
  if (!x) return FLCE_ERR_ARG;
  if (!aligned(x, element_size(dtype))) return FLCE_ERR_ALIGN;
  int rc = mx_buffers(rows, codes, scales);
  if (rc != FLCE_OK) return rc;
  int sms = 0;
  if ((rc = device_check(&sms)) != FLCE_OK) return rc;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  MxQuantParams q = {x, dtype, rows, cols, ld_x, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales)};
  FLCE_LAUNCH(K_MX_QUANT, launch_mx_quantize(q, sms, stream));
  return FLCE_OK;
}

int flce_microscale_dequantize(const void* codes, const void* scales, int64_t rows, int64_t cols, void* out,
                               int out_dtype, void* stream_handle) {
  if (!dtype_ok(out_dtype) || !mx_shape_ok(rows, cols)) return FLCE_ERR_ARG;
  if (rows == 0) return FLCE_OK;
  if (!out) return FLCE_ERR_ARG;
  if (!aligned(out, 32)) return FLCE_ERR_ALIGN;
  int rc = mx_buffers(rows, codes, scales);
  if (rc != FLCE_OK) return rc;
  int sms = 0;
  if ((rc = device_check(&sms)) != FLCE_OK) return rc;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  FLCE_LAUNCH(K_MX_DEQUANT, launch_mx_dequantize(static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales),
                                                 rows, cols, out, out_dtype, stream));
  return FLCE_OK;
}

size_t flce_microscale_workspace_size(int64_t rows, int64_t cols) {
  if (!mx_shape_ok(rows, cols)) return 0;
  return kHeaderBytes + round256(mx_codes(rows, cols)) + round256(mx_scales(rows, cols));
}

int flce_microscale_matmul(const void* a_codes, const void* a_scales, int64_t rows, const void* w_codes,
                           const void* w_scales, int64_t vocab, int64_t cols, float out_mult, float softcap, void* out,
                           int out_dtype, int64_t ld_out, void* workspace, size_t workspace_bytes,
                           void* stream_handle) {
  int rc = check_product(rows, vocab, cols, w_codes, w_scales, out_mult, softcap, out, out_dtype, &ld_out, workspace);
  if (rc != FLCE_OK) return rc;
  if ((rc = mx_buffers(rows, a_codes, a_scales)) != FLCE_OK) return rc;
  if (rows == 0) return FLCE_OK;
  if (workspace_bytes < kHeaderBytes) return FLCE_ERR_WORKSPACE;
  int sms = 0;
  if ((rc = device_check(&sms)) != FLCE_OK) return rc;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  return launch_mx_gemm(product(rows, vocab, cols, a_codes, a_scales, w_codes, w_scales, out_mult, softcap, out,
                                out_dtype, ld_out, workspace),
                        sms, stream);
}

int flce_microscale_linear(const void* x, int dtype, int64_t ld_x, int64_t rows, const void* w_codes,
                           const void* w_scales, int64_t vocab, int64_t cols, float out_mult, float softcap, void* out,
                           int out_dtype, int64_t ld_out, void* workspace, size_t workspace_bytes,
                           void* stream_handle) {
  return flce_microscale_linear_limited(x, dtype, ld_x, rows, w_codes, w_scales, vocab, cols, out_mult, softcap, out,
                                        out_dtype, ld_out, workspace, workspace_bytes, 0, 0, stream_handle);
}

int flce_microscale_linear_limited(const void* x, int dtype, int64_t ld_x, int64_t rows, const void* w_codes,
                                   const void* w_scales, int64_t vocab, int64_t cols, float out_mult, float softcap,
                                   void* out, int out_dtype, int64_t ld_out, void* workspace, size_t workspace_bytes,
                                   int64_t timeout_ns, int flags, void* stream_handle) {
  if (timeout_ns < 0 || (flags & ~FLCE_FLAG_TEST_STALL)) return FLCE_ERR_ARG;
  int rc = check_product(rows, vocab, cols, w_codes, w_scales, out_mult, softcap, out, out_dtype, &ld_out, workspace);
  if (rc != FLCE_OK) return rc;
  if (!dtype_ok(dtype) || ld_x < cols) return FLCE_ERR_ARG;
  if (rows == 0) return FLCE_OK;
  if (!x) return FLCE_ERR_ARG;
  if (!aligned(x, element_size(dtype))) return FLCE_ERR_ALIGN;
  if (workspace_bytes < flce_microscale_workspace_size(rows, cols)) return FLCE_ERR_WORKSPACE;
  int sms = 0;
  if ((rc = device_check(&sms)) != FLCE_OK) return rc;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  uint8_t* codes = static_cast<uint8_t*>(workspace) + kHeaderBytes;
  uint8_t* scales = codes + round256(mx_codes(rows, cols));
  MxGemmParams g = product(rows, vocab, cols, codes, scales, w_codes, w_scales, out_mult, softcap, out, out_dtype, ld_out,
                           workspace);
  if (timeout_ns > 0) g.timeout_ns = static_cast<uint64_t>(timeout_ns);
  g.stall = (flags & FLCE_FLAG_TEST_STALL) != 0;
  if (mx_gemm_encodes(rows, cols)) {
    g.x = x;
    g.x_dtype = dtype;
    g.ld_x = ld_x;
  } else {
    MxQuantParams q = {x, dtype, rows, cols, ld_x, codes, scales};
    FLCE_LAUNCH(K_MX_QUANT, launch_mx_quantize(q, sms, stream));
  }
  return launch_mx_gemm(g, sms, stream);
}

int flce_sample(const void* logits, int logits_dtype, int64_t rows, int64_t vocab, int64_t ld_logits, const float* u,
                const float* temperatures, float temperature, const int32_t* top_ks, int32_t top_k,
                const float* top_ps, float top_p, const float* min_ps, float min_p, int64_t* tokens, float* logprobs,
                void* stream_handle) {
  if (!dtype_ok(logits_dtype) || rows < 0 || rows > kMaxRows / 8 || vocab <= 0 || vocab >= (int64_t{1} << 22) ||
      ld_logits < vocab)
    return FLCE_ERR_ARG;
  if ((!temperatures && std::isnan(temperature)) || (!top_ps && std::isnan(top_p)) || (!min_ps && std::isnan(min_p)))
    return FLCE_ERR_ARG;
  if (rows == 0) return FLCE_OK;
  if (!logits || !u || !tokens) return FLCE_ERR_ARG;
  if (!aligned(logits, element_size(logits_dtype)) || !aligned(u, 4) || !aligned(temperatures, 4) ||
      !aligned(top_ks, 4) || !aligned(top_ps, 4) || !aligned(min_ps, 4) || !aligned(tokens, 8) || !aligned(logprobs, 4))
    return FLCE_ERR_ALIGN;
  int sms = 0;
  const int rc = device_check(&sms);
  if (rc != FLCE_OK) return rc;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  SampleParams p = {};
  p.x = logits;
  p.dtype = logits_dtype;
  p.rows = rows;
  p.vocab = vocab;
  p.ld = ld_logits;
  p.u = u;
  p.temperatures = temperatures;
  p.temperature = temperature;
  p.top_ks = top_ks;
  p.top_k = top_k;
  p.top_ps = top_ps;
  p.top_p = top_p;
  p.min_ps = min_ps;
  p.min_p = min_p;
  p.tokens = tokens;
  p.logprobs = logprobs;
  FLCE_LAUNCH(K_SAMPLE, launch_sample(p, sms, stream));
  return FLCE_OK;
}

}  // extern "C"
