// Host entries of the operators at a model's two ends (include/flce_model.h): argument
// checks, workspace carving and launches. No allocation, no host synchronisation,
// errors returned before any launch.
#include <cuda_runtime.h>

#include <cmath>

#include "flce_host.h"
#include "flce_internal.h"
#include "model_internal.h"

using namespace flce;

namespace {

constexpr int64_t kMaxHidden = int64_t{1} << 24;
constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1;
constexpr int64_t kMostDrafts = 1024;
constexpr int64_t kBlock = 32;  // elements of a checkpoint that share a scale

inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }
inline bool dtype_ok(int d) { return d == FLCE_DTYPE_BF16 || d == FLCE_DTYPE_F32; }
inline size_t element_size(int d) { return d == FLCE_DTYPE_F32 ? 4 : 2; }
inline bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
inline bool shape_ok(int64_t rows, int64_t hidden) { return rows >= 0 && rows <= kMaxRows && hidden > 0 && hidden <= kMaxHidden; }
inline int64_t blocks(int64_t hidden) { return (hidden + kBlock - 1) / kBlock; }

// A matrix in memory; NULL lies apart from everything.
struct Span {
  const void* p;
  size_t bytes;
};
inline Span matrix(const void* p, int64_t rows, int64_t ld, int64_t hidden, size_t es) {
  return {p, rows > 0 ? (static_cast<size_t>(rows - 1) * ld + hidden) * es : 0};
}
inline bool apart(const Span& a, const Span& b) {
  if (!a.p || !b.p) return true;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x + a.bytes <= y || y + b.bytes <= x;
}
// Outputs apart from the inputs and from each other.
template <int O, int I>
bool outputs_apart(const Span (&out)[O], const Span (&in)[I]) {
  for (int o = 0; o < O; ++o) {
    for (int i = 0; i < I; ++i)
      if (!apart(out[o], in[i])) return false;
    for (int i = 0; i < o; ++i)
      if (!apart(out[o], out[i])) return false;
  }
  return true;
}

int device_check(int* sms) {
  int cc = 0;
  const int rc = device_info(sms, &cc);
  if (rc != FLCE_OK) return rc;
  return cc == 103 ? FLCE_OK : FLCE_ERR_UNSUPPORTED;
}

// Workspace of the embedding's gradient.
struct EmbeddingSpace {
  size_t keys, sums, joins;
  size_t total() const { return 4 * keys + 2 * sums + joins; }
};
EmbeddingSpace embedding_space(int64_t rows, int64_t hidden) {
  const size_t tiles = static_cast<size_t>((rows + kEmbeddingTile - 1) / kEmbeddingTile);
  return {round256(sizeof(uint32_t) * static_cast<size_t>(rows)), round256(sizeof(float) * tiles * static_cast<size_t>(hidden)),
          rows > 0 ? round256(sizeof(uint32_t) * (tiles + 2)) : 0};
}

// Rows that a verification looks at, -1 if there are too many.
int64_t verify_rows(int64_t batch, int64_t drafts, bool with_draft) {
  if (batch < 0 || drafts < 0 || drafts > kMostDrafts || batch > kMaxRows / 8 / (2 * drafts + 1)) return -1;
  return batch * (with_draft ? 2 * drafts + 1 : drafts + 1);
}

}  // namespace

extern "C" {

int flce_checkpoint_store(const void* x, int dtype, int64_t rows, int64_t hidden, int64_t ld_x, void* codes, void* scales,
                          void* stream_handle) {
  if (!dtype_ok(dtype) || !shape_ok(rows, hidden) || ld_x < hidden) return FLCE_ERR_ARG;
  if (rows == 0) return FLCE_OK;
  if (!x || !codes || !scales) return FLCE_ERR_ARG;
  const size_t es = element_size(dtype);
  if (!aligned(x, es)) return FLCE_ERR_ALIGN;
  const Span in[] = {matrix(x, rows, ld_x, hidden, es)};
  const Span out[] = {matrix(codes, rows, hidden, hidden, 1), matrix(scales, rows, blocks(hidden), blocks(hidden), 1)};
  if (!outputs_apart(out, in)) return FLCE_ERR_ARG;
  int sms = 0;
  const int rc = device_check(&sms);
  if (rc != FLCE_OK) return rc;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  CheckpointParams p = {};
  p.x = x;
  p.dtype = dtype;
  p.rows = rows;
  p.hidden = hidden;
  p.ld = ld_x;
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = static_cast<uint8_t*>(scales);
  FLCE_LAUNCH(K_CHECKPOINT_STORE, launch_checkpoint_store(p, stream));
  return FLCE_OK;
}

int flce_checkpoint_load(const void* codes, const void* scales, int64_t rows, int64_t hidden, void* out, int out_dtype,
                         void* stream_handle) {
  if (!dtype_ok(out_dtype) || !shape_ok(rows, hidden)) return FLCE_ERR_ARG;
  if (rows == 0) return FLCE_OK;
  if (!codes || !scales || !out) return FLCE_ERR_ARG;
  const size_t es = element_size(out_dtype);
  if (!aligned(out, es)) return FLCE_ERR_ALIGN;
  const Span in[] = {matrix(codes, rows, hidden, hidden, 1), matrix(scales, rows, blocks(hidden), blocks(hidden), 1)};
  const Span to[] = {matrix(out, rows, hidden, hidden, es)};
  if (!outputs_apart(to, in)) return FLCE_ERR_ARG;
  int sms = 0;
  const int rc = device_check(&sms);
  if (rc != FLCE_OK) return rc;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  CheckpointParams p = {};
  p.out = out;
  p.dtype = out_dtype;
  p.rows = rows;
  p.hidden = hidden;
  p.ld = hidden;
  p.codes = static_cast<uint8_t*>(const_cast<void*>(codes));
  p.scales = static_cast<uint8_t*>(const_cast<void*>(scales));
  FLCE_LAUNCH(K_CHECKPOINT_LOAD, launch_checkpoint_load(p, stream));
  return FLCE_OK;
}

int flce_add_layer_norm(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual, int dtype, int64_t rows,
                        int64_t hidden, const void* weight, const void* bias, int weight_dtype, float eps, int rms, void* y,
                        void* sum, void* codes, void* scales, float* mean, float* rstd, void* stream_handle) {
  if (!dtype_ok(dtype) || !dtype_ok(weight_dtype) || !shape_ok(rows, hidden) || ld_x < hidden ||
      (residual && ld_residual < hidden) || !(eps >= 0.f) || !std::isfinite(eps) || !codes != !scales)
    return FLCE_ERR_ARG;
  if (rows == 0) return FLCE_OK;
  if (!x || !y) return FLCE_ERR_ARG;
  const size_t es = element_size(dtype), ws = element_size(weight_dtype);
  if (!aligned(x, es) || !aligned(residual, es) || !aligned(y, es) || !aligned(sum, es) || !aligned(weight, ws) ||
      !aligned(bias, ws) || !aligned(mean, 4) || !aligned(rstd, 4))
    return FLCE_ERR_ALIGN;
  const Span in[] = {matrix(x, rows, ld_x, hidden, es), matrix(residual, rows, ld_residual, hidden, es),
                     matrix(weight, 1, hidden, hidden, ws), matrix(bias, 1, hidden, hidden, ws)};
  const Span out[] = {matrix(y, rows, hidden, hidden, es), matrix(sum, rows, hidden, hidden, es),
                      matrix(codes, rows, hidden, hidden, 1), matrix(scales, rows, blocks(hidden), blocks(hidden), 1),
                      matrix(rms ? nullptr : mean, rows, 1, 1, 4), matrix(rstd, rows, 1, 1, 4)};
  if (!outputs_apart(out, in)) return FLCE_ERR_ARG;
  int sms = 0;
  const int rc = device_check(&sms);
  if (rc != FLCE_OK) return rc;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  AddNormParams p = {};
  p.x = x;
  p.dtype = dtype;
  p.rows = rows;
  p.hidden = hidden;
  p.ld_x = ld_x;
  p.residual = residual;
  p.ld_res = residual ? ld_residual : hidden;
  p.weight = weight;
  p.bias = bias;
  p.w_f32 = weight_dtype == FLCE_DTYPE_F32;
  p.eps = eps;
  p.rms = rms != 0;
  p.out = y;
  p.sum = sum;
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = static_cast<uint8_t*>(scales);
  p.mean = mean;
  p.rstd = rstd;
  FLCE_LAUNCH(K_ADD_NORM, launch_add_norm(p, sms, stream));
  return FLCE_OK;
}

size_t flce_add_layer_norm_workspace_size(int64_t rows, int64_t hidden) {
  int sms = 0;
  if (!shape_ok(rows, hidden) || device_check(&sms) != FLCE_OK) return 0;
  const int64_t parts = add_norm_partial_rows(rows, hidden, sms);
  return 2 * round256(sizeof(float) * static_cast<size_t>(parts > 0 ? parts : 1) * hidden);
}

int flce_add_layer_norm_backward(const void* grad_y, int64_t ld_grad_y, const void* grad_sum, int64_t ld_grad_sum, const void* x,
                                 int64_t ld_x, const void* codes, const void* scales, int dtype, int64_t rows, int64_t hidden,
                                 const void* weight, int weight_dtype, const float* mean, const float* rstd, int rms, void* grad_x,
                                 float* grad_weight, float* grad_bias, int accumulate, void* workspace, size_t workspace_bytes,
                                 void* stream_handle) {
  if (!dtype_ok(dtype) || !dtype_ok(weight_dtype) || !shape_ok(rows, hidden) || (x && ld_x < hidden) || ld_grad_y < hidden ||
      (grad_sum && ld_grad_sum < hidden) || !codes != !scales || (x && codes))
    return FLCE_ERR_ARG;
  if (!grad_x && !grad_weight && !grad_bias) return FLCE_OK;
  const bool sums = grad_weight || grad_bias;
  if (rows > 0 && ((!x && !codes) || !grad_y || !rstd || (!rms && !mean))) return FLCE_ERR_ARG;
  if (sums && !workspace) return FLCE_ERR_ARG;
  const size_t es = element_size(dtype), wes = element_size(weight_dtype);
  if (!aligned(x, es) || !aligned(grad_y, es) || !aligned(grad_sum, es) || !aligned(grad_x, es) || !aligned(weight, wes) ||
      !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(grad_weight, 4) || !aligned(grad_bias, 4) || !aligned(workspace, 16))
    return FLCE_ERR_ALIGN;
  const Span in[] = {matrix(x, rows, ld_x, hidden, es), matrix(grad_y, rows, ld_grad_y, hidden, es),
                     matrix(grad_sum, rows, ld_grad_sum, hidden, es), matrix(codes, rows, hidden, hidden, 1),
                     matrix(scales, rows, blocks(hidden), blocks(hidden), 1), matrix(weight, 1, hidden, hidden, wes),
                     matrix(rms ? nullptr : mean, rows, 1, 1, 4), matrix(rstd, rows, 1, 1, 4)};
  const Span out[] = {matrix(grad_x, rows, hidden, hidden, es), matrix(grad_weight, 1, hidden, hidden, 4),
                      matrix(grad_bias, 1, hidden, hidden, 4), {sums ? workspace : nullptr, workspace_bytes}};
  if (!outputs_apart(out, in)) return FLCE_ERR_ARG;
  int sms = 0;
  const int rc = device_check(&sms);
  if (rc != FLCE_OK) return rc;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  const size_t half = round256(sizeof(float) * static_cast<size_t>(rows > 0 ? add_norm_partial_rows(rows, hidden, sms) : 1) * hidden);
  if (sums && workspace_bytes < 2 * half) return FLCE_ERR_WORKSPACE;
  AddNormParams p = {};
  p.x = x;
  p.ld_x = x ? ld_x : hidden;
  p.codes = static_cast<uint8_t*>(const_cast<void*>(codes));
  p.scales = static_cast<uint8_t*>(const_cast<void*>(scales));
  p.gy = grad_y;
  p.ld_gy = ld_grad_y;
  p.gs = grad_sum;
  p.ld_gs = grad_sum ? ld_grad_sum : hidden;
  p.dtype = dtype;
  p.rows = rows;
  p.hidden = hidden;
  p.weight = weight;
  p.w_f32 = weight_dtype == FLCE_DTYPE_F32;
  p.rms = rms != 0;
  p.out = grad_x;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  char* ws = static_cast<char*>(workspace);
  p.part_w = grad_weight ? reinterpret_cast<float*>(ws) : nullptr;
  p.part_b = grad_bias ? reinterpret_cast<float*>(ws + half) : nullptr;
  int partials = 0;
  if (rows > 0)
    FLCE_LAUNCH(K_ADD_NORM_BWD, codes ? launch_add_norm_bwd_8bit(p, sms, &partials, stream) : launch_add_norm_bwd(p, sms, &partials, stream));
  if (sums)
    FLCE_LAUNCH(K_NORM_WGRAD, launch_norm_wgrad(p.part_w, p.part_b, partials, hidden, grad_weight, grad_bias, accumulate, stream));
  return FLCE_OK;
}

int flce_embedding(const int64_t* tokens, int64_t rows, const void* W, int dtype, int64_t ld_w, int64_t vocab, int64_t hidden,
                   float scale, void* out, int out_dtype, void* stream_handle) {
  if (!dtype_ok(dtype) || !dtype_ok(out_dtype) || !shape_ok(rows, hidden) || vocab <= 0 || vocab >= kMaxRows || ld_w < hidden ||
      !std::isfinite(scale))
    return FLCE_ERR_ARG;
  if (rows == 0) return FLCE_OK;
  if (!tokens || !W || !out) return FLCE_ERR_ARG;
  const size_t es = element_size(dtype), os = element_size(out_dtype);
  if (!aligned(tokens, 8) || !aligned(W, es) || !aligned(out, os)) return FLCE_ERR_ALIGN;
  const Span in[] = {{tokens, static_cast<size_t>(rows) * 8}, matrix(W, vocab, ld_w, hidden, es)};
  const Span to[] = {matrix(out, rows, hidden, hidden, os)};
  if (!outputs_apart(to, in)) return FLCE_ERR_ARG;
  int sms = 0;
  const int rc = device_check(&sms);
  if (rc != FLCE_OK) return rc;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  EmbeddingParams p = {};
  p.tokens = tokens;
  p.rows = rows;
  p.vocab = vocab;
  p.hidden = hidden;
  p.ld = ld_w;
  p.scale = scale;
  p.dtype = dtype;
  p.out_dtype = out_dtype;
  p.in = W;
  p.out = out;
  FLCE_LAUNCH(K_EMBEDDING, launch_embedding(p, stream));
  return FLCE_OK;
}

size_t flce_embedding_workspace_size(int64_t rows, int64_t hidden) {
  return shape_ok(rows, hidden) ? embedding_space(rows, hidden).total() : 0;
}

int flce_embedding_backward(const void* grad_out, int dtype, int64_t ld_grad, const int64_t* tokens, int64_t rows, int64_t vocab,
                            int64_t hidden, float scale, float* grad_W, int accumulate, void* workspace, size_t workspace_bytes,
                            void* stream_handle) {
  if (!dtype_ok(dtype) || !shape_ok(rows, hidden) || vocab <= 0 || vocab >= kMaxRows || ld_grad < hidden || !std::isfinite(scale) ||
      !grad_W)
    return FLCE_ERR_ARG;
  if (rows > 0 && (!grad_out || !tokens || !workspace)) return FLCE_ERR_ARG;
  // (grids: at most a CTA per tile and 512 columns and one per token of the vocabulary, 65535 groups of 32768 tokens)
  if (rows > int64_t{65535} * 32768 || (rows / kEmbeddingTile + 1) * (hidden / 512 + 1) + vocab > kMaxRows) return FLCE_ERR_ARG;
  const size_t es = element_size(dtype);
  if (!aligned(grad_out, es) || !aligned(tokens, 8) || !aligned(grad_W, 4) || !aligned(workspace, 16)) return FLCE_ERR_ALIGN;
  const EmbeddingSpace space = embedding_space(rows, hidden);
  if (rows > 0 && workspace_bytes < space.total()) return FLCE_ERR_WORKSPACE;
  const Span in[] = {{rows > 0 ? tokens : nullptr, static_cast<size_t>(rows) * 8}, matrix(rows > 0 ? grad_out : nullptr, rows, ld_grad, hidden, es)};
  const Span out[] = {matrix(grad_W, vocab, hidden, hidden, 4), {rows > 0 ? workspace : nullptr, space.total()}};
  if (!outputs_apart(out, in)) return FLCE_ERR_ARG;
  int sms = 0;
  const int rc = device_check(&sms);
  if (rc != FLCE_OK) return rc;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  EmbeddingParams p = {};
  p.tokens = tokens;
  p.rows = rows;
  p.vocab = vocab;
  p.hidden = hidden;
  p.ld = ld_grad;
  p.scale = scale;
  p.dtype = dtype;
  p.in = grad_out;
  p.out = grad_W;
  p.accumulate = accumulate != 0;
  if (rows > 0) {
    char* ws = static_cast<char*>(workspace);
    p.sorted = reinterpret_cast<uint32_t*>(ws);
    p.places = reinterpret_cast<uint32_t*>(ws + space.keys);
    p.sorted2 = reinterpret_cast<uint32_t*>(ws + 2 * space.keys);
    p.places2 = reinterpret_cast<uint32_t*>(ws + 3 * space.keys);
    p.head = reinterpret_cast<float*>(ws + 4 * space.keys);
    p.tail = reinterpret_cast<float*>(ws + 4 * space.keys + space.sums);
    p.joins = reinterpret_cast<uint32_t*>(ws + 4 * space.keys + 2 * space.sums);
    const int sorted = launch_embedding_sort(&p, sms, stream);
    if (sorted != FLCE_OK) return sorted;
  }
  return launch_embedding_grad(p, stream);
}

size_t flce_verify_workspace_size(int64_t batch, int64_t drafts) {
  const int64_t rows = verify_rows(batch, drafts, true);
  return rows < 0 ? 0 : (sizeof(RowCut) + sizeof(uint32_t)) * static_cast<size_t>(rows);
}

int flce_verify(const void* target, int logits_dtype, int64_t batch, int64_t drafts, int64_t vocab, int64_t ld_target,
                int64_t batch_ld_target, const int64_t* draft_tokens, const void* draft, int64_t ld_draft, int64_t batch_ld_draft,
                const float* u, const float* temperatures, float temperature, const int32_t* top_ks, int32_t top_k,
                const float* top_ps, float top_p, const float* min_ps, float min_p, int64_t* tokens, int64_t* accepted,
                float* logprobs, void* workspace, size_t workspace_bytes, void* stream_handle) {
  if (drafts == 0) draft = nullptr;
  const int64_t rows = verify_rows(batch, drafts, draft != nullptr);
  if (!dtype_ok(logits_dtype) || rows < 0 || vocab <= 0 || vocab >= (int64_t{1} << 22) || ld_target < 0 || batch_ld_target < 0 ||
      (draft && (ld_draft < 0 || batch_ld_draft < 0)))
    return FLCE_ERR_ARG;
  if ((!temperatures && std::isnan(temperature)) || (!top_ps && std::isnan(top_p)) || (!min_ps && std::isnan(min_p)))
    return FLCE_ERR_ARG;
  if (batch == 0) return FLCE_OK;
  if (!target || !u || !tokens || !accepted || !workspace || (drafts > 0 && !draft_tokens)) return FLCE_ERR_ARG;
  const size_t es = element_size(logits_dtype);
  if (!aligned(target, es) || !aligned(draft, es) || !aligned(u, 4) || !aligned(draft_tokens, 8) || !aligned(temperatures, 4) ||
      !aligned(top_ks, 4) || !aligned(top_ps, 4) || !aligned(min_ps, 4) || !aligned(tokens, 8) || !aligned(accepted, 8) ||
      !aligned(logprobs, 4) || !aligned(workspace, 16))
    return FLCE_ERR_ALIGN;
  // (as many words as rows of the target follow the cuts)
  const size_t space = (sizeof(RowCut) + sizeof(uint32_t)) * static_cast<size_t>(rows);
  if (workspace_bytes < space) return FLCE_ERR_WORKSPACE;
  const size_t b = static_cast<size_t>(batch), places = b * (static_cast<size_t>(drafts) + 1);
  const Span in[] = {{target, ((b - 1) * batch_ld_target + drafts * ld_target + vocab) * es},
                     {draft, draft ? ((b - 1) * batch_ld_draft + (drafts - 1) * ld_draft + vocab) * es : 0},
                     {u, places * 4}, {draft_tokens, b * drafts * 8}, {temperatures, b * 4}, {top_ks, b * 4}, {top_ps, b * 4},
                     {min_ps, b * 4}};
  const Span out[] = {{tokens, places * 8}, {accepted, b * 8}, {logprobs, places * 4}, {workspace, space}};
  if (!outputs_apart(out, in)) return FLCE_ERR_ARG;
  int sms = 0;
  const int rc = device_check(&sms);
  if (rc != FLCE_OK) return rc;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  VerifyParams p = {};
  p.x = target;
  p.dtype = logits_dtype;
  p.rows = rows;
  p.vocab = vocab;
  p.ld = ld_target;
  p.batch_ld = batch_ld_target;
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
  p.draft = draft;
  p.draft_ld = ld_draft;
  p.draft_batch_ld = batch_ld_draft;
  p.draft_tokens = draft_tokens;
  p.drafts = drafts;
  p.target_rows = batch * (drafts + 1);
  p.cuts = static_cast<RowCut*>(workspace);
  p.progress = reinterpret_cast<uint32_t*>(p.cuts + rows);
  FLCE_LAUNCH(K_VERIFY_CUT, launch_verify_cuts(p, sms, stream));
  FLCE_LAUNCH(K_VERIFY, launch_verify(p, batch, accepted, sms, stream));
  return FLCE_OK;
}

}  // extern "C"
