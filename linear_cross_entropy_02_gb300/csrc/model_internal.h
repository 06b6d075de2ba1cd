// Internal interface between the host entries of the operators at a model's two ends
// (model_api.cpp) and their kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "flce_model.h"
#include "head_internal.h"

namespace flce {

enum ModelKernelId {
  K_ADD_NORM = FLCE_MODEL_KERNEL_FIRST,
  K_ADD_NORM_BWD,
  K_CHECKPOINT_STORE,
  K_CHECKPOINT_LOAD,
  K_EMBEDDING,
  K_EMBEDDING_SORT,
  K_EMBEDDING_GRAD,
  K_VERIFY_CUT,
  K_VERIFY,
};

// ------------------------------------------------------------ residual and norm
// (K_NORM_WGRAD joins the partial sums. A struct of its own, as is VerifyParams: the norm's and sampling's
// kernels, with more parameters than they use, were compiled to slower code.)
struct AddNormParams : NormParams {
  const void* residual;  // nullable
  int64_t ld_res;
  void* sum;             // nullable
  uint8_t* codes;        // 8-bit checkpoint: written (nullable), or read in the place of x
  uint8_t* scales;
  const void* gs;        // backward: gradient of the sum, or null
  int64_t ld_gs;
};
// Most partial rows that the backward passes write for a call on this device.
int add_norm_partial_rows(int64_t rows, int64_t hidden, int sms);
cudaError_t launch_add_norm(const AddNormParams& p, int sms, cudaStream_t s);
cudaError_t launch_add_norm_bwd(const AddNormParams& p, int sms, int* partials, cudaStream_t s);
cudaError_t launch_add_norm_bwd_8bit(const AddNormParams& p, int sms, int* partials, cudaStream_t s);

// ------------------------------------------------------------ 8-bit checkpoints
struct CheckpointParams {
  const void* x;  // store: input
  void* out;      // load: output
  int dtype;
  int64_t rows, hidden, ld;
  uint8_t* codes;
  uint8_t* scales;
};
cudaError_t launch_checkpoint_store(const CheckpointParams& p, cudaStream_t s);
cudaError_t launch_checkpoint_load(const CheckpointParams& p, cudaStream_t s);

// ------------------------------------------------------------ embeddings
struct EmbeddingParams {
  const int64_t* tokens;
  int64_t rows, vocab, hidden, ld;  // ld: row stride of W (forward) or of grad_out (backward)
  float scale;
  int dtype, out_dtype;
  const void* in;  // W, or grad_out
  void* out;       // embeddings, or grad_W (fp32)
  int accumulate;  // backward
  // backward: tokens in rising order, their positions rising within one, and the sums of
  // segments that cross tiles of kEmbeddingTile of them
  uint32_t* sorted;
  uint32_t* places;
  uint32_t* sorted2;  // the other side of a merge
  uint32_t* places2;
  float* head;
  float* tail;
  // runs that cross tiles: number of short ones, of long ones, then the tiles in which they begin, the short
  // ones' from the front, the long ones' from the end
  uint32_t* joins;
};
constexpr int kEmbeddingTile = 32;
cudaError_t launch_embedding(const EmbeddingParams& p, cudaStream_t s);
// Sorts the tokens into p->sorted and p->places, which it may swap with the other side.
int launch_embedding_sort(EmbeddingParams* p, int sms, cudaStream_t stream);
int launch_embedding_grad(const EmbeddingParams& p, cudaStream_t stream);

// ------------------------------------------------------------ verification
// What the filters keep of a row of logits: those up to `last` in rank order (list
// entries: complemented order key, index) whose exponential is at least min_p.
struct RowCut {
  uint64_t last;
  uint64_t whole;   // sum of the kept weights; 0: no distribution, the rest says nothing
  float top, inv;   // largest logit, 1 / temperature
  float min_p;
  float over;       // 1 / whole, rounded to 64 bits and then to 32
};
// Rows of the target [batch][drafts + 1] (x, with row stride ld), then of the draft [batch][drafts], if it
// has any; p.rows: all of them. u, tokens and logprobs are [batch][drafts + 1].
struct VerifyParams : SampleParams {
  const void* draft;
  const int64_t* draft_tokens;
  int64_t target_rows, drafts;
  int64_t batch_ld, draft_ld, draft_batch_ld;
  RowCut* cuts;        // of every row
  uint32_t* progress;  // [batch][drafts + 1]
};
// launch_verify_cuts fills p.cuts, launch_verify reads it.
cudaError_t launch_verify_cuts(const VerifyParams& p, int sms, cudaStream_t s);
cudaError_t launch_verify(const VerifyParams& p, int64_t batch, int64_t* accepted, int sms, cudaStream_t s);

}  // namespace flce
