/*
 * flce_model.h - C ABI of the operators at the two ends of a model whose head is
 * the fused linear cross-entropy: embeddings in the head's weight, the residual's
 * addition with the norm behind it, 8-bit checkpoints of what that norm keeps for
 * its backward pass, and the verification of drafted tokens.
 *
 * The conventions of flce.h and flce_head.h hold: device pointers owned by the
 * caller, no allocation, no host synchronisation, asynchronous on `stream`, FLCE_*
 * return codes found on the host before any launch, nothing trapped or thrown, the
 * current device owns the stream and every pointer. Element types are
 * FLCE_DTYPE_BF16 and FLCE_DTYPE_F32; every sum and statistic is held in 32 bits
 * or more, and bf16 results are rounded once (to nearest even). Outputs overlap
 * neither each other nor an input. The calls find no errors on the device; their
 * workspaces hold no status.
 */
#ifndef FLCE_MODEL_H
#define FLCE_MODEL_H

#include "flce_head.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- 8-bit checkpoints
 * A matrix [rows, H] of activations in 8 bits with a scale for each 32 consecutive
 * elements of a row (the last block of a row may be shorter):
 *   e    = the least whole number >= -127 with max |x| of the block <= 448 2^e
 *   code = x 2^-e rounded to nearest (ties to even) in E4M3, to 240 at most where e = 120,
 *          as 256 2^120 is beyond fp32: what is finite reads back finite
 * codes [rows, H] bytes and scales [rows, ceil(H / 32)] bytes (e + 127, E8M0), both
 * contiguous. A block with an infinity or NaN gets the NaN scale (255) and reads
 * back as NaN. H up to 2^24. flce_checkpoint_load writes what they stand for,
 * out [rows, H] contiguous, in out_dtype (exact but below its normal range). */
int flce_checkpoint_store(const void* x, int dtype, int64_t rows, int64_t hidden, int64_t ld_x, void* codes, void* scales,
                          void* stream);
int flce_checkpoint_load(const void* codes, const void* scales, int64_t rows, int64_t hidden, void* out, int out_dtype,
                         void* stream);

/* ---------------------------------------------------------------- residual and norm
 *   s = x + residual, rounded to x's type;  y = norm(s), as flce_layer_norm of s
 * residual [rows, ld_residual], NULL for s = x. sum [rows, H] gets s, codes and
 * scales its 8-bit checkpoint; sum, and codes with scales, are nullable. The rest is
 * as in flce_layer_norm; y, sum, codes are contiguous. */
int flce_add_layer_norm(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual, int dtype, int64_t rows,
                        int64_t hidden, const void* weight, const void* bias, int weight_dtype, float eps, int rms, void* y,
                        void* sum, void* codes, void* scales, float* mean, float* rstd, void* stream);

/* Backward, from s (x [rows, ld_x]) or, where x is NULL, from its checkpoint, and the
 * saved statistics:
 *   grad_x = grad_sum + the norm's gradient (flce_layer_norm_backward of grad_y),
 * rounded once to `dtype`, the type of grad_y, grad_sum, grad_x and x; it is the gradient
 * of x and of the residual alike. grad_sum is the gradient of s from its other uses, NULL
 * for none. The rest is as in flce_layer_norm_backward. */
size_t flce_add_layer_norm_workspace_size(int64_t rows, int64_t hidden);
int flce_add_layer_norm_backward(const void* grad_y, int64_t ld_grad_y, const void* grad_sum, int64_t ld_grad_sum, const void* x,
                                 int64_t ld_x, const void* codes, const void* scales, int dtype, int64_t rows, int64_t hidden,
                                 const void* weight, int weight_dtype, const float* mean, const float* rstd, int rms, void* grad_x,
                                 float* grad_weight, float* grad_bias, int accumulate, void* workspace, size_t workspace_bytes,
                                 void* stream);

/* ---------------------------------------------------------------- embeddings
 *   out[i] = scale W[tokens[i]],  W [vocab, ld_w], out [rows, H] contiguous in out_dtype
 * A negative token stands for none and gives a row of zeros; one at or behind the
 * vocabulary gives a row of NaN. */
int flce_embedding(const int64_t* tokens, int64_t rows, const void* W, int dtype, int64_t ld_w, int64_t vocab, int64_t hidden,
                   float scale, void* out, int out_dtype, void* stream);

/* Its gradient: grad_W[t] = scale (sum of grad_out[i] over i with tokens[i] = t), fp32
 * [vocab, H] contiguous, summed in an order that depends on the tokens alone: results do
 * not change from run to run. accumulate != 0 adds it to what grad_W holds (the fused
 * head's accumulator, for a weight that is both), else absent tokens' rows are zeroed.
 * That addition takes numbers below 2^-126 as zero, in grad_W and in its result.
 * Tokens outside of the vocabulary count for nothing. vocab < 2^31 - 1, rows up to
 * 65535 x 32768. */
size_t flce_embedding_workspace_size(int64_t rows, int64_t hidden);
int flce_embedding_backward(const void* grad_out, int dtype, int64_t ld_grad, const int64_t* tokens, int64_t rows, int64_t vocab,
                            int64_t hidden, float scale, float* grad_W, int accumulate, void* workspace, size_t workspace_bytes,
                            void* stream);

/* ---------------------------------------------------------------- verification
 * For each of `batch` requests: `drafts` drafted tokens d_i, drawn one after another
 * from a draft model, and the target's logits at their places and at the one behind
 * them. With p_i the distribution that flce_sample draws from for the target's row i
 * (whole weights w of the tokens that the request's temperature, top_k, top_p and min_p
 * keep, W their sum, p = w / W), and q_i that for the draft's row i under the same settings
 * (logits of a draft sampled at another temperature are scaled first), or, where `draft` is
 * NULL, all weight on d_i:
 *   accepted  the drafts before the first with not u_i q_i(d_i) < p_i(d_i)  (in fp64)
 *   then one token more, at place n = accepted: where d_n was compared and not accepted,
 *   drawn from the weights r = floor(max(p_n - q_n, 0) 2^40), p and q as w (1 / W) in fp32
 *   (from those of p_n if all are 0); else, n = drafts or d_n no token, from p_n's weights:
 *   the first index at which the running sum of the weights is above u_drafts times
 *   their sum, as in flce_sample.
 * That way the tokens are distributed as if drawn from the target alone. A draft outside
 * of [0, vocab) stands for none: requests may have fewer drafts than others. tokens
 * [batch, drafts + 1]: the accepted drafts, the token drawn, -1 behind it. accepted
 * [batch]. logprobs [batch, drafts + 1], nullable: log p of each token, 0 behind the last.
 * Where a request comes to a row without a distribution (as in flce_sample: NaN or
 * +infinity, no finite logit, a NaN setting) or to a NaN u, its token there is -1, with a NaN
 * log-probability, and its last.
 * target [batch, drafts + 1, vocab] with strides of ld_target (rows) and batch_ld_target
 * (requests), draft [batch, drafts, vocab] likewise, both of logits_dtype; u [batch, drafts + 1];
 * draft_tokens [batch, drafts]. temperature and the rest: arrays of one value per request, or
 * NULL for the scalar beside it. drafts up to 1024, vocab < 2^22. */
size_t flce_verify_workspace_size(int64_t batch, int64_t drafts);
int flce_verify(const void* target, int logits_dtype, int64_t batch, int64_t drafts, int64_t vocab, int64_t ld_target,
                int64_t batch_ld_target, const int64_t* draft_tokens, const void* draft, int64_t ld_draft, int64_t batch_ld_draft,
                const float* u, const float* temperatures, float temperature, const int32_t* top_ks, int32_t top_k,
                const float* top_ps, float top_p, const float* min_ps, float min_p, int64_t* tokens, int64_t* accepted,
                float* logprobs, void* workspace, size_t workspace_bytes, void* stream);

/* Kernel ids of these operators for flce_profile_read and flce_kernel_name: a
 * read of n > FLCE_MODEL_KERNEL_FIRST entries reaches them. */
#define FLCE_MODEL_KERNEL_FIRST 48
#define FLCE_MODEL_KERNEL_COUNT 9

#ifdef __cplusplus
}
#endif

#endif /* FLCE_MODEL_H */
