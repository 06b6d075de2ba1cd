/*
 * flce_head.h - C ABI of the operators around the fused linear cross-entropy
 * head: the norm in front of it (layer norm or RMS norm, forward and
 * backward), its product on a microscaled 4-bit weight for answering, and the
 * choice of the next token from its logits.
 *
 * The conventions of flce.h hold: device pointers owned by the caller, no
 * allocation, no host synchronisation, asynchronous on `stream`, FLCE_* return
 * codes found on the host before any launch, nothing trapped or thrown, the
 * current device owns the stream and every pointer. Element types are
 * FLCE_DTYPE_BF16 and FLCE_DTYPE_F32; every sum and statistic is held in
 * 32 bits or more, and bf16 results are rounded once (to nearest even).
 */
#ifndef FLCE_HEAD_H
#define FLCE_HEAD_H

#include "flce.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- norm
 * For rows x of length H (statistics in fp32, the variance from the centred
 * values, not from a difference of squares):
 *   layer norm  y = (x - mean) rstd w + b,  rstd = (var(x) + eps)^(-1/2)
 *   RMS norm    y = x rstd w + b,           rstd = (mean(x^2) + eps)^(-1/2)
 * x [rows, ld_x] (ld_x >= H, any alignment of whole elements; 16-byte aligned
 * rows take the vector path), y [rows, H] contiguous and not overlapping x
 * unless it is x itself with ld_x = H. weight and bias [H], both of
 * weight_dtype, each NULL for 1 and 0. mean and rstd [rows] fp32: the saved
 * statistics, nullable (mean is not written with rms). H up to 2^24. */
int flce_layer_norm(const void* x, int dtype, int64_t rows, int64_t hidden, int64_t ld_x, const void* weight,
                    const void* bias, int weight_dtype, float eps, int rms, void* y, float* mean, float* rstd,
                    void* stream);

/* Backward, from x and the saved statistics (mean is not read with rms and
 * must be given without). With xhat = (x - mean) rstd and g = grad_y w:
 *   grad_x      = rstd (g - mean(g) - xhat mean(g xhat))    (rms: no mean(g))
 *   grad_weight = sum over rows of grad_y xhat               (fp32 [H])
 *   grad_bias   = sum over rows of grad_y                    (fp32 [H])
 * grad_x [rows, H] contiguous in x's dtype, not overlapping x or grad_y unless it
 * is one of them itself with a row stride of H; any of the three may be NULL.
 * accumulate != 0 adds the two sums to what grad_weight and grad_bias hold,
 * as the fused head does with grad_W. The sums are taken in a fixed order:
 * results do not change from run to run. rows = 0 gives zero sums. The workspace
 * is needed for the two sums only. The call finds no errors on the device and
 * leaves the workspace's first 256 bytes, with the status word of flce_get_status,
 * as they are: a workspace that the fused head used keeps that call's status. */
size_t flce_layer_norm_workspace_size(int64_t rows, int64_t hidden);
int flce_layer_norm_backward(const void* grad_y, int64_t ld_grad_y, const void* x, int64_t ld_x, int dtype,
                             int64_t rows, int64_t hidden, const void* weight, int weight_dtype, const float* mean,
                             const float* rstd, int rms, void* grad_x, float* grad_weight, float* grad_bias,
                             int accumulate, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------- microscaled 4-bit
 * A matrix [rows, K] held as 4-bit floating point with one scale for each 32
 * consecutive elements of a row (OCP Microscaling Formats v1.0, MXFP4: E2M1
 * elements, E8M0 scales):
 *   e      = floor(log2(max |x| of the block)) - 2, in [-127, 125]
 *   code   = x 2^-e rounded to nearest (ties to the even code) among
 *            0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives, at most 6
 * A block of zeros has e = -127; a block with an infinity or NaN gets the NaN
 * scale (255) and reads back as NaN. K is a multiple of 32.
 * codes [rows, K / 2]: contiguous, 16-byte aligned, the even element in the
 * low four bits. scales: E8M0 bytes (e + 127) in tiles of 128 rows x 4 blocks,
 * [ceil(rows / 128)][ceil(K / 128)][32][4][4], where row r, block c is at
 * [r / 128][c / 4][r % 32][r % 128 / 32][c % 4]; 16-byte aligned; places
 * without a block hold 127. That is the order in which tensor memory takes
 * scales, so a tile travels as one 512-byte copy. */
size_t flce_microscale_codes_size(int64_t rows, int64_t cols);
size_t flce_microscale_scales_size(int64_t rows, int64_t cols);
int flce_microscale_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld_x, void* codes,
                             void* scales, void* stream);
/* out [rows, cols] contiguous, 32-byte aligned = what the codes stand for, in out_dtype. */
int flce_microscale_dequantize(const void* codes, const void* scales, int64_t rows, int64_t cols, void* out,
                               int out_dtype, void* stream);

/* Logits of a microscaled weight: out = cap(out_mult A W^T), A [rows, K],
 * W [vocab, K], cap(z) = T tanh(z / T) for softcap T > 0, else z. Block products
 * are taken by the tensor cores from the 4-bit values and summed in fp32. out
 * [rows, vocab] with row stride ld_out (>= vocab, 0 => vocab), out_dtype.
 * flce_microscale_matmul takes A microscaled; flce_microscale_linear takes
 * x [rows, K] in bf16 or fp32 (16-byte aligned rows or not) and microscales it
 * into the workspace first. The workspace (16-byte aligned) begins with the
 * status word of flce_get_status (FLCE_ERR_TIMEOUT if a bounded wait gave up). */
size_t flce_microscale_workspace_size(int64_t rows, int64_t cols);
int flce_microscale_matmul(const void* a_codes, const void* a_scales, int64_t rows, const void* w_codes,
                           const void* w_scales, int64_t vocab, int64_t cols, float out_mult, float softcap, void* out,
                           int out_dtype, int64_t ld_out, void* workspace, size_t workspace_bytes, void* stream);
int flce_microscale_linear(const void* x, int dtype, int64_t ld_x, int64_t rows, const void* w_codes,
                           const void* w_scales, int64_t vocab, int64_t cols, float out_mult, float softcap, void* out,
                           int out_dtype, int64_t ld_out, void* workspace, size_t workspace_bytes, void* stream);
/* The same with the limit of each bounded device wait (0 => 2 s) and flags: 0, or
 * FLCE_FLAG_TEST_STALL, a test hook: no product is taken, so that the waits run
 * out and the call ends with FLCE_ERR_TIMEOUT in the status word. */
int flce_microscale_linear_limited(const void* x, int dtype, int64_t ld_x, int64_t rows, const void* w_codes,
                                   const void* w_scales, int64_t vocab, int64_t cols, float out_mult, float softcap,
                                   void* out, int out_dtype, int64_t ld_out, void* workspace, size_t workspace_bytes,
                                   int64_t timeout_ns, int flags, void* stream);

/* ---------------------------------------------------------------- sampling
 * One token per row of logits [rows, vocab] (row stride ld_logits) from given
 * random numbers u [rows] (fp32 in [0, 1)). Per row, with m the largest logit
 * and t_i = (x_i - m) (1 / temperature) in fp32:
 *   w_i = floor(exp(t_i) 2^40)                     (whole numbers, so every sum is
 *                                                   exact in any order)
 *   tokens are ranked by falling logit, ties by index
 *   top_k  keeps the first top_k                   (<= 0 or >= vocab: all)
 *   top_p  keeps those of them before which less than top_p of their weight
 *          lies                                    (>= 1: all)
 *   min_p  keeps those of them with exp(t_i) >= min_p  (<= 0: all)
 * the first token is always kept. The answer is the first index at which the
 * running sum of the kept weights, in index order, is above u times their sum.
 * temperature <= 0 takes the first token (the lowest index of the largest
 * logit). Logits of -infinity are never chosen. A row with a NaN or +infinity,
 * without any finite logit, or with a NaN setting or u gets token -1 and a NaN
 * log-probability; the other rows are unaffected.
 * temperature, top_k, top_p, min_p: the arrays hold one value per row (device);
 * NULL takes the scalar beside it for every row. tokens [rows] int64.
 * logprobs [rows] fp32, nullable: log of the answer's probability among the
 * kept tokens. A temperature so small that its reciprocal overflows counts as 0;
 * for +infinity the reciprocal is taken as the smallest positive number, so that
 * finite logits weigh alike and those of -infinity nothing.
 * vocab < 2^22. */
int flce_sample(const void* logits, int logits_dtype, int64_t rows, int64_t vocab, int64_t ld_logits, const float* u,
                const float* temperatures, float temperature, const int32_t* top_ks, int32_t top_k,
                const float* top_ps, float top_p, const float* min_ps, float min_p, int64_t* tokens, float* logprobs,
                void* stream);

/* Kernel ids of these operators for flce_profile_read and flce_kernel_name: a
 * read of n > FLCE_HEAD_KERNEL_FIRST entries reaches them. */
#define FLCE_HEAD_KERNEL_FIRST 32
#define FLCE_HEAD_KERNEL_COUNT 7

#ifdef __cplusplus
}
#endif

#endif /* FLCE_HEAD_H */
