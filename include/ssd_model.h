/*
 * ssd_model.h -- C ABI of the operators that stand around the blocks of a
 * language model in training and serving: the norm in front of a block with
 * the residual's addition (and an output in 8 bits), the cross entropy over a
 * large vocabulary without its logits, and the orthogonalisation of an update.
 * Part of libssd_gb300.
 *
 * Conventions: those of ssd_layer.h (views, alignment, fp32 arithmetic, fixed
 * orders of sums, workspaces, errors through ssd_device_error).  Workspaces
 * must start on 256 bytes, need no initialisation and keep nothing between
 * calls; two calls at once need two.
 *
 * Sizes, beyond which a call returns SSD_ERR_UNSUPPORTED: the norm 2^31 - 1 tokens in all
 * and 16384 channels; the loss 2^30 tokens, 65536 channels, 2^24 words and 2^30 tiles of
 * 128 tokens x 128 words; orthogonalisation 32767 matrices with sides of 2^20 and 2^30
 * tiles of 128 x 128 in all.
 */
#ifndef SSD_GB300_MODEL_H
#define SSD_GB300_MODEL_H

#include "ssd_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------- residual addition and norm */

typedef struct {
  int64_t batch, seqlen, channels;
  float eps;
} ssd_add_norm_dims;

/*
 * total = x + residual (rounded once to stream_dtype), y = t / sqrt(mean(t^2)
 * + eps) weight over each token's channels, with t the sum before its
 * rounding.
 *
 * x, y [batch, seqlen, channels] of dtype; residual, total of stream_dtype,
 * which is dtype or SSD_F32; weight [channels] fp32.  residual NULL: t = x, and
 * total (if given) is x in stream_dtype.  total NULL: not written.  y may be x,
 * total may be residual (the same view each); other overlaps are not allowed.
 */
SSD_API ssd_status ssd_add_norm(const ssd_add_norm_dims *dims, ssd_dtype dtype, ssd_dtype stream_dtype,
                        const ssd_seq *x, const ssd_seq *residual, const float *weight,
                        const ssd_seq *y, const ssd_seq *total, void *stream);

/*
 * The same with y in 8 bits: of every `block` consecutive channels of a token
 * (the last block may be shorter) scale = max|y| / 448 and q = y / scale rounded
 * to e4m3 (4 exponent bits, 3 mantissa bits, largest value 448); a block of zeros has scale 0.
 *
 * block: 32, 64, 128, or 0 (a scale for each token).  q: a view of bytes;
 * scales: dense fp32 [batch, seqlen, ceil(channels / block)].  Both overlap nothing.
 */
SSD_API ssd_status ssd_add_norm_quantized(const ssd_add_norm_dims *dims, ssd_dtype dtype,
                                  ssd_dtype stream_dtype, int64_t block, const ssd_seq *x,
                                  const ssd_seq *residual, const float *weight, const ssd_seq *q,
                                  float *scales, const ssd_seq *total, void *stream);

/*
 * Gradients through ssd_add_norm from its total, given gy = dL/dy (dtype) and
 * gtotal = dL/dtotal (stream_dtype; NULL = 0): dx (dtype) and dresidual
 * (stream_dtype), the same values each rounded to its type, and dweight fp32.
 * Each of the three may be NULL.  dx may be gy and dresidual gtotal.
 */
SSD_API size_t ssd_add_norm_backward_workspace_size(const ssd_add_norm_dims *dims, ssd_dtype dtype,
                                            ssd_dtype stream_dtype);
SSD_API ssd_status ssd_add_norm_backward(const ssd_add_norm_dims *dims, ssd_dtype dtype,
                                 ssd_dtype stream_dtype, const ssd_seq *total,
                                 const float *weight, const ssd_seq *gy, const ssd_seq *gtotal,
                                 const ssd_seq *dx, const ssd_seq *dresidual, float *dweight,
                                 void *workspace, size_t ws_bytes, void *stream);

/* ------------------------------------ cross entropy over a vocabulary */

enum { SSD_REDUCE_NONE = 0, SSD_REDUCE_SUM = 1, SSD_REDUCE_MEAN = 2 };

typedef struct {
  int64_t batch, seqlen, channels, vocab;
  int64_t ignore_index; /* tokens with this target have no loss */
  int reduction;        /* SSD_REDUCE_*; the mean is over the tokens with a target */
} ssd_loss_dims;

/*
 * z = x W^T, lse = log sum exp z, loss = lse - z[target] of every token.
 *
 * x [batch, seqlen, channels] of dtype; weight: vocab rows of `channels`
 * elements of dtype, token_stride apart (batch_stride is not read); targets
 * dense int64 [batch, seqlen].  loss and lse: dense fp32 [batch, seqlen], zero
 * for tokens without a target, whose rows of x are not read; loss may be NULL with
 * a reduction, whose result is *total (else NULL): the sum, or the mean (0
 * without any target).  A target that is neither ignore_index nor within
 * [0, vocab) gives a NaN.
 *
 * The logits are never stored.  fp32 operands are taken in two planes of 11
 * bits after a scaling by powers of two: products as exact as fp32 ones of
 * values down to 2^-28 of the largest finite one of x's rows with a target, or
 * of W; smaller ones are off by 2^-39 of that.  An infinity counts as a NaN there:
 * in a token's row it spoils its own results, in W every token's.  bf16 products are
 * exact; a word whose logit is -inf has no share of a token, +inf gives NaN.  The fp32
 * sums of either type are the tensor cores', cut at 24 bits towards zero (bf16: with each
 * 16 channels, which leaves logits up to channels / 16 times 2^-23 of the sum of their
 * terms off).
 */
SSD_API size_t ssd_linear_cross_entropy_workspace_size(const ssd_loss_dims *dims, ssd_dtype dtype,
                                               const ssd_seq *weight);
SSD_API ssd_status ssd_linear_cross_entropy(const ssd_loss_dims *dims, ssd_dtype dtype, const ssd_seq *x,
                                    const ssd_seq *weight, const int64_t *targets, float *loss,
                                    float *total, float *lse, void *workspace, size_t ws_bytes,
                                    void *stream);

/*
 * Gradients from the forward pass's lse.  gloss: dL/dloss, dense fp32
 * [batch, seqlen] without a reduction, else dL/dtotal, one fp32 value on the
 * device; NULL = 1.  dx: a view of dtype (rows of tokens without a target are
 * zero); dweight: dense [vocab, channels] of dtype.  Either may be NULL.
 *
 * fp32: softmax terms below 2^-28 are off by 2^-39.  A token's factor is applied
 * to its dx after the product, whatever the others' are; for dweight the products
 * gloss x have the limits of x.
 */
SSD_API size_t ssd_linear_cross_entropy_backward_workspace_size(const ssd_loss_dims *dims,
                                                        ssd_dtype dtype, const ssd_seq *weight);
SSD_API ssd_status ssd_linear_cross_entropy_backward(const ssd_loss_dims *dims, ssd_dtype dtype,
                                             const ssd_seq *x, const ssd_seq *weight,
                                             const int64_t *targets, const float *lse,
                                             const float *gloss, const ssd_seq *dx, void *dweight,
                                             void *workspace, size_t ws_bytes, void *stream);

/* ----------------------------------------------- orthogonalised updates */

typedef struct {
  int64_t count, rows, cols; /* matrices of rows x cols */
  int steps;                 /* 1 .. 100 */
  float a, b, c, eps;
} ssd_orth_dims;

/*
 * Newton-Schulz: X = G / (|G| + eps) with the Frobenius norm of each matrix,
 * then `steps` times X <- a X + b (X X^T) X + c (X X^T)^2 X.
 *
 * update: `count` matrices batch_stride apart, rows token_stride apart, of
 * in_dtype; result likewise of out_dtype.  result may be update where types
 * and strides are the same.
 *
 * Precision goes by out_dtype.  SSD_BF16: products of operands rounded to fp16
 * (11 bits), X carried in 22 bits until the last two steps.  SSD_F32: everything
 * in 22 bits.  Entries and eps may lie anywhere in their types' range; entries below
 * 2^-28 of |G| keep 2^-39 of it.  A matrix that holds an infinity or a NaN gives NaN, the
 * others of a stack are not touched by it.  Steps that take X beyond 4 or b A + c A A
 * beyond 16 (the usual coefficients stay below 1.3 and 3) overflow.
 */
SSD_API size_t ssd_orthogonalize_workspace_size(const ssd_orth_dims *dims, ssd_dtype in_dtype,
                                        ssd_dtype out_dtype);
SSD_API ssd_status ssd_orthogonalize(const ssd_orth_dims *dims, ssd_dtype in_dtype, ssd_dtype out_dtype,
                             const ssd_seq *update, const ssd_seq *result, void *workspace,
                             size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSD_GB300_MODEL_H */
