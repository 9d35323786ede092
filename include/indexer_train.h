/*
 * libindexer_bwd, second header -- the operators around the indexer when a
 * model with sparse attention is trained or converted: the layer norm of the
 * indexer's keys (or of hidden states), the log probabilities of a model's
 * logits, and the distillation of a student from a teacher's top logits.
 * Status codes, streams and device status are those of indexer_bwd.h.  Pointers
 * are to memory of the current device, or managed memory: another device's is
 * refused.
 *
 * Conventions of this header (where they differ from indexer_bwd.h)
 *  - A matrix is [rows, width] with unit stride along a row and `stride`
 *    elements (>= width) from a row to the next, so a slice of a wider buffer
 *    is taken as it is.  Pointers need the alignment of their element type
 *    only; rows that all start on 16-byte boundaries take wider accesses.
 *  - rows = 0 is a valid call: nothing is read, column sums are set to 0.
 *  - Element types are ibwd_dtype codes.  Statistics, sums, losses and the
 *    gradients of weights are fp32; every result in a 16-bit type is rounded
 *    once, to nearest even, from the fp32 result.
 *  - Outputs must not overlap inputs except where a function says so.
 *  - All results are bitwise reproducible from run to run.
 *  - Nothing is allocated; only ibwd_layer_norm_bwd takes a workspace.
 */
#ifndef INDEXER_TRAIN_H
#define INDEXER_TRAIN_H

#include "indexer_bwd.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { IBWD_F32 = 0, IBWD_BF16 = 1, IBWD_F16 = 2 } ibwd_dtype;

/* Limits of the operators below. */
#define IBWD_MAX_TOP 128   /* top alternatives of a row */
#define IBWD_MAX_KEPT 1024 /* teacher tokens of a row */

/*
 * Layer norm over the rows of x:
 *   mean = sum x / N,  rstd = 1 / sqrt(sum (x - mean)^2 / N + eps),
 *   y = (x - mean) * rstd * gamma + beta        (N = width >= 1)
 *   x            x_type [rows, width], stride x_stride
 *   gamma, beta  w_type [width], each NULL for 1 / 0; w_type is IBWD_F32 or x_type
 *   y            y_type [rows, width], stride y_stride; y_type is x_type, or any type for an fp32 x;
 *                may be x itself (same pointer, type and stride)
 *   mean, rstd   fp32 [rows], each NULL when not wanted (the backward pass needs both)
 *   eps          finite, >= 0
 */
IBWD_API int ibwd_layer_norm_fwd(const void* x, int x_type, int64_t x_stride, const void* gamma, const void* beta,
                                 int w_type, void* y, int y_type, int64_t y_stride, float* mean, float* rstd,
                                 int64_t rows, int width, float eps, void* stream);

/* Bytes of device workspace ibwd_layer_norm_bwd needs for dgamma and dbeta
 * (column sums of groups of rows, fp32); 0 for unsupported arguments. */
IBWD_API size_t ibwd_layer_norm_bwd_workspace_size(int64_t rows, int width);

/*
 * Backward pass of the layer norm: with xh = (x - mean) * rstd and d = dy * gamma,
 *   dx = rstd * (d - sum(d)/N - xh * sum(d xh)/N),
 *   dgamma = sum over rows of dy * xh,   dbeta = sum over rows of dy
 *   dy      dy_type [rows, width]: x_type or fp32, or any type for an fp32 x
 *   x, gamma, mean, rstd  as the forward pass took and gave them
 *   dx      x_type [rows, width]; may be x, or dy where that has x_type, itself (same stride)
 *   dgamma, dbeta  fp32 [width], each NULL when not wanted, written (not accumulated);
 *           widths of up to 2^30 - 64 with either
 *   workspace  at least ibwd_layer_norm_bwd_workspace_size bytes, 16-byte
 *              aligned (may be NULL when dgamma and dbeta are)
 */
IBWD_API int ibwd_layer_norm_bwd(const void* dy, int dy_type, int64_t dy_stride, const void* x, int x_type,
                                 int64_t x_stride, const void* gamma, int w_type, const float* mean,
                                 const float* rstd, void* dx, int64_t dx_stride, float* dgamma, float* dbeta,
                                 int64_t rows, int width, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Log probabilities of a row of logits x over its vocabulary, y = x / temperature:
 *   lse = log sum_v exp(y_v),  p_v = exp(y_v - lse)
 *   logprob = y[token] - lse,  entropy = -sum_v p_v log p_v
 *   top: the top_n largest logits, ties by the lowest index, as token ids and
 *        log probabilities, best first
 * A logit of -inf is a masked token: probability 0, log probability -inf,
 * never among the top (free places at the end hold id -1 and -inf).  A row
 * with every token masked has lse = logprob = -inf and entropy 0.  A NaN or
 * +inf makes the row's lse, logprob, entropy and top log probabilities NaN; the
 * top ids are those of the largest numbers, never of a NaN.
 *   logits   type [rows, vocab], stride `stride`
 *   tokens   int32 [rows] or NULL; an id outside [0, vocab) is padding: logprob 0
 *   logprob  fp32 [rows], NULL exactly when tokens is
 *   entropy, lse  fp32 [rows], each NULL when not wanted
 *   top_ids int32, top_logprobs fp32 [rows, top_n]; 0 <= top_n <= min(vocab, IBWD_MAX_TOP), both NULL for 0
 *   temperature   finite, > 0
 */
IBWD_API int ibwd_token_logprobs_fwd(const void* logits, int type, int64_t stride, const int32_t* tokens,
                                     float temperature, float* logprob, float* entropy, float* lse,
                                     int32_t* top_ids, float* top_logprobs, int top_n, int64_t rows, int vocab,
                                     void* stream);

/*
 * Gradient of the log probabilities and entropies:
 *   dlogits_v = (dlogprob * ([v = token] - p_v) - dentropy * p_v * (log p_v + entropy)) / temperature
 *   lse, entropy  as the forward pass gave them (entropy NULL when dentropy is)
 *   tokens and dlogprob, dentropy: fp32 [rows], NULL for no such part; a
 *        padding token's dlogprob counts as 0
 *   dlogits  type [rows, vocab], stride dlogits_stride; may be logits itself (same stride)
 * A fully masked row (lse = -inf) gets 0.
 */
IBWD_API int ibwd_token_logprobs_bwd(const void* logits, int type, int64_t stride, const int32_t* tokens,
                                     float temperature, const float* lse, const float* entropy,
                                     const float* dlogprob, const float* dentropy, void* dlogits,
                                     int64_t dlogits_stride, int64_t rows, int vocab, void* stream);

/*
 * Distillation from a teacher's top logits.  A row keeps up to K teacher
 * tokens; ids outside [0, vocab) are padding.  With T = temperature,
 *   p = softmax over the kept slots of teacher / T   (teacher: logits or log probabilities)
 *   q = softmax over the vocabulary of logits / T
 *   loss = T^2 * sum_j p_j (log p_j - log q[ids_j])
 * A slot whose teacher value is -inf counts for nothing (0 log 0 = 0), a
 * token kept in several slots has the sum of their probabilities in the
 * gradient, and a row that keeps nothing, or whose logits are all -inf, has
 * loss 0 and gradient 0.  A kept token of p > 0 whose logit is -inf makes the
 * loss +inf (its gradient stays finite).  A kept slot's NaN is the row's loss
 * and the kept tokens' gradient; a padding slot's value is not looked at.
 *   logits   type [rows, vocab], stride `stride`
 *   ids int32, teacher fp32 [rows, K]; 1 <= K <= IBWD_MAX_KEPT
 *   loss, lse  fp32 [rows] (lse of logits / T)
 */
IBWD_API int ibwd_distill_fwd(const void* logits, int type, int64_t stride, const int32_t* ids,
                              const float* teacher, int K, float temperature, float* loss, float* lse,
                              int64_t rows, int vocab, void* stream);

/* Its gradient, dlogits_v = dloss * T * (q_v - sum_{ids_j = v} p_j):
 *   lse    as ibwd_distill_fwd gave it;  dloss  fp32 [rows]
 *   dlogits  type [rows, vocab], stride dlogits_stride; may be logits itself (same stride) */
IBWD_API int ibwd_distill_bwd(const void* logits, int type, int64_t stride, const int32_t* ids,
                              const float* teacher, int K, float temperature, const float* lse,
                              const float* dloss, void* dlogits, int64_t dlogits_stride, int64_t rows, int vocab,
                              void* stream);

/* Loss and gradient in one call, for a loss that is a weighted sum over the
 * rows: dloss = grad_scale * row_weight (row_weight fp32 [rows], NULL for 1).
 * loss is written without the weight.  dlogits may be logits itself (same
 * stride); loss may be NULL when only the gradient is wanted. */
IBWD_API int ibwd_distill_grad(const void* logits, int type, int64_t stride, const int32_t* ids,
                               const float* teacher, int K, float temperature, const float* row_weight,
                               float grad_scale, float* loss, void* dlogits, int64_t dlogits_stride, int64_t rows,
                               int vocab, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* INDEXER_TRAIN_H */
