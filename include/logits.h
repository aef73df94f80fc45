/*
 * logits.h -- C ABI of the operators on the rows of a logits matrix: what a
 * product with an output head (gemm.h) is followed by.
 *
 *   logits_logprobs       log-probability of a given token of each row, the
 *                         row's entropy and log-sum-exp, its top alternatives
 *   logits_logprobs_grad  the first three, and the gradient for the logits
 *   logits_distill        distillation loss against a teacher's top logits
 *   logits_distill_grad   that, and the gradient for the logits
 *
 * The logits are T rows of V values, row-major, element (i, j) at
 * [i * ld + j], ld >= V, of type GEMM_F32, GEMM_F16 or GEMM_BF16; nothing
 * beyond column V of a row is read.  With x_j = logits_j / temperature,
 *
 *   lse = log sum_j exp(x_j),   p_j = exp(x_j - lse).
 *
 * A logit of -inf is a token that is masked out: p_j = 0 and it contributes
 * nothing.  A row with nothing but -inf (or V == 0) has lse = -inf, entropy 0
 * and a gradient of zeros.  A NaN or +inf logit makes its row's results NaN.
 * Softmax statistics and all results but the gradient are fp32; the gradient
 * is computed in fp32 and rounded once (to nearest even) to its type, which
 * is that of the logits.
 *
 * Memory and streams.  All pointers are DEVICE pointers owned by the caller
 * and aligned to their element; nothing is kept after a call returns, there
 * is no workspace and no allocation.  A call launches one kernel on `stream`
 * (a cudaStream_t; NULL = the legacy default stream) of `device` (a CUDA
 * ordinal, made current while the call runs and then restored) and
 * synchronises nothing, so it may be captured in a graph.  Calls are
 * independent: any number may run at once, from any threads and streams.
 * Results do not depend on timing: the same inputs give the same bits.  Every
 * wait inside a kernel is bounded: a copy that has not arrived after 2 s is
 * made up for by plain loads, a row whose CTAs then still wait for one another's
 * statistics becomes NaN, its alternatives NaN and -1.
 *
 * Errors.  Arguments are checked on the host before anything is launched:
 * GEMM_ERR_INVALID_ARG (null pointer, negative size, stride below its row
 * length, bad type or temperature, counts out of range), GEMM_ERR_UNSUPPORTED
 * (V or T above 2^31 - 4097), GEMM_ERR_MISALIGNED (a pointer not aligned to
 * its element), GEMM_ERR_NO_DEVICE (not a compute capability 10.3 device),
 * GEMM_ERR_CUDA (a CUDA call failed).  T == 0 launches nothing.
 */
#ifndef TCDT_LOGITS_H
#define TCDT_LOGITS_H

#include <stdint.h>

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LOGITS_MAX_TOP 128       /* largest number of alternatives */
#define LOGITS_MAX_TEACHER 1024  /* largest number of teacher tokens of a row */

/* Per row i, with y = tokens[i]:
 *   logprob[i]  x_y - lse, or 0 where y is outside 0..V-1 (say -1: nothing is
 *               given for this row); -inf for a masked token
 *   entropy[i]  -sum_j p_j log p_j
 *   lse[i]
 *   top_logprob[i * top + r], top_token[i * top + r], r = 0..top-1: the
 *               log-probabilities of the row's largest logits in descending
 *               order, equal logits by the lowest token.  Tokens of -inf (and
 *               NaN) are no alternatives: places that are left hold -inf and -1.
 * tokens may be NULL (then logprob is not written); each of logprob, entropy
 * and lse may be NULL; top is 0..LOGITS_MAX_TOP and the two top arrays may be
 * NULL when it is 0.  temperature is a positive finite number. */
gemm_status_t logits_logprobs(int device, gemm_dtype_t dtype, const void *logits, int64_t T, int64_t V, int64_t ld,
                              const int64_t *tokens, float temperature, int top, float *logprob, float *entropy,
                              float *lse, float *top_logprob, int64_t *top_token, void *stream);

/* logits_logprobs without alternatives, and the gradient for the logits of
 * sum_i (g[i] logprob[i] + h[i] entropy[i]):
 *   dlogits[i * ldd + j] = (g (1[j = y] - p_j) - h p_j (log p_j + entropy)) / temperature,
 * its g terms left out where y is outside 0..V-1.  g or h may be NULL (zeros);
 * tokens may be NULL only with g.  dlogits is written once; of the logits, what
 * a row has beyond the 64 KB or less that each of its CTAs keeps on chip is read
 * twice, the second time from L2 while the rows worked on at once fit it.  dlogits may be
 * the logits themselves (same pointer and stride), and overlaps them in no
 * other way.  A row of dlogits that starts elsewhere within 16 bytes than its
 * logits is stored element by element: right, and up to three times slower. */
gemm_status_t logits_logprobs_grad(int device, gemm_dtype_t dtype, const void *logits, int64_t T, int64_t V,
                                   int64_t ld, const int64_t *tokens, float temperature, const float *g,
                                   const float *h, float *logprob, float *entropy, float *lse, void *dlogits,
                                   int64_t ldd, void *stream);

/* Distillation from the K largest logits of a teacher.  teacher_tokens and
 * teacher_logits are T x K, row-major with the row stride ldt (elements, both
 * the same); the logits are of type teacher_dtype (GEMM_F32, GEMM_F16 or
 * GEMM_BF16) and may be log-probabilities as well (a row's constant does not
 * matter).  A token outside 0..V-1 is padding, its logit is not used (it may
 * be NaN).  With P the softmax of teacher_logits / temperature over a row's
 * real entries (0 at the others) and Q the p above,
 *   loss[i] = temperature^2 sum_k P_k (log P_k - log Q_{token k}),
 * 0 where there is no real entry (or only -inf ones); +inf where the student
 * has masked a token with P_k > 0.  A token given twice counts as two terms.
 * lse may be NULL.  K is 0..LOGITS_MAX_TEACHER. */
gemm_status_t logits_distill(int device, gemm_dtype_t dtype, const void *logits, int64_t T, int64_t V, int64_t ld,
                             int64_t K, const int64_t *teacher_tokens, gemm_dtype_t teacher_dtype,
                             const void *teacher_logits, int64_t ldt, float temperature, float *loss, float *lse,
                             void *stream);

/* logits_distill, and the gradient for the logits of sum_i w[i] loss[i]:
 *   dlogits[i * ldd + j] = w temperature (Q_j - sum over k with token j of P_k),
 * zeros where the loss has no real entry.  Reads, and in place, as for
 * logits_logprobs_grad. */
gemm_status_t logits_distill_grad(int device, gemm_dtype_t dtype, const void *logits, int64_t T, int64_t V,
                                  int64_t ld, int64_t K, const int64_t *teacher_tokens, gemm_dtype_t teacher_dtype,
                                  const void *teacher_logits, int64_t ldt, float temperature, const float *w,
                                  float *loss, float *lse, void *dlogits, int64_t ldd, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TCDT_LOGITS_H */
