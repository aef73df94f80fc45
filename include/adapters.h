/*
 * adapters.h -- C ABI of low-rank adapters beside a shared product (gemm.h):
 * rows of many requests, each with its own adapter or none, and the gradients
 * of a training step.
 *
 *   gemm_run_adapters      D = X W + bias + (the rows' adapters)
 *   gemm_adapters_grad     gradients of the adapters' two factors
 *   gemm_adapters_hidden_width  columns of the rows that the two share
 *
 * Row i has the adapter g = index[i]; a value outside 0..count-1 (say -1) means
 * none.  With A = down[g] (rank x K), U = up[g] (N x rank), s = scale[g],
 *
 *   h[i]    = s A X[i]                       (rank values)
 *   D[i, :] = X[i, :] W + bias + U h[i]
 *
 * Of sum(dD * D), with p[i] = s U^T dD[i]:
 *
 *   dX[i]     = dD[i] W^T + A^T p[i]
 *   d_down[g] = sum over the rows i of g of p[i] X[i]^T
 *   d_up[g]   = sum over the rows i of g of dD[i] h[i]^T
 *
 * so dX and p come from gemm_run_adapters too: dD in the place of X, W^T of W,
 * U^T of A and A^T of U (the same memory, the other layout), and the two others
 * from gemm_adapters_grad with h and p.  A row's results depend on that row,
 * W and its own adapter alone: infinities and NaN of other rows and
 * adapters do not reach it, nor those of other adapters' rows an
 * adapter's gradients.  (Its own ones do, an infinity of U, X or dD as a NaN where the low
 * part of h or p that it meets is 0.)  Rows of an adapter need not be neighbours.
 *
 * h and p are handed on as `hidden`: M rows of P = gemm_adapters_hidden_width(rank) / 2
 * high parts, the values rounded to the plan's type, and P low parts, what that
 * rounding lost (columns from the rank on are 0): 16 bits would be the
 * only rounding before D's own, the two parts together keep 16 (bf16) or up to 22 (fp16)
 * bits.
 *
 * fp16 values are to be within its range, 65504 at most; and its low parts end at 2^-24, so
 * that a value is off by up to 2^-25 however small it is: one of 1e-3 keeps 15 bits, one of
 * 1e-5 eight.  In D and dX that is 2^-25 of a row's sum of |U| or |A|, but p = s U^T dD is that
 * small itself while U is near 0, or where dD comes from a mean, and then d_down is as far
 * off.  With `wide`, on fp16 plans, rows have 3 P columns: low parts, high parts, and what the high
 * parts lost times 2^11, which gemm_adapters_grad takes instead of the low ones: 22 bits from
 * 2^-14 on, off by 2^-36 below.
 *
 * Types.  X, W, down, up, dD and hidden are of the plan's type, GEMM_F16 or
 * GEMM_BF16; scale and bias fp32; D and the two gradients GEMM_F32 or the plan's
 * type (D of an fp16 plan also GEMM_BF16).  Sums are fp32, each output is
 * rounded once.
 *
 * Memory, streams and errors are gemm.h's: device pointers of the caller;
 * X, W, down, up, dD and hidden start on 16-byte boundaries and so do
 * their rows and an adapter's factors (GEMM_ERR_MISALIGNED); one plan is
 * used by one stream at a time; a wait inside a kernel that ran out is in
 * gemm_plan_device_status.  D, hidden and the gradients overlap no input and not one
 * another.  Nothing is allocated, so calls may be captured.
 */
#ifndef TCDT_ADAPTERS_H
#define TCDT_ADAPTERS_H

#include <stdint.h>

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GEMM_ADAPTERS_MAX_RANK 128

/* down: element (g, r, k) at [g * down_stride + r * down_ld + k] (GEMM_ROW_MAJOR,
 * down_ld >= K) or [... + k * down_ld + r] (GEMM_COL_MAJOR, down_ld >= rank);
 * up: element (g, n, r) at [g * up_stride + n * up_ld + r] (GEMM_ROW_MAJOR,
 * up_ld >= rank) or [... + r * up_ld + n] (GEMM_COL_MAJOR, up_ld >= N). */
typedef struct {
    int64_t count;             /* adapters, 0 or more */
    int64_t rank;              /* 1..GEMM_ADAPTERS_MAX_RANK */
    const void *down;
    int64_t down_ld, down_stride;
    gemm_layout_t down_layout;
    const void *up;
    int64_t up_ld, up_stride;
    gemm_layout_t up_layout;
    const float *scale;        /* [count], or NULL (ones) */
    const int32_t *index;      /* [M] */
    int64_t ldp;               /* gemm_adapters_grad: row stride of p, 0 for ldh */
    int32_t wide;              /* 1: gemm_run_adapters's hidden, gemm_adapters_grad's p is wide (fp16 plans) */
    int32_t wide_h;            /* 1: gemm_adapters_grad's h is */
} gemm_adapters_t;

/* Columns of `hidden` (not wide): 2 P, P = 16, 32, 64 or 128, the smallest that holds the
 * rank; 0 for a rank out of range. */
int64_t gemm_adapters_hidden_width(int64_t rank);

/* D (M x N, row-major) of X (M x K, row-major) and W (K x N, either layout).
 * bias is [N] or NULL.  hidden (M rows of ldh elements) is written. */
gemm_status_t gemm_run_adapters(gemm_plan_t plan, const void *X, const void *W, void *D, int64_t M, int64_t N,
                                int64_t K, int64_t ldx, int64_t ldw, int64_t ldd, gemm_layout_t layoutW,
                                gemm_dtype_t out_dtype, const float *bias, const gemm_adapters_t *adapters,
                                void *hidden, int64_t ldh, void *stream);

/* d_down[g * down_stride + r * down_ld + k] and d_up[g * up_stride + n * up_ld + r],
 * of all `count` adapters (zeros for one without rows), from X (M x K), dD
 * (M x N), both row-major, h and p.  The adapters' gradients lie one after
 * another, or their rows in turn (down_ld >= (count - 1) down_stride + K); in a
 * stack whose matrices overlap their CTAs would write the same memory
 * (GEMM_ERR_INVALID_ARG).  Of `adapters` count, rank, index, ldp, wide and
 * wide_h are used.
 * Either of d_down and d_up may be NULL, with what only it needs. */
gemm_status_t gemm_adapters_grad(gemm_plan_t plan, const void *X, const void *dD, int64_t M, int64_t N, int64_t K,
                                 int64_t ldx, int64_t lddd, const gemm_adapters_t *adapters, const void *h,
                                 const void *p, int64_t ldh, gemm_dtype_t out_dtype, void *d_down, int64_t down_ld,
                                 int64_t down_stride, void *d_up, int64_t up_ld, int64_t up_stride, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TCDT_ADAPTERS_H */
