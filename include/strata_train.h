/*
 * strata_train.h -- C ABI of the operators that score and train the end of a model.
 *
 *   strata_layer_norm_rows      layer norm of hidden rows, with the residual's addition
 *   strata_layer_norm_grad      and its way back: gradients of the rows, the weight and the bias
 *   strata_cross_entropy_rows   the head's product and the cross entropy of one given token a row (its
 *                               negative is the token's log-probability), without keeping the logits
 *   strata_cross_entropy_grad   and its way back: gradients of the rows and of the head
 *   strata_distill_rows         the same product and the distance from a teacher's top logits
 *   strata_distill_grad         and its way back
 *
 * The conventions are those of strata_tail.h: device pointers owned by the caller, work enqueued on
 * `stream` only, STRATA_OK or a negative STRATA_E* code with strata_last_error(), argument checks
 * before any work is enqueued, no context, and calls on several streams independent as long as their
 * buffers (a workspace is one) are.  The calls may be captured in a CUDA graph; graphs that replay at
 * the same time need workspaces of their own.  Results do not depend on timing: the same call gives the
 * same bits.  Their launches overlap the kernel before them as those of strata_tail.h do, and
 * strata_tail_errors tells their kernels' error bits too.
 */
#ifndef STRATA_TRAIN_H
#define STRATA_TRAIN_H

#include <stdint.h>

#include "strata_tail.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- limits -------------------------------------------------------------------------------- */
#define STRATA_LOSS_MAX_ROWS    131072 /* T of the losses (of the norms: 2^31 - 1)                    */
#define STRATA_LOSS_MAX_WIDTH   32768  /* H of the losses (of the norms: STRATA_TAIL_MAX_WIDTH)       */
#define STRATA_DISTILL_MAX_TOKENS 128  /* K: a teacher's tokens for a row                             */

/*
 * For each of T rows of H elements:
 *   h = x + residual                                                   (32 bits; residual NULL: h = x)
 *   y = (h - mean) * rstd * weight + bias,    mean = mean(h),  rstd = 1 / sqrt(mean((h - mean)^2) + eps)
 * and writes what has a pointer: residual_out = h and y, rounded to `dtype` (x's, the residual's, the weight's
 * and the bias's: F32 or BF16; bias NULL: none), and mean and rstd, one float for each row, which the
 * way back takes.  (They are of h before its rounding to residual_out.)
 * Strides count elements; rows may be any distance >= H apart and need only their element's
 * alignment (rows that start on 16 bytes run faster).  residual_out may be the residual or x
 * itself; y may not overlap an input.  A NaN or an infinity stays within its row.
 */
int strata_layer_norm_rows(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                           const void* bias, int dtype, int T, int H, float eps, void* residual_out, int64_t ldro,
                           void* y, int64_t ldy, float* mean, float* rstd, void* stream);

/*
 * With v = (x - mean) * rstd and a = dy * weight, for the rows x that were normed (h, where there was a residual):
 *   dx = rstd * (a - mean(a) - v * mean(a * v)) + dresidual      (dresidual NULL: not added)
 *   dweight = sum over rows of dy * v,    dbias = sum over rows of dy
 * dx, dweight and dbias are `dtype`, as dy, x, weight and dresidual are; each may be NULL, but not all.  Sums are
 * held in 32 bits.  dx may be dy, x or dresidual itself.  With T = 0 dweight and dbias are set to zeros.
 * `workspace` (for dweight and dbias): strata_layer_norm_workspace(T, H) bytes on 256 bytes of alignment.
 */
int64_t strata_layer_norm_workspace(int T, int H);
int strata_layer_norm_grad(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* weight, const float* mean,
                           const float* rstd, const void* dresidual, int64_t lddr, int dtype, int T, int H, void* dx,
                           int64_t lddx, void* dweight, void* dbias, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * For each of T rows x[t] of H elements and a head w of V rows, z[t][v] = sum_h x[t][h] w[v][h], and
 *   lse[t] = log sum_v exp(z[t][v]),    loss[t] = lse[t] - z[t][ids[t]]
 * x and w are bfloat16, sums, lse and loss 32 bits; no more of the logits than a tile is held anywhere.
 * A row whose id is negative is left out: loss 0 and lse 0, and its x is not looked at (nor a NaN in it).  An id of V
 * or more gives NaN for both.
 * x and w start on 16 bytes; H and the strides ldx and ldw are multiples of 8.
 * `workspace`: strata_loss_workspace(T, V, H, 0, 0) bytes on 256 bytes of alignment, free to be reused
 * when the stream has passed the call; K = 0 says that it is for a cross entropy, grad = 1 that it is for a gradient (and 0 is
 * the size for a call that would be refused).
 */
int64_t strata_loss_workspace(int T, int V, int H, int K, int grad);
int strata_cross_entropy_rows(const void* x, int64_t ldx, const void* w, int64_t ldw, int T, int V, int H,
                              const int32_t* ids, float* loss, float* lse, void* workspace, int64_t workspace_bytes,
                              void* stream);

/*
 * The gradients of sum_t g[t] * loss[t], from the lse that the call above gave:
 *   dz[t][v] = g[t] * (exp(z[t][v] - lse[t]) - [v = ids[t]]),    dx = dz w,    dw = dz^T x
 * dx [T][H] and dw [V][H] are bfloat16 (either may be NULL).  The logits are computed again, in pieces of the vocabulary;
 * dz / g is rounded to bfloat16 between the products, and so is x[t] g[t] / max|g| (x itself where
 * all g are equal).  With the T, V and H of the call that gave lse they are the same bits of z; so what is left of dz / g where a
 * row is all but sure of its token is off by the rounding of lse, 3 * 2^-24 (|lse| + 1) at most (with the lse of a call of
 * another size: by 1e-6 of z, too).  A row that is left out, whose id is V or more or whose g is 0 gets dx = 0 and adds nothing to dw.
 * With T = 0 dw is set to zeros.  dx and dw start on 16 bytes, their strides are multiples of 8, and they do not overlap an
 * input or one another.
 * `workspace`: strata_loss_workspace(T, V, H, 0, 1) bytes, which hold a piece of dz (at most 512 MB, or 511 columns more where
 * that is all of the vocabulary) and parts of dx (256 MB, or one of them) beside copies of the rows.
 */
int strata_cross_entropy_grad(const void* x, int64_t ldx, const void* w, int64_t ldw, int T, int V, int H,
                              const int32_t* ids, const float* lse, const float* g, void* dx, int64_t lddx, void* dw,
                              int64_t lddw, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * A teacher gives K tokens ids[t][k] for each row and their logits or log-probabilities teacher[t][k] (what is common to
 * a row's falls out).  With the temperature s (0.001 to 1000), over the tokens given
 *   q[t] = softmax(teacher[t] / s),   lse[t] = log sum_v exp(z[t][v] / s),
 *   loss[t] = s^2 * sum_k q[t][k] * (log q[t][k] - (z[t][ids[t][k]] / s - lse[t]))
 * An id that is negative or whose teacher value is -inf is not there; a row without ids is left out, as above.  An id of
 * V or more makes its row's loss and lse NaN.  The same id may come twice: both count.
 * ids and teacher are packed.  workspace: strata_loss_workspace(T, V, H, K, 0).  Else as strata_cross_entropy_rows.
 */
int strata_distill_rows(const void* x, int64_t ldx, const void* w, int64_t ldw, int T, int V, int H, int K,
                        const int32_t* ids, const float* teacher, float temperature, float* loss, float* lse, void* workspace,
                        int64_t workspace_bytes, void* stream);

/*
 * The gradients of sum_t g[t] * loss[t] (a student as sure as its teacher: dz / (g s) off by 8 * 2^-24 (|lse| + 1) at most):
 *   dz[t][v] = g[t] * s * (exp(z[t][v] / s - lse[t]) - sum of q[t][k] with ids[t][k] = v),    dx = dz w,    dw = dz^T x
 * workspace: strata_loss_workspace(T, V, H, K, 1).  Else as strata_cross_entropy_grad.
 */
int strata_distill_grad(const void* x, int64_t ldx, const void* w, int64_t ldw, int T, int V, int H, int K,
                        const int32_t* ids, const float* teacher, float temperature, const float* lse, const float* g, void* dx,
                        int64_t lddx, void* dw, int64_t lddw, void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* STRATA_TRAIN_H */
