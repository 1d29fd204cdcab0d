/*
 * strata_tail.h -- C ABI of the operators around the sampler: the end of a decode step.
 *
 *   strata_norm_rows     root-mean-square norm of hidden rows, with the residual's addition, and an
 *                        output in 8 bits with one scale per row
 *   strata_project_rows  a projection shared by all rows (the head, or a layer's) plus each row's
 *                        own low-rank adapter, in bfloat16 or from the norm's 8-bit rows
 *   strata_draw_rows     temperature, top_k, top_p and min_p sampling of logit rows from random
 *                        numbers that the caller brings; no limit on top_k
 *
 * The conventions are those of strata_sample.h: device pointers owned by the caller, work enqueued
 * on `stream` only, STRATA_OK or a negative STRATA_E* code with strata_last_error(), and argument
 * checks before any work is enqueued (a call that returns an error has launched nothing).  These
 * calls need no context: they run on the calling thread's current device, every buffer they use is
 * an argument, and calls on several streams are independent as long as their buffers are.  The three
 * operators may be captured in a CUDA graph (strata_tail_errors waits, and may not).  A call with no rows
 * does nothing and returns STRATA_OK.
 * Their launches are set up while the kernel before them on the stream runs (programmatic dependent
 * launch) and wait on the GPU for it to end before they touch memory.  Beside sampling calls of the
 * same stream: the first of them behind a call with STRATA_FLAG_OWN_OUTPUTS (which waits for nothing)
 * and the first call with STRATA_FLAG_EARLY_LOAD behind one of them are launched without that overlap.
 */
#ifndef STRATA_TAIL_H
#define STRATA_TAIL_H

#include <stdint.h>

#include "strata_sample.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- element types beside STRATA_DTYPE_F32 and STRATA_DTYPE_BF16 --------------------------- */
#define STRATA_DTYPE_F8          2      /* 8-bit floating point, e4m3 without infinities (|v| <= 448) */

/* ---- limits -------------------------------------------------------------------------------- */
#define STRATA_TAIL_MAX_WIDTH    131072 /* H of strata_norm_rows, K of strata_project_rows           */
#define STRATA_TAIL_MAX_ADAPTERS 1024   /* S of strata_project_rows                                  */
#define STRATA_TAIL_MAX_RANK     256    /* R of strata_project_rows, a multiple of 16                */

/*
 * For each of T rows of H elements:
 *   h = x + residual            (32 bits; residual NULL: h = x)
 *   y = h * rsqrt(mean(h * h) + eps) * weight
 * and writes what has a pointer: residual_out = h and y, rounded to `dtype` (x's, the residual's and
 * the weight's: F32 or BF16), and the 8-bit row q = e4m3(y * (1 / scale)) with
 * scale = max(max|y| / 448, 2^-100), computed from y in 32 bits, before any rounding.
 * Strides count elements; rows may be any distance >= H apart and need only their element's
 * alignment (rows that start on 16 bytes run faster).  residual_out may be the residual or x
 * itself; q and y may not overlap an input.  A NaN or an infinity stays within its row.
 */
int strata_norm_rows(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight, int dtype,
                     int T, int H, float eps, void* residual_out, int64_t ldro, void* y, int64_t ldy, void* q,
                     int64_t ldq, float* scale, void* stream);

/*
 * y[t][n] = x_scale[t] * w_scale[n] * sum_k x[t][k] w[n][k]
 *           + adapter_scale[c] * sum_r (x_scale[t] * sum_k x[t][k] a[c][r][k]) * b[c][n][r],   c = row_adapter[t]
 * x and w are `dtype`: BF16 (no scales: pass NULL) or F8 (both scales).  a [S][R][K], b [S][N][R]
 * and y are bfloat16, a and b packed; a row whose row_adapter is outside 0..S-1 has no adapter.
 * S = 0 (the adapter pointers may be NULL) is the projection alone.  Sums are held in 32 bits; the inner row
 * (adapter_scale * x_scale * x a^T) is held as two bfloat16 (2^-16) between its two products.
 * An adapter's infinities and NaNs reach the rows that use it and no others.  T is at most 524,288, N 2^31 - 257.
 * x, w, a and b start on 16 bytes, and K and the strides ldx and ldw are multiples of 16 bytes; R is
 * a multiple of 16 (pad smaller ranks with zeros).  ldy >= N is any stride, y any bfloat16 address.
 * `workspace`: strata_project_workspace(T, S, R) bytes on 256 bytes of alignment, free to be reused
 * when the stream has passed the call.  It grows with rows times adapters up to 256 MB (or what 2,048
 * rows take); larger calls go through their rows in slabs.
 */
int64_t strata_project_workspace(int T, int S, int R);
int strata_project_rows(const void* x, int64_t ldx, const float* x_scale, const void* w, int64_t ldw,
                        const float* w_scale, int dtype, int T, int N, int K, const void* a, const void* b, int S,
                        int R, const int32_t* row_adapter, const float* adapter_scale, void* y, int64_t ldy,
                        void* workspace, int64_t workspace_bytes, void* stream);

/*
 * One id for each of B logit rows (F32 or BF16), by the sampler's chain without its limit on top_k:
 *   order: logit descending, ties to the lowest index; NaN and -inf are never chosen
 *   top_k (<= 0: off)  ->  min_p (<= 0: off): logit >= logit0 + logf(min_p)
 *   ->  top_p (>= 1: off): of the temperature-1 mass left, the smallest prefix that reaches top_p
 *   ->  temperature: weights exp((logit - logit0) / temperature); <= 0 or NaN: the first in order
 * No cut removes the first in order.  The draw walks what is left in index order: the first id whose
 * summed weight exceeds u times the total.  Weights are whole numbers, floor(exp(.) * 2^43), and
 * u and top_p count in units of 2^-24 (rounded down), so that every sum is exact and the answer
 * does not depend on how a row is split.  u outside [0, 1) is taken to its nearest value inside.
 * out_lps (NULL: not wanted) is the id's log-probability under the weights that it was drawn from
 * (0 for a first in order by temperature).  A row without a finite or +inf logit: id -1, NaN.
 * temperature, top_k, top_p and min_p hold one value per row on the device; NULL means 1, off, off,
 * off.  Rows start on 16 bytes, and ld * element is a multiple of 16 bytes (columns V .. ld - 1 are
 * not looked at).
 */
int strata_draw_rows(const void* logits, int dtype, int B, int V, int64_t ld, const float* u,
                     const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                     int32_t* out_ids, float* out_lps, void* stream);

/*
 * Bits that the kernels of the calls above raised on the current device since the last call, read
 * after the stream's work so far (this call waits for it) and cleared in one step: STRATA_DEVERR_TIMEOUT,
 * a bounded wait inside a kernel ran out and the call's output is not valid (a draw gives each such row id
 * -1 and NaN).  The bits are those of all
 * streams: each is told to one caller.
 */
int strata_tail_errors(uint32_t* bits, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* STRATA_TAIL_H */
