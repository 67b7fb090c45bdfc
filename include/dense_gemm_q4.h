/*
 * dense_gemm_q4.h -- products with weights held in 4 bits with a scale for each
 * group of them, for the GB300 dense GEMM library: a linear layer whose
 * activations stay in 16 bits, for one weight matrix or one for each expert.
 *
 * Weights (out x in, N x K; `experts` of them, one behind the other, where rows
 * are grouped by expert):
 *   codes   N rows of ldq bytes (a multiple of 16, at least (K + 1) / 2), 16-byte
 *           aligned: columns 2j and 2j + 1 in the low and high half of byte j.
 *           Nothing past a row's last code is read, so the last row may end there.
 *   scales  ceil(K / group) rows of N values of X's type, contiguous
 *   zeros   ceil(K / group) rows of N bytes, contiguous, of which the low four bits
 *           count; or NULL: 8 for all
 *   W[n][k] = scales[k / group][n] * (code(n, k) - zeros[k / group][n])
 * group is a multiple of 32 (one at least K: a scale for each row).
 *
 * dtype codes are those of gemm_plan: 1 = FP16, 2 = BF16.  Pointers, streams, errors
 * and the device fault word follow dense_gemm.h, offsets of experts
 * dense_gemm_group.h: argument problems are reported synchronously before anything
 * is queued, work is queued on `stream`, and every device-side wait is bounded.
 * Inputs must not overlap outputs.  Sizes are at most GEMM_GROUP_MAX_SIZE.
 *
 * Device memory: calls with more than 2048 rows (of an expert, were all alike), or with sums
 * too long for the tensor cores (see below), take a workspace for the weights in 16 bits, a
 * power of two of bytes, at most GEMM_Q4_WORKSPACE (more only where a single row of an
 * expert's weights needs more): one per (device, stream), under the rules of dense_gemm.h
 * (replaced by a larger one when a call needs more, never freed, shared by the graphs
 * captured on the stream, whose replays must not overlap).  Those replaced take less
 * than the last one together.  Before a stream capture, make one call of the same sizes
 * on that stream.
 */
#ifndef DENSE_GEMM_Q4_H_
#define DENSE_GEMM_Q4_H_

#include "dense_gemm.h"
#include "dense_gemm_group.h"

#if defined(__cplusplus)
extern "C" {
#endif

#define GEMM_Q4_WORKSPACE (256ll << 20)

/*
 * Y[i] := X[i] . W^T for X (rows x K) and Y (rows x N) of dtype: with experts == 0
 * for all rows, W the only matrix (offsets is NULL); else for the rows i of each
 * expert g, W its matrix, as gemm_grouped does.  X is 16-byte aligned and ldx a
 * multiple of 8, or X is packed (ldx == K) at any alignment of its type, which takes
 * a copy with aligned rows in a workspace first; else GEMM_ERR_MISALIGNED.  Y has any
 * alignment of its type.  FP32 accumulation; one rounding of the result.  K == 0: zeros.
 *
 * Up to 8 rows, 16 of a matrix of at most 2^24 weights, or 8 for each expert, the integers
 * code - zero, exact in 16 bits, are multiplied and each group's FP32 sum is scaled.  For
 * more rows the weights are rounded to dtype first: a row's result then differs by their
 * rounding from what it is among few rows, and an FP16 weight that rounds beyond 65504 is an
 * infinity, where among few rows only the result has to fit.  (There the tensor cores also
 * truncate the running sum at each step of 16 terms.  It is cut into parts that are added in
 * FP32, of at most 16384 terms; up to 2048 rows in BF16, which rounds eight times as coarsely
 * as FP16, of 131072.)
 */
gemm_status_t gemm_q4_linear(int dtype, int group, int rows, int N, int K, int experts,
                             const void *X, int ldx, const void *codes, int ldq,
                             const void *scales, const void *zeros, const int *offsets, void *Y,
                             int ldy, cudaStream_t stream);

#if defined(__cplusplus)
}
#endif

#endif /* DENSE_GEMM_Q4_H_ */
