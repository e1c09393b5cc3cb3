/*
 * gemv_tokens.h -- C ABI of the INT8 product for several tokens: the weights
 * of gemv_q8 (include/gemv.h) against activations that are quantised to INT8
 * with one scale per token, for prompts and batches, where gemv_q8 takes one
 * binary16 vector.
 *
 *     q_tj = round(x_tj / s_t),  s_t = max_j |x_tj| / 127
 *     y_ti = (sum_j q_tj A_ij) * (s_t * scale_i)
 *
 * Conventions as in gemv.h: device pointers, caller-owned buffers, work
 * enqueued on `stream`, gemv_status codes, nothing allocated, no workspace,
 * deterministic (the sums are whole numbers, so they do not depend on their
 * order).  Outputs must not overlap inputs.
 */
#ifndef MBGR_GEMV_TOKENS_H
#define MBGR_GEMV_TOKENS_H

#include <stdint.h>

#include "gemv.h"
#include "gemv_types.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations x[T][N] of type `dtype` (gemv_dtype), rows `stride` elements
 * apart (stride >= N), -> q int8[T][N] and scale float[T], both dense.
 *   scale_t = absmax / 127, one binary32 division;
 *   q_tj    = the whole number nearest to the exact quotient x_tj / scale_t,
 *             ties to even, clipped to [-127, 127]; a zero scale gives zeros.
 * A row that holds an infinity or a NaN has no scale: it gets scale NaN and
 * codes 0, so that every product of it is NaN.  N == 0 writes scale = 0.
 * T == 0 is a no-op.  The bandwidth path needs 16-byte-aligned x rows and
 * 8-byte-aligned q rows with N % 8 == 0; others take an element-wise path.
 * GEMV_E_INVAL for negative sizes, stride < N, an unknown dtype or a missing
 * pointer. */
int gemv_quantize_tokens_q8(const void* x, int dtype, int64_t stride, int8_t* q, float* scale, int T, int N,
                            hipStream_t stream);

/* y[T][M] of type `dtype` (gemv_dtype), dense:
 *   A int8[M][N] row-major and scale binary16[M] as for gemv_q8,
 *   x int8[T][N] row-major, x_scale float[T],
 *   y_ti = rn(float(sum_j x_tj A_ij) * (x_scale_t * scale_i)),
 * the sum exact in 32-bit integers, the rest in binary32, one rounding to
 * the output's type.  Every int8 value is accepted on both sides; N is at most
 * 131071, where no sum can leave 32 bits (GEMV_E_UNSUPPORTED beyond).
 * N == 0 writes products of zero.  M == 0 or T == 0 is a no-op.
 * GEMV_E_UNSUPPORTED too where a launch would pass 2^30 work-items (never below
 * 2^25 elements of y); GEMV_E_INVAL for negative sizes, an unknown dtype or a
 * missing pointer.
 * The bandwidth path needs 16-byte-aligned A and x and N % 16 == 0; others
 * take a slower path, whose operands go through registers. */
int gemv_gemm_q8(const int8_t* A, const uint16_t* scale, const int8_t* x, const float* x_scale, void* y, int dtype,
                 int T, int M, int N, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MBGR_GEMV_TOKENS_H */
