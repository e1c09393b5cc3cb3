/*
 * gemv_rotate.h -- C ABI of what stands between the projections of a token and
 * its attention: the norm of each query and key head and the rotation by the
 * token's position, in one pass, into tensors or straight into a paged cache
 * (include/gemv_attention.h).
 *
 *   n_d = x_d * rsqrt(sum_d x_d^2 / head_dim + eps) * weight_d
 *   y_a = n_a cos(t f_i) - n_b sin(t f_i),   y_b = n_b cos(t f_i) + n_a sin(t f_i)
 *
 * for a token at position t and the pairs (a, b) of the first `rotated`
 * elements of a head, i = 0 .. rotated / 2 - 1: (i, i + rotated / 2), or
 * (2 i, 2 i + 1) where `interleaved`.  The other elements stay n.  Angles are
 * formed and reduced in binary64, so far positions lose nothing; all else is
 * binary32, rounded once to the output's type.
 *
 * Conventions as in gemv.h: device pointers, caller-owned buffers, work
 * enqueued on `stream`, gemv_status codes, nothing allocated, no workspace,
 * deterministic.
 */
#ifndef MBGR_GEMV_ROTATE_H
#define MBGR_GEMV_ROTATE_H

#include <stdint.h>

#include "gemv_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Host memory, read before the call returns. */
typedef struct gemv_rotation {
    int head_dim;          /* 1 to 256 */
    int rotated;           /* even, 0 to head_dim */
    int interleaved;       /* pairs (2 i, 2 i + 1) where not 0 */
    const double* freqs;   /* device, [rotated / 2]: f_i, radians per position */
    int norm;              /* 0: no norm and no weights, the rotation only */
    float eps;
    int weight_dtype;      /* gemv_dtype of the weights */
} gemv_rotation;

/* Heads of `rows` tokens: [rows][heads][head_dim], the heads of a token dense, tokens
 * `stride` elements apart (at least heads * head_dim).  heads may be 0. */
typedef struct gemv_heads {
    const void* x;
    int64_t stride;
    int heads;
    const void* weight;    /* [head_dim], or NULL: ones */
    void* out;             /* laid out alike, with out_stride; may be x itself where types and strides are the same */
    int64_t out_stride;
} gemv_heads;

/* q and k of type `dtype` (gemv_dtype) -> their out of type `out_dtype`;
 * positions int32 [rows], negative ones too.  k may be NULL.  The outputs
 * overlap neither each other nor, but for the above, the inputs.
 * The bandwidth path needs 16-byte-aligned x, out and weights, and strides and
 * head_dim that are multiples of 8; others go element by element.
 * GEMV_E_INVAL for negative sizes, a stride below heads * head_dim, rotated odd
 * or outside [0, head_dim], an unknown type, a missing pointer, or an out whose
 * rows share memory with x's in another type or stride, with the other's or with
 * the other out's;
 * GEMV_E_UNSUPPORTED for head_dim over 256 and for more than 2^30 heads of a row. */
int gemv_norm_rotate(const gemv_rotation* how, const gemv_heads* q, const gemv_heads* k, int dtype, int out_dtype,
                     const int32_t* positions, int rows, hipStream_t stream);

/* The same, with k's results and v put into the cache instead of k's out, and
 * results of the cache's type: token r's go to slot slots[r], which counts
 * through the pages (page slots[r] / page_size, at slots[r] % page_size).  A slot
 * outside the cache is left out (its query is written all the same); no slot
 * stands twice.  v has no norm and no rotation; its weight, out and out_stride
 * are not used, nor k's out and out_stride.  k and v have the cache's heads
 * (GEMV_E_INVAL otherwise); the cache's limits are those of gemv_attention.h. */
int gemv_norm_rotate_append(const gemv_rotation* how, const gemv_heads* q, const gemv_heads* k, const gemv_heads* v,
                            int dtype, const int32_t* positions, int rows, const gemv_kv_cache* cache,
                            const int64_t* slots, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MBGR_GEMV_ROTATE_H */
