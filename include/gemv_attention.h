/*
 * gemv_attention.h -- C ABI of decode attention over a paged key-value
 * cache, and of the cache's upkeep: append and eviction.
 *
 * The cache is a pool of pages, each of `page_size` slots; a slot holds one
 * token's key and value for every key-value head.  Slot j of sequence b lies
 * in page table[b][j / page_size] at j % page_size.  Sequence b holds
 * lens[b] tokens, in slots 0 .. lens[b] - 1.
 *
 * Conventions as in gemv.h: device pointers, caller-owned buffers, work
 * enqueued on `stream`, gemv_status codes, nothing allocated, deterministic.
 * The descriptor gemv_kv_cache itself is host memory, read before the call
 * returns.  Where a call needs scratch memory the caller passes it
 * (`workspace`, 16-byte aligned, of at least the bytes that the matching
 * *_workspace function returns); its contents mean nothing between calls,
 * and calls that may run at once need one each.
 *
 * Nothing on the device is trusted for addressing: a page number outside
 * [0, pages) is a hole (its slots are not read, written or attended to), a
 * length is taken as at most max_len, the table's width and 2^31 - 4096, a
 * negative one as 0.
 *
 * Addressing needs 16-byte-aligned keys and values: k, v and every row, so
 * strides and head_dim are multiples of 8 elements; GEMV_E_UNSUPPORTED
 * otherwise, and for head_dim over 256.
 */
#ifndef MBGR_GEMV_ATTENTION_H
#define MBGR_GEMV_ATTENTION_H

#include <stddef.h>
#include <stdint.h>

#include "gemv.h"
#include "gemv_types.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gemv_kv_cache {
    void* k;              /* keys and values: the same layout, two buffers or two parts of one */
    void* v;
    int dtype;            /* GEMV_F16 or GEMV_BF16 */
    int pages;
    int page_size;        /* slots in a page, any number from 1 */
    int heads;            /* key-value heads */
    int head_dim;
    int64_t stride_page;  /* elements between pages, slots of a page and heads: any order, */
    int64_t stride_slot;  /* each at least head_dim                                        */
    int64_t stride_head;
} gemv_kv_cache;

/* The sequences of a call. */
typedef struct gemv_kv_batch {
    const int32_t* table;  /* [batch][width], rows table_stride entries apart */
    int64_t table_stride;
    int width;             /* pages per sequence */
    const int32_t* lens;   /* [batch] */
    int batch;
    int max_len;           /* no length is above it: what launches are sized for */
} gemv_kv_batch;

/* Attention of one new token per sequence:
 *   o_bh = sum_j p_bhj v_bj(h'),  p_bh = softmax_j(scale * q_bh . k_bj(h')),  j < lens[b],
 * query head h using key-value head h' = h / (q_heads / heads).
 *   q     [batch][q_heads][head_dim] of the cache's type, sequences q_stride
 *         elements apart (a multiple of 8); q_heads a multiple of heads;
 *   out   [batch][q_heads][head_dim] of the cache's type, dense; it may be q
 *         itself, where q is dense, and overlaps nothing else.
 * A sequence of length 0, with holes only, or with no logit above -inf gets
 * zeros.  Products are summed and the softmax is taken in binary32; the
 * probabilities are not rounded before they meet the values.
 * `weights`, if not NULL: float [batch][heads][slots], slots >= max_len;
 *   weights[b][h'][j] += sum over the query heads h of h' of p_bhj, j < lens[b]
 * (0 for holes); other entries stay as they are.
 * Lengths are split over workgroups, and the parts joined in order of
 * position, in a second launch; short ones are not split.  Both, and the
 * workspace, are sized for max_len and the current device; GEMV_E_UNSUPPORTED
 * where a launch would pass 2^30 work-items (about 4 million parts of 1024
 * slots). */
size_t gemv_attention_workspace(const gemv_kv_cache* cache, const gemv_kv_batch* batch, int q_heads, int weighted);

int gemv_attention(const gemv_kv_cache* cache, const gemv_kv_batch* batch, const void* q, int64_t q_stride,
                   int q_heads, float scale, void* out, float* weights, int64_t slots, void* workspace,
                   size_t workspace_bytes, hipStream_t stream);

/* Writes new tokens to the cache.  Rows starts[b] .. starts[b+1] - 1 of k and
 * v ([rows][heads][head_dim] of the cache's type, rows k_stride / v_stride
 * elements apart, multiples of 8) are sequence b's new tokens; lens[b]
 * counts them already, so the last of them goes to slot lens[b] - 1.  Rows
 * before starts[0] or from starts[batch] on are not read, and a row whose
 * slot lies before 0, past the table's width or in a hole is left out.
 * `starts`: int32 [batch + 1], ascending.  max_len is not used.
 * With `weights` (float) and `positions` (int32), both [batch][heads][slots],
 * and seen (int32 [batch]: the tokens that the sequence has had in all, the
 * new ones included), a written slot also gets weight 0 and the token's
 * position, counted from 0: the state that gemv_kv_evict goes by; a slot from
 * `slots` on is written without them.  All three or none (GEMV_E_INVAL).
 * A page that is written must belong to one sequence of the call and stand in
 * its table once; k and v must not overlap the cache. */
int gemv_kv_append(const gemv_kv_cache* cache, const gemv_kv_batch* batch, const int32_t* starts, const void* k,
                   int64_t k_stride, const void* v, int64_t v_stride, int rows, float* weights, int32_t* positions,
                   const int32_t* seen, int64_t slots, hipStream_t stream);

/* Eviction by accumulated attention weight.  Each key-value head of a
 * sequence with lens[b] > budget keeps `budget` of its tokens: those whose
 * position is at least seen[b] - recent, then those of the largest weight
 * (NaN counts as larger than any number); between equals the lower slot
 * stays.  The kept tokens in slots from `budget` on move, in order, to the
 * slots below `budget` that the evicted ones leave, in order; the others
 * stay where they are, so no more than what was evicted is moved.  Heads keep
 * tokens of their own: a slot then holds different positions per head.
 *   weights, positions [batch][heads][slots], slots >= max_len: read;
 *   weights_out, positions_out, the same shape: the kept tokens' in their new
 *     slots, 0 and -1 in every slot from min(lens[b], budget) on;
 *   lens_out int32 [batch]: min(lens[b], budget).
 * The outputs must not overlap the inputs.  Keys and values move in place;
 * slots from `budget` on keep their contents.  A kept token in a hole moves
 * nothing, and nothing moves into a hole.  Pages must belong to one sequence
 * of the call, once: copy a shared page before evicting from it.
 * 0 <= budget, 0 <= recent (GEMV_E_INVAL otherwise).  Keep recent <= budget:
 * the newest tokens are equals, so where they alone are more than the budget
 * those in the lower slots stay, which are not the latest of them.
 * GEMV_E_UNSUPPORTED beyond 2^20 heads of sequences (batch * heads). */
size_t gemv_kv_evict_workspace(const gemv_kv_cache* cache, const gemv_kv_batch* batch, int budget);

int gemv_kv_evict(const gemv_kv_cache* cache, const gemv_kv_batch* batch, const int32_t* seen, const float* weights,
                  const int32_t* positions, int64_t slots, int budget, int recent, float* weights_out,
                  int32_t* positions_out, int32_t* lens_out, void* workspace, size_t workspace_bytes,
                  hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MBGR_GEMV_ATTENTION_H */
