/*
 * gemv_prompt.h -- C ABI of attention over a paged key-value cache for more
 * than gemv_attention (include/gemv_attention.h) takes: several new tokens per
 * sequence (prompts, chunks of them, drafted tokens), a window with first
 * tokens that stay visible, and groups of sequences that share a prefix.
 *
 * The cache, the descriptors and the conventions are those of
 * gemv_attention.h: device pointers, caller-owned buffers, work enqueued on
 * `stream`, gemv_status codes, nothing allocated, deterministic, nothing on the
 * device trusted for addressing, a workspace (16-byte aligned) per call that
 * may run at once with others.  Slot j of a sequence is its token at position
 * j; after gemv_kv_evict, whose heads keep tokens in an order of their own, a
 * window and several new tokens have no meaning.
 */
#ifndef MBGR_GEMV_PROMPT_H
#define MBGR_GEMV_PROMPT_H

#include <stddef.h>
#include <stdint.h>

#include "gemv_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Causal attention of the newest tokens of each sequence, whose keys and
 * values stand in the cache already:
 *   o_th = sum_j p_thj v_j(h'),  p_th = softmax_j(scale * q_th . k_j(h')),
 * over the slots j <= P that token t at position P sees: all of them, or with
 * window > 0 those with j > P - window or j < sinks.
 *   starts  int32 [batch + 1], ascending: rows starts[b] .. starts[b+1] - 1 of q
 *           and out are the last tokens of sequence b, which with them holds
 *           lens[b]; the newest is at position lens[b] - 1.  May be NULL where
 *           every sequence has one new token: row b (max_new 1, rows >= batch).
 *   rows    of q and out in all; starts are taken as at most that.
 *   max_new no sequence has more new tokens: rows before a sequence's last
 *           max_new are left out.
 *   q       [rows][q_heads][head_dim] of the cache's type, rows q_stride
 *           elements apart (a multiple of 8); q_heads a multiple of heads;
 *   out     [rows][q_heads][head_dim] of the cache's type, dense.  Rows of no
 *           sequence, and those left out, stay as they are.  It may be q itself,
 *           where q is dense, and overlaps nothing else.
 * A row that sees nothing (more new tokens than lens[b], holes only, no logit
 * above -inf) gets zeros; what a row does not see does not touch it, NaN and
 * infinities included.  Sums and the softmax are kept in binary32; where max_new
 * is above 1 the powers are rounded to the cache's type before they meet the
 * values: by half a step, or in binary16, where that is more, by 2^-32 of the row's
 * largest power.
 * GEMV_E_INVAL for negative sizes, a missing pointer (starts too, where max_new
 * is not 1 or rows < batch), window < 0 or sinks < 0, an out that shares memory with
 * q's rows otherwise than as said, or too small a workspace;
 * GEMV_E_UNSUPPORTED as for gemv_attention, for out not 16-byte aligned,
 * for more than 2^30 rows of heads, and where a launch would pass 2^30 work-items
 * (about 4 million tiles of 128 query rows, or joins of 4). */
size_t gemv_prompt_attention_workspace(const gemv_kv_cache* cache, const gemv_kv_batch* batch, int rows, int max_new,
                                       int q_heads, int window, int sinks);

int gemv_prompt_attention(const gemv_kv_cache* cache, const gemv_kv_batch* batch, const int32_t* starts, int rows,
                          int max_new, const void* q, int64_t q_stride, int q_heads, float scale, int window, int sinks,
                          void* out, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Attention of one new token per sequence, where groups of sequences share a
 * prefix: sequence b of group g sees the prefixes->lens[g] tokens of the
 * prefix, then its own lens[b] (the new one among them):
 *   o_bh = sum_j p_bhj v_j(h') over both, softmax over both together.
 * The prefix's keys and values are read once for the whole group.
 *   prefixes  the prefixes as sequences: batch is the number of groups,
 *             max_len the longest;
 *   starts    int32 [prefixes->batch + 1], ascending: sequences starts[g] ..
 *             starts[g+1] - 1 are group g's; a sequence of no group sees its own
 *             tokens only;
 *   batch, q, out, zeros, special values and statuses as for gemv_attention
 *   (without weights); out 16-byte aligned.
 * The two may share pages.  The powers of the prefix are rounded to the
 * cache's type before they meet its values, as above; others are not. */
size_t gemv_prefix_attention_workspace(const gemv_kv_cache* cache, const gemv_kv_batch* prefixes,
                                       const gemv_kv_batch* batch, int q_heads);

int gemv_prefix_attention(const gemv_kv_cache* cache, const gemv_kv_batch* prefixes, const int32_t* starts,
                          const gemv_kv_batch* batch, const void* q, int64_t q_stride, int q_heads, float scale, void* out,
                          void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MBGR_GEMV_PROMPT_H */
