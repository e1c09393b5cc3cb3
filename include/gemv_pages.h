/*
 * gemv_pages.h -- C ABI of the pages of a paged key-value cache
 * (include/gemv_attention.h): tables of pages and the slots of new tokens, made
 * on the device from the sequences' lengths, and pages given back.
 *
 * Free pages are a stack: free[0 .. count[0]) are page numbers that no table
 * holds.  Pages are taken from its top, and put there.
 *
 * Conventions as in gemv.h: device pointers, caller-owned buffers, work
 * enqueued on `stream`, gemv_status codes, nothing allocated, deterministic.
 * Nothing on the device is trusted for addressing.
 */
#ifndef MBGR_GEMV_PAGES_H
#define MBGR_GEMV_PAGES_H

#include <stddef.h>
#include <stdint.h>

#include "gemv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The tables of sequences, and the free pages of their pool. */
typedef struct gemv_page_pool {
    int32_t* free_pages;    /* [pages] */
    const int32_t* count;   /* [1 or more]: how many of them there are */
    int pages;              /* of the pool */
    int page_size;
    int32_t* table;         /* [batch][width], rows table_stride entries apart */
    int64_t table_stride;
    int width;
    int batch;
} gemv_page_pool;

/* Room for new tokens: sequence b, of lens[b] tokens, gets added[b] more (negative
 * numbers count as 0).  Its pages are those of the table's first ceil(lens[b] /
 * page_size) entries; the entries after these are written, up to ceil((lens[b]
 * + added[b]) / page_size) or the table's width, with pages from the stack, in the
 * order of sequences and positions.  Where the stack is empty the entry becomes
 * -1: a hole, whose tokens are neither kept nor seen.
 *   rows       of positions and slots, at least the sum of added: new tokens from
 *              that on are not counted, and get no pages;
 *   count_out  int32 [2]: free pages left, and pages that were missing;
 *   lens_out   int32 [batch]: lens[b] and the tokens that it got;
 *   starts     int32 [batch + 1]: the first row of each sequence, and their sum;
 *   positions  int32 [rows]: of each row's token, lens[b] on;
 *   slots      int64 [rows]: page * page_size + position % page_size, or -1 where
 *              its page is a hole or past the table's width.
 * Rows from starts[batch] on get position 0 and slot -1.  The stack is not
 * written: what lies from count_out[0] to count[0] has been taken.  The outputs overlap
 * neither each other nor the inputs.  Lengths are taken as 0 to 2^31 - 1 with
 * what is added.
 * GEMV_E_INVAL for negative sizes, page_size below 1, table_stride below width, a
 * missing pointer or outputs that overlap (of a table whose rows lie apart, its first
 * row is looked at); GEMV_E_UNSUPPORTED for more than 2^30 rows. */
int gemv_reserve_pages(const gemv_page_pool* pool, const int32_t* lens, const int32_t* added, int rows,
                       int32_t* count_out, int32_t* lens_out, int32_t* starts, int32_t* positions, int64_t* slots,
                       hipStream_t stream);

/* Gives pages back: sequence b keeps the table's first ceil(keep[b] / page_size)
 * entries (keep 0 releases it, its length after an eviction drops what that left;
 * negative numbers count as 0); the pages of its other entries, up to the width,
 * are put on the stack in the order of sequences and entries, and the entries
 * become -1.  Entries that name no page are not put there, nor pages past the
 * stack's room: a page given back must stand in one table, once.
 *   count_out  int32 [2]: free pages now, and 0; it overlaps no input;
 *   workspace  of at least gemv_release_pages_workspace bytes, 16-byte aligned,
 *              one for each call that may run at once.
 * GEMV_E_INVAL as above, and for too small a workspace; GEMV_E_UNSUPPORTED for
 * more than 65536 sequences. */
size_t gemv_release_pages_workspace(const gemv_page_pool* pool);

int gemv_release_pages(const gemv_page_pool* pool, const int32_t* keep, int32_t* count_out, void* workspace,
                       size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MBGR_GEMV_PAGES_H */
