/*
 * cache_serving.h -- C ABI of libsel, paged key cache: what a serving step
 * does besides cache.h's operators.  New tokens' rows are appended at their
 * positions, rotated by them on the way; attention over a window of the
 * latest positions and a few first ones; attention of a batch whose sequences
 * share a long prefix, which is attended to once for all of them where their
 * heads leave room in a tile and that makes less of the work.
 *
 * Conventions, cache format, page table and errors are cache.h's.
 */
#ifndef SEL_CACHE_SERVING_H_
#define SEL_CACHE_SERVING_H_

#include "cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The position rotation.  table: fp32, row p (of `positions`, `stride` elements
 * apart, on 16 bytes) holds the rot / 2 cosines and then the rot / 2 sines of
 * position p's angles.  Elements [first, first + rot) of a row are rotated in
 * pairs: pair i is (first + i, first + rot / 2 + i), with `interleaved` (first
 * + 2 i, first + 2 i + 1); (u, v) becomes (u cos - v sin, v cos + u sin), the
 * products and their sum rounded to fp32.  first is a multiple of 8, rot of 16. */
typedef struct {
    const float *table;
    int64_t positions, stride;
    int64_t first, rot;
    int interleaved;
} sel_rotation;

/* Appends new rows to the sequences of a paged cache, rotated, and rotates the
 * same tokens' queries.
 *   x          [tokens, x_stride] of x_dtype (SEL_F32 | SEL_BF16), d elements a
 *              token, rows on 16 bytes; token t belongs to sequence t / (tokens / b).
 *              Neither it nor another input may overlap the rows that are written.
 *   page_table int32 [b, table_stride], max_pages columns used.
 *   positions  [tokens] of pos_dtype (SEL_I32 | SEL_I64): the row goes to row
 *              p % page_size of page page_table[s, p / page_size].  A negative
 *              position is a padding token: nothing is written.  A position past
 *              the page table or the rotation's table, or whose page is not in
 *              [0, pages), writes nothing and sets *err_flag = SEL_EINVAL.  Two
 *              tokens' places have to differ (of two equal ones either row, or a
 *              mix, is kept).
 *   q          NULL, or the tokens' queries, of q_dtype (SEL_F32 | SEL_BF16),
 *              element (t, i, e) at t * q_row_stride + i * q_head_stride + e, i < h,
 *              rows of d on 16 bytes.
 *   q_out      bf16 [tokens, h, d] contiguous, on 16 bytes (unused without q).
 *              It may be q itself (bf16, contiguous): then only what is rotated
 *              is touched.  Else the two may not overlap, nor may q_out overlap
 *              another input or the cache.  A token whose position is negative
 *              or past the rotation's table has its queries copied as they are.
 * Rows are rounded (SEL_BF16) or quantised (SEL_E4M3) as by sel_cache_write,
 * from the rotated fp32 values; queries are rounded to bf16 once.
 * SEL_EUNSUPPORTED: tokens * ceil(d / SEL_CACHE_GROUP) >= 2^27, d >= 2^30, h * d
 * > 2^31 - 1 or tokens * h * d >= 2^40. */
SEL_API int sel_cache_append(const void *x, int x_dtype, int64_t tokens, int64_t x_stride, const sel_cache *cache,
                             const int32_t *page_table, int64_t b, int64_t max_pages, int64_t table_stride,
                             const void *positions, int pos_dtype, const sel_rotation *rotation, const void *q,
                             int q_dtype, int64_t h, int64_t q_row_stride, int64_t q_head_stride, void *q_out,
                             int32_t *err_flag, void *stream);

/* sel_cache_attention (idx == NULL) of rows that see, of the positions below
 * their end, the last `window` and those below `sinks`:
 *     p < end[r] and (p >= end[r] - window or p < sinks).
 * window >= 1, sinks >= 0.  The page table's entries for pages that hold no
 * position of any of the sequence's rows may be anything (freed pages): they are
 * no finding and have no influence.  (Those between the windows of rows whose
 * ends lie apart may be looked up all the same.) */
SEL_API int sel_cache_attention_window(const void *q, int64_t rows, int64_t h, int64_t q_row_stride,
                                       int64_t q_head_stride, const sel_cache *cache, const int32_t *page_table,
                                       int64_t b, int64_t max_pages, int64_t table_stride, const int32_t *end,
                                       int64_t window, int64_t sinks, int64_t dv, float scale, void *out, float *lse,
                                       void *workspace, size_t workspace_bytes, int32_t *err_flag, void *stream);

/* Scratch bytes of such a call on the current device; 0 on invalid arguments. */
SEL_API size_t sel_cache_attention_window_workspace_size(int64_t rows, int64_t h, int64_t d, int64_t dv, int64_t b,
                                                         int64_t max_pages, int64_t page_size, int64_t window,
                                                         int64_t sinks);

/* sel_cache_attention (idx == NULL) where the first `shared` positions are the
 * same rows for all sequences, usually because their page tables start with the
 * same pages: each of these rows may be read by way of the page table of any
 * sequence with a row that sees it.  shared >= 0; more than the page table's
 * positions means all of them.  It saves work where a tile of 64 (row, head)
 * columns (128 where d <= 192) holds more rows than a sequence has: with more than
 * 32 heads (64), or a sequence's rows filling it, each sequence attends to the
 * prefix for itself. */
SEL_API int sel_cache_attention_shared(const void *q, int64_t rows, int64_t h, int64_t q_row_stride,
                                       int64_t q_head_stride, const sel_cache *cache, const int32_t *page_table,
                                       int64_t b, int64_t max_pages, int64_t table_stride, const int32_t *end,
                                       int64_t shared, int64_t dv, float scale, void *out, float *lse, void *workspace,
                                       size_t workspace_bytes, int32_t *err_flag, void *stream);

/* Scratch bytes of such a call on the current device; 0 on invalid arguments. */
SEL_API size_t sel_cache_attention_shared_workspace_size(int64_t rows, int64_t h, int64_t d, int64_t dv, int64_t b,
                                                         int64_t max_pages, int64_t page_size, int64_t shared);

#ifdef __cplusplus
}
#endif

#endif /* SEL_CACHE_SERVING_H_ */
