/*
 * cache.h -- C ABI of libsel, paged key cache: rows quantised as they are
 * written, read back at positions, and the attention of new tokens over them.
 *
 * The selection of sel.h works on the scores of one key; its gather reads a
 * contiguous bf16 key.  A serving program keeps that key in a paged cache,
 * usually in 8 bits, and attends to the rows that a selection chose (or to
 * every row so far).  These entry points do that with the conventions of
 * sel.h: caller-owned device pointers, asynchronous on `stream`, no
 * allocation, argument errors found on the host before a launch, device
 * findings in err_flag, strides in elements.
 *
 * Cache.  One row of d elements a position, shared by all heads (the
 * attention's value is the first dv elements of the row).  Rows lie in pages
 * of page_size rows:
 *   SEL_BF16  bf16 rows.
 *   SEL_E4M3  8-bit floating-point rows (4 exponent bits, 3 mantissa bits,
 *             largest value 448) with one fp32 scale for each run of
 *             SEL_CACHE_GROUP elements: value = code * scale.  sel_cache_write
 *             stores powers of two, so that the value is exact in bf16; with
 *             other scales the value is rounded to bf16 once.
 * Position p of sequence s is row p % page_size of page
 * page_table[s, p / page_size].  Row r of a call belongs to sequence
 * r / (rows / b): rows are batch-major, as in sel_gather_rows.
 */
#ifndef SEL_CACHE_H_
#define SEL_CACHE_H_

#include "../sel.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { SEL_E4M3 = 2 }; /* cache element type, next to SEL_BF16 */

#define SEL_CACHE_GROUP 128      /* elements of a row that share a scale */
#define SEL_CACHE_ATTN_MAX_D 512 /* widest row sel_cache_attention takes */

/* A paged cache.  data: element (page, i, e) at page * page_stride + i *
 * row_stride + e; rows start on 16 bytes and hold whole 16-byte vectors (d a
 * multiple of 8 in SEL_BF16, of 16 in SEL_E4M3; data, row_stride and
 * page_stride to match).  scales (SEL_E4M3 only, else NULL): scale (page, i,
 * g) at page * scale_page_stride + i * scale_row_stride + g, g < ceil(d /
 * SEL_CACHE_GROUP). */
typedef struct {
    void *data;
    float *scales;
    int dtype;
    int64_t pages, page_size, d;
    int64_t page_stride, row_stride;
    int64_t scale_page_stride, scale_row_stride;
} sel_cache;

/* Writes new rows into the cache.
 *   x        [tokens, x_stride] of x_dtype (SEL_F32 | SEL_BF16), d elements a
 *            token, rows on 16 bytes.
 *   slots    [tokens] of slot_dtype (SEL_I32 | SEL_I64): the row's place, page
 *            * page_size + row in the page.  A negative slot is a padding
 *            token: nothing is written.  A slot >= pages * page_size writes
 *            nothing and sets *err_flag = SEL_EINVAL.  Slots of one call have
 *            to differ (of two equal ones either row, or a mix, is kept).
 * SEL_BF16: fp32 rows are rounded to nearest even.  SEL_E4M3: each run of 128
 * gets the smallest power of two 2^e, e >= -126, with 448 * 2^e >= its largest
 * finite magnitude, and the codes are value / 2^e rounded to nearest even; an
 * infinity is stored as +-448 * 2^e, a NaN as NaN.
 * SEL_EUNSUPPORTED: tokens * ceil(d / SEL_CACHE_GROUP) >= 2^27. */
SEL_API int sel_cache_write(const void *x, int x_dtype, int64_t tokens, int64_t x_stride, const void *slots,
                            int slot_dtype, const sel_cache *cache, int32_t *err_flag, void *stream);

/* Reads rows back:  out[r, j, :] = bf16 row at position max(idx[r, j], 0) of
 * sequence r / (rows / b).
 *   page_table  int32 [b, table_stride], max_pages columns used.
 *   idx         [rows, idx_row_stride] of idx_dtype, n columns.
 *   out         bf16 [rows, n, d] contiguous, on 16 bytes.
 * A position >= max_pages * page_size, or one whose page is not in [0, pages),
 * gives a zero row and sets *err_flag = SEL_EINVAL. */
SEL_API int sel_cache_gather(const sel_cache *cache, const int32_t *page_table, int64_t b, int64_t max_pages,
                             int64_t table_stride, const void *idx, int idx_dtype, int64_t rows, int64_t n,
                             int64_t idx_row_stride, void *out, int32_t *err_flag, void *stream);

/* Attention of new tokens over the cache: for each row r and head i,
 *     z_k = scale * <q[r, i, :], K_k>,  out[r, i, :] = sum_k softmax(z)_k K_k[0 .. dv),
 *     lse[r, i] = log sum_k exp z_k,
 * over the row's positions k:
 *   idx == NULL  every position below end[r] (a causal chunk, or single tokens);
 *   idx != NULL  the positions idx[r, 0 .. n) (a selection's output); a
 *                negative one stands for none, one at or past end[r] is left
 *                out, one that is listed twice counts twice.
 *   q        bf16, element (r, i, e) at r * q_row_stride + i * q_head_stride + e,
 *            rows of d on 16 bytes; h >= 1 heads.
 *   end      int32 [rows] exclusive ends, clamped to [0, max_pages *
 *            page_size]; NULL means that limit for every row.
 *   dv       1 <= dv <= d, a multiple of 8.
 *   scale    finite, of any sign, at most 2e38 in magnitude.
 *   out      bf16 [rows, h, dv] contiguous, on 16 bytes.
 *   lse      fp32 [rows, h] contiguous, or NULL (natural logarithm).
 *   workspace  device scratch of at least sel_cache_attention_workspace_size
 *            bytes, 256-byte aligned, any contents; may be NULL when that is 0.
 * A row without positions gives zeros and lse = -inf.  Positions that a row
 * does not attend to have no influence on it, whatever their cache rows hold.
 * An infinity past the first dv elements counts by its score alone (a score of
 * -inf has the weight 0).  A row that attends to a cache row with an infinity
 * or NaN among the first dv elements gets results that are not finite; whether
 * only the elements that the formula makes so, or all and lse, is not specified.
 * Positions past the page table, or whose page is not in [0, pages), are left
 * out and set *err_flag = SEL_EINVAL.  Sums and the softmax are in fp32; the
 * weights are rounded to bf16 for the product with the values.
 * The waits between a CTA's warps end: one that runs out (after about 2 s, where
 * microseconds are usual) sets *err_flag = SEL_ETIMEOUT, and the rows whose
 * results were lost by it hold NaN in out and lse, with or without an err_flag.
 * SEL_EUNSUPPORTED: d > SEL_CACHE_ATTN_MAX_D, rows * h > 2^31 - 1, or
 * n or max_pages * page_size > 2^31 - 256. */
SEL_API int sel_cache_attention(const void *q, int64_t rows, int64_t h, int64_t q_row_stride, int64_t q_head_stride,
                                const sel_cache *cache, const int32_t *page_table, int64_t b, int64_t max_pages,
                                int64_t table_stride, const int32_t *end, const void *idx, int idx_dtype, int64_t n,
                                int64_t idx_row_stride, int64_t dv, float scale, void *out, float *lse,
                                void *workspace, size_t workspace_bytes, int32_t *err_flag, void *stream);

/* Scratch bytes of such a call on the current device (idx_given: whether idx
 * is not NULL): non-zero when rows are few and their positions are shared out
 * over several CTAs.  0 on invalid arguments. */
SEL_API size_t sel_cache_attention_workspace_size(int64_t rows, int64_t h, int64_t d, int64_t dv, int64_t b,
                                                  int64_t max_pages, int64_t page_size, int idx_given, int64_t n);

/* Test hook: GPU clock cycles after which a wait of sel_cache_attention gives
 * up, for the calls that follow, in the whole process; negative: the usual
 * 4e9.  Always SEL_OK. */
SEL_API int sel_cache_set_wait_limit(int64_t cycles);

#ifdef __cplusplus
}
#endif

#endif /* SEL_CACHE_H_ */
