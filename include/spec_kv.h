/*
 * spec_kv.h -- the key/value cache of the verify step and the attention that
 * reads it (libspecverify.so).
 *
 * A verify step scores gamma_b + 1 tokens of every sequence at once: the
 * target's forward pass appends their keys and values to the cache and lets
 * each of them attend to the sequence so far.  spec_commit then returns the
 * cache length to keep (kv_len): the entries of rejected drafts are simply
 * overwritten by the next step.  Many sequences sampled from one prompt share
 * the prompt's entries (the prefix), which are held, and read, once.
 *
 * Cache.  Pages of page_size tokens: element (page, head, slot, d) of the keys
 * is k_pages[page*k_page_stride + (head*page_size + slot)*head_dim + d], of
 * the values likewise.  Position p of sequence b is token p of the prefix
 * (p < prefix_len, page prefix_table[p / page_size]) or token p - prefix_len
 * of the sequence's own pages (page_table[b*table_row_stride + ...]).
 * Formats: bfloat16, or e4m3 with one exponent e (k_exp / v_exp, int8,
 * [n_pages, n_kv_heads, page_size]) for each token and head: a stored y stands
 * for y * 2^e, e the least integer in [-100, 119] with max|x| <= 448 * 2^e.
 *
 * Conventions are those of spec_verify.h: device pointers owned by the
 * caller, no allocation, asynchronous on the stream, arguments checked before
 * any launch, per-row errors reported in row_status (optional), bitwise
 * reproducible results.  Cache pointers and page strides are multiples of 16
 * bytes; other tensors need their element's alignment only (multiples of 16
 * bytes run faster).
 */
#ifndef SPEC_KV_H
#define SPEC_KV_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { SPEC_KV_BF16 = 0, SPEC_KV_E4M3 = 1 } spec_kv_format;

/* Row status bits, beside those of spec_verify.h (SPEC_ROW_BAD_GAMMA). */
#define SPEC_ROW_BAD_LENGTH (1 << 7) /* kv_len[b] below prefix_len, or the step's
                                        tokens pass the row's page table */
#define SPEC_ROW_BAD_PAGE   (1 << 8) /* a page id in use outside [0, n_pages) */

typedef struct {
  void *k_pages, *v_pages;
  int8_t *k_exp, *v_exp; /* e4m3 only (ignored for bfloat16) */
  int64_t k_page_stride, v_page_stride; /* elements; >= n_kv_heads*page_size*head_dim */
  int32_t n_pages;
  int32_t page_size;  /* 16, 32, 64 or 128 */
  int32_t n_kv_heads; /* >= 1 */
  int32_t head_dim;   /* 64, 80, 96 or 128 */
  int32_t format;     /* spec_kv_format */
} spec_kv_cache;

typedef struct {
  int32_t B;          /* sequences, 0 .. 4096; 0 => no-op */
  int32_t gamma_max;  /* the step holds gamma_max + 1 tokens per sequence (ignored by spec_kv_read) */
  int32_t max_pages;  /* columns of page_table (>= 0) */
  int32_t prefix_len; /* shared tokens (>= 0; 0 => no prefix) */
  int64_t table_row_stride;     /* elements, >= max_pages */
  const int32_t *page_table;    /* device [B, max_pages]: the sequences' own pages */
  const int32_t *prefix_table;  /* device [ceil(prefix_len / page_size)] */
  const int32_t *kv_len;        /* device [B]: tokens held, prefix included */
  const int32_t *gamma_per_row; /* device [B], NULL => gamma_max: sequence b has
                                   gamma_b + 1 tokens in this step */
} spec_kv_batch;

/*
 * Append a step's keys and values: token t <= gamma_b of sequence b goes to
 * position kv_len[b] + t.  k, v: device [B, gamma_max+1, n_kv_heads, head_dim]
 * in float32 or bfloat16 (spec_dtype), element (b, t, h, d) at
 * b*strides[0] + t*strides[1] + h*strides[2] + d.  A whole prompt is one
 * call with gamma_max + 1 its length (the prefix itself: B = 1, page_table the
 * prefix's, prefix_len 0).  To e4m3 every value is rounded once, to nearest
 * even, saturating; NaN and infinities become NaN, and the exponent is that
 * of the row's finite values.  To bfloat16 values are rounded to nearest even.
 * A row with a bad gamma or length writes nothing; with a bad page id its
 * tokens on that page are not written, the others are.  No two tokens
 * of a call may share a place.
 */
spec_status spec_kv_append(const spec_kv_cache *cache, const spec_kv_batch *batch, const void *k,
                           const void *v, int32_t dtype, const int64_t *k_strides,
                           const int64_t *v_strides, int32_t *row_status, void *stream);

/*
 * Read back positions begin .. begin + n - 1 of every sequence, in float32 or
 * bfloat16 (rounded to nearest even): k_out, v_out device
 * [B, n, n_kv_heads, head_dim], contiguous.  Positions at or past kv_len[b]
 * give zeros.  A bad length gives NaN in the whole row, a bad page id in the
 * positions on that page.
 */
spec_status spec_kv_read(const spec_kv_cache *cache, const spec_kv_batch *batch, int32_t begin,
                         int32_t n, int32_t dtype, void *k_out, void *v_out, int32_t *row_status,
                         void *stream);

/*
 * The verify step's attention.  q: device bfloat16 [B, gamma_max+1, n_heads,
 * head_dim] (strides as above), n_heads a multiple of n_kv_heads: query head h
 * reads key/value head h / (n_heads / n_kv_heads).  The step's own tokens are
 * in the cache already (spec_kv_append with the same batch): query i of
 * sequence b attends to positions 0 .. kv_len[b] + i:
 *   z_j = scale * sum_d q_d k_jd,  lse = log sum_j exp z_j,
 *   out_d = sum_j exp(z_j - lse) v_jd.
 * out: device bfloat16 [B, gamma_max+1, n_heads, head_dim]; lse: optional
 * device float32 [B, gamma_max+1, n_heads]; both contiguous.  Queries past
 * gamma_b give 0 and -inf; a row with an error gives NaN.  The prefix is read
 * once for the whole batch.  Scores, softmax sums and outputs are accumulated
 * in single precision.  The softmax weights enter the product with the values
 * in 16 bits, as the values do: over a bfloat16 cache as bfloat16 (2^-8 of
 * each), over an e4m3 cache as float16 and times 2^e, e the exponent of the
 * token's values (in a prefix that more than 64 query rows of a key/value head
 * share, the largest one of its 128 tokens).  Such a product loses bits below
 * 2^-22 of the row's largest (in such a prefix 2^-25) and may vanish below
 * 2^-33 (2^-36), also for an element that is 0 in the token of the largest;
 * below 2^-134 the weight may be missing from lse.  e4m3 entries and queries enter
 * their products exactly where an element is at least 2^-28 of its query's
 * largest and, in a prefix that more than 64 query rows of a key/value head
 * share, an entry at least 2^-22 of the largest within its 128 tokens; smaller
 * ones are rounded.  NaN and infinities in keys and values that a query does
 * not attend to do not reach it.  A row whose kernel gave up a wait reports
 * SPEC_ROW_WAIT_TIMEOUT and gives NaN.
 *
 * workspace: required, 256-byte aligned, spec_attend_workspace_size bytes (it
 * depends on the shapes only, not on kv_len); contents do not matter.
 */
size_t spec_attend_workspace_size(const spec_kv_cache *cache, const spec_kv_batch *batch,
                                  int32_t n_heads);

spec_status spec_attend(const spec_kv_cache *cache, const spec_kv_batch *batch, const void *q,
                        int32_t n_heads, const int64_t *q_strides, float scale, void *out,
                        float *lse, int32_t *row_status, void *workspace, size_t workspace_bytes,
                        void *stream);

#ifdef __cplusplus
}
#endif
#endif /* SPEC_KV_H */
