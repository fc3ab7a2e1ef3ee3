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
#define SPEC_ROW_NO_PAGES   (1 << 9) /* the pool has not enough free pages for the row */

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

/*
 * The attention of a step whose tokens are a tree's nodes (spec_tree.h): as
 * spec_attend, but query i of sequence b attends to the positions before the
 * step, 0 .. kv_len[b] - 1, and to those nodes j <= gamma_b of the step
 * (position kv_len[b] + j) whose bit is set in its mask row.  mask: device int32
 * [B, gamma_max+1, W], contiguous, W = ceil((gamma_max+1) / 32), bit j & 31 of
 * word j >> 5: spec_tree_mask's, or any other (a query that sees nothing gives
 * 0 and -inf).  gamma_max < SPEC_TREE_MAX.  All else is as for spec_attend; with
 * more than 64 query rows of a key/value head ((gamma_max + 1) n_heads /
 * n_kv_heads) the sequences' own tokens have the roundings of a prefix that as many
 * share (exponents by 128 tokens of a sequence, its nodes among them).
 */
size_t spec_attend_tree_workspace_size(const spec_kv_cache *cache, const spec_kv_batch *batch,
                                       int32_t n_heads);

spec_status spec_attend_tree(const spec_kv_cache *cache, const spec_kv_batch *batch,
                             const int32_t *mask, const void *q, int32_t n_heads,
                             const int64_t *q_strides, float scale, void *out, float *lse,
                             int32_t *row_status, void *workspace, size_t workspace_bytes,
                             void *stream);

/*
 * Move the entries of an accepted path together: for j = 1 .. accepted_len[b]
 * the entry at position kv_len[b] + path[b, j] goes to position kv_len[b] + j,
 * kv_len the lengths before the step.  path: device int32 [B, gamma_max+1],
 * contiguous, path[b, 0] = 0, increasing (spec_tree_accept's); accepted_len:
 * device int32 [B].  Entries elsewhere stay as they are.  One call for every
 * cache (layer) of the model.  gamma_per_row is not read.  A row whose
 * accepted_len is not in [0, gamma_max] or whose path is not increasing from 0
 * within the step (SPEC_ROW_BAD_TREE, 1 << 10), or whose positions pass its
 * table (SPEC_ROW_BAD_LENGTH), moves nothing; an entry on or for a page that
 * is not there is not moved (SPEC_ROW_BAD_PAGE).
 */
spec_status spec_kv_compact(const spec_kv_cache *cache, const spec_kv_batch *batch,
                            const int32_t *path, const int32_t *accepted_len,
                            int32_t *row_status, void *stream);

/*
 * Page tables over a pool of pages.  refs: device int32 [n_pages], how many
 * table entries hold each page; a page with a count of 0 (or less) is free.
 * Pages that the tables below do not hold (a shared prefix's, say) have their
 * counts set by the caller.  table: device int32 [B, max_pages], row stride in
 * elements, of the sequences' own pages; held: device int32 [B], the entries
 * of each row in use.  What stands behind them in a row is not read, and is
 * overwritten as the row grows.  All caches (layers) of a model share one pool,
 * one table and these calls; page contents are per cache (spec_kv_copy).
 */
typedef struct {
  int32_t B;          /* sequences, 0 .. 4096; 0 => no-op */
  int32_t max_pages;  /* columns of table (>= 0) */
  int32_t n_pages;    /* of the pool */
  int32_t page_size;  /* 16, 32, 64 or 128 */
  int32_t prefix_len; /* tokens that kv_len counts and the table does not hold */
  int64_t table_row_stride;
  int32_t *refs, *table, *held;
} spec_kv_pool;

/*
 * Let row b hold kv_len[b] + n_step tokens (prefix included); kv_len[b] = -1:
 * none.  Pages that are too many are given back (their counts fall by one);
 * pages that are missing are the free ones of the lowest numbers, of those
 * that are free once all rows have given back, in the order of the rows and
 * of the positions.  A row is served if the pool has pages for it and for all
 * rows before it; else it keeps what it has (SPEC_ROW_NO_PAGES).  A row with
 * kv_len below -1 or, unless it is -1, with kv_len[b] + n_step < prefix_len, with
 * more pages than columns, or held outside [0, max_pages] is left as it is
 * (SPEC_ROW_BAD_LENGTH).  A page id outside [0, n_pages) that is to be given
 * back is passed over (SPEC_ROW_BAD_PAGE).
 */
spec_status spec_kv_resize(const spec_kv_pool *pool, const int32_t *kv_len, int32_t n_step,
                           int32_t *row_status, void *stream);

/*
 * Let rows dst[j], j < n, which hold no pages, become forks of rows src[j]: the
 * pages that are full (kv_len[src[j]] tokens) are shared, their counts rise by
 * one; of a last page that is not full the fork has its own, the free page of
 * the lowest number that the forks before it leave, and copies [n, 3] (device
 * int32) says what to copy to it in every cache: page, new page, tokens
 * (spec_kv_copy); -1, -1, 0 where there is nothing to copy.  held and kv_len
 * of dst[j] are set.  A fork whose page the pool does not have
 * (SPEC_ROW_NO_PAGES) changes nothing, and so does one with a row outside
 * [0, B), src[j] = dst[j], dst[j] holding pages or named by an earlier fork of
 * the call (SPEC_ROW_BAD_FORK), or whose source's kv_len does not fit what it
 * holds (SPEC_ROW_BAD_LENGTH).  A source's page id outside [0, n_pages) is
 * copied to the fork, not counted, its contents not copied (SPEC_ROW_BAD_PAGE).
 * fork_status: optional device int32 [n].  n in [0, 4096].
 */
#define SPEC_ROW_BAD_FORK (1 << 12)

spec_status spec_kv_fork(const spec_kv_pool *pool, int32_t *kv_len, const int32_t *src,
                         const int32_t *dst, int32_t n, int32_t *copies, int32_t *fork_status,
                         void *stream);

/*
 * Copy entries between pages of a cache: for each of n triples (page, new page,
 * tokens) of copies (device int32 [n, 3], contiguous) slots 0 .. tokens - 1
 * (at most page_size) of all heads.  Triples with a page outside [0, n_pages)
 * or no tokens are passed over.  No page is the target of two triples of a
 * call, or the source of one and the target of another.  n in [0, 2^20].
 */
spec_status spec_kv_copy(const spec_kv_cache *cache, const int32_t *copies, int32_t n,
                         void *stream);

#ifdef __cplusplus
}
#endif
#endif /* SPEC_KV_H */
