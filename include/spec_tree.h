/*
 * spec_tree.h -- trees of drafted tokens, and the logits that they are judged
 * by (libspecverify.so).
 *
 * A step of sequence b holds nodes 0 .. gamma_b: node 0 is the last committed
 * token (its cache entry comes with this step, as in spec_kv.h), node j >= 1 is
 * draft j - 1 of draft_tokens [B, gamma_max], the child of node
 * parents[b, j - 1] in [0, j).  A chain has parents[b, j - 1] = j - 1.  Drafts
 * that are alternatives of one another share a parent.
 *
 * One step: spec_tree_mask turns the parents into what each node sees and its
 * depth (its position is kv_len[b] + depth); the target's forward pass appends
 * the nodes' keys and values in node order (spec_kv_append) and attends with
 * the masks (spec_attend_tree); spec_adjust applies penalties, biases and a
 * grammar to every node's logits; spec_sample draws a token at every node;
 * spec_tree_accept follows these draws along the tree; spec_kv_compact moves
 * the accepted nodes' entries together, and spec_commit appends the tokens.
 * The emitted tokens are the target's own draws, one at each node that the
 * walk visits, so they follow the target's law whatever the drafts are.
 *
 * Conventions are those of spec_verify.h: device pointers owned by the caller,
 * no allocation, asynchronous on the stream, arguments checked before any
 * launch, per-row errors reported in row_status (optional), bitwise
 * reproducible results.
 */
#ifndef SPEC_TREE_H
#define SPEC_TREE_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_TREE_MAX 512 /* nodes of a step at most, the root included */

/* Row status bits, beside those of spec_verify.h and spec_kv.h. */
#define SPEC_ROW_BAD_TREE    (1 << 10) /* a parent outside [0, j), or a path that is not one */
#define SPEC_ROW_BAD_PENALTY (1 << 11) /* a penalty that is not finite, a repetition penalty <= 0 */

/*
 * Masks and depths of trees.  parents: device int32 [B, gamma_max]; mask: device
 * int32 [B, N, W], N = gamma_max + 1, W = ceil(N / 32): bit j & 31 of word
 * j >> 5 of row i is set if node j is node i or an ancestor of it; depth:
 * optional device int32 [B, N], 0 for the root; all contiguous.  Nodes past
 * gamma_b have empty masks and depth 0, and so have all nodes of a row with an
 * error (SPEC_ROW_BAD_GAMMA, SPEC_ROW_BAD_TREE).  parents may be NULL when
 * gamma_max is 0.
 */
spec_status spec_tree_mask(int32_t B, int32_t gamma_max, const int32_t *parents,
                           const int32_t *gamma_per_row, int32_t *mask, int32_t *depth,
                           int32_t *row_status, void *stream);

/*
 * The walk along the target's draws.  target_tokens: device int32 [B, N], the
 * token drawn from the target's law at each node; draft_tokens and parents as
 * above.  From node 0: at node i, the child whose draft is target_tokens[b, i]
 * (the lowest of several) is accepted and visited next; without one the walk
 * ends, and target_tokens[b, i] is next_token[b].  accepted_len [B]: drafts
 * accepted.  path (optional) [B, N]: the visited nodes in order, beginning
 * with 0, then -1.  path_tokens (optional) [B, gamma_max]: the accepted drafts
 * in order, then -1: with accepted_len and next_token what spec_commit takes.
 * A row with an error (SPEC_ROW_BAD_GAMMA, SPEC_ROW_BAD_TREE, a negative target
 * token at a visited node: SPEC_ROW_BAD_TOKEN) has accepted_len 0, next_token
 * -1 and an empty path.
 */
spec_status spec_tree_accept(int32_t B, int32_t gamma_max, const int32_t *target_tokens,
                             const int32_t *draft_tokens, const int32_t *parents,
                             const int32_t *gamma_per_row, int32_t *accepted_len,
                             int32_t *next_token, int32_t *path, int32_t *path_tokens,
                             int32_t *row_status, void *stream);

/*
 * Penalties, biases and masks on the logits of a step.  What comes before the
 * token that node i's logits are for: the sequence seq[b, 0 .. seq_len[b]),
 * the first prompt_len[b] tokens of it the prompt, then the drafts on the way
 * to node i (node i's own among them).  With s the tokens of all of that, n_v
 * the number of times that v occurs in it behind the prompt, r, f, p the
 * sequence's penalties:
 *   1. v in s: z > 0 ? z / r : z * r         (repetition penalty r > 0)
 *   2. n_v > 0: z - f n_v - p                (frequency, presence)
 *   3. z + the bias of v
 *   4. -inf where v is not allowed
 * in single precision, rounded once to the logits' type.  Logits that no step
 * applies to are copied as they are.  A mask that allows nothing leaves a row
 * of -inf, which the samplers report (SPEC_ROW_NO_FINITE).
 */
typedef struct {
  int32_t B, gamma_max, V; /* B = 0: no-op; V in [1, 2^24] */
  int32_t dtype;           /* spec_dtype of logits and out */
  int32_t capacity;        /* columns of seq, below 2^30 */
  int32_t n_bias;          /* entries of a row's bias list, 0 .. 65534 */
  /* strides in elements: logits and out [B, gamma_max + 1, V], seq [B, capacity],
     allowed [B, gamma_max + 1, ceil(V / 32)] (words; 0: one for all).  No two
     positions of out overlap. */
  int64_t logits_row_stride, logits_pos_stride, out_row_stride, out_pos_stride;
  int64_t seq_row_stride, allowed_row_stride, allowed_pos_stride;
  /* device arrays; the optional ones may be NULL */
  const int32_t *seq, *seq_len;  /* tokens outside [0, V) count for nothing; [B] */
  const int32_t *prompt_len;     /* optional [B], in [0, seq_len[b]]; NULL: 0 */
  const int32_t *draft_tokens;   /* [B, gamma_max], contiguous; NULL when gamma_max is 0 */
  const int32_t *tree_mask;      /* optional [B, N, W] of spec_tree_mask; NULL: a chain */
  const int32_t *gamma_per_row;  /* optional [B]; NULL: gamma_max */
  const float *repetition, *presence, *frequency; /* optional [B] each */
  const int32_t *bias_ids;       /* [B, n_bias]: tokens outside [0, V) are skipped; */
  const float *bias;             /* of a token that is listed twice the last entry counts */
  const int32_t *allowed;        /* optional: bit v & 31 of word v >> 5: v is allowed */
} spec_adjust_params;

/*
 * out may be logits itself (in place: only what changes is then read and
 * written), or a tensor that has no element in common with it (refused
 * otherwise).  Positions past gamma_b are copied as they are.  A row with an
 * error (SPEC_ROW_BAD_GAMMA, SPEC_ROW_BAD_PENALTY, SPEC_ROW_BAD_LENGTH (1 << 7):
 * seq_len outside [0, capacity], prompt_len outside [0, seq_len]) gives NaN in
 * all its positions.
 * Both tensors need their element's alignment; rows of both that are equally
 * far from a multiple of 16 bytes run faster.
 */
spec_status spec_adjust(const void *logits, const spec_adjust_params *params, void *out,
                        int32_t *row_status, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* SPEC_TREE_H */
