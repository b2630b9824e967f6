/*
 * locksgen.h — the calls of liblocks.so for generation with more than one
 * hypothesis per request (beam search) and for tokens whose positions have
 * several axes (images, video), over the paged cache of locks.h and lockskv.h,
 * whose conventions they share.
 *
 * Beam search.  A request has `beams` rows of the cache, one after the other:
 * row r of locks_cache_t is beam r % beams of request r / beams.  A step:
 *   lockskv_append        one token per row
 *   locksgen_attend       or locks_dense_decode, or locks_decode_step
 *   (the model's logits)
 *   locksgen_select       the best continuations
 *   locksgen_reorder      the rows follow their parents
 * A row of length 0 is an idle one: it has no token and no pages in use.
 *
 * Pages of a request.  Rows may refer to the same page as long as it is full;
 * from its open page on (column seq_lens / page_size of the block table, the
 * page that the row's next token goes to) a row's pages are its own.  That is
 * how locksgen_reorder leaves them, without a page being allocated or counted:
 * a beam that is continued twice gives its copy the pages of one that is not
 * continued, from the open page on.  So a request begins with its prompt in row 0
 * and the other rows idle (length 0): they hold the prompt's full pages, by
 * reference or not at all, and pages of their own from the prompt's open page on,
 * and the scores of rows other than 0 are -infinity.  From then on every row, an
 * idle one too, has to have a page of its own in the column of the live rows' open
 * page when the rows are reordered.  What the row that gives its pages held before
 * that column leaves the tables: full pages, and, where it had ended or been idle for
 * a while, the open page it was left with and those after it.  A page, full or not,
 * is the caller's to give out again when no row's table holds it any more, or only
 * idle rows', in columns before the open pages of all live rows of the request.
 */
#ifndef LOCKSGEN_H_
#define LOCKSGEN_H_

#include "lockskv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further bits of the device error word. */
#define LOCKSGEN_DEVERR_LOGITS 0x40  /* a NaN or +infinity among a live beam's logits, or as its score */
#define LOCKSGEN_DEVERR_PARENT 0x80  /* a parent outside [-1, beams) */

/* Most rows of a request, and most continuations kept of one. */
#define LOCKSGEN_MAX_BEAMS 32
#define LOCKSGEN_MAX_KEEP 64
/* Most rows (batch * beams) and tokens of a choice. */
#define LOCKSGEN_MAX_ROWS 65535
#define LOCKSGEN_MAX_VOCAB (1 << 22)
/* Most axes of a position. */
#define LOCKSGEN_MAX_AXES 4

/* Positions with several axes:
 *   positions     device int32 [num_axes][total], rows axis_stride elements
 *                 apart: the rotation table's row of each token on each axis.
 *                 A row outside [0, rope_rows) on any axis sets
 *                 LOCKS_DEVERR_POSITION and the token is skipped
 *   axis_of_pair  the axis of rotated pair i, for i < rotary_dim / 2 (host) */
typedef struct locksgen_axes {
  const int32_t* positions;
  int64_t axis_stride;
  int32_t num_axes;
  uint8_t axis_of_pair[64];
} locksgen_axes_t;

/* lockskv_append with positions of several axes: pair i takes its cosine and
 * sine, columns i and rotary_dim/2 + i of the table, from the row of its own
 * axis.  append->rope is required and append->positions must be NULL.  With
 * the same row on every axis this is lockskv_append. */
LOCKS_API locks_status_t locksgen_append_axes(const locks_cache_t* cache, const lockskv_tokens_t* tokens,
                                              const lockskv_append_t* append, const locksgen_axes_t* axes, void* ws,
                                              size_t ws_bytes, void* stream);

/* A choice among the continuations of `batch` requests of `beams` rows:
 *   logits       [batch * beams][vocab], LOCKS_DTYPE_BF16 or LOCKS_DTYPE_F32
 *                (dtype), rows row_stride elements apart (at least vocab),
 *                aligned to an element
 *   scores       float32 [batch][beams]: the hypotheses' log probabilities;
 *                -infinity for a row without a hypothesis, whose logits may
 *                be anything
 *   ended        int32 [batch][beams], or NULL: nonzero for a hypothesis that
 *                has ended, whose logits may be anything (needs an end_token)
 *   end_token    the token that ends a hypothesis, or -1 for none
 *   keep         continuations kept per request, 1..LOCKSGEN_MAX_KEEP
 * and what it gives, all [batch][keep], best first:
 *   out_scores   float32;  out_parents  int32: the beam, 0..beams-1;
 *   out_tokens   int32;    out_ended    int32, or NULL: 1 where the hypothesis
 *                has ended now (its parent had, or its token is end_token)
 * out_scores and out_ended may be scores and ended where keep is beams or batch is 1. */
typedef struct locksgen_choice {
  const void* logits;
  const float* scores;
  const int32_t* ended;
  float* out_scores;
  int32_t* out_parents;
  int32_t* out_tokens;
  int32_t* out_ended;
  int64_t row_stride;
  int32_t batch, beams, vocab, keep;
  int32_t dtype, end_token;
} locksgen_choice_t;

/* Bytes of workspace locksgen_select needs for these sizes.  It is no bound for smaller
 * ones: few rows are cut into more parts, so ask for each set of sizes (the pointers
 * and row_stride do not matter).  What exceeds a limit above is LOCKS_ERR_UNSUPPORTED. */
LOCKS_API locks_status_t locksgen_select_workspace_size(const locksgen_choice_t* choice, size_t* bytes);

/* The best continuations of every request: token v of live beam w scores
 *   scores[w] + x_v - ln sum_u exp(x_u)        (x: the beam's logits)
 * where x_v is above -infinity; a beam that has ended continues as it is, with
 * its own score and the token end_token.  Out come the `keep` largest.  Ties go
 * to the lower beam, and within a beam to the larger logit (logits that differ
 * may score the same), then to the lower token.  Places for which there is no
 * continuation get the score -infinity, parent and token -1 and ended 0.  Scores are
 * compared in 64 bits, of which the sums of exponentials are float32 (two beams'
 * continuations closer than 2^-16 may change places), and rounded once.  A live beam
 * with a NaN or +infinity among its logits, or with such a score, has no
 * continuation and sets LOCKSGEN_DEVERR_LOGITS.  `ws`: 256-byte aligned, its
 * first word the device error word, zeroed once before its first use. */
LOCKS_API locks_status_t locksgen_select(const locksgen_choice_t* choice, void* ws, size_t ws_bytes, void* stream);

/* Bytes of workspace locksgen_reorder needs. */
LOCKS_API locks_status_t locksgen_reorder_workspace_size(const locks_cache_t* cache, int32_t beams, size_t* bytes);

/* The rows of a cache follow their parents (in place; block_table, seq_lens and
 * n_summarized, where given, are written): with parents int32 [batch] (device;
 * beams of the row's own request, as locksgen_select writes them) row r
 * becomes a copy of its parent p:
 *   - its length and summarised pages are p's;
 *   - its pages before p's open page are p's (the same physical pages);
 *   - the lowest row of those with parent p takes p's pages from the open one
 *     on as they are.  The n-th other row of the request that is not the lowest of
 *     its parent takes, from that column on, the pages of the n-th row that is
 *     nobody's parent, and the open page's tokens are copied there, in whole
 *     groups of 16.
 * A row with parent -1 becomes idle: length 0, and the whole table row of one
 * of the rows that are nobody's parent and are left.  Rows of a request that
 * are live should have one length: one that takes the pages of a row with a
 * later open page than its parent's becomes idle instead and sets
 * LOCKS_DEVERR_LENGTHS, as does the copy of a row whose length the table cannot hold.
 *
 * `caches` (host) holds num_caches caches, the layers of a model, that differ
 * in their pools only: one block table, one set of lengths.  batch must be a
 * multiple of beams.  `ws` as for locksgen_select. */
LOCKS_API locks_status_t locksgen_reorder(const locks_cache_t* caches, int32_t num_caches, int32_t beams,
                                          const int32_t* parents, void* ws, size_t ws_bytes, void* stream);

/* Bytes of workspace locksgen_attend needs. */
LOCKS_API locks_status_t locksgen_attend_workspace_size(const locks_cache_t* cache, const locks_params_t* params,
                                                        int32_t beams, size_t* bytes);

/* locks_dense_decode (same arguments and results, up to rounding) for rows that
 * share pages: shared_pages (device int32 [batch / beams]) says how many leading
 * columns of the block table are the same for all rows of a request that are
 * not idle.  Those pages are read once per request (for each 32 of its query
 * heads of a KV head) and not once per row.  No row may be shorter than what it shares: the count is
 * cut to the shortest row's full pages.  Where the columns differ after all,
 * LOCKS_DEVERR_BLOCK_TABLE is set and the request's results are those of some row's pages.
 * Logits, sums and outputs are accumulated in float32; the softmax weights are
 * rounded to bf16 for bf16 pages (2^-8 of each) and to half precision for 4-bit
 * ones (2^-11, and 2^-32 of the row's largest), whose values s * code are rounded
 * to half precision too. */
LOCKS_API locks_status_t locksgen_attend(const locks_cache_t* cache, const locks_params_t* params, int32_t beams,
                                         const int32_t* shared_pages, const void* q, void* out, float* lse, void* ws,
                                         size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LOCKSGEN_H_ */
