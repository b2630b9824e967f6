/*
 * lockskv.h — the calls of liblocks.so that write tokens into the paged KV cache
 * and attend whole prompts over it; locks.h holds the decode step that reads the
 * same cache one token at a time, and the conventions that these calls share
 * (device pointers, bf16 elements, caller-owned buffers and stream, no
 * allocation, no synchronisation, host-side checks before any launch, a device
 * error word for what only the device can see, CUDA-graph capture).
 *
 * Serving order.  A prompt: lockskv_append (its keys rotated and stored, its
 * queries rotated), lockskv_prompt_attend, locks_build_summaries for the pages
 * that are now full.  A decode step: lockskv_append with one token per
 * sequence, then locks_decode_step or locks_dense_decode.
 *
 * Ragged token rows.  The calls take the newest tokens of every sequence as
 * rows of one array, sequence after sequence: rows cu_tokens[b] ..
 * cu_tokens[b+1]-1 belong to sequence b (n_b of them, possibly none) and are
 * the tokens at positions seq_lens[b] - n_b .. seq_lens[b] - 1 (seq_lens
 * counts the new tokens, as in locks.h).  With cu_tokens NULL row b is the one
 * newest token of sequence b, `total` is the batch, and a sequence of length 0
 * (an idle slot of a padded batch) has none.  Rows from cu_tokens[batch] on
 * belong to nobody: what they hold has no effect, and nothing is written to
 * them or for them.
 */
#ifndef LOCKSKV_H_
#define LOCKSKV_H_

#include "locks.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The newest tokens of a batch:
 *   cu_tokens   device int32 [batch + 1], nondecreasing, cu_tokens[batch] <=
 *               total; or NULL (one token per sequence)
 *   total       rows of the token arrays
 *   max_tokens  at least every n_b (host knowledge that shapes the launch; 1
 *               when cu_tokens is NULL); any larger number is right too, but
 *               makes a larger launch.  A sequence with more sets
 *               LOCKS_DEVERR_LENGTHS and its rows past max_tokens are skipped.
 * total = 0 (whose arrays may be NULL) or max_tokens = 0 is a call that does
 * nothing. */
typedef struct lockskv_tokens {
  const int32_t* cu_tokens;
  int32_t total;
  int32_t max_tokens;
} lockskv_tokens_t;

/* What lockskv_append writes:
 *   k, v          bf16 [total][num_kv_heads][128], rows k_stride, v_stride
 *                 elements apart (so they may be slices of a fused projection)
 *   q, q_out      bf16 [total][num_q_heads][128] queries to rotate, rows
 *                 q_stride and q_out_stride elements apart, or both NULL;
 *                 q_out may be q itself (same stride), else the two must not
 *                 overlap
 *   rope          float32 [rope_rows][rotary_dim]: row p holds rotary_dim/2
 *                 cosines, then rotary_dim/2 sines of position p's angles; NULL
 *                 for no rotation (rotary_dim 0)
 *   positions     device int32 [total]: the table row of each token; NULL for
 *                 its position in the sequence.  A row outside [0, rope_rows)
 *                 sets LOCKS_DEVERR_POSITION and the token is skipped
 *   rotary_dim    leading dimensions that rotate: a multiple of 16 up to 128
 *   interleaved   0: pair i is dimensions (i, i + rotary_dim/2); 1: (2i, 2i+1)
 * Pointers are 16-byte aligned; strides are multiples of 8 and at least
 * num_heads * 128. */
typedef struct lockskv_append {
  const void* k;
  const void* v;
  const void* q;
  void* q_out;
  const float* rope;
  const int32_t* positions;
  int64_t k_stride, v_stride, q_stride, q_out_stride;
  int32_t num_q_heads;
  int32_t rope_rows;
  int32_t rotary_dim;
  int32_t interleaved;
} lockskv_append_t;

/* Append the newest tokens to the cache (its pools are written; seq_lens and
 * block_table must already cover them).  With (a, b) a pair of a key and (c, s)
 * its row of the table,
 *   a' = a c - b s,  b' = b c + a s
 * in float32, each product and the sum rounded once and the result rounded to
 * bf16; values are stored as they are.  A bf16 cache holds those bf16 numbers.
 * A LOCKS_KV_Q4 cache holds, for each 32 dimensions of them, s = half(max|x| / 7)
 * and the codes rint(x / s) clamped to [-7, 7] (ties to even; zeros where s is
 * zero).  s is at most LOCKS_KV_Q4_MAX_SCALE, so larger numbers saturate at +-65464; a group with
 * an infinity or a NaN gets a NaN scale.  `ws` may be NULL, or any 256-byte
 * aligned memory whose first word is the device error word
 * (locks_get_device_error).  Two sequences must not share a page that either of
 * them writes. */
LOCKS_API locks_status_t lockskv_append(const locks_cache_t* cache, const lockskv_tokens_t* tokens,
                                        const lockskv_append_t* append, void* ws, size_t ws_bytes, void* stream);

/* Read the newest tokens back out of the cache: k_out, v_out bf16
 * [total][num_kv_heads][128] (contiguous; either may be NULL), the numbers that
 * attention sees, s * code rounded to bf16 for a LOCKS_KV_Q4 cache.  With
 * cu_tokens from the lengths themselves this copies whole sequences out of
 * their pages. */
LOCKS_API locks_status_t lockskv_read(const locks_cache_t* cache, const lockskv_tokens_t* tokens, void* k_out,
                                      void* v_out, void* ws, size_t ws_bytes, void* stream);

/* Bytes of workspace lockskv_prompt_attend needs for these shapes (at least
 * 256).  It is planned for sequences as long as the block table is wide, not
 * for their lengths: from 385 (token, head) rows of a KV head on, 4-bit pages
 * are turned into fp16 planes of 768 bytes per KV head and token of the table (16-token
 * bf16 pages: 512 bytes, from 897 rows on), unless those exceed 4 GiB.
 * A narrower table (fewer max_pages, the same pages) needs less.  Zero it once (locks_workspace_init) before its first use; calls of any
 * shapes that it is large enough for may then share it, one after another.  Two
 * calls, or replays of two captured graphs, that may run at the same time need
 * a workspace each. */
LOCKS_API locks_status_t lockskv_prompt_workspace_size(const locks_cache_t* cache, const locks_params_t* params,
                                                       const lockskv_tokens_t* tokens, size_t* bytes);

/* Causal attention of the newest tokens over the cache, which already holds
 * them: for row i of sequence b at position p = seq_lens[b] - n_b + i,
 *   out[row][hq][:] = sum_{t <= p} softmax_t(scale * q.k_t) v_t
 *   lse[row][hq]    = ln sum_{t <= p} exp(scale * q.k_t)      (optional)
 * q: bf16 [total][num_q_heads][128], rows q_stride elements apart (a multiple
 * of 8, at least num_q_heads * 128; base 16-byte aligned); out bf16
 * [total][num_q_heads][128] and lse float32 [total][num_q_heads], contiguous.
 * params->budget_tokens and flags are not used.  Logits, sums and the output's
 * accumulation are float32; softmax weights are rounded to bf16 for bf16 pages
 * (2^-8 of each) and to half precision for 4-bit ones (2^-11, and 2^-31 of the
 * row's largest), whose values s * code are rounded to half precision too. */
LOCKS_API locks_status_t lockskv_prompt_attend(const locks_cache_t* cache, const locks_params_t* params,
                                               const lockskv_tokens_t* tokens, const void* q, int64_t q_stride,
                                               void* out, float* lse, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LOCKSKV_H_ */
