/*
 * spec_attention.h -- C ABI of the attention operators around the paged
 * key-value cache (sm_103a): the newest tokens of every sequence over its
 * cache (one token, a drafted chain, or a tree of candidates: the target
 * pass that spec_verify and spec_tree_verify follow), and packed prompts.
 *
 * For a query row q_i of head h and the keys k_j and values v_j of its group's
 * key-value head (heads / kv_heads query heads share one):
 *   s_ij  = scale * (q_i . k_j)            over the keys j that i may see
 *   out_i = sum_j exp(s_ij - m_i) v_j / sum_j exp(s_ij - m_i),  m_i = max_j s_ij
 *   lse_i = m_i + log sum_j exp(s_ij - m_i)
 * A row that sees no key (or only keys of score -inf) gets out = 0, lse =
 * -inf.  A row with a score that is not a number gets NaN in out and lse; a
 * value that is infinite or not a number and seen makes its column of the row
 * not finite.  Keys and values that no row may see are never used:
 * not-a-number and infinite values in them have no effect.
 *
 * spec_kv_attention.  S new tokens per sequence (a row of q_len[b] <= S of
 * them where q_len is given; the rows behind are left as they were), L =
 * seq_len[b] committed positions before them.  Token i sees every committed
 * position and, of the new entries, j <= i (chain, parents = NULL) or node i
 * and its ancestors (tree: parents [B][S], parents[b][0] = -1, parents[b][i]
 * in [0, i), as in spec_tree.h).
 *   q    [B][S][heads][head_dim], token rows q_stride elements apart (token
 *        b*S+i starts at (b*S+i)*q_stride; heads of a token are dense)
 *   pool [num_pages][page_size][entry]: ONE layer's plane of the cache of
 *        spec_kv_commit.h, an entry being [2][kv_heads][head_dim] (keys, then
 *        values) of the type of q
 *   staged [B][S][entry]: the new tokens' entries (one layer's plane), or
 *        NULL: they are in the pool at positions L .. L+S-1
 *   block_table, seq_len, q_len int32 as in spec_kv_commit.h
 *   out  [B][S][heads][head_dim] dense; out_lse f32 [B][S][heads] or NULL
 * A sequence with a negative seq_len, a q_len outside [0, S], positions
 * behind the block table, a page id outside [0, num_pages) at a position
 * that is seen, or a bad parent gets out = 0 and lse = -inf in its rows and
 * sets bits of the error word (SPEC_ATTN_DEVERR_*).  (With a q_len outside
 * [0, S] all S rows; a sequence of q_len 0 is not looked at.)
 *
 * spec_prompt_attention.  B sequences packed behind each other: sequence b's
 * queries are rows cu_q[b] .. cu_q[b+1]-1 of q [total_q][heads][head_dim] and
 * its keys and values rows cu_k[b] .. cu_k[b+1]-1 of k, v
 * [total_k][kv_heads][head_dim] (cu_k = NULL: the same as cu_q).  Causal,
 * aligned at the end: of n queries and m keys, query i sees the keys j <= i +
 * m - n (with m > n the queries are the last part of a prompt whose first
 * m - n tokens were processed before).  Token rows are q_stride, k_stride and
 * v_stride elements apart (heads of a token are dense), out is dense.  Rows
 * of out that belong to no sequence are left as they were.  A sequence whose
 * offsets are negative, decrease or pass total_q / total_k is skipped (its
 * rows left as they were) and sets SPEC_ATTN_DEVERR_LENGTH.  Rows named by
 * two sequences (offsets that overlap) are computed for either.
 *
 * Types: q, k, v, pool, staged and out are all bf16 (SPEC_ATTN_BF16) or all
 * fp16 (SPEC_ATTN_FP16).  Scores, maxima, sums and outputs accumulate in
 * f32; the weights exp(s - m) are rounded to the input type for the product
 * with the values (a relative error of at most half a step of the type per
 * weight, the size of the rounding of the result), the result once.  In fp16
 * a weight of less than 2^-21 is off by up to 2^-32 instead: n keys add at
 * most n 2^-32 max|v| to the error of out.
 *
 * Ownership and asynchrony as in spec_verify.h: caller-owned device memory,
 * work enqueued on `stream`, nothing allocated.  Zero a workspace once before
 * its first use (every call leaves it ready for the next, of either operator
 * and of any sizes that it is large enough for); calls that share one, and
 * captured graphs that do, must not run concurrently.  Equal calls give equal
 * bits.
 * Alignment: 16 bytes for q, k, v, pool, staged, out and workspace; strides
 * multiples of 8 elements, at least heads*head_dim (kv_heads*head_dim); 4
 * bytes for the rest.  Sizes: head_dim 64 or 128, 1 <= kv_heads, heads a
 * multiple of kv_heads with heads / kv_heads <= 64, heads <= 1024, 1 <= B <=
 * 65535, 1 <= S <= 256, B*S <= 2^24, total_q and total_k <= 2^24, the
 * position ranges of spec_kv_commit.h, 0 < scale, scale * log2 e finite.
 */
#ifndef SPEC_ATTENTION_H_
#define SPEC_ATTENTION_H_

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_ATTN_BF16 0
#define SPEC_ATTN_FP16 1

/* error-word bits */
#define SPEC_ATTN_DEVERR_CAPACITY 1 /* positions behind the block table */
#define SPEC_ATTN_DEVERR_PAGE 2     /* a page id outside the pool */
#define SPEC_ATTN_DEVERR_LENGTH 4   /* a length or an offset out of range */
#define SPEC_ATTN_DEVERR_TREE 8     /* a parent out of range */
#define SPEC_ATTN_DEVERR_TIMEOUT 16 /* a bounded on-chip wait gave up */

typedef struct {
  int32_t B;         /* sequences */
  int32_t S;         /* new tokens per sequence */
  int32_t heads;     /* query heads */
  int32_t kv_heads;  /* key-value heads */
  int32_t head_dim;  /* 64 or 128 */
  int32_t page_size; /* positions per page */
  int32_t num_pages; /* pages of the pool */
  int32_t max_pages; /* block-table columns */
  int32_t dtype;     /* SPEC_ATTN_BF16 or SPEC_ATTN_FP16 */
  int64_t q_stride;  /* elements from one token of q to the next */
} spec_kv_attn_dims;

typedef struct {
  int32_t B;        /* sequences */
  int32_t heads;    /* query heads */
  int32_t kv_heads; /* key-value heads */
  int32_t head_dim; /* 64 or 128 */
  int32_t total_q;  /* rows of q and out */
  int32_t total_k;  /* rows of k and v */
  int32_t dtype;    /* SPEC_ATTN_BF16 or SPEC_ATTN_FP16 */
  int64_t q_stride, k_stride, v_stride; /* elements from one token to the next */
} spec_prompt_dims;

/* Workspace bytes (0 if the sizes are invalid); the lengths do not matter. */
SPEC_API size_t spec_kv_attention_workspace_bytes(spec_kv_attn_dims dims);
SPEC_API size_t spec_prompt_attention_workspace_bytes(spec_prompt_dims dims);

/* See above.  Both return SPEC_ERR_ARG for a null required pointer or a bad
 * scale, SPEC_ERR_DIMS for sizes outside the ranges above, SPEC_ERR_ALIGN,
 * SPEC_ERR_WORKSPACE, SPEC_ERR_CUDA for a launch failure. */
SPEC_API spec_status spec_kv_attention(const void *q, const void *pool, const int32_t *block_table,
                                       const int32_t *seq_len, const void *staged, const int32_t *parents,
                                       const int32_t *q_len, float scale, void *out, float *out_lse,
                                       spec_kv_attn_dims dims, void *workspace, size_t workspace_bytes,
                                       spec_stream_t stream);

SPEC_API spec_status spec_prompt_attention(const void *q, const void *k, const void *v, const int32_t *cu_q,
                                           const int32_t *cu_k, float scale, void *out, float *out_lse,
                                           spec_prompt_dims dims, void *workspace, size_t workspace_bytes,
                                           spec_stream_t stream);

/* Synchronises `stream` and copies the error word of the latest call of
 * either operator on this workspace to *error_word. */
SPEC_API spec_status spec_attention_read_error(void *workspace, int32_t *error_word, spec_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_ATTENTION_H_ */
