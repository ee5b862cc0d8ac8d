/*
 * spec_kv8.h -- C ABI of the paged key-value cache held in 8 bits (sm_103a):
 * the commit of accepted entries into it, its pages, and the attention of a
 * sequence's newest tokens over it.
 *
 * State (device, caller-owned; block_table, seq_len and ref_count as in
 * spec_kv_commit.h and spec_kv_pages.h):
 *   pool   [layers][num_pages][page_size][2][kv_heads][head_dim] codes of one
 *          byte (keys, then values): SPEC_KV8_E4M3 (largest 448) or
 *          SPEC_KV8_E5M2 (largest 57344)
 *   scales f32 [layers][num_pages][2][kv_heads]: one for each page, kind and
 *          key-value head; a code stands for its value times the scale
 *
 * spec_kv8_commit: the entries that a round keeps, quantised.
 *   staged [layers][B][S][2][kv_heads][head_dim] in 16 bits (bf16 or fp16)
 *   path = NULL: entry i of sequence b, i < keep = min(num_accepted[b] + 1, S),
 *     becomes position L + i, L = seq_len[b] (spec_kv_commit.h); a prompt of n
 *     tokens is committed with num_accepted = n - 1.
 *   path int32 [B][S]: entry 0 is node 0, entry i node path[b][i-1], i = 1 ..
 *     num_accepted[b] (spec_kv_commit_path of spec_kv_pages.h); S <= 256.
 *   seq_len[b] = L + keep; num_accepted < 0 keeps nothing.
 * For a page, kind and head of which entries are written, with `most` the
 * largest finite magnitude among them:
 *   e = the smallest integer >= -126 with most <= largest code * 2^e (-126 for
 *       most = 0)
 *   scale = 2^e, or the page's present scale where that is larger and the page
 *       holds committed entries (positions below L)
 *   code = x / scale, rounded to nearest, ties to even
 * Where a page's scale rises, the codes of its committed entries are rounded
 * again to the new scale.  Scales are powers of two, so that is exact but for
 * codes that become subnormal: the error of any entry stays below the rounding
 * of its own code plus half a subnormal step for each rise that reaches it.
 * Slots behind the committed entries, and pages that get no entry, stay as
 * they were.  A value that is not a number becomes a code that is not; an
 * infinity becomes one in E5M2 and not a number in E4M3.  Scales of another
 * origin may be any positive normal number: then x / scale is computed as
 * x * (1 / scale) in f32.
 * A sequence with a negative seq_len, positions behind the block table, a page
 * id outside the pool, or a path that is not strictly ascending within 1 ..
 * S-1 (or as long as S) is left untouched and sets a SPEC_KV_DEVERR_* bit.  Of
 * one call, no page may be written through two places of the table
 * (spec_kv8_reserve gives a shared page's writers pages of their own).
 *
 * spec_kv8_reserve, spec_kv8_compact: spec_kv_reserve and spec_kv_compact of
 * spec_kv_pages.h on this pool; the scales of a page that is copied or moved
 * go with it.  (spec_kv_fork and spec_kv_release touch neither.)
 *
 * spec_kv8_attention: the attention of spec_kv_attention (spec_attention.h):
 * S new tokens per sequence over L = seq_len[b] committed positions of the
 * 8-bit pool (ONE layer's plane) and, of the new entries, those that are
 * staged in 16 bits at j <= i (chain, parents = NULL) or node i and its
 * ancestors (tree).
 *   q    [B][S][heads][head_dim], token rows q_stride elements apart
 *   staged [B][S][2][kv_heads][head_dim] of the type of q
 *   out  [B][S][heads][head_dim] dense, of the type of q; out_lse f32
 *        [B][S][heads] or NULL
 * A row that sees only scores of -inf gets out = 0, lse = -inf; a score that
 * is not a number makes its row NaN, and so does a query row with a value that
 * is not finite or of 2^100 and more; a value that is not finite and seen
 * makes its column of the row not finite.  Entries that no row may see never
 * matter, whatever their codes, scales and staged values are.  Sequences are
 * refused, with out = 0 and lse = -inf in their rows, as in spec_attention.h
 * (SPEC_ATTN_DEVERR_*); q_len as there.
 * Precision: the products of the query with 8-bit keys, and of the weights
 * with 8-bit values, are taken with the 16-bit operand split into 8-bit parts;
 * those with staged entries are products of 16-bit operands, the weights
 * rounded to the type of q.  A query element is good to 2^-27 of its row's
 * largest.  A weight times its value's scale is good to 2^-11 of itself or
 * 2^-26 of the row's largest (staged entries count with a scale of 1),
 * whichever is more, so n small ones are off by n 2^-26 of it at most.  Behind
 * positions whose weights are far above all before them (new tokens that
 * outweigh the cache, a cached key with nearly all of the weight) it is good to
 * 2^-17 of the largest among the next 128 where that is less (but not beyond
 * 2^-57 of the row's).  Products, maxima and sums accumulate in f32 and the
 * result is rounded once.  Scales must be 0 or positive normal numbers for
 * positions that are seen; a seen value scale beyond 2^96 makes its rows NaN (a
 * key's may), and the bound above holds from 2^-84 on.  Staged values of 2^64
 * and more may overflow.  The scores of a cached key with an infinite code may
 * be NaN where the definition has an infinity.
 *
 * Ownership and asynchrony as in spec_verify.h: work is enqueued on `stream`,
 * nothing is allocated.  Workspaces are zeroed once before their first use and
 * left ready for the next call, of any sizes that they are large enough for;
 * a workspace of the commit, of the pages and of the attention are three.
 * Calls that share one, and captured graphs that do, must not run
 * concurrently.  Equal calls give equal bits.
 * Alignment: 16 bytes for q, pool, staged, out and workspaces; 4 for the rest.
 * Sizes: 1 <= B <= 65535, head_dim 64 or 128, 1 <= kv_heads <= 1024, 1 <= layers
 * <= 65535, page_size, num_pages, max_pages >= 1, max_pages*page_size and
 * num_pages*page_size < 2^31.  Commit: 1 <= S <= 2^20 (256 with a path).
 * Attention: 1 <= S <= 256, B*S <= 2^24, heads a multiple of kv_heads with
 * heads / kv_heads <= 64, heads <= 1024, q_stride a multiple of 8 and at least
 * heads*head_dim, 0 < scale <= 65536.
 */
#ifndef SPEC_KV8_H_
#define SPEC_KV8_H_

#include "spec_attention.h"
#include "spec_kv_pages.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_KV8_E4M3 0
#define SPEC_KV8_E5M2 1

typedef struct {
  int32_t B;         /* sequences */
  int32_t S;         /* staged entries per sequence */
  int32_t layers;    /* layers (pool, scales and staged planes) */
  int32_t kv_heads;  /* key-value heads */
  int32_t head_dim;  /* 64 or 128 */
  int32_t page_size; /* positions per page */
  int32_t num_pages; /* pages per layer plane of the pool */
  int32_t max_pages; /* block-table columns */
  int32_t dtype;     /* of staged: SPEC_ATTN_BF16 or SPEC_ATTN_FP16 */
  int32_t format;    /* of the codes: SPEC_KV8_E4M3 or SPEC_KV8_E5M2 */
} spec_kv8_dims;

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
  int32_t format;    /* SPEC_KV8_E4M3 or SPEC_KV8_E5M2 */
  int64_t q_stride;  /* elements from one token of q to the next */
} spec_kv8_attn_dims;

/* Workspace bytes (0 if the sizes are invalid); the lengths do not matter. */
SPEC_API size_t spec_kv8_commit_workspace_bytes(spec_kv8_dims dims);
SPEC_API size_t spec_kv8_attention_workspace_bytes(spec_kv8_attn_dims dims);

/* See above.  All return SPEC_ERR_ARG for a null required pointer or a bad
 * scale, SPEC_ERR_DIMS for sizes outside the ranges above, SPEC_ERR_ALIGN,
 * SPEC_ERR_WORKSPACE, SPEC_ERR_CUDA for a launch failure. */
SPEC_API spec_status spec_kv8_commit(const int32_t *num_accepted, const int32_t *path, int32_t *seq_len,
                                     const int32_t *block_table, const void *staged, void *pool, float *scales,
                                     spec_kv8_dims dims, void *workspace, size_t workspace_bytes,
                                     spec_stream_t stream);

SPEC_API spec_status spec_kv8_attention(const void *q, const void *pool, const float *scales,
                                        const int32_t *block_table, const int32_t *seq_len, const void *staged,
                                        const int32_t *parents, const int32_t *q_len, float scale, void *out,
                                        float *out_lse, spec_kv8_attn_dims dims, void *workspace,
                                        size_t workspace_bytes, spec_stream_t stream);

/* spec_kv_reserve and spec_kv_compact (and their workspace) with the scales
 * of kv_heads heads; entry_bytes = 2 * kv_heads * head_dim. */
SPEC_API spec_status spec_kv8_reserve(const int32_t *num_new, const int32_t *seq_len, int32_t *block_table,
                                      int32_t *ref_count, void *pool, float *scales, int32_t layers,
                                      int32_t kv_heads, int64_t entry_bytes, spec_kv_pages_dims dims, void *workspace,
                                      size_t workspace_bytes, spec_stream_t stream);

SPEC_API spec_status spec_kv8_compact(int32_t *block_table, int32_t *ref_count, void *pool, float *scales,
                                      int32_t layers, int32_t kv_heads, int64_t entry_bytes, int32_t *out_num_live,
                                      spec_kv_pages_dims dims, void *workspace, size_t workspace_bytes,
                                      spec_stream_t stream);

/* Synchronises `stream` and copies the error word of the latest call on this
 * workspace (of the commit or of the attention) to *error_word. */
SPEC_API spec_status spec_kv8_read_error(void *workspace, int32_t *error_word, spec_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_KV8_H_ */
