/*
 * spec_kv_pages.h -- C ABI of the page management of the paged key-value
 * cache (sm_103a): sharing a sequence's pages with a copy, reserving pages
 * for new positions (copy on write), giving pages back, and moving the live
 * pages to the front of the pool.
 *
 * State (device, caller-owned, the layouts of spec_kv_commit.h):
 *   pool        [layers][num_pages][page_size][entry_bytes]
 *   block_table int32 [B][max_pages]: page of positions p*page_size ..
 *               (p+1)*page_size-1 of sequence b, negative where it holds none
 *   seq_len     int32 [B]: committed length
 *   ref_count   int32 [num_pages]: how many block-table entries hold a page;
 *               a page is free iff its count is 0
 * A sequence's pages are the non-negative entries of its row.  Allocation
 * always takes the free pages of lowest id, so the state after a call is a
 * function of the state before it.
 *
 * spec_kv_release: for every b with new_len[b] >= 0 the sequence keeps the
 * columns below ceil(new_len[b] / page_size); every page behind them is given
 * back (count - 1, entry -1) and seq_len[b] = new_len[b].  new_len[b] < 0
 * leaves the sequence alone; new_len = NULL stands for seq_len itself (pages
 * reserved ahead are given back).  new_len[b] > seq_len[b] is an error.
 *
 * spec_kv_fork: for every pair i < n, sequence dst[i], which must hold no
 * page, becomes a copy of sequence src[i]: its row names the same pages (the
 * columns below ceil(len / page_size), counts + 1; the rest -1) and its
 * length is the same.  Nothing is copied: reserve copies a shared page when
 * it is to be written.  A pair is refused when an index is out of range, when
 * src[i] is the dst of any pair of the call, or when an earlier pair of the
 * call has the same dst.
 *
 * spec_kv_reserve: makes positions seq_len[b] .. seq_len[b]+num_new[b]-1 of
 * every sequence with num_new[b] > 0 writable.  A column of that range that
 * holds no page gets one; a column whose page is shared (count > 1) gets a
 * new page, into which the committed slots of the old one (positions below
 * seq_len[b]) are copied in every layer, and the old page's count drops.  As
 * if the sequences, and the columns of each, were served in order, the last
 * holder of a page keeps it.
 * Pages are handed out by ascending sequence and column.  seq_len does not
 * change.  All or nothing: when the call needs more pages than are free,
 * nothing changes (SPEC_KV_DEVERR_POOL).
 *
 * spec_kv_compact: with m live pages, every live page with an id >= m moves,
 * in ascending order, to the free ids below m in ascending order: contents of
 * every layer, count and every block-table entry.  Afterwards the live pages
 * are 0 .. m-1.  out_num_live (int32 [1], may be NULL) receives m.
 *
 * Invalid data (SPEC_KV_DEVERR_* bits): a sequence or pair with a negative
 * length, a length behind what is allowed, a page id >= num_pages, a page
 * missing where committed positions lie, or a held page whose count is below
 * 1 is left untouched, sets a bit of the error word, and the others are
 * served.  (spec_kv_release looks at the entries that it gives back.)  In
 * spec_kv_compact an entry that names no live page stays as it is
 * and sets SPEC_KV_DEVERR_PAGE.  What else a wrong count does is the caller's:
 * counts that disagree with the table make pages look free that are not, and
 * of several sequences that give back a page with fewer counts than holders
 * it is not determined which are refused.
 *
 * Ownership and asynchrony as in spec_verify.h: work is enqueued on `stream`,
 * nothing is allocated.  `workspace` holds spec_kv_pages_workspace_bytes(dims)
 * bytes, zeroed once before its first use; calls that share a workspace, and
 * calls on the same state, must not run concurrently (the same stream is
 * fine).  The error word is rewritten by every call.
 * Alignment: pool and workspace 16 bytes, the others 4; entry_bytes % 16 ==
 * 0.  Sizes: 1 <= B <= 65535, page_size, num_pages, max_pages >= 1,
 * max_pages*page_size and num_pages*page_size < 2^31, 1 <= layers <= 65535,
 * 1 <= n <= 65535.
 */
#ifndef SPEC_KV_PAGES_H_
#define SPEC_KV_PAGES_H_

#include "spec_kv_commit.h"

#ifdef __cplusplus
extern "C" {
#endif

/* error-word bits, beside SPEC_KV_DEVERR_CAPACITY, _PAGE and _LENGTH */
#define SPEC_KV_DEVERR_PATH 8  /* spec_kv_commit_path: not an ascending path of the tree */
#define SPEC_KV_DEVERR_REF 16  /* a held page has a count below 1 */
#define SPEC_KV_DEVERR_PAIR 32 /* spec_kv_fork: indexes out of range or repeated */
#define SPEC_KV_DEVERR_BUSY 64 /* spec_kv_fork: the destination holds pages */
#define SPEC_KV_DEVERR_POOL 128 /* spec_kv_reserve: not enough free pages */

typedef struct {
  int32_t B;         /* sequences (rows of the block table) */
  int32_t max_pages; /* block-table columns */
  int32_t num_pages; /* pages of the pool */
  int32_t page_size; /* positions per page */
} spec_kv_pages_dims;

/* Workspace bytes for `dims` (0 if the sizes are invalid). */
SPEC_API size_t spec_kv_pages_workspace_bytes(spec_kv_pages_dims dims);

/* Errors of the four calls: SPEC_ERR_ARG for a null required pointer,
 * SPEC_ERR_DIMS for sizes outside the ranges above, SPEC_ERR_ALIGN,
 * SPEC_ERR_WORKSPACE for a short workspace, SPEC_ERR_CUDA for a launch
 * failure. */
SPEC_API spec_status spec_kv_release(const int32_t *new_len, int32_t *seq_len, int32_t *block_table,
                                     int32_t *ref_count, spec_kv_pages_dims dims, void *workspace,
                                     size_t workspace_bytes, spec_stream_t stream);

SPEC_API spec_status spec_kv_fork(const int32_t *src, const int32_t *dst, int32_t n, int32_t *seq_len,
                                  int32_t *block_table, int32_t *ref_count, spec_kv_pages_dims dims, void *workspace,
                                  size_t workspace_bytes, spec_stream_t stream);

SPEC_API spec_status spec_kv_reserve(const int32_t *num_new, const int32_t *seq_len, int32_t *block_table,
                                     int32_t *ref_count, void *pool, int32_t layers, int64_t entry_bytes,
                                     spec_kv_pages_dims dims, void *workspace, size_t workspace_bytes,
                                     spec_stream_t stream);

SPEC_API spec_status spec_kv_compact(int32_t *block_table, int32_t *ref_count, void *pool, int32_t layers,
                                     int64_t entry_bytes, int32_t *out_num_live, spec_kv_pages_dims dims,
                                     void *workspace, size_t workspace_bytes, spec_stream_t stream);

/* Synchronises `stream` and copies the error word of the latest call on this
 * workspace to *error_word. */
SPEC_API spec_status spec_kv_pages_read_error(void *workspace, int32_t *error_word, spec_stream_t stream);

/*
 * The commit of a tree round: after spec_tree_verify accepted the nodes
 * path[b][0 .. n-1] (its out_path; n = num_accepted[b]) of sequence b, the
 * entries that survive are the root's and the path's, in that order:
 *   entry 0 = node 0, entry i = node path[b][i-1], i = 1 .. n,
 * and entry i becomes position L+i, L = seq_len[b]; seq_len[b] = L + n + 1.
 * n < 0 (a sequence flagged by the verify step) keeps nothing.
 *
 * staged [layers][B][N][entry_bytes]: entry of node i of sequence b; or NULL
 * for in-place mode, where the tree pass wrote node i's entry at position
 * L+i, and the kept ones move down to L .. L+n (node 0 is in its place).
 * The other arguments, sizes and errors are those of spec_kv_commit with
 * dims.S = N; `path` is int32 [B][N].  A sequence with n >= N, or whose
 * path[b][0 .. n-1] is not strictly ascending within 1 .. N-1
 * (SPEC_KV_DEVERR_PATH), and one that spec_kv_commit would refuse, is left
 * untouched.  Workspace: spec_kv_path_workspace_bytes(dims) bytes, zeroed
 * once; its error word is read with spec_kv_pages_read_error.
 */
SPEC_API size_t spec_kv_path_workspace_bytes(spec_kv_dims dims);
SPEC_API spec_status spec_kv_commit_path(const int32_t *num_accepted, const int32_t *path, int32_t *seq_len,
                                         const int32_t *block_table, const void *staged, void *pool,
                                         spec_kv_dims dims, void *workspace, size_t workspace_bytes,
                                         spec_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_KV_PAGES_H_ */
