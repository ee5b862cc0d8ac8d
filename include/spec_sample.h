/*
 * spec_sample.h -- tokens drawn from filtered distributions (sm_103a): the
 * temperature, top-k, top-p (nucleus) and min-p of each row, and the filtered
 * logits, which make the verify step exact for filtered models.
 *
 * For a row of logits z [V] with temperature T > 0 and m = max z:
 *   w_v = exp((z_v - m) / T); tokens with z_v = -inf have weight 0 and are
 *   never kept (a grammar's bans).  In the order of descending z, ties by
 *   ascending token id, the kept tokens are those within all of
 *     top-k: the first top_k (top_k <= 0: all)
 *     top-p: the shortest prefix of those whose weights sum to at least top_p
 *            times theirs, one token at least (top_p >= 1: all)
 *     min-p: w_v >= min_p (min_p <= 0: all; above 1 as 1)
 *   token = smallest id v with C_v > u * S, C the running sum of the kept
 *   weights in ascending id and S their sum (the rule of the verify step's
 *   draws); u outside [0, 1) counts as its nearest end.
 * T = 0: the token of the largest logit, the lowest id among equals; the
 * filters do not matter.
 *
 * out_logits (may be NULL, may be logits itself with ld = out_ld): z_v of kept tokens, m - 512 T
 * of all others (m - 512 for T = 0, where the token alone is kept): their
 * weights underflow to 0 in spec_verify_from_logits and
 * spec_tree_verify_from_logits at the same T, so a round on filtered draft and
 * target rows draws exactly from the filtered target (for |z| / T up to 2^22,
 * as far as the verify step's exponents go).  (The value is finite: it is
 * rounded to f32, away from m where f32 is coarser than the difference, and not
 * below -FLT_MAX.)
 *
 * Weights are computed to 2^-31 of themselves and summed as integers of 2^-46
 * of the largest (2^-(63 - ceil log2 V) where V exceeds 2^17), so sums do not
 * depend on their order; prefix sums are compared with top_p and u without
 * rounding.  Equal calls give equal bits.
 *
 * Arguments (device pointers, caller-owned, as in spec_verify.h):
 *   logits      f32, row r at logits + r*ld (ld >= V)
 *   uniforms    f32 [rows]; NULL draws nothing (out_tokens must be NULL then)
 *   params      settings of all rows, or arrays [rows] in their place
 *   out_tokens  int32 [rows], -1 for a row that is refused; may be NULL
 *   out_logits  f32, row r at out_logits + r*out_ld; may be NULL (one of the
 *               two outputs is required)
 * A row with a logit that is NaN or +inf, or without a finite one
 * (SPEC_SAMPLE_DEVERR_NONFINITE), or whose array settings are NaN or a negative
 * or infinite temperature (SPEC_SAMPLE_DEVERR_PARAM), gets token -1, its row of
 * out_logits is left as it was, and the error word's bit is set.  The same
 * settings given for all rows are refused by the call (SPEC_ERR_ARG).
 * Temperatures between 0 and 2^-100 count as 2^-100, those above 2^100 as it.
 *
 * workspace: spec_sample_workspace_bytes(dims) bytes, 16-byte aligned, zeroed
 * once before its first use (every call leaves it ready for the next, of any
 * sizes); calls that share one must not run concurrently.  Alignment: 4 bytes
 * for the rest.  Sizes: 1 <= rows <= 2^24, 1 <= V <= 2^19.
 */
#ifndef SPEC_SAMPLE_H_
#define SPEC_SAMPLE_H_

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* error-word bits */
#define SPEC_SAMPLE_DEVERR_NONFINITE 1
#define SPEC_SAMPLE_DEVERR_PARAM 2

typedef struct {
  int32_t rows;
  int32_t V;
  int64_t ld;     /* floats from one row of logits to the next */
  int64_t out_ld; /* of out_logits */
} spec_sample_dims;

typedef struct {
  float temperature;
  int32_t top_k;
  float top_p;
  float min_p;
  /* int32 or f32 [rows] (device) in place of the value above, or NULL */
  const float *temperatures;
  const int32_t *top_ks;
  const float *top_ps;
  const float *min_ps;
} spec_sample_params;

/* Workspace bytes (0 if the sizes are invalid). */
SPEC_API size_t spec_sample_workspace_bytes(spec_sample_dims dims);

/* See above.  SPEC_ERR_ARG for a null required pointer or bad settings,
 * SPEC_ERR_DIMS for sizes outside the ranges above, SPEC_ERR_ALIGN,
 * SPEC_ERR_WORKSPACE, SPEC_ERR_CUDA for a launch failure. */
SPEC_API spec_status spec_sample(const float *logits, const float *uniforms, const spec_sample_params *params,
                                 int32_t *out_tokens, float *out_logits, spec_sample_dims dims, void *workspace,
                                 size_t workspace_bytes, spec_stream_t stream);

/* Synchronises `stream` and copies the error word of the latest call on this
 * workspace to *error_word. */
SPEC_API spec_status spec_sample_read_error(void *workspace, int32_t *error_word, spec_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_SAMPLE_H_ */
