/*
 * spec_filter.h -- C ABI of sampling and of filtered logits under a policy of temperature, top-k,
 * min-p and top-p, each row with settings of its own where they are wanted (MI355X, gfx950).
 *
 * A row's policy, in this order, over its finite logits z (-inf is never kept):
 *   temperature  e_v = exp((z_v - max z) / T)
 *   top_k        0 < top_k < V keeps z_v >= the top_k-th largest logit
 *   min_p        keeps e_v >= min_p (a token's probability against the largest)
 *   top_p        top_p < 1 keeps v if what is kept so far and larger, sum of e_w over z_w > z_v, is
 *                less than top_p times the sum of all that is kept so far
 * Tokens with equal logits are kept or dropped together, so that the kept set is all logits at or
 * above one of them, whatever their order.  T == 0 keeps the lowest-index largest logit alone.
 * Weights are taken in 64 bits and summed as whole numbers: the same call gives the same bits, and
 * draws and thresholds are those of the definition but where a cumulative weight lies within 10^-10
 * of the total of its threshold, for any V.
 *
 * spec_filter_logits writes the logits that are kept, and -inf elsewhere: spec_verify,
 * spec_tree_verify, spec_overlap and spec_typical_verify take such rows with top_k = 0 and the same
 * temperature, so that target and draft go through one policy.
 *
 * Conventions are those of spec_verify.h.  Any call may be captured into a HIP graph; the workspace
 * needs no particular contents, and calls that overlap in time need workspaces of their own.
 */
#ifndef SPEC_FILTER_H
#define SPEC_FILTER_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SV_ROW_BAD_POLICY (-11) /* a row's setting outside its range                          */
#define SV_FILTER_MAX_V (1 << 24)

/* A setting is the scalar, or where the pointer is not NULL the row's entry of a device array.
 *   temperature  finite, >= 0;  top_k  any (<= 0: off);  top_p  in (0, 1];  min_p  in [0, 1]
 * Scalars outside are refused: SV_ERR_TEMPERATURE, SV_ERR_PARAM.  So is an output that shares memory
 * with the other, with the logits (but for rows filtered in place), with u or with an array of
 * settings: SV_ERR_PARAM. */
typedef struct {
  float temperature;
  int32_t top_k;
  float top_p;
  float min_p;
  const float *temperatures; /* [rows] */
  const int32_t *top_ks;     /* [rows] */
  const float *top_ps;       /* [rows] */
  const float *min_ps;       /* [rows] */
} sv_policy;

/* Workspace of either call, 256-byte aligned, any contents. */
size_t sv_filter_workspace_bytes(int32_t rows, int32_t V, sv_dtype dtype);

/* One draw per row, as spec_sample: tokens[b] is the first kept v, in index order, whose cumulative
 * weight exceeds u[b] times the total.
 *   logits      [B, V] dtype, V at most SV_FILTER_MAX_V
 *   u           [B] float32 in [0, 1); may be NULL if every temperature is the scalar 0
 *   tokens      [B] int32 out, -1 for a row with a code
 *   row_status  [B] int32 out: 0, or SV_ROW_BAD_POLICY, SV_ROW_BAD_LOGITS (a NaN or +inf logit, or
 *               no finite one), SV_ROW_BAD_UNIFORM (T > 0 and u outside [0, 1)), tested in this order
 * events as in spec_verify_timed, or NULL. */
sv_status spec_sample_filtered(const void *logits, sv_dtype dtype, const float *u, int32_t B,
                               int32_t V, const sv_policy *policy, int32_t *tokens,
                               int32_t *row_status, void *workspace, size_t workspace_bytes,
                               void *stream, void *const *events, int32_t n_events,
                               int32_t *n_launched);

/* Rows of logits with -inf outside the kept set.
 *   logits      [rows, V] dtype
 *   out         [rows, V] dtype out; may be logits itself, else they do not overlap.  A row with
 *               a code becomes NaN
 *   row_status  [rows] int32 out: 0, SV_ROW_BAD_POLICY or SV_ROW_BAD_LOGITS */
sv_status spec_filter_logits(const void *logits, sv_dtype dtype, int32_t rows, int32_t V,
                             const sv_policy *policy, void *out, int32_t *row_status,
                             void *workspace, size_t workspace_bytes, void *stream,
                             void *const *events, int32_t n_events, int32_t *n_launched);

/* Names of the kernels either call launches, ';'-separated (static storage). */
const char *sv_filter_launch_plan(int32_t draw);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_FILTER_H */
