/*
 * cdb_ops.h — operators of one decode step for programs that drive the model
 * themselves: write a token's keys and values to the paged cache, attend to
 * the cache, pick the next token from the logits.  The engine of cdb.h runs
 * the same steps inside cdb_step_core and cdb_step_boundary; requests admitted
 * with cdb_admit_sampled use the sampler below.
 *
 * Conventions.  All pointers inside the argument structs are device pointers
 * on the current device unless marked otherwise; nothing is allocated, nothing
 * is kept between calls, no call synchronizes.  Work is enqueued on `stream`
 * (cudaStream_t, NULL: the legacy default stream) and can be captured into a
 * CUDA graph.  Calls return CDB_OK, CDB_ERR_ARG (refused before any launch;
 * cdb_ops_last_error() says why) or CDB_ERR_CUDA (a launch failed).
 */
#ifndef CDB_OPS_H
#define CDB_OPS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Why the last cdb_* operator call of this host thread was refused ("" if it was not). */
const char *cdb_ops_last_error(void);

/* ---------------------------------------------------------------- sampling
 * One token per row from its logits x, by a uniform number the caller gives.
 * With m = max x and T the row's temperature, w_i = exp((x_i - m) / T).  Kept
 * are, one filter after the other over the row's tokens in the order (logit
 * descending, index ascending):
 *   top_k   the first top_k tokens (top_k <= 0 or >= vocab: all);
 *   top_p   of those, the shortest prefix whose mass reaches top_p times the
 *           mass of those (top_p >= 1: all; at least one token stays);
 *   min_p   of those, tokens with w_i >= min(min_p, 1) (min_p <= 0: all).
 * The token is the lowest index i whose running mass over the kept tokens, in
 * index order, exceeds u times their total mass; logprob = log(w_i / total).
 * A temperature that is not > 0 takes the argmax (lowest index of a tie) with
 * logprob 0.  A logit of -inf or NaN is never chosen; a row without any other
 * gives token -1 and logprob -inf.  If a row holds +inf, its +inf entries
 * share the whole mass.  u is clamped to [0, 1); u = 0 takes the lowest kept
 * token whose weight is above e^-700.  T below 2^-126 counts as 2^-126.  Masses
 * are exact sums of 64-bit fixed-point weights (unit 2^-44 of the largest, each
 * within 2^-35 of its value), so a row's token depends on nothing but the row. */
#define CDB_SAMPLE_MAX_VOCAB 262144
typedef struct {
  int rows, vocab;           /* vocab <= CDB_SAMPLE_MAX_VOCAB */
  const void *logits;        /* [rows][ld] */
  int dtype;                 /* CDB_FP32 or CDB_BF16 */
  int64_t ld;                /* elements between rows, >= vocab */
  const float *u;            /* [rows] */
  const float *temperature;  /* [rows] */
  const int32_t *top_k;      /* [rows], or NULL: off */
  const float *top_p;        /* [rows], or NULL: off */
  const float *min_p;        /* [rows], or NULL: off */
  int32_t *token;            /* [rows] */
  float *logprob;            /* [rows], or NULL */
} cdb_sample_args;
int cdb_sample(const cdb_sample_args *a, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* CDB_OPS_H */
