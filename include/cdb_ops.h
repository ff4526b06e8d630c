/*
 * cdb_ops.h — operators of one decode step for programs that drive the model
 * themselves: write a token's keys and values to the paged cache, attend to
 * the cache, pick the next token from the logits.  The engine of cdb.h runs
 * the same steps inside cdb_step_core and cdb_step_boundary; requests admitted
 * with cdb_admit_sampled use the sampler below.
 *
 * Conventions.  All pointers inside the argument structs are device pointers
 * on the current device unless marked otherwise, inputs and outputs do not
 * overlap; nothing is allocated, nothing is kept between calls, no call
 * synchronizes.  Work is enqueued on `stream` (cudaStream_t, NULL: the legacy
 * default stream) and can be captured into a CUDA graph (with CUDA's lazy
 * loading, make the first call of an operator outside of the capture).  Calls
 * of several host threads or streams may run at once if they share no output,
 * workspace or status.  rows = 0 does nothing.  Calls return CDB_OK,
 * CDB_ERR_ARG (refused before any launch; cdb_ops_last_error() says why),
 * CDB_ERR_CUDA (a launch failed) or CDB_ERR_STATE (out of host memory).
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
 * token whose weight is above e^-700.  T is clamped to 2^-126..2^126.  Masses
 * are exact sums of 64-bit fixed-point weights (unit 2^-44 of the largest; each
 * off by at most 2^-33 of its value and one unit, so that weights below the unit
 * count nothing unless u = 0), so a row's token depends on nothing but the row. */
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

/* ------------------------------------------------------------- paged cache
 * A pool of 16-token pages, laid out as the engine's: per block and slot, K
 * then V, each head's 16 positions contiguous.  A slot is one KV entry per
 * token: looped models keep one per (layer, loop step).  Position p of sequence
 * s lives in block block_table[s][p / 16].
 * An e4m3 pool (CDB_E4M3) holds 8-bit codes and, per (position, head) of K and
 * of V, a float32 scale; a cached value is scale * code. */
#define CDB_E4M3 2
typedef struct {
  void *pool;                 /* [kv_blocks][n_kv_slots][2][n_kv_heads][16][head_dim] */
  float *scales;              /* e4m3: [kv_blocks][n_kv_slots][2][n_kv_heads][16]; else NULL */
  const int32_t *block_table; /* [n_seqs][max_blocks], entries behind a sequence's last page unused */
  int dtype;                  /* CDB_BF16 or CDB_E4M3 */
  int kv_blocks, n_kv_slots, n_kv_heads, head_dim; /* head_dim 32, 64, 96 or 128 */
  int n_seqs, max_blocks;
} cdb_paged_cache;

/* Device status bits that the cache operators OR into *status (a device int32
 * the caller zeroes; NULL: not reported).  The row concerned is skipped; where
 * attention meets a bad block (a shared prefix: all rows), outputs are undefined. */
#define CDB_OPS_BAD_BLOCK 1   /* block table entry out of range */
#define CDB_OPS_BAD_SLOT 2    /* slot_base + depth out of range */
#define CDB_OPS_BAD_ROW 8     /* sequence or position out of range */
#define CDB_OPS_TIMEOUT 32    /* a bounded wait inside a kernel expired */
#define CDB_OPS_NOT_SHARED 128 /* rows name different blocks inside shared_len */

/* ------------------------------------------------------------- cache write
 * Row i of qkv holds n_heads query heads, n_kv_heads key heads and n_kv_heads
 * value heads of head_dim elements.  In one pass, in fp32:
 *   with gains, every query and key head is normalised, x / sqrt(mean x^2 +
 *   eps) * gain;  with a table, queries and keys are rotated by the row's
 *   position, element j < rot_dim / 2 with j + rot_dim / 2, by (cos, sin) =
 *   rope[pos][j] (elements behind rot_dim are left);
 *   queries are rounded to bf16 into q; keys and values go to position pos of
 *   sequence seq, slot slot_base + depth: rounded to bf16, or as e4m3 with
 *   scale = max(max|x| / 448, 2^-126) and code = e4m3(x / scale), the scale
 *   rounded to float32 where it is stored but not in the quotient.
 * A row with seq < 0 is padding: nothing of it is read or written.  Two rows
 * of one call must not name the same position of the same sequence and slot. */
typedef struct {
  cdb_paged_cache cache;
  int rows, n_heads;
  const void *qkv;        /* [rows][ldqkv], ldqkv >= (n_heads + 2 n_kv_heads) head_dim; 16-byte aligned rows */
  int dtype;              /* CDB_FP32 or CDB_BF16 */
  int64_t ldqkv;
  const float *q_gain, *k_gain; /* [head_dim] each, or both NULL: no norm */
  float eps;
  const float *rope;      /* [rope_positions][rot_dim / 2][2], or NULL: no rotation */
  int rope_positions, rot_dim; /* rot_dim a multiple of 16, <= head_dim */
  const int32_t *seq, *pos;    /* [rows] */
  const int32_t *depth;   /* [rows], or NULL: all 0 */
  int slot_base;
  void *q;                /* bf16 [rows][ldq], ldq >= n_heads head_dim; 16-byte aligned rows */
  int64_t ldq;
  int32_t *status;
} cdb_cache_write_args;
int cdb_cache_write(const cdb_cache_write_args *a, void *stream);

/* -------------------------------------------------------- decode attention
 * One query token per row over the cached positions 0..pos of its sequence:
 * o = sum_j softmax_j(scale * q . k_j) v_j per head, query head h reading KV
 * head h / (n_heads / n_kv_heads).  Softmax statistics and sums are fp32.
 * Weights enter the products as 16-bit numbers: bf16 cache, two of them, within
 * 2^-17 of the weight; e4m3 cache, weight times value scale within 2^-22 of its
 * value or 2^-33 of the row's largest (behind a shared prefix 2^-11 or 2^-33).
 * With an e4m3 cache a query's elements are exact down to 2^-17 of the head's
 * largest one, smaller ones within 2^-25 of that.
 * A row with seq < 0 is padding: its output is left as it was.  A row with
 * pos < 0 has no keys: zeros.  Without a shared prefix, keys are taken a fixed
 * number at a time and joined in order, so a row's bits do not depend on the
 * other rows.
 * shared_len > 0 (a multiple of 16) says that every row's sequence names the
 * same blocks for positions 0..shared_len-1 (a common prompt, all of it
 * written, its values finite): those keys are then read once for all rows (head_dim 64 and 128,
 * two rows or more, at most 128 query heads per KV head; else the prefix is
 * read per row), and cut by the number of rows, which changes a row's roundings.
 * The sequence of the first row with seq >= 0 names the blocks that are read; a
 * row that names others sets CDB_OPS_NOT_SHARED where they are read once.  A row
 * may end inside the prefix.  depth must be NULL then (all rows in one slot).
 * workspace: cdb_attention_workspace() bytes, 256-byte aligned, any contents;
 * used by one call at a time.
 * max_ctx costs time and memory whether rows reach it or not: the grid and the
 * workspace hold every split of max_ctx for every row (128 rows of 1000 keys, 32/8
 * heads, bf16: 82 us and 19 MB with max_ctx 1024, 126 us and 283 MB with 32768,
 * 252 us and 1.1 GB with 131072).  Take the longest row of the batch, rounded up
 * to as few lengths as the program captures graphs for. */
typedef struct {
  cdb_paged_cache cache;
  int rows, n_heads;
  const void *q;          /* bf16 [rows][ldq]; 16-byte aligned rows */
  int64_t ldq;
  const int32_t *seq, *pos;
  const int32_t *depth;
  int slot_base;
  float scale;            /* finite */
  int max_ctx;            /* every pos < max_ctx (checked on the device), <= max_blocks * 16; see above for its cost */
  int shared_len;
  void *out;              /* bf16 [rows][ldo]; 16-byte aligned rows */
  int64_t ldo;
  int32_t *status;
  void *workspace;
  size_t workspace_bytes;
} cdb_attention_args;
int cdb_attention(const cdb_attention_args *a, void *stream);
/* Workspace for a call of this many rows; shared_len < 0: for any shared_len
 * and any number of rows up to this.  0 for arguments cdb_attention refuses. */
size_t cdb_attention_workspace(int rows, int n_heads, int n_kv_heads, int head_dim, int max_ctx, int shared_len);

#ifdef __cplusplus
}
#endif
#endif /* CDB_OPS_H */
