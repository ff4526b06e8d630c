/*
 * cdb_ops.h — operators of a step for programs that drive the model
 * themselves: plan pages and rows, rotate queries and keys, write a token's keys
 * and values to the paged cache, attend to the cache (one token per row, whole
 * prompts, drafted tokens), pick the next token from the logits, keep the
 * accepted part of a draft.  The engine of cdb.h runs
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
#define CDB_OPS_NO_BLOCKS 256 /* pages: fewer free blocks than the requests need */
#define CDB_OPS_NO_ROWS 512   /* pages: more new tokens than max_rows */

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

/* --------------------------------------------------------- pages and rows
 * Block tables and packed rows from the lengths of a step's requests, and the
 * blocks of dropped tokens back to the free list.  Request i is sequence seq[i]
 * with lens[i] cached tokens.  new_tokens[i] >= 0 adds that many: blocks for its
 * pages ceil(lens / 16) .. ceil((lens + new) / 16) - 1 are taken, and it gets
 * rows row_start[i] .. row_start[i + 1] - 1, row r with row_seq[r] = seq[i], the
 * next positions in row_pos[r], and row_slot[r] = 16 * block + position % 16.
 * new_tokens[i] < 0 drops that many of its last tokens (all, if it has fewer):
 * blocks of its pages from ceil(what is left / 16) on are given back.
 * Free blocks are the entries state[0] .. state[1] - 1, modulo free_slots, of the
 * ring `free_blocks`: blocks are taken at state[0] and given at state[1], requests
 * and pages in ascending order, and blocks that a call gives are not taken by it.
 * lens_out[i] is the new length and state_out the new counters; they may be lens
 * and state themselves.  Rows from row_start[requests] to max_rows - 1 are padding:
 * row_seq, row_pos and row_slot -1.  Table entries behind a sequence's last page
 * are left as they were.  A sequence is named by one request at most, but for
 * requests with lens and new_tokens 0, which do nothing (padding).
 * A call that cannot be served in full changes nothing: it sets a status bit
 * (CDB_OPS_NO_BLOCKS; CDB_OPS_NO_ROWS; CDB_OPS_BAD_ROW: a sequence, length or
 * counter out of range, or pages past max_blocks), lens_out and state_out are as
 * before, row_start is 0 and every row padding. */
#define CDB_PLAN_MAX_REQUESTS 8192
typedef struct {
  int requests;                 /* <= CDB_PLAN_MAX_REQUESTS */
  const int32_t *lens, *new_tokens; /* [requests] */
  const int32_t *seq;           /* [requests], or NULL: request i is sequence i */
  int32_t *block_table;         /* [n_seqs][max_blocks] */
  int n_seqs, max_blocks;
  int32_t *free_blocks;         /* [free_slots] */
  int free_slots;               /* <= 2^28 */
  const int64_t *state;         /* [2]: blocks taken and given so far */
  int64_t *state_out;           /* [2] */
  int32_t *lens_out;            /* [requests] */
  int32_t *row_start;           /* [requests + 1] */
  int32_t *row_seq, *row_pos;   /* [max_rows] */
  int64_t *row_slot;            /* [max_rows], or NULL */
  int max_rows;                 /* <= 2^30 */
  int32_t *status;
} cdb_plan_pages_args;
int cdb_plan_pages(const cdb_plan_pages_args *a, void *stream);

/* --------------------------------------------------------------- rotation
 * Query / key norm and rotary positions of rows whose positions are not their
 * places in the cache, or that cdb_cache_write's table does not cover: pairs of
 * neighbours, scaled angles, far positions, drafted tokens (which share a depth).
 * A row of x holds n_heads query heads, then n_kv_heads key heads.  In fp32: with
 * gains, each head becomes x / sqrt(mean x^2 + eps) * gain; then pair j < rot_dim /
 * 2 is turned by the angle of 2 pi * (pos * steps[j] mod 2^64) / 2^64 and
 * multiplied by `factor`; elements behind rot_dim are left as they are.  A pair
 * is (j, j + rot_dim / 2), or (2j, 2j + 1) if interleaved.  Angles are exact sums of
 * a 64-bit fraction of a turn, whatever the position; sine and cosine are taken of
 * its distance from the nearest quarter of a turn, rounded to fp32 (2.4e-8 at most).
 * out may be x itself; otherwise they do not overlap.  A row with pos < 0 is
 * padding: nothing of it is read or written. */
typedef struct {
  int rows, n_heads, n_kv_heads, head_dim; /* head_dim 32, 64, 96 or 128 */
  const void *x;          /* [rows][ldx], ldx >= (n_heads + n_kv_heads) head_dim; 16-byte aligned rows */
  int dtype;              /* CDB_FP32 or CDB_BF16, of out too */
  int64_t ldx;
  const int32_t *pos;     /* [rows] */
  const uint64_t *steps;  /* [rot_dim / 2]: turns per position, times 2^64 */
  int rot_dim;            /* a multiple of 16, <= head_dim */
  int interleaved;
  float factor;           /* of cos and sin; finite */
  const float *q_gain, *k_gain; /* [head_dim] each, or both NULL: no norm */
  float eps;
  void *out;              /* [rows][ldo]; 16-byte aligned rows */
  int64_t ldo;
} cdb_rotate_args;
int cdb_rotate(const cdb_rotate_args *a, void *stream);

/* ------------------------------------------- attention of prompts and drafts
 * Request i has query rows row_start[i] .. row_start[i + 1] - 1, its last
 * tokens: lens[i] counts its cached tokens, these among them, so row t of n is at
 * position lens - n + t.  Their keys and values are in the cache (slot `slot`) before the
 * call.  o = sum_j softmax_j(scale * q . k_j) v_j per head, query head h reading
 * KV head h / (n_heads / n_kv_heads), over the positions j that the row sees:
 *   cdb_prompt_attention  all up to its own;
 *   cdb_draft_attention   all before the request's rows, and of those the ones
 *                         whose bits are set in the row's mask: bit u % 64 of
 *                         visible[row][u / 64] for row u of the request (a tree's
 *                         nodes: its ancestors and itself).  Bits of rows that the
 *                         request does not have are ignored.
 * A row that sees nothing, or nothing with a score above -inf, gives zeros.  Rows
 * behind row_start[requests] are left as they were.  Where row_start descends
 * anywhere, CDB_OPS_BAD_ROW is set and `out` is undefined.
 * Softmax statistics and sums are fp32; weights enter the products as 16-bit
 * numbers: bf16 cache, two of them, within 2^-17 of the weight; e4m3 cache, one,
 * weight times value scale, within 2^-11 of it or 2^-33 of the row's largest.
 * With an e4m3 cache a query's elements are exact down to 2^-14 of the head's largest
 * one, smaller ones within 2^-21 of that; a head with an infinite element counts as NaN.
 * Keys and values that no row sees may hold anything.  A value with an infinite or
 * NaN element makes that element infinite or NaN in the rows that see it, and may make
 * the head's other elements NaN there (it does where its block of 128 keys is not
 * seen whole by all rows of a tile); a value scale that is not finite does so to all
 * elements of the head.  Rows that do not see it keep their bits.
 * Where a call has few rows for the GPU, keys are cut among CTAs and joined, by the
 * lengths of all its requests: this changes roundings, never from one run to the
 * next.  max_ctx costs nothing but that a call within 256 tokens is never cut.
 * workspace: cdb_prompt_attention_workspace() bytes, 256-byte aligned, any
 * contents; used by one call at a time. */
#define CDB_DRAFT_MAX 256
typedef struct {
  cdb_paged_cache cache;
  int rows, n_heads;        /* rows of q and out; at most 128 query heads per KV head */
  const void *q;            /* bf16 [rows][ldq]; 16-byte aligned rows */
  int64_t ldq;
  int requests;
  const int32_t *row_start; /* [requests + 1], ascending, row_start[0] >= 0 */
  const int32_t *lens;      /* [requests] */
  const int32_t *seq;       /* [requests], or NULL: request i is sequence i; < 0: skipped */
  int slot;
  float scale;              /* finite */
  int max_ctx;              /* every length <= max_ctx (checked on the device), <= max_blocks * 16 */
  const uint64_t *visible;  /* draft: [rows][mask_words]; prompt: NULL */
  int mask_words;           /* draft: 1 .. CDB_DRAFT_MAX / 64; a request has at most 64 mask_words rows */
  void *out;                /* bf16 [rows][ldo]; 16-byte aligned rows */
  int64_t ldo;
  int32_t *status;
  void *workspace;
  size_t workspace_bytes;
} cdb_prompt_attention_args;
int cdb_prompt_attention(const cdb_prompt_attention_args *a, void *stream);
int cdb_draft_attention(const cdb_prompt_attention_args *a, void *stream);
/* Workspace for any call of up to this many rows and requests.  0 for arguments that are refused. */
size_t cdb_prompt_attention_workspace(int rows, int requests, int n_heads, int n_kv_heads, int head_dim, int max_ctx);

/* ---------------------------------------------------------- accepted drafts
 * Moves the cached keys, values and scales of a draft's accepted nodes to the
 * positions they have in the text, in every slot: entry k < keep[i] of request i
 * from position base[i] + path[i][k] to base[i] + k.  path ascends strictly from
 * path[i][0] >= 0.  keep[i] = 0 moves nothing.  The positions behind are left
 * as they were (drop them with cdb_plan_pages).  A request with seq < 0 is
 * skipped; one with a sequence, node or position out of range sets
 * CDB_OPS_BAD_ROW and moves nothing.  A sequence is named by one request at most. */
typedef struct {
  cdb_paged_cache cache;
  int requests;
  const int32_t *base;     /* [requests] */
  const int32_t *path;     /* [requests][ld_path] */
  int64_t ld_path;         /* >= max_path */
  int max_path;            /* 1 .. CDB_DRAFT_MAX */
  const int32_t *keep;     /* [requests], <= max_path */
  const int32_t *seq;      /* [requests], or NULL: request i is sequence i */
  int32_t *status;
} cdb_keep_path_args;
int cdb_keep_path(const cdb_keep_path_args *a, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* CDB_OPS_H */
