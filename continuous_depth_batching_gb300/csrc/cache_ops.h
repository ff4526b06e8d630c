// Launchers of the paged-cache operators: arguments as checked by the entry
// points of cdb_ops.h.
#pragma once

#include <cuda_runtime.h>

#include "../../include/cdb_ops.h"

namespace cdb {

cudaError_t launch_cache_write(cudaStream_t s, const cdb_cache_write_args& a);
cudaError_t launch_decode_attention(cudaStream_t s, const cdb_attention_args& a);
// Bytes of the partials of such a call.
size_t attention_workspace(int rows, int n_heads, int n_kv_heads, int head_dim, int max_ctx, int shared_len);

// How a row's own keys are split.
struct AttnPlan {
  int hpc;             // KV heads of one CTA
  int qblocks;         // groups of at most 8 query heads per KV head
  int split;           // keys of one CTA
  int warps_per_head;  // of a CTA
  int own_parts;       // partials a row can have
};
// How a shared prefix is cut; chunks 0: it is not, every row reads it itself.
struct SharedPlan {
  int tile_rows;  // batch rows of a tile of at most 128 query rows
  int chunk;      // keys of a CTA, a multiple of 64
  int chunks;     // partials per (row, head)
};
// The prefix's partials (shared_prefix.cu): [row][head][parts], the first
// p.chunks of each; head_dim 64 or 128.  Launched right after the kernel for the
// rows' own keys, beside which it runs; its end is the end of both.
cudaError_t launch_shared_prefix(cudaStream_t s, const cdb_attention_args& a, const SharedPlan& p, int parts, float* part_o,
                                 float2* part_ml);

}  // namespace cdb
