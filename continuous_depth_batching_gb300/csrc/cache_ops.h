// Launchers of the paged-cache operators (cache_ops.cu): arguments as checked
// by the entry points of cdb_ops.h.
#pragma once

#include <cuda_runtime.h>

#include "../../include/cdb_ops.h"

namespace cdb {

cudaError_t launch_cache_write(cudaStream_t s, const cdb_cache_write_args& a);

// Geometry of a decode-attention call: how a row's keys are split.
struct AttnPlan {
  int hpc;      // KV heads of one CTA
  int qblocks;  // groups of at most 8 query heads per KV head
  int split;    // keys of one CTA
  int warps_per_head;  // partials of one CTA per head
  int own_parts;       // partials a row can have
};
AttnPlan attention_plan(int n_heads, int n_kv_heads, int head_dim, int max_ctx);
cudaError_t launch_decode_attention(cudaStream_t s, const cdb_attention_args& a);

}  // namespace cdb
