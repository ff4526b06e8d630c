// Launchers of the operators that prepare and settle a step's rows: arguments
// as checked by the entry points of cdb_ops.h.
#pragma once

#include <cuda_runtime.h>

#include "../../include/cdb_ops.h"

namespace cdb {

cudaError_t launch_rotate(cudaStream_t s, const cdb_rotate_args& a);
cudaError_t launch_plan_pages(cudaStream_t s, const cdb_plan_pages_args& a);
cudaError_t launch_keep_path(cudaStream_t s, const cdb_keep_path_args& a);

// Packed prompts, or drafts where a.visible is given (prompt_attention.cu).
cudaError_t launch_prompt_attention(cudaStream_t s, const cdb_prompt_attention_args& a);
size_t prompt_attention_workspace(int rows, int requests, int n_heads, int n_kv_heads, int head_dim, int max_ctx);

}  // namespace cdb
