// Sampling kernel (sample.cu): the operator of cdb_ops.h and the engine's
// sampled requests share it.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace cdb {

// Settings of one engine sequence slot.
struct SampleParams {
  int on;  // 0: greedy, the row is left alone
  float temperature;
  int top_k;
  float top_p, min_p;
};

struct SampleRows {
  int rows, vocab;
  const void* logits;
  int64_t ld;
  const float* u;
  const float* temperature;
  const int* top_k;    // nullable
  const float* top_p;  // nullable
  const float* min_p;  // nullable
  int* token;
  float* logprob;      // nullable
  int empty_token;     // token of a row that has nothing to choose from
  // Engine rows (slot non-null): row i belongs to sequence slot[i] and makes
  // its token t[i]; settings come from params[slot], the number, the forced
  // token and the result from index slot * cap + t.
  const int* slot;
  const int* t;
  const SampleParams* params;
  const int* forced;
  int cap;
};

// rows <= INT_MAX / 8, vocab <= CDB_SAMPLE_MAX_VOCAB.
cudaError_t launch_sample(cudaStream_t s, const SampleRows& a, bool bf16);

}  // namespace cdb
