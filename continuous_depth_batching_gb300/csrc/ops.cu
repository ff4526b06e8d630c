// C entry points of the decode-step operators (include/cdb_ops.h): argument
// checks and launches.
#include <climits>
#include <string>

#include "../../include/cdb.h"
#include "../../include/cdb_ops.h"
#include "kernels.cuh"
#include "sample.h"

namespace {

thread_local std::string g_err;

int refuse(const char* why) {
  g_err = why;
  return CDB_ERR_ARG;
}

int launched(cudaError_t e) {
  if (e == cudaSuccess) return CDB_OK;
  g_err = cudaGetErrorString(e);
  return CDB_ERR_CUDA;
}

}  // namespace

// The body of an entry point: no C++ exception crosses the C boundary.
#define CDB_ENTRY_BEGIN \
  try {                 \
    g_err.clear();
#define CDB_ENTRY_END                \
  }                                  \
  catch (...) {                      \
    return CDB_ERR_STATE;            \
  }

extern "C" {

const char* cdb_ops_last_error(void) { return g_err.c_str(); }

int cdb_sample(const cdb_sample_args* a, void* stream) {
  CDB_ENTRY_BEGIN
  if (!a) return refuse("no arguments");
  if (a->rows < 0 || a->rows > INT_MAX / 8) return refuse("rows out of range");
  if (a->vocab < 1 || a->vocab > CDB_SAMPLE_MAX_VOCAB) return refuse("vocab must be in 1..262144");
  if (a->ld < a->vocab) return refuse("ld is smaller than vocab");
  if (a->dtype != CDB_FP32 && a->dtype != CDB_BF16) return refuse("logits must be fp32 or bf16");
  if (!a->logits || !a->u || !a->temperature || !a->token) return refuse("logits, u, temperature and token are needed");
  if ((uintptr_t)a->logits % (a->dtype == CDB_FP32 ? 4 : 2)) return refuse("logits are not aligned to their type");
  cdb::SampleRows r = {};
  r.rows = a->rows;
  r.vocab = a->vocab;
  r.logits = a->logits;
  r.ld = a->ld;
  r.u = a->u;
  r.temperature = a->temperature;
  r.top_k = a->top_k;
  r.top_p = a->top_p;
  r.min_p = a->min_p;
  r.token = a->token;
  r.logprob = a->logprob;
  r.empty_token = -1;
  return launched(cdb::launch_sample(static_cast<cudaStream_t>(stream), r, a->dtype == CDB_BF16));
  CDB_ENTRY_END
}

}  // extern "C"
