// C entry points of the decode-step operators (include/cdb_ops.h): argument
// checks and launches.
#include <climits>
#include <cmath>
#include <string>

#include "../../include/cdb.h"
#include "../../include/cdb_ops.h"
#include "cache_ops.h"
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

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Why the cache cannot be used, or nullptr.
const char* bad_cache(const cdb_paged_cache& c) {
  if (c.dtype != CDB_BF16 && c.dtype != CDB_E4M3) return "the cache must be bf16 or e4m3";
  if (c.head_dim != 32 && c.head_dim != 64 && c.head_dim != 96 && c.head_dim != 128)
    return "head_dim must be 32, 64, 96 or 128";
  if (c.kv_blocks < 1 || c.n_kv_slots < 1 || c.n_kv_heads < 1 || c.n_seqs < 1 || c.max_blocks < 1)
    return "cache dimensions must be >= 1";
  if (c.max_blocks > INT_MAX / 16) return "max_blocks out of range";
  if (!c.pool || !aligned(c.pool, 16)) return "pool is missing or not 16-byte aligned";
  if (!c.block_table) return "block_table is missing";
  if (c.dtype == CDB_E4M3 && (!c.scales || !aligned(c.scales, 16))) return "scales are missing or not 16-byte aligned";
  return nullptr;
}

}  // namespace

// The body of an entry point: no C++ exception crosses the C boundary.
#define CDB_ENTRY_BEGIN \
  try {                 \
    g_err.clear();
#define CDB_ENTRY_END                \
  }                                  \
  catch (...) {                      \
    return CDB_ERR_STATE; /* out of host memory */ \
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
  if (a->rows == 0) return CDB_OK;
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

int cdb_cache_write(const cdb_cache_write_args* a, void* stream) {
  CDB_ENTRY_BEGIN
  if (!a) return refuse("no arguments");
  if (const char* why = bad_cache(a->cache)) return refuse(why);
  const int hd = a->cache.head_dim;
  if (a->rows < 0) return refuse("rows out of range");
  if (a->n_heads < 1 || a->n_heads > (1 << 20) || a->cache.n_kv_heads > (1 << 20)) return refuse("n_heads out of range");
  if (a->dtype != CDB_FP32 && a->dtype != CDB_BF16) return refuse("qkv must be fp32 or bf16");
  const int64_t es = a->dtype == CDB_FP32 ? 4 : 2;
  if (a->ldqkv < ((int64_t)a->n_heads + 2 * a->cache.n_kv_heads) * hd) return refuse("ldqkv is smaller than a row");
  if (a->rows == 0) return CDB_OK;
  if (!a->qkv || !aligned(a->qkv, 16) || a->ldqkv * es % 16) return refuse("qkv is missing or its rows are not 16-byte aligned");
  if (!a->q || !aligned(a->q, 16) || a->ldq % 8 || a->ldq < (int64_t)a->n_heads * hd)
    return refuse("q is missing, too narrow, or its rows are not 16-byte aligned");
  if (!a->q_gain != !a->k_gain) return refuse("q_gain and k_gain come together");
  if (a->q_gain && (!aligned(a->q_gain, 16) || !aligned(a->k_gain, 16))) return refuse("gains are not 16-byte aligned");
  if (a->q_gain && !(a->eps >= 0.f)) return refuse("eps must be >= 0");
  if (a->rope) {
    if (a->rot_dim < 16 || a->rot_dim % 16 || a->rot_dim > hd) return refuse("rot_dim must be a multiple of 16, <= head_dim");
    if (a->rope_positions < 1 || !aligned(a->rope, 16)) return refuse("the rotation table is empty or not 16-byte aligned");
  }
  if (!a->seq || !a->pos) return refuse("seq and pos are needed");
  return launched(cdb::launch_cache_write(static_cast<cudaStream_t>(stream), *a));
  CDB_ENTRY_END
}

// Largest call: 31-bit grids and TMA row coordinates, 16-bit split index.
static const char* bad_attention(int rows, int n_heads, int n_kv_heads, int head_dim, int max_ctx, int shared_len) {
  if (n_kv_heads < 1 || n_heads < 1 || n_heads % n_kv_heads) return "n_heads must be a multiple of n_kv_heads";
  if (head_dim != 32 && head_dim != 64 && head_dim != 96 && head_dim != 128) return "head_dim must be 32, 64, 96 or 128";
  if (rows < 0 || (int64_t)rows * n_heads > INT_MAX / 2) return "rows out of range";
  if (max_ctx < 1 || max_ctx > (1 << 22)) return "max_ctx must be in 1..4194304";
  if (shared_len < 0 || shared_len % 16) return "shared_len must be a multiple of 16";
  if (shared_len > max_ctx) return "shared_len is longer than max_ctx";
  return nullptr;
}

size_t cdb_attention_workspace(int rows, int n_heads, int n_kv_heads, int head_dim, int max_ctx, int shared_len) {
  if (bad_attention(rows, n_heads, n_kv_heads, head_dim, max_ctx, shared_len < 0 ? 0 : shared_len)) return 0;
  return cdb::attention_workspace(rows, n_heads, n_kv_heads, head_dim, max_ctx, shared_len);
}

int cdb_attention(const cdb_attention_args* a, void* stream) {
  CDB_ENTRY_BEGIN
  if (!a) return refuse("no arguments");
  if (const char* why = bad_cache(a->cache)) return refuse(why);
  const cdb_paged_cache& c = a->cache;
  if (const char* why = bad_attention(a->rows, a->n_heads, c.n_kv_heads, c.head_dim, a->max_ctx, a->shared_len))
    return refuse(why);
  if ((uint64_t)c.kv_blocks * c.n_kv_slots * 2 * c.n_kv_heads * 16 >= (1ull << 31) - 64)
    return refuse("the pool has more than 2^31 key rows");
  if (a->max_ctx > (int64_t)c.max_blocks * 16) return refuse("max_ctx is longer than the block table");
  if (a->rows == 0) return CDB_OK;
  const int64_t width = (int64_t)a->n_heads * c.head_dim;
  if (!a->q || !aligned(a->q, 16) || a->ldq % 8 || a->ldq < width)
    return refuse("q is missing, too narrow, or its rows are not 16-byte aligned");
  if (!a->out || !aligned(a->out, 16) || a->ldo % 8 || a->ldo < width)
    return refuse("out is missing, too narrow, or its rows are not 16-byte aligned");
  if (!a->seq || !a->pos) return refuse("seq and pos are needed");
  if (!std::isfinite(a->scale)) return refuse("scale must be finite");
  if (a->shared_len && (a->depth || a->slot_base < 0 || a->slot_base >= c.n_kv_slots))
    return refuse("a shared prefix needs all rows in one slot (depth NULL, slot_base a slot of the cache)");
  if (!a->workspace || !aligned(a->workspace, 256) ||
      a->workspace_bytes < cdb_attention_workspace(a->rows, a->n_heads, c.n_kv_heads, c.head_dim, a->max_ctx, a->shared_len))
    return refuse("workspace is missing, too small or not 256-byte aligned");
  return launched(cdb::launch_decode_attention(static_cast<cudaStream_t>(stream), *a));
  CDB_ENTRY_END
}

}  // extern "C"
