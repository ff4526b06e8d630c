// Operators that prepare and settle a step's rows (include/cdb_ops.h): pages and
// rows from request lengths, rotary positions, the accepted path of a draft.
#include <algorithm>

#include "../../include/cdb.h"
#include "common.cuh"
#include "kernels.cuh"
#include "row_ops.h"
#include "tc.cuh"

namespace cdb {

// ---------------------------------------------------------------------------
// pages and rows
// ---------------------------------------------------------------------------
namespace pages {

constexpr int kThreads = 512;
constexpr int kPage = 16;

__device__ __forceinline__ long long pages_of(long long tokens) { return (tokens + kPage - 1) / kPage; }

// Exclusive sums over the block of three counts at once, and their totals in `total`.
__device__ __forceinline__ void scan3(long long v[3], long long total[3], long long (*sh)[3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long own[3] = {v[0], v[1], v[2]};
#pragma unroll
  for (int o = 1; o < 32; o *= 2)
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const long long x = __shfl_up_sync(0xffffffffu, v[i], o);
      if (lane >= o) v[i] += x;
    }
  __syncthreads();
  if (lane == 31)
    for (int i = 0; i < 3; ++i) sh[warp][i] = v[i];
  __syncthreads();
  for (int i = 0; i < 3; ++i) {
    long long before = 0, all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      const long long x = sh[w][i];
      before += w < warp ? x : 0;
      all += x;
    }
    total[i] = all;
    v[i] += before - own[i];
  }
}

// For each of N numbers the last i with start[i] <= x; start ascends and start[0] <= x < start[n].  Side by side,
// where one bisection after the other took twice the time of the whole kernel.
template <int N>
__device__ __forceinline__ void find(const int* (&start)[N], int (&x)[N], int n, int (&at)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) at[e] = 0;
  for (int half = 1 << (31 - __clz(n)); half; half >>= 1)
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (at[e] + half < n && start[e][at[e] + half] <= x[e]) at[e] += half;
}

// Every CTA of the cluster sums up all requests (a few thousand additions, where
// sharing them out would cost a second round of cluster barriers), then takes its
// part of the rows and pages, found by bisection in shared memory.  Nothing is
// written before every CTA has read lens and state, which outputs may be.
// Latency bounds it: the chain of loads, sums, barrier, lookups and stores (64 requests
// 4.1 us, 1000 with 21702 rows 9.7; those in clusters of four CTAs 16).
template <int B>  // rows of a thread at a time
__global__ void __launch_bounds__(kThreads) k_plan_pages(const __grid_constant__ cdb_plan_pages_args a, int ctas) {
  extern __shared__ int dyn[];
  __shared__ long long sh[kThreads / 32][3];
  const int n = a.requests, tid = threadIdx.x;
  int* row0 = dyn;             // [n + 1] first row of each request
  int* take0 = row0 + n + 1;   // [n + 1] first block taken
  int* give0 = take0 + n + 1;  // [n + 1] first block given back
  int* len = give0 + n + 1;    // [n]
  pdl_wait();
  pdl_trigger();
  const long long head = a.state[0], tail = a.state[1];
  const int per = (n + kThreads - 1) / kThreads;
  const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
  long long v[3] = {0, 0, 0}, total[3];
  bool bad = head < 0 || tail < head || tail - head > a.free_slots;
#pragma unroll 4
  for (int i = i0; i < i1; ++i) {
    const int l = a.lens[i], d = a.new_tokens[i], s = a.seq ? a.seq[i] : i;
    const long long after = max(0ll, (long long)l + d), have = pages_of(l), want = pages_of(after);
    bad |= l < 0 || s < 0 || s >= a.n_seqs || have > a.max_blocks || want > a.max_blocks;
    v[0] += max(0, d);
    v[1] += max(0ll, want - have);
    v[2] += max(0ll, have - want);
    len[i] = l;
  }
  scan3(v, total, sh);
  bad = __syncthreads_or(bad);
  const bool few = total[1] > tail - head, full = total[0] > a.max_rows;
  bad |= total[2] > a.free_slots - (tail - head);
  const bool ok = !bad && !few && !full;  // then every total fits an int
  if (ok) {
    for (int i = i0; i < i1; ++i) {
      const int l = len[i], d = a.new_tokens[i];
      const long long have = pages_of(l), want = pages_of(max(0ll, (long long)l + d));
      row0[i] = (int)v[0], take0[i] = (int)v[1], give0[i] = (int)v[2];
      v[0] += max(0, d);
      v[1] += max(0ll, want - have);
      v[2] += max(0ll, have - want);
    }
    if (tid == 0) row0[n] = (int)total[0], take0[n] = (int)total[1], give0[n] = (int)total[2];
  }
  if (ctas > 1) {
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
  const int at = blockIdx.x * kThreads + tid, step = ctas * kThreads;
  const int rows = ok ? (int)total[0] : 0;
  // One 64-bit remainder for each end of the ring, none for its entries.
  const unsigned slots = a.free_slots, head_at = (unsigned)((unsigned long long)head % slots),
                 tail_at = (unsigned)((unsigned long long)tail % slots);
  auto ring = [&](unsigned from, unsigned k) { return from + k < slots ? from + k : from + k - slots; };  // k < slots
  // Rows, blocks taken and blocks given go by side by side: their lookups and loads do not wait for one another (1000
  // requests with 21702 rows: 11.5 us one after the other, 9.6 four rows at a time).
  const int taken = ok ? (int)total[1] : 0, given = ok ? (int)total[2] : 0, most = max(a.max_rows, max(B * taken, B * given));
  for (int k = 0; k < most; k += B * step) {
    int i[B], seq[B], pos[B], block[B];
    const int t = k / B + at;
    int x[B + 2], in[B + 2];
    const int* where[B + 2];
#pragma unroll
    for (int e = 0; e < B; ++e) x[e] = k + e * step + at, where[e] = row0;
    x[B] = x[B + 1] = t, where[B] = take0, where[B + 1] = give0;
    if (n) find<B + 2>(where, x, n, in);
#pragma unroll
    for (int e = 0; e < B; ++e) i[e] = x[e] < rows ? in[e] : -1;
    const int ti = t < taken ? in[B] : -1, gi = t < given ? in[B + 1] : -1;
#pragma unroll
    for (int e = 0; e < B; ++e) seq[e] = i[e] < 0 ? -1 : a.seq ? a.seq[i[e]] : i[e];
    const int ts = ti < 0 ? 0 : a.seq ? a.seq[ti] : ti, gs = gi < 0 ? 0 : a.seq ? a.seq[gi] : gi;
    const int taken_block = ti < 0 ? 0 : a.free_blocks[ring(head_at, t)], drop = gi < 0 ? 0 : a.new_tokens[gi];
#pragma unroll
    for (int e = 0; e < B; ++e) {
      pos[e] = -1, block[e] = 0;
      if (i[e] < 0) continue;
      const int l = len[i[e]], have = (int)pages_of(l);
      pos[e] = l + k + e * step + at - row0[i[e]];
      const int page = pos[e] / kPage;
      block[e] = page < have ? a.block_table[(size_t)seq[e] * a.max_blocks + page]
                             : a.free_blocks[ring(head_at, take0[i[e]] + page - have)];
    }
    int given_block = 0;
    if (gi >= 0) {
      const long long want = pages_of(max(0ll, (long long)len[gi] + drop));
      given_block = a.block_table[(size_t)gs * a.max_blocks + want + t - give0[gi]];
    }
#pragma unroll
    for (int e = 0; e < B; ++e) {
      const int r = k + e * step + at;
      if (r >= a.max_rows) continue;
      a.row_seq[r] = seq[e];
      a.row_pos[r] = pos[e];
      if (a.row_slot) a.row_slot[r] = i[e] < 0 ? -1 : (long long)block[e] * kPage + pos[e] % kPage;
    }
    if (ti >= 0) a.block_table[(size_t)ts * a.max_blocks + pages_of(len[ti]) + t - take0[ti]] = taken_block;
    if (gi >= 0) a.free_blocks[ring(tail_at, t)] = given_block;
  }
  for (int i = at; i <= n; i += step) {
    a.row_start[i] = ok ? row0[i] : 0;
    if (i < n) a.lens_out[i] = ok ? (int)max(0ll, (long long)len[i] + a.new_tokens[i]) : len[i];
  }
  if (at == 0) {
    a.state_out[0] = ok ? head + total[1] : head;
    a.state_out[1] = ok ? tail + total[2] : tail;
    if (bad) report(a.status, CDB_OPS_BAD_ROW);
    else if (few) report(a.status, CDB_OPS_NO_BLOCKS);
    else if (full) report(a.status, CDB_OPS_NO_ROWS);
  }
}

}  // namespace pages

cudaError_t launch_plan_pages(cudaStream_t s, const cdb_plan_pages_args& a) {
  using namespace pages;
  const size_t smem = (size_t)(4 * a.requests + 3) * 4;
  static bool set[kMaxDevices] = {};
  const int dev = current_device();
  if (!set[dev]) {
    for (auto k : {k_plan_pages<1>, k_plan_pages<4>}) {
      const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (4 * CDB_PLAN_MAX_REQUESTS + 3) * 4);
      if (e != cudaSuccess) return e;
    }
    set[dev] = true;
  }
  // A row for each thread of up to eight CTAs (64 rows: 4.0 us, 4.6 with the kernel for four); beyond that four.
  int ctas = 1;
  while (ctas < 8 && a.max_rows > ctas * kThreads) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = ctas;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  count_launch();
  return cudaLaunchKernelEx(&cfg, a.max_rows <= ctas * kThreads ? k_plan_pages<1> : k_plan_pages<4>, a, ctas);
}

// ---------------------------------------------------------------------------
// rotation
// ---------------------------------------------------------------------------
namespace rot {

// 16 elements of a head: in the rotated part of a half layout, 8 of each half,
// so that a thread holds both numbers of its pairs; else 16 in a row.
template <typename T>
struct Unit {
  static constexpr int W = 16 / sizeof(T);  // elements of a 16-byte load
  static constexpr int N = 16 / W;          // loads
};

template <typename T>
__device__ __forceinline__ void load16(const T* p, int second, float* v) {
  constexpr int W = Unit<T>::W, N = Unit<T>::N;
#pragma unroll
  for (int i = 0; i < N; ++i) Chunk<T>::load(p + (i < N / 2 ? i * W : second + (i - N / 2) * W), v + i * W);
}
__device__ __forceinline__ void store_chunk(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store_chunk(__nv_bfloat16* p, const float* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(tc::pack_bf16(v[0], v[1]), tc::pack_bf16(v[2], v[3]), tc::pack_bf16(v[4], v[5]),
                                            tc::pack_bf16(v[6], v[7]));
}
template <typename T>
__device__ __forceinline__ void store16(T* p, int second, const float* v) {
  constexpr int W = Unit<T>::W, N = Unit<T>::N;
#pragma unroll
  for (int i = 0; i < N; ++i) store_chunk(p + (i < N / 2 ? i * W : second + (i - N / 2) * W), v + i * W);
}

// A warp takes heads_per_warp heads of a row; G lanes take a head, 16 elements
// each.  A lane's eight angles are the same for every head, so their sines and
// cosines are computed once: pos * step wraps around at whole turns, which
// leaves the exact fraction, whatever the position.  A row's angles, the
// norm's sums and loads come one after the other in a warp, of which 16 fit an SM (120 registers); that
// bounds it (8192 rows of 40 heads of 128 with norm, bf16 40 us, 4.2 of 6.7 TB/s, fp32 56, 6.0; four heads of
// a lane on their way 38 us in bf16, but 500 such rows without norm 5.8 for 5.1).
template <typename T, int HD>
__global__ void __launch_bounds__(128) k_rotate(const __grid_constant__ cdb_rotate_args a, int heads_per_warp, int parts) {
  constexpr int G = HD == 96 ? 8 : HD / 16;  // lanes of a head; of 96 elements, six lanes work
  constexpr int A = 32 / G;                  // heads of a warp at a time
  const int lane = threadIdx.x & 31, u = lane % G;
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const long long row = w / parts;
  pdl_wait();
  pdl_trigger();
  if (row >= a.rows) return;
  const int pos = a.pos[row];
  if (pos < 0) return;
  const int heads = a.n_heads + a.n_kv_heads;
  const int h0 = (int)(w % parts) * heads_per_warp, h1 = min(heads, h0 + heads_per_warp);
  const bool in = u * 16 < HD;
  const int rd = a.rot_dim, units = rd / 16;
  const bool turns = u < units, halves = turns && !a.interleaved;
  const int first = halves ? 8 * u : 16 * u;           // of the unit's first 8 elements
  const int second = halves ? rd / 2 : 8;              // from those to the other 8
  float c[8], s[8];
  if (turns) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint64_t phase = a.steps[8 * u + j] * (uint64_t)(uint32_t)pos;
      // Whole quarters of a turn are taken off first: what is left, at most 1/4 half turn either way, rounds to fp32 by
      // 2^-27 half turns at most (of a whole half turn 2^-25).
      const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
      float sr, cr;
      sincospif(__ll2float_rn((long long)(phase - ((uint64_t)quarter << 62))) * 0x1p-63f, &sr, &cr);
      const float sq = quarter & 1 ? cr : sr, cq = quarter & 1 ? sr : cr;
      s[j] = (quarter & 2 ? -sq : sq) * a.factor, c[j] = ((quarter + 1) & 2 ? -cq : cq) * a.factor;
    }
  }
  float gq[16], gk[16];
  const bool norm = a.q_gain != nullptr;
  if (norm && in) {
    load16(a.q_gain + first, second, gq);
    load16(a.k_gain + first, second, gk);
  }
  const T* x = static_cast<const T*>(a.x) + row * a.ldx + first;
  T* y = static_cast<T*>(a.out) + row * a.ldo + first;
  constexpr int B = 2;  // heads in flight
  for (int h = h0 + lane / G; h - lane / G < h1; h += A * B) {
    float v[B][16];
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (in && h + b * A < h1) load16(x + (size_t)(h + b * A) * HD, second, v[b]);
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int hb = h + b * A;
      const bool on = in && hb < h1;
      if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = on ? fmaf(v[b][e], v[b][e], ss) : 0.f;
#pragma unroll
        for (int o = 1; o < G; o *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(ss / HD + a.eps);
#pragma unroll
        for (int e = 0; e < 16; ++e) v[b][e] = v[b][e] * r * (hb < a.n_heads ? gq[e] : gk[e]);
      }
      if (halves) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float p = v[b][j], q = v[b][8 + j];
          v[b][j] = p * c[j] - q * s[j];
          v[b][8 + j] = q * c[j] + p * s[j];
        }
      } else if (turns) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float p = v[b][2 * j], q = v[b][2 * j + 1];
          v[b][2 * j] = p * c[j] - q * s[j];
          v[b][2 * j + 1] = q * c[j] + p * s[j];
        }
      }
      if (on) store16(y + (size_t)hb * HD, second, v[b]);
    }
  }
}

template <typename T, int HD>
cudaError_t launch(cudaStream_t s, const cdb_rotate_args& a) {
  constexpr int A = 32 / (HD == 96 ? 8 : HD / 16);
  // Few rows: a row's heads over several warps, so that no SM is without one.
  const int heads = a.n_heads + a.n_kv_heads;
  int parts = 1;
  while ((long long)a.rows * parts < 152 * 16 && (heads + parts - 1) / parts > A) parts *= 2;
  const int hpw = ((heads + parts - 1) / parts + A - 1) / A * A;
  parts = (heads + hpw - 1) / hpw;
  const long long warps = (long long)a.rows * parts;
  count_launch();
  return launch_pdl(k_rotate<T, HD>, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, s, a, hpw, parts);
}

template <typename T>
cudaError_t launch_as(cudaStream_t s, const cdb_rotate_args& a) {
  switch (a.head_dim) {
    case 32: return launch<T, 32>(s, a);
    case 64: return launch<T, 64>(s, a);
    case 96: return launch<T, 96>(s, a);
    case 128: return launch<T, 128>(s, a);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace rot

cudaError_t launch_rotate(cudaStream_t s, const cdb_rotate_args& a) {
  return a.dtype == CDB_FP32 ? rot::launch_as<float>(s, a) : rot::launch_as<__nv_bfloat16>(s, a);
}

// ---------------------------------------------------------------------------
// accepted drafts
// ---------------------------------------------------------------------------
namespace keep {

constexpr int kThreads = 256;

// A thread owns 16 bytes of a (slot, K or V, head) row, or a scale, and takes
// them along the path.  The path ascends, so what is overwritten was read before
// (entry k goes to k <= path[k], and no later entry comes from there): loads of
// several entries may run ahead of their stores.  16 paths of 96 slots from HBM: 14.3 us, half of
// the copy rate (64 registers: four CTAs of an SM at a time, each with a chain of lookups before its first load);
// one path of 4 slots: 1.6 us, the latency of those, one load and one store.
__global__ void __launch_bounds__(kThreads) k_keep_path(const __grid_constant__ cdb_keep_path_args a) {
  __shared__ long long from[CDB_DRAFT_MAX], to[CDB_DRAFT_MAX];  // 16 * block + offset, past 32 bits in large pools
  __shared__ int moves;
  const cdb_paged_cache& c = a.cache;
  const int i = blockIdx.y, tid = threadIdx.x;
  if (tid == 0) moves = 0;
  pdl_wait();
  pdl_trigger();
  const int seq = a.seq ? a.seq[i] : i, n = a.keep[i];
  const long long base = a.base[i];
  if (seq < 0) return;
  const int32_t* path = a.path + i * a.ld_path;
  int bad = (seq >= c.n_seqs || n < 0 || n > a.max_path || base < 0) ? CDB_OPS_BAD_ROW : 0;
  __syncthreads();
  if (!bad && tid < n) {
    const int p = path[tid];
    const long long src = base + p, dst = base + tid;
    if (p < tid || (tid > 0 && path[tid - 1] >= p) || src >= (long long)c.max_blocks * 16) {
      bad = CDB_OPS_BAD_ROW;
    } else if (p > tid) {
      const int32_t* t = c.block_table + (size_t)seq * c.max_blocks;
      const int bs = t[src / 16], bd = t[dst / 16];
      if (bs < 0 || bs >= c.kv_blocks || bd < 0 || bd >= c.kv_blocks) bad = CDB_OPS_BAD_BLOCK;
      from[tid] = bs * 16ll + src % 16;
      to[tid] = bd * 16ll + dst % 16;
      atomicMin(&moves, tid - CDB_DRAFT_MAX);  // entries before the first that moves are in place
    }
  }
  bad = __syncthreads_or(bad & CDB_OPS_BAD_ROW) ? CDB_OPS_BAD_ROW : __syncthreads_or(bad) ? CDB_OPS_BAD_BLOCK : 0;
  if (bad) {
    if (tid == 0 && blockIdx.x == 0) report(a.status, bad);
    return;
  }
  const int k0 = moves == 0 ? n : moves + CDB_DRAFT_MAX;  // strictly ascending: all behind the first move too
  const int rb = c.head_dim * (c.dtype == CDB_BF16 ? 2 : 1), vec = rb / 16;  // bytes and pieces of a position of a head
  const long long heads = (long long)c.n_kv_slots * 2 * c.n_kv_heads;        // (slot, K or V, head)
  const long long pieces = heads * vec, all = pieces + (c.dtype == CDB_E4M3 ? heads : 0);
  uint4* pool = static_cast<uint4*>(c.pool);
  constexpr int B = 8;
  for (long long p = (long long)blockIdx.x * kThreads + tid; p < all; p += (long long)gridDim.x * kThreads) {
    if (p < pieces) {
      const long long h = p / vec;
      const int piece = (int)(p - h * vec);
      auto at = [&](long long cell) { return (((cell >> 4) * heads + h) * 16 + (cell & 15)) * vec + piece; };
      for (int k = k0; k < n; k += B) {
        uint4 v[B];
#pragma unroll
        for (int e = 0; e < B; ++e)
          if (k + e < n) v[e] = pool[at(from[k + e])];
#pragma unroll
        for (int e = 0; e < B; ++e)
          if (k + e < n) pool[at(to[k + e])] = v[e];
      }
    } else {
      const long long h = p - pieces;
      auto at = [&](long long cell) { return ((cell >> 4) * heads + h) * 16 + (cell & 15); };
      for (int k = k0; k < n; k += B) {
        float v[B];
#pragma unroll
        for (int e = 0; e < B; ++e)
          if (k + e < n) v[e] = c.scales[at(from[k + e])];
#pragma unroll
        for (int e = 0; e < B; ++e)
          if (k + e < n) c.scales[at(to[k + e])] = v[e];
      }
    }
  }
}

}  // namespace keep

cudaError_t launch_keep_path(cudaStream_t s, const cdb_keep_path_args& a) {
  const cdb_paged_cache& c = a.cache;
  const long long heads = (long long)c.n_kv_slots * 2 * c.n_kv_heads;
  const long long pieces = heads * (c.head_dim * (c.dtype == CDB_BF16 ? 2 : 1) / 16 + (c.dtype == CDB_E4M3));
  // Eight CTAs for each SM, of which four fit at a time: a CTA's look at the path is shared by several pieces of its threads (16 paths of 96 slots,
  // from HBM: 18.5 us with a CTA for every 256 pieces, 14.3 so).
  const unsigned x = (unsigned)std::min((pieces + keep::kThreads - 1) / keep::kThreads, std::max(1ll, 152ll * 8 / a.requests));
  count_launch();
  return launch_pdl(keep::k_keep_path, dim3(x, a.requests), dim3(keep::kThreads), 0, s, a);
}

}  // namespace cdb
