// Attention of a batch over a prefix that all its rows share (the shared_len
// part of cdb_attention, include/cdb_ops.h), on the 5th-generation tensor
// cores: head_dim 64 or 128, bf16 or e4m3 cache.
//
// With one query row per sequence, the rows of the batch (times the query
// heads of one KV head) are the rows of a matrix product with the prefix's
// keys, so the prefix is read once per 128 such rows instead of once per row.
// What bounds it: the bytes of the prefix below some 250 query rows per KV
// head, beyond that the exponentials and the tensor cores together.
//
// One CTA per (KV head, tile of 128 query rows, chunk of keys).  The chunk is
// walked in blocks of 64 keys that go to two softmax groups in turn (even
// blocks, odd blocks), each with an output accumulator, a running maximum and
// a running sum of its own: a thread owns a whole row of a block, so no value
// crosses lanes or warps, and the tensor cores work on one group's block while
// the other group is in its exponentials.  The two are joined at the end.
//   warps 0-3, 4-7  softmax groups: thread t owns query row t (its TMEM lane);
//                   it reads its 64 scores, and writes the weights back over
//                   them as bf16 (rounding each weight by at most 2^-9 of it,
//                   less than the bf16 output's own rounding; the sum that
//                   normalises is of the fp32 weights): the weights are the A
//                   operand of the second product straight from TMEM;
//   warp 8          TMA producer (q tile, key blocks);
//   warp 9          MMA issuer: S = Q K^T (128 x 64), O += P V;
//   warps 10-13     e4m3 only: turn code blocks into bf16 K and V in the MMA's
//                   swizzled layout.  Codes are exact in bf16; a key's scale
//                   multiplies its fp32 score, a value's scale its weight
//                   before that is rounded, so e4m3 costs no further rounding.
// TMEM: two output accumulators of head_dim columns, two score buffers of 64
// columns per group.  V is an N-major B operand in its stored order.  Every
// mbarrier wait is bounded; on expiry the kernel reports CDB_OPS_TIMEOUT, lets
// its own copies and MMAs finish (bounded), frees TMEM and returns.
#include "../../include/cdb.h"
#include "cache_ops.h"
#include "common.cuh"
#include "kernels.cuh"
#include "tc.cuh"
#include "tmap.h"

#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace cdb {
namespace sp {

using namespace tc;

constexpr int kRows = 128;  // query rows of a tile
constexpr int kKeys = 64;   // keys of a block: four pages

template <int HD, bool Q8>
struct Geo {
  static_assert(HD == 64 || HD == 128, "head dim");
  static constexpr int NX = HD / 64;                  // 128-byte slices of a bf16 row
  static constexpr int QSLICE = kRows * 128;
  static constexpr int QBYTES = NX * QSLICE;
  static constexpr int KSLICE = kKeys * 128;
  static constexpr int KVB = NX * KSLICE;             // K (or V) of a block
  // K and V have rings of their own: K is given back as soon as its scores are
  // computed, two blocks before its V is used, so more blocks are in flight.
  static constexpr int KS = Q8 ? 3 : 5;
  static constexpr int VS = Q8 ? 4 : 6;
  static constexpr int RAWKV = kKeys * HD;            // codes of K (or V) of a block
  static constexpr int RAW = Q8 ? 2 * RAWKV + 2 * kKeys * 4 : 0;
  static constexpr int NR = Q8 ? 3 : 0;               // code blocks in flight
  static constexpr int OFF_K = QBYTES;
  static constexpr int OFF_V = OFF_K + KS * KVB;
  static constexpr int OFF_RAW = OFF_V + VS * KVB;
  static constexpr int OFF_SC = OFF_RAW + NR * RAW;   // e4m3: scales of the blocks in use, [VS][K, V][kKeys]
  static constexpr int OFF_XCH = OFF_SC + (Q8 ? VS * 2 * kKeys * 4 : 0);  // float2 [2][kRows]
  static constexpr int OFF_BAR = OFF_XCH + 2 * kRows * 8;
  static constexpr int NBAR = 2 + 2 * KS + 2 * VS + 4 + 4 + 2 + 2 * 3;
  static constexpr size_t SMEM = 1024 + OFF_BAR + NBAR * 8 + 16;
  static constexpr int THREADS = 320 + (Q8 ? 128 : 0);
  static constexpr int O_COL = 0;                     // [2][HD]
  static constexpr int S_COL = 2 * HD;                // [2 groups][2 buffers][64]
  static constexpr int TMEM_COLS = 512;
};

struct Args {
  cdb_attention_args a;
  int group;     // query heads per KV head
  int tile_rows; // batch rows of a tile (group * tile_rows <= 128)
  int chunk;     // keys of a CTA, a multiple of 64
  int parts;     // partials per (row, head); this kernel writes the first ones
  float* part_o;
  float2* part_ml;
};

template <int HD, bool Q8>
__global__ void __launch_bounds__(Geo<HD, Q8>::THREADS, 1)
    k_shared_prefix(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                    const __grid_constant__ Args A) {
  using G = Geo<HD, Q8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qs = smem;
  float2* xch = reinterpret_cast<float2*>(smem + G::OFF_XCH);
  uint64_t* qbar = reinterpret_cast<uint64_t*>(smem + G::OFF_BAR);
  uint64_t* done = qbar + 1;
  uint64_t* k_full = done + 1;
  uint64_t* k_empty = k_full + G::KS;
  uint64_t* v_full = k_empty + G::KS;
  uint64_t* v_empty = v_full + G::VS;
  uint64_t* s_full = v_empty + G::VS;   // [group][buffer]
  uint64_t* p_full = s_full + 4;        // [group][buffer]
  uint64_t* o_done = p_full + 4;        // [group]
  uint64_t* raw_full = o_done + 2;
  uint64_t* raw_empty = raw_full + 3;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(raw_empty + 3);

  const cdb_attention_args& a = A.a;
  const cdb_paged_cache& c = a.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kh = blockIdx.x, row0 = blockIdx.y * A.tile_rows, chunk = blockIdx.z;
  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmq) : "memory");
    if (!Q8) asm volatile("prefetch.tensormap [%0];" ::"l"(&tmk) : "memory");
    mbar_init(qbar, 1);
    mbar_init(done, 1);
    for (int s = 0; s < G::KS; ++s) {
      mbar_init(&k_full[s], Q8 ? 4 : 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < G::VS; ++s) {
      mbar_init(&v_full[s], Q8 ? 4 : 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
    }
    mbar_init(&o_done[0], 1);
    mbar_init(&o_done[1], 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(tmem_slot)),
                 "r"(G::TMEM_COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  const int k_lo = chunk * A.chunk, k_hi = min(a.shared_len, k_lo + A.chunk);
  const int nb = (k_hi - k_lo + kKeys - 1) / kKeys;  // >= 1
  const int npg = (k_hi - k_lo) / 16;

  if (warp == 8) {
    // ---------------- producer ----------------
    // The first sequence of the batch names the prefix's blocks.
    int base = -1;
    for (int r0 = 0; r0 < a.rows && base < 0; r0 += 32) {
      const int s = r0 + lane < a.rows ? a.seq[r0 + lane] : -1;
      const uint32_t has = __ballot_sync(0xffffffffu, s >= 0 && s < c.n_seqs);
      if (has) base = __shfl_sync(0xffffffffu, s, __ffs(has) - 1);
    }
    const int* bt = c.block_table + (size_t)max(base, 0) * c.max_blocks + k_lo / 16;
    uint64_t pol;  // the prefix is read again by the other tiles and by the next steps
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
    if (lane == 0) {
      mbar_arrive_tx(qbar, (uint32_t)(G::NX * A.group * A.tile_rows * 128));
      for (int x = 0; x < G::NX; ++x) tma_3d(su32(qs + x * G::QSLICE), &tmq, qbar, x * 64, kh * A.group, row0);
    }
    bool ok = true;
    int issued = 0;
    int blk_l = -1;
    for (int j = 0; j < nb; ++j) {
      if ((j & 7) == 0) {  // table entries of the next eight blocks, one per lane
        const int pg = 4 * j + lane;
        blk_l = base >= 0 && pg < npg ? bt[pg] : -1;
        if (base >= 0 && pg < npg && (blk_l < 0 || blk_l >= c.kv_blocks)) report(a.status, CDB_OPS_BAD_BLOCK), blk_l = -1;
      }
      const int blk = __shfl_sync(0xffffffffu, blk_l, ((j & 7) * 4 + lane) & 31);
      const bool mine = lane < 4 && blk >= 0;
      const uint32_t n = (uint32_t)__popc(__ballot_sync(0xffffffffu, mine));
      const long long head = ((long long)blk * c.n_kv_slots + a.slot_base) * 2 * c.n_kv_heads + kh;
      if constexpr (Q8) {
        const int s = j % G::NR;
        if (j >= G::NR && !(ok = __all_sync(0xffffffffu, mbar_wait(&raw_empty[s], ((j / G::NR) - 1) & 1)))) break;
        if (lane == 0) mbar_arrive_tx(&raw_full[s], n * (2 * 16 * HD + 2 * 64));
        __syncwarp();
        if (mine) {
          const uint32_t st = su32(smem + G::OFF_RAW + (size_t)s * G::RAW);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const long long at = (head + kv * c.n_kv_heads) * 16;
            bulk_1d(st + kv * G::RAWKV + lane * 16 * HD, static_cast<const uint8_t*>(c.pool) + at * HD, 16 * HD, &raw_full[s]);
            bulk_1d(st + 2 * G::RAWKV + (kv * kKeys + lane * 16) * 4, c.scales + at, 64, &raw_full[s]);
          }
        }
      } else {
        const int sk = j % G::KS, sv = j % G::VS;
        const int y = (int)(head * 16);
        if (j >= G::KS && !(ok = __all_sync(0xffffffffu, mbar_wait(&k_empty[sk], ((j / G::KS) - 1) & 1)))) break;
        if (lane == 0) mbar_arrive_tx(&k_full[sk], n * (G::NX * 16 * 128));
        __syncwarp();
        if (mine)
          for (int x = 0; x < G::NX; ++x)
            tma_2d(su32(smem + G::OFF_K + sk * G::KVB) + x * G::KSLICE + lane * 16 * 128, &tmk, &k_full[sk], x * 128, y, pol);
        issued = 2 * j + 1;
        if (j >= G::VS && !(ok = __all_sync(0xffffffffu, mbar_wait(&v_empty[sv], ((j / G::VS) - 1) & 1)))) break;
        if (lane == 0) mbar_arrive_tx(&v_full[sv], n * (G::NX * 16 * 128));
        __syncwarp();
        if (mine)
          for (int x = 0; x < G::NX; ++x)
            tma_2d(su32(smem + G::OFF_V + sv * G::KVB) + x * G::KSLICE + lane * 16 * 128, &tmk, &v_full[sv], x * 128,
                   y + c.n_kv_heads * 16, pol);
      }
      issued = 2 * j + 2;
    }
    if (!ok && lane == 0) report(a.status, CDB_OPS_TIMEOUT);
    // Copies in flight land before the CTA may leave (at once when everything was used).
    mbar_wait(qbar, 0);
    const int nk = (issued + 1) / 2, nv = issued / 2;
    if constexpr (Q8) {
      for (int j = max(0, nv - G::NR); j < nv; ++j) mbar_wait(&raw_full[j % G::NR], (j / G::NR) & 1);
    } else {
      for (int j = max(0, nk - G::KS); j < nk; ++j) mbar_wait(&k_full[j % G::KS], (j / G::KS) & 1);
      for (int j = max(0, nv - G::VS); j < nv; ++j) mbar_wait(&v_full[j % G::VS], (j / G::VS) & 1);
    }
  } else if (warp == 9) {
    // ---------------- MMA issuer ----------------
    if (lane == 0) {
      constexpr uint32_t idS = idesc_bf16(kRows, kKeys, false), idO = idesc_bf16(kRows, HD, true);
      const uint32_t qa = su32(qs);
      bool ok = mbar_wait(qbar, 0);
      auto scores = [&](int i) -> bool {  // S of block i: group i & 1, buffer (i >> 1) & 1
        const int s = i % G::KS, g = i & 1, n = i >> 1;
        if (!mbar_wait(&k_full[s], (i / G::KS) & 1)) return false;
        // The buffer held the weights of the group's block n - 2.
        if (n >= 2 && !mbar_wait(&o_done[g], (n - 2) & 1)) return false;
        fence_after();
        const uint32_t kb = su32(smem + G::OFF_K + s * G::KVB);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          mma_ss(tmem + G::S_COL + (g * 2 + (n & 1)) * kKeys, desc_k(qa + (kk / 4) * G::QSLICE + (kk % 4) * 32),
                 desc_k(kb + (kk / 4) * G::KSLICE + (kk % 4) * 32), idS, kk > 0 ? 1u : 0u);
        commit(&s_full[g * 2 + (n & 1)]);
        commit(&k_empty[s]);
        return true;
      };
      if (ok) ok = scores(0);
      if (ok && nb > 1) ok = scores(1);
      for (int i = 0; ok && i < nb; ++i) {
        if (i + 2 < nb && !(ok = scores(i + 2))) break;
        const int s = i % G::VS, g = i & 1, n = i >> 1;
        if (!(ok = mbar_wait(&v_full[s], (i / G::VS) & 1))) break;
        if (!(ok = mbar_wait(&p_full[g * 2 + (n & 1)], (n >> 1) & 1))) break;
        fence_after();
        const uint32_t vb = su32(smem + G::OFF_V + s * G::KVB);
        const int steps = min(4, npg - 4 * i);  // pages behind the chunk were not copied
        for (int kk = 0; kk < steps; ++kk)
          mma_ts(tmem + G::O_COL + g * HD, tmem + G::S_COL + (g * 2 + (n & 1)) * kKeys + kk * 8,
                 desc_mn(vb + kk * 2048, G::KSLICE), idO, (n > 0 || kk > 0) ? 1u : 0u);
        commit(&o_done[g]);
        commit(&v_empty[s]);
      }
      if (!ok) report(a.status, CDB_OPS_TIMEOUT);
      commit(done);  // every MMA issued above completes before TMEM is released
      mbar_wait(done, 0);
    }
  } else if (warp >= 10) {
    // ---------------- code converters (e4m3) ----------------
    if constexpr (Q8) {
      const int tid = threadIdx.x - 320;
      bool ok = true;
      for (int j = 0; j < nb; ++j) {
        const int sk = j % G::KS, sv = j % G::VS, r = j % G::NR;
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&raw_full[r], (j / G::NR) & 1)))) break;
        const uint8_t* raw = smem + G::OFF_RAW + (size_t)r * G::RAW;
        constexpr int C = HD / 16;  // 16-code pieces of a key row
        auto turn = [&](const uint8_t* src, uint32_t dst) {
#pragma unroll 4
          for (int u = tid; u < kKeys * C; u += 128) {
            const int key = u / C, p = u % C;
            const uint4 w = *reinterpret_cast<const uint4*>(src + key * HD + p * 16);
            uint32_t o[8];
            const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 x = widen2(in[e]), y = widen2(in[e] >> 16);
              o[2 * e] = pack_bf16(x.x, x.y);
              o[2 * e + 1] = pack_bf16(y.x, y.y);
            }
            const uint32_t line = dst + (p / 4) * G::KSLICE + key * 128;
            const int c0 = (p % 4) * 2;
            st_shared_v4(line + ((c0 ^ (key & 7)) << 4), o[0], o[1], o[2], o[3]);
            st_shared_v4(line + (((c0 + 1) ^ (key & 7)) << 4), o[4], o[5], o[6], o[7]);
          }
        };
        if (j >= G::KS && !(ok = __all_sync(0xffffffffu, mbar_wait(&k_empty[sk], ((j / G::KS) - 1) & 1)))) break;
        turn(raw, su32(smem + G::OFF_K + sk * G::KVB));
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_full[sk]);
        if (j >= G::VS && !(ok = __all_sync(0xffffffffu, mbar_wait(&v_empty[sv], ((j / G::VS) - 1) & 1)))) break;
        // The scales move along: the code block is given back before the softmax group reads them.
        reinterpret_cast<float*>(smem + G::OFF_SC)[sv * 2 * kKeys + tid] = reinterpret_cast<const float*>(raw + 2 * G::RAWKV)[tid];
        turn(raw + G::RAWKV, su32(smem + G::OFF_V + sv * G::KVB));
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&v_full[sv]);
          mbar_arrive(&raw_empty[r]);
        }
      }
      if (!ok && lane == 0) report(a.status, CDB_OPS_TIMEOUT);
    }
  } else {
    // ---------------- softmax groups ----------------
    const int q4 = warp & 3, g = warp >> 2;
    const int r = q4 * 32 + lane;
    const int br = row0 + r / A.group;  // batch row of this tile row
    const bool in = r < A.group * A.tile_rows && br < a.rows;
    const int seq = in ? a.seq[br] : -1, pos = in ? a.pos[br] : -1;
    const bool live = in && seq >= 0 && seq < c.n_seqs && pos < a.max_ctx;
    const int lim = min(pos, k_hi - 1) - k_lo;  // last key of this row, from the chunk's first
    // Scores in the log2 domain; a negative factor turns the scores around first, so that the
    // maximum can be taken before the factor is applied.
    const bool turn_round = a.scale < 0.f;
    const float scale = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-37f);  // not 0: a masked score stays -inf
    constexpr float kTau = 8.f;  // rescale O only when the row maximum grows by more than 2^8
    const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
    const uint32_t to = trow + G::O_COL + g * HD;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    int n = 0;  // blocks of this group so far
    for (int i = g; i < nb; i += 2, ++n) {
      const int b = g * 2 + (n & 1);
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&s_full[b], (n >> 1) & 1)))) break;
      fence_after();
      const uint32_t ts = trow + G::S_COL + b * kKeys;
      float sv[64];
      tmem_ld32(ts, sv);
      tmem_ld32(ts + 32, sv + 32);
      if (turn_round) {
#pragma unroll
        for (int k = 0; k < 64; ++k) sv[k] = -sv[k];
      }
      const float4* ks = nullptr;  // scales of the block's keys, then of its values
      if constexpr (Q8) {
        const int st = i % G::VS;
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&v_full[st], (i / G::VS) & 1)))) break;
        ks = reinterpret_cast<const float4*>(smem + G::OFF_SC + st * 2 * kKeys * 4);
#pragma unroll
        for (int k = 0; k < kKeys / 4; ++k) {
          const float4 f = ks[k];
          sv[4 * k] *= f.x, sv[4 * k + 1] *= f.y, sv[4 * k + 2] *= f.z, sv[4 * k + 3] *= f.w;
        }
      }
      const int left = lim - i * kKeys;  // keys 0..left of the block are this row's
      if (!__all_sync(0xffffffffu, left >= kKeys - 1)) {
#pragma unroll
        for (int k = 0; k < 64; ++k) sv[k] = k <= left ? sv[k] : -INFINITY;
      }
      float x4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int k = 0; k < 64; k += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) x4[e] = max3(x4[e], sv[k + 2 * e], sv[k + 2 * e + 1]);
      const float mx = fmaxf(fmaxf(x4[0], x4[1]), fmaxf(x4[2], x4[3])) * scale;
      const float mnew = mx > m + kTau ? mx : m;
      if (n > 0 && __any_sync(0xffffffffu, mnew != m)) {
        // O holds the group's earlier blocks against the old maximum.
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&o_done[g], (n - 1) & 1)))) break;
        fence_after();
        const float f = m == -INFINITY ? 0.f : ex2(m - mnew);
#pragma unroll 1
        for (int c0 = 0; c0 < HD; c0 += 32) {
          float v[32];
          tmem_ld32(to + c0, v);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] *= f;
          tmem_st32(to + c0, reinterpret_cast<const uint32_t*>(v));
        }
        l *= f;
      }
      m = mnew;
      const float mm = m == -INFINITY ? 0.f : m;
      uint32_t p[32];
      const uint64_t s2 = pair(scale, scale), m2 = pair(-mm, -mm);
      uint64_t l2[2] = {pair(l, 0.f), pair(0.f, 0.f)};
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        float x0, x1, x2, x3;
        unpair(fma2(pair(sv[2 * e], sv[2 * e + 1]), s2, m2), x0, x1);
        unpair(fma2(pair(sv[2 * e + 2], sv[2 * e + 3]), s2, m2), x2, x3);
        x0 = ex2(x0), x1 = ex2(x1), x2 = ex2(x2), x3 = ex2(x3);
        l2[0] = add2(l2[0], pair(x0, x1));
        l2[1] = add2(l2[1], pair(x2, x3));
        if constexpr (Q8) {
          const float4 f = ks[kKeys / 4 + e / 2];
          // No weight times a scale that may be NaN (pages behind the chunk).
          p[e] = pack_bf16(x0 > 0.f ? x0 * f.x : 0.f, x1 > 0.f ? x1 * f.y : 0.f);
          p[e + 1] = pack_bf16(x2 > 0.f ? x2 * f.z : 0.f, x3 > 0.f ? x3 * f.w : 0.f);
        } else {
          p[e] = pack_bf16(x0, x1);
          p[e + 1] = pack_bf16(x2, x3);
        }
      }
      float la, lb, lc, ld;
      unpair(l2[0], la, lb);
      unpair(l2[1], lc, ld);
      l = (la + lb) + (lc + ld);
      tmem_st32(ts, p);
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[b]);
    }
    if (ok && n > 0) ok = __all_sync(0xffffffffu, mbar_wait(&o_done[g], (n - 1) & 1));
    fence_after();
    xch[g * kRows + r] = make_float2(m, l);
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (!ok) {
      if (lane == 0) report(a.status, CDB_OPS_TIMEOUT);
    } else {
      // Join the groups; warps of group g write columns g HD/2 .. of the partial.
      const float2 e0 = xch[r], e1 = xch[kRows + r];
      const float mj = fmaxf(e0.x, e1.x);
      const float f0 = e0.x == -INFINITY ? 0.f : ex2(e0.x - mj), f1 = e1.x == -INFINITY ? 0.f : ex2(e1.x - mj);
      const int h = kh * A.group + r % A.group;
      const size_t pi = ((size_t)br * a.n_heads + h) * A.parts + chunk;
      float* po = A.part_o + pi * HD + g * (HD / 2);
      const uint32_t t0 = trow + G::O_COL + g * (HD / 2);
#pragma unroll 1
      for (int c0 = 0; c0 < HD / 2; c0 += 32) {
        float v[32], w[32];
        tmem_ld32(t0 + c0, v);
        if (nb > 1) {
          tmem_ld32(t0 + HD + c0, w);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = v[e] * f0 + w[e] * f1;
        }
        if (live) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4*>(po + c0 + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
      }
      // A single block leaves group 1 without a state: f0 is 1 (or the row has no key at all).
      if (live && g == 0) A.part_ml[pi] = make_float2(mj, e0.y * f0 + e1.y * f1);
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 9) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(G::TMEM_COLS));
  }
}

template <int HD, bool Q8>
cudaError_t launch(cudaStream_t s, const Args& A, int chunks) {
  using G = Geo<HD, Q8>;
  const cdb_attention_args& a = A.a;
  const cdb_paged_cache& c = a.cache;
  CUtensorMap tq, tk = {};
  if (!tmap_bf16_3d(&tq, a.q, HD, a.n_heads, a.rows, (uint64_t)HD * 2, (uint64_t)a.ldq * 2, 64, A.group, A.tile_rows))
    return cudaErrorInvalidValue;
  const uint64_t rows = (uint64_t)c.kv_blocks * c.n_kv_slots * 2 * c.n_kv_heads * 16;
  if (!Q8 && !tmap_u8_2d(&tk, c.pool, HD * 2, rows, HD * 2, 128, 16, 128)) return cudaErrorInvalidValue;
  static bool set[kMaxDevices] = {};
  const int dev = current_device();
  if (!set[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(k_shared_prefix<HD, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)G::SMEM);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  const int tiles = (a.rows + A.tile_rows - 1) / A.tile_rows;
  count_launch();
  return launch_pdl(k_shared_prefix<HD, Q8>, dim3(c.n_kv_heads, tiles, chunks), dim3(G::THREADS), G::SMEM, s, tq, tk, A);
}

}  // namespace sp

cudaError_t launch_shared_prefix(cudaStream_t s, const cdb_attention_args& a, const SharedPlan& p, int parts, float* part_o,
                                 float2* part_ml) {
  sp::Args A;
  A.a = a;
  A.group = a.n_heads / a.cache.n_kv_heads;
  A.tile_rows = p.tile_rows;
  A.chunk = p.chunk;
  A.parts = parts;
  A.part_o = part_o;
  A.part_ml = part_ml;
  const bool q8 = a.cache.dtype == CDB_E4M3;
  if (a.cache.head_dim == 64) return q8 ? sp::launch<64, true>(s, A, p.chunks) : sp::launch<64, false>(s, A, p.chunks);
  return q8 ? sp::launch<128, true>(s, A, p.chunks) : sp::launch<128, false>(s, A, p.chunks);
}

}  // namespace cdb
