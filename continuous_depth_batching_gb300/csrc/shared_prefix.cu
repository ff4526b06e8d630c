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
//                   them in 16 bits: the weights are the A operand of the
//                   second product straight from TMEM.  bf16 weights are two
//                   numbers, what the first one leaves in the second, which
//                   take the space of the 64 scores and a product each: within
//                   2^-17, as in the kernel for a row's own keys (256 rows x
//                   32/8 heads behind 16384 tokens: 117 us, 112 with one; 8
//                   rows behind 512: 10.1 and 9.4; an output's error then is
//                   its own rounding's alone);
//   warps 8, 11     TMA producers: q tile and K blocks, V blocks.  A copy takes
//                   its warp some 70 cycles to issue, so a page is one copy: a
//                   4-dimensional box lays its 128-byte slices out as
//                   [8 keys][slice][key][128 bytes], which both operands read;
//   warp 9          issues S = Q K^T (128 x 64), up to three blocks ahead, with q
//                   from TMEM too (the softmax groups put it there): shared
//                   memory has to feed K and V only, 64 KB a block with the
//                   copies, where q would add 32;
//   warp 10         issues O += P V, with a bf16 cache for both parts of P;
//   warps 12-15     e4m3 only: widen code blocks to fp16 in the MMA's swizzled
//                   layout (exactly; one conversion per two codes, where bf16
//                   would take four instructions).  A key's scale multiplies
//                   its fp32 score, a value's scale its weight; weights are
//                   relative to the largest weight times scale of their row,
//                   as in k_decode, and one fp16 number (within 2^-11, or
//                   2^-33 of that largest one); q becomes
//                   fp16, each row divided by a power of two.  (Values scaled by
//                   the converters instead, rounded to fp16: 168 us where this
//                   took 125, 256 rows x 32/8 heads behind 16384 tokens: the
//                   converters then hold the others up.)
// Waits and issues of one block cost a warp some 500 cycles (a commit about
// 140, a wait 100), as much as the products themselves: hence two issuing warps,
// one commit per product, and pairs of barriers that two lanes wait for at once.
// TMEM: two output accumulators of head_dim columns, q in head_dim / 2, three
// score buffers of 64 columns (all 512 with head_dim 128).  V is an N-major B operand in its stored order.  Every
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
  static constexpr int OCT = NX * 1024;               // 8 keys of a block, slice by slice
  static constexpr int PAGE = 2 * OCT;
  static constexpr int KVB = 4 * PAGE;                // K (or V) of a block
  // K and V have rings of their own: K is given back as soon as its scores are
  // computed, two blocks before its V is used, so more blocks are in flight.
  static constexpr int KS = Q8 ? 3 : 5;
  static constexpr int VS = Q8 ? 4 : 6;
  static constexpr int RAWKV = kKeys * HD;            // codes of K (or V) of a block
  static constexpr int RAW = Q8 ? 2 * RAWKV + 2 * kKeys * 4 : 0;
  static constexpr int NR = Q8 ? 4 : 0;               // code blocks in flight
  static constexpr int OFF_K = QBYTES;
  static constexpr int OFF_V = OFF_K + KS * KVB;
  static constexpr int OFF_RAW = OFF_V + VS * KVB;
  static constexpr int SCN = 3 * kKeys + 4;
  static constexpr int OFF_SC = OFF_RAW + NR * RAW;   // e4m3: [VS] scales of K, of V, the latter's logarithms, two maxima of those
  static constexpr int OFF_XCH = OFF_SC + (Q8 ? VS * SCN * 4 : 0);  // float2 [2][kRows]
  static constexpr int OFF_BAR = OFF_XCH + 2 * kRows * 8;
  static constexpr int NBAR = 4 + 2 * KS + 2 * VS + 3 + 2 * 4;
  static constexpr size_t SMEM = 1024 + OFF_BAR + NBAR * 8 + 16;
  static constexpr int THREADS = 384 + (Q8 ? 128 : 0);
  static constexpr int O_COL = 0;                     // [2][HD]
  static constexpr int Q_COL = 2 * HD;                // head_dim / 2, two 16-bit elements per column
  static constexpr int S_COL = Q_COL + HD / 2;        // [3][64]: block i's scores, then weights, in buffer i % 3
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

// The first sequence of the batch, which names the prefix's blocks (-1: none).
__device__ __forceinline__ int first_sequence(const cdb_attention_args& a) {
  const int lane = threadIdx.x & 31;
  int base = -1;
  for (int r0 = 0; r0 < a.rows && base < 0; r0 += 32) {
    const int s = r0 + lane < a.rows ? a.seq[r0 + lane] : -1;
    const uint32_t has = __ballot_sync(0xffffffffu, s >= 0 && s < a.cache.n_seqs);
    if (has) base = __shfl_sync(0xffffffffu, s, __ffs(has) - 1);
  }
  return base;
}

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
  uint64_t* q_ready = qbar + 1;         // q is in TMEM
  uint64_t* done = q_ready + 1;         // [2]: both issuing warps' last MMAs
  uint64_t* k_full = done + 2;
  uint64_t* s_full = k_full + G::KS;    // scores of the block in this K slot are complete: the slot is free
  uint64_t* v_full = s_full + G::KS;
  uint64_t* o_done = v_full + G::VS;    // the product with the V slot is complete: slot and weights are free
  uint64_t* p_full = o_done + G::VS;    // the weights in the score buffer are complete
  uint64_t* raw_full = p_full + 3;
  uint64_t* raw_empty = raw_full + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(raw_empty + 4);

  const cdb_attention_args& a = A.a;
  const cdb_paged_cache& c = a.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kh = blockIdx.x, row0 = blockIdx.y * A.tile_rows, chunk = blockIdx.z;
  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmq) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmk) : "memory");
    mbar_init(qbar, 1);
    mbar_init(q_ready, 8);
    mbar_init(&done[0], 1);
    mbar_init(&done[1], 1);
    for (int s = 0; s < G::KS; ++s) {
      mbar_init(&k_full[s], Q8 ? 2 : 1);
      mbar_init(&s_full[s], 1);
    }
    for (int s = 0; s < G::VS; ++s) {
      mbar_init(&v_full[s], Q8 ? 2 : 1);
      mbar_init(&o_done[s], 1);
    }
    for (int i = 0; i < 3; ++i) mbar_init(&p_full[i], 4);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&raw_full[i], 2);
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
  pdl_trigger();  // no wait yet: see the end
  const int k_lo = chunk * A.chunk, k_hi = min(a.shared_len, k_lo + A.chunk);
  const int nb = (k_hi - k_lo + kKeys - 1) / kKeys;  // >= 1
  const int npg = (k_hi - k_lo) / 16;

  // e4m3: registers from the other warpgroups to the softmax groups (128 each at launch), which read the scales of
  // a block's keys before its scores and those of its values before they are wanted: read where they are used, one
  // read waits for another (256 rows x 32/8 heads behind 16384 tokens, few keys of their own: 125 us, 108 so; it is
  // 112 now, bf16 97).
  static_assert(!Q8 || (G::THREADS == 512 && 256 * 184 + 256 * 72 <= 512 * 128), "registers of the launch");
  if (warp >= 8) {
    if constexpr (Q8) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 8 || warp == 11) {
      // ---------------- producers ----------------
      constexpr int kPage = 16 * HD * (Q8 ? 1 : 2);  // bytes of a page of one head, K or V
      const int kv = warp == 8 ? 0 : 1;
      const int base = first_sequence(a);
      const int* bt = c.block_table + (size_t)max(base, 0) * c.max_blocks + k_lo / 16;
      uint64_t pol;  // the prefix is read again by the other tiles and by the next steps
      asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
      if (kv == 0 && elect_one()) {
        mbar_arrive_tx(qbar, (uint32_t)(G::NX * A.group * A.tile_rows * 128));
        for (int x = 0; x < G::NX; ++x) tma_3d(su32(qs + x * G::QSLICE), &tmq, qbar, x * 64, kh * A.group, row0);
      }
      __syncwarp();
      // The ring this warp fills: K or V slots, or its half of the code slots.
      const int slots = Q8 ? G::NR : kv ? G::VS : G::KS;
      uint64_t* full = Q8 ? raw_full : kv ? v_full : k_full;
      uint64_t* empty = Q8 ? raw_empty : kv ? o_done : s_full;
      const uint32_t ring = su32(smem + (Q8 ? G::OFF_RAW + kv * G::RAWKV : kv ? G::OFF_V : G::OFF_K));
      bool ok = true;
      int issued = 0, blk_l = -1, s = 0;
      uint32_t parity = 1;  // of the slot's last use, from the second round on
      for (int j = 0; j < nb; ++j) {
        if ((j & 7) == 0) {  // table entries of the next eight blocks, one per lane
          const int pg = 4 * j + lane;
          blk_l = base >= 0 && pg < npg ? bt[pg] : -1;
          if (base >= 0 && pg < npg && (blk_l < 0 || blk_l >= c.kv_blocks)) report(a.status, CDB_OPS_BAD_BLOCK), blk_l = -1;
        }
        int blk[4], n = 0;
  #pragma unroll
        for (int i = 0; i < 4; ++i) {
          blk[i] = __shfl_sync(0xffffffffu, blk_l, (j & 7) * 4 + i);
          n += blk[i] >= 0;
        }
        if (j >= slots && !(ok = __all_sync(0xffffffffu, mbar_wait(&empty[s], parity)))) break;
        if (elect_one()) {
          mbar_arrive_tx(&full[s], (uint32_t)n * (kPage + (Q8 ? 64 : 0)));
  #pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (blk[i] < 0) continue;
            // Key rows before this head's page (V follows n_kv_heads pages after K).
            const long long at = ((((long long)blk[i] * c.n_kv_slots + a.slot_base) * 2 + kv) * c.n_kv_heads + kh) * 16;
            if constexpr (Q8) {
              tma_2d(ring + s * G::RAW + i * kPage, &tmk, &full[s], 0, (int)at, pol);
              bulk_1d(ring + s * G::RAW + (2 - kv) * G::RAWKV + (kv * kKeys + i * 16) * 4, c.scales + at, 64, &full[s]);
            } else
              tma_4d(ring + s * G::KVB + i * G::PAGE, &tmk, &full[s], 0, 0, 0, (int)(at / 8), pol);
          }
        }
        __syncwarp();
        issued = j + 1;
        if (++s == slots) s = 0, parity ^= 1;
      }
      if (!ok && lane == 0) report(a.status, CDB_OPS_TIMEOUT);
      // Copies in flight land before the CTA may leave (at once when everything was used).
      if (kv == 0) mbar_wait(qbar, 0);
      for (int j = max(0, issued - slots); j < issued; ++j) mbar_wait(&full[j % slots], (j / slots) & 1);
    } else if (warp == 9) {
      // ---------------- scores ----------------
      constexpr uint32_t id = idesc_16(!Q8, kRows, kKeys, false);
      const uint64_t kd = desc_k(su32(smem + G::OFF_K), G::OCT);  // addresses in 16-byte units
      bool ok = __all_sync(0xffffffffu, mbar_wait(q_ready, 0));
      for (int i = 0; ok && i < nb; ++i) {
        const int s = i % G::KS;
        // Lane 1 waits for the product with the weights that the buffer held, block i - 3's; the others for K.
        uint64_t* bar = &k_full[s];
        uint32_t parity = (i / G::KS) & 1;
        if (lane == 1 && i >= 3) bar = &o_done[(i - 3) % G::VS], parity = ((i - 3) / G::VS) & 1;
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar, parity)))) break;
        fence_after();
        const uint64_t kb = kd + (uint32_t)(s * (G::KVB / 16));
        const uint32_t d = tmem + G::S_COL + (i % 3) * kKeys;
        if (elect_one()) {
  #pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            mma_ts(d, tmem + G::Q_COL + kk * 8, kb + ((kk / 4) * 1024 + (kk % 4) * 32) / 16, id, kk > 0 ? 1u : 0u);
          commit(&s_full[s]);
        }
        __syncwarp();
      }
      if (!ok && lane == 0) report(a.status, CDB_OPS_TIMEOUT);
      if (elect_one()) commit(&done[0]);  // every MMA issued above completes before TMEM is released
      __syncwarp();
      mbar_wait(&done[0], 0);
    } else if (warp == 10) {
      // ---------------- weights times values ----------------
      constexpr uint32_t id = idesc_16(!Q8, kRows, HD, true);
      const uint64_t vd = desc_mn(su32(smem + G::OFF_V), 1024, G::OCT);
      bool ok = true;
      for (int i = 0; i < nb; ++i) {
        const int s = i % G::VS, g = i & 1, n = i >> 1;
        const bool other = lane == 1;  // lane 1 waits for V, the others for the weights
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(other ? &v_full[s] : &p_full[i % 3], (other ? i / G::VS : i / 3) & 1)))) break;
        fence_after();
        const uint64_t vb = vd + (uint32_t)(s * (G::KVB / 16));
        const uint32_t d = tmem + G::O_COL + g * HD, p = tmem + G::S_COL + (i % 3) * kKeys;
        const int steps = npg - 4 * i;  // pages behind the chunk were not copied
        if (elect_one()) {
  #pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            if (kk < steps) mma_ts(d, p + kk * 8, vb + (kk * G::PAGE) / 16, id, (n > 0 || kk > 0) ? 1u : 0u);
          if constexpr (!Q8) {
  #pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              if (kk < steps) mma_ts(d, p + 32 + kk * 8, vb + (kk * G::PAGE) / 16, id, 1u);
          }
          commit(&o_done[s]);
        }
        __syncwarp();
      }
      if (!ok && lane == 0) report(a.status, CDB_OPS_TIMEOUT);
      if (elect_one()) commit(&done[1]);
      __syncwarp();
      mbar_wait(&done[1], 0);
    } else if (warp >= 12) {
      // ---------------- code converters (e4m3) ----------------
      if constexpr (Q8) {
        // Two warps for K, two for V.  8 codes to 16 bytes at a time: the lanes of a half warp (hd 64: a quarter)
        // take a key's row, so loads and stores of a warp meet every bank once, and the addresses of one thread
        // are a constant apart.
        const int kv = warp >= 14 ? 1 : 0, tid = (threadIdx.x - 384) & 63;
        constexpr int C = HD / 8, KI = 64 / C;  // 8-code pieces of a row, rows of one step
        const int key = tid / C, p = tid % C;
        const int slots = kv ? G::VS : G::KS;
        uint64_t* full = kv ? v_full : k_full;
        uint64_t* empty = kv ? o_done : s_full;
        const uint32_t to = su32(smem + (kv ? G::OFF_V : G::OFF_K)) + (p / 8) * 1024;
        bool ok = true;
        for (int j = 0; j < nb; ++j) {
          const int s = j % slots, r = j % G::NR;
          const bool other = lane == 1 && j >= slots;  // lane 1 waits for the slot, the others for the codes
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(other ? &empty[s] : &raw_full[r],
                                                       other ? ((j / slots) - 1) & 1 : (j / G::NR) & 1))))
            break;
          const uint8_t* raw = smem + G::OFF_RAW + (size_t)r * G::RAW;
          const uint8_t* src = raw + kv * G::RAWKV + key * HD + p * 8;
          uint2 w[kKeys / KI];
  #pragma unroll
          for (int u = 0; u < kKeys / KI; ++u) w[u] = *reinterpret_cast<const uint2*>(src + u * KI * HD);
          if (kv) {
            // The scales move along: the code block is given back before the softmax group reads them.
            float* sc = reinterpret_cast<float*>(smem + G::OFF_SC) + s * G::SCN;
            const float* f = reinterpret_cast<const float*>(raw + 2 * G::RAWKV);
            const float fv = f[kKeys + tid];
            sc[tid] = f[tid];
            sc[kKeys + tid] = fv;
            sc[2 * kKeys + tid] = __log2f(fabsf(fv));
            // The largest magnitude of the value scales that were copied, by halves: its logarithm, at least -82.
            const uint32_t fm = __reduce_max_sync(0xffffffffu, tid / 16 < npg - 4 * j ? __float_as_uint(fabsf(fv)) : 0u);
            if (lane == 0) sc[3 * kKeys + tid / 32] = fmaxf(__log2f(__uint_as_float(fm)), -82.f);
          }
  #pragma unroll
          for (int u = 0; u < kKeys / KI; ++u) {
            const int k = key + u * KI;
            st_shared_v4(to + s * G::KVB + (k / 8) * G::OCT + (k % 8) * 128 + (((p % 8) ^ (k % 8)) << 4), widen(w[u].x),
                         widen_hi(w[u].x), widen(w[u].y), widen_hi(w[u].y));
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&full[s]);
            mbar_arrive(&raw_empty[r]);
          }
        }
        if (!ok && lane == 0) report(a.status, CDB_OPS_TIMEOUT);
      }
    }
  } else {
    if constexpr (Q8) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    // ---------------- softmax groups ----------------
    const int q4 = warp & 3, g = warp >> 2;
    const int r = q4 * 32 + lane;
    const int br = row0 + r / A.group;  // batch row of this tile row
    const bool in = r < A.group * A.tile_rows && br < a.rows;
    const int seq = in ? a.seq[br] : -1, pos = in ? a.pos[br] : -1;
    const bool live = in && seq >= 0 && seq < c.n_seqs && pos < a.max_ctx;
    const int lim = min(max(pos, -1), k_hi - 1) - k_lo;  // last key of this row, from the chunk's first
    // Scores in the log2 domain; a negative factor turns the scores around first, so that the
    // maximum can be taken before the factor is applied.
    const bool turn_round = a.scale < 0.f;
    float scale = fabsf(a.scale) * 1.4426950408889634f;
    constexpr float kTau = 8.f;  // rescale O only when the row maximum grows by more than 2^8
    const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
    const uint32_t to = trow + G::O_COL + g * HD;
    // What O and l are relative to (log2; bf16: the row's maximum score, within 8; e4m3: its maximum of score +
    // log2(value scale), see k_decode), and the sum of the weights.
    float m = -INFINITY, l = 0.f;
    float up = 1.f;  // e4m3: what q was divided by
    bool ok = true;
    {
      // q to TMEM, row by row (two 16-bit elements per column): the groups take a 64-element slice each.
      ok = __all_sync(0xffffffffu, mbar_wait(qbar, 0));
      float down = 1.f;
      if constexpr (Q8) {
        float mx = 0.f;
#pragma unroll
        for (int x = 0; x < G::NX; ++x)
#pragma unroll
          for (int ch = 0; ch < 8; ++ch) {
            const uint4 w = *reinterpret_cast<const uint4*>(qs + x * G::QSLICE + r * 128 + ((ch ^ (r & 7)) << 4));
            const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mx = max3(mx, fabsf(__uint_as_float(v[e] << 16)), fabsf(__uint_as_float(v[e] & 0xFFFF0000u)));
          }
        // 2^-e and 2^e for mx = 2^e f; 1 for zero, tiny, infinite or NaN maxima.
        const uint32_t eb = __float_as_uint(mx) & 0x7F800000u;
        const bool norm = eb > 0x00800000u && eb < 0x7E000000u;
        down = norm ? __uint_as_float(0x7F000000u - eb) : 1.f;
        up = norm ? __uint_as_float(eb) : 1.f;
      }
      if (g < G::NX) {
        uint32_t h[32];
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          const uint4 w = *reinterpret_cast<const uint4*>(qs + g * G::QSLICE + r * 128 + ((ch ^ (r & 7)) << 4));
          const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            h[4 * ch + e] = Q8 ? pack_f16(__uint_as_float(v[e] << 16) * down, __uint_as_float(v[e] & 0xFFFF0000u) * down) : v[e];
        }
        tmem_st32(trow + G::Q_COL + g * 32, h);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
    }
    scale = fmaxf(scale * up, 1e-37f);  // not 0: a masked score stays -inf
    int n = 0;  // blocks of this group so far
    for (int i = g; ok && i < nb; i += 2, ++n) {
      const uint32_t ts = trow + G::S_COL + (i % 3) * kKeys;
      const int left = lim - i * kKeys;  // keys 0..left of the block are this row's
      float sv[64];
      uint32_t p[32];
      auto mask = [&] {
        if (!__all_sync(0xffffffffu, left >= kKeys - 1)) {
#pragma unroll
          for (int k = 0; k < 64; ++k) sv[k] = k <= left ? sv[k] : -INFINITY;
        }
      };
      auto greatest = [&] {
        float x4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 64; k += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) x4[e] = max3(x4[e], sv[k + 2 * e], sv[k + 2 * e + 1]);
        return fmaxf(fmaxf(x4[0], x4[1]), fmaxf(x4[2], x4[3])) * scale;
      };
      // Moves the row to the reference `to`; O holds the group's earlier blocks against the old one.
      auto move = [&](float to_m) {
        const float f = m == -INFINITY ? 0.f : ex2(m - to_m);
        l *= f;
        m = to_m;
        if (n == 0) return true;
        if (!__all_sync(0xffffffffu, mbar_wait(&o_done[(i - 2) % G::VS], ((i - 2) / G::VS) & 1))) return false;
        fence_after();
#pragma unroll 1
        for (int c0 = 0; c0 < HD; c0 += 32) {
          float v[32];
          tmem_ld32(to + c0, v);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] *= f;
          tmem_st32(to + c0, reinterpret_cast<const uint32_t*>(v));
        }
        return true;
      };
      if constexpr (Q8) {
        // The scales of the block's keys, which come with V, before its scores; those of its values below.
        float4 sf[16];
        const uint32_t scales = su32(smem + G::OFF_SC + (i % G::VS) * G::SCN * 4);
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&v_full[i % G::VS], (i / G::VS) & 1)))) break;
#pragma unroll
        for (int k = 0; k < 16; ++k) sf[k] = ld_shared_v4(scales + k * 16);
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&s_full[i % G::KS], (i / G::KS) & 1)))) break;
        fence_after();
        tmem_ld32(ts, sv);
        tmem_ld32(ts + 32, sv + 32);
        if (turn_round) {
#pragma unroll
          for (int k = 0; k < 64; ++k) sv[k] = -sv[k];
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float4 f = sf[k];
          unpair(mul2(pair(sv[4 * k], sv[4 * k + 1]), pair(f.x, f.y)), sv[4 * k], sv[4 * k + 1]);
          unpair(mul2(pair(sv[4 * k + 2], sv[4 * k + 3]), pair(f.z, f.w)), sv[4 * k + 2], sv[4 * k + 3]);
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) sf[k] = ld_shared_v4(scales + 256 + k * 16);
        const float4 vm = ld_shared_v4(scales + 768);
        mask();
        // No weight times scale may pass 2^15 (fp16 ends at 2^16), no weight 2^97.  The largest score with the largest
        // scale (2^-82 if that is less) bounds them; only where that passes, and so at a row's first keys, is the
        // largest product looked for (for every block: 141 us where this takes 126, 256 rows x 32/8 heads behind
        // 16384 tokens; logarithms of the scales taken here and not by the converters: 129).
        const float mx = greatest();
        if (__any_sync(0xffffffffu, mx + fmaxf(vm.x, vm.y) > m + 15.f)) {
          float t4[4] = {mx - 82.f, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float4 f = ld_shared_v4(scales + 512 + k * 16);
            t4[k % 4] = max3(t4[k % 4], fmaf(sv[4 * k], scale, f.x), fmaf(sv[4 * k + 1], scale, f.y));
            t4[k % 4] = max3(t4[k % 4], fmaf(sv[4 * k + 2], scale, f.z), fmaf(sv[4 * k + 3], scale, f.w));
          }
          float t = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) - 8.f;
          t = t > m + 7.f ? t : m;
          if (__any_sync(0xffffffffu, t != m) && !(ok = move(t))) break;
        }
        const float mm = m == -INFINITY ? 0.f : m;
        const uint64_t s2 = pair(scale, scale), m2 = pair(-mm, -mm);
        uint64_t l2[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float x0, x1, x2, x3;
          unpair(fma2(pair(sv[2 * e], sv[2 * e + 1]), s2, m2), x0, x1);
          unpair(fma2(pair(sv[2 * e + 2], sv[2 * e + 3]), s2, m2), x2, x3);
          x0 = ex2(x0), x1 = ex2(x1), x2 = ex2(x2), x3 = ex2(x3);
          l2[0] = add2(l2[0], pair(x0, x1));
          l2[1] = add2(l2[1], pair(x2, x3));
          // Keys behind the chunk may have any scale, NaN too, but their pages are not multiplied.
          const float4 f = sf[e / 2];
          unpair(mul2(pair(f.x, f.y), pair(x0, x1)), x0, x1);
          unpair(mul2(pair(f.z, f.w), pair(x2, x3)), x2, x3);
          p[e] = pack_f16(x0, x1);
          p[e + 1] = pack_f16(x2, x3);
        }
        float la, lb, lc, ld;
        unpair(l2[0], la, lb);
        unpair(l2[1], lc, ld);
        l += (la + lb) + (lc + ld);
      } else {
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&s_full[i % G::KS], (i / G::KS) & 1)))) break;
        fence_after();
        tmem_ld32(ts, sv);
        tmem_ld32(ts + 32, sv + 32);
        if (turn_round) {
#pragma unroll
          for (int k = 0; k < 64; ++k) sv[k] = -sv[k];
        }
        mask();
        const float mx = greatest();
        const float mnew = mx > m + kTau ? mx : m;
        if (__any_sync(0xffffffffu, mnew != m) && !(ok = move(mnew))) break;
        const float mm = m == -INFINITY ? 0.f : m;
        const uint64_t s2 = pair(scale, scale), m2 = pair(-mm, -mm);
        uint64_t l2[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
        uint32_t low[32];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float x0, x1, x2, x3;
          unpair(fma2(pair(sv[2 * e], sv[2 * e + 1]), s2, m2), x0, x1);
          unpair(fma2(pair(sv[2 * e + 2], sv[2 * e + 3]), s2, m2), x2, x3);
          x0 = ex2(x0), x1 = ex2(x1), x2 = ex2(x2), x3 = ex2(x3);
          l2[0] = add2(l2[0], pair(x0, x1));
          l2[1] = add2(l2[1], pair(x2, x3));
          p[e] = pack_bf16(x0, x1);
          p[e + 1] = pack_bf16(x2, x3);
          low[e] = bf16_rest(x0, x1, p[e]);
          low[e + 1] = bf16_rest(x2, x3, p[e + 1]);
        }
        tmem_st32(ts + 32, low);
        float la, lb, lc, ld;
        unpair(l2[0], la, lb);
        unpair(l2[1], lc, ld);
        l += (la + lb) + (lc + ld);
      }
      tmem_st32(ts, p);
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[i % 3]);
    }
    const int last = g + 2 * (n - 1);
    if (ok && n > 0) ok = __all_sync(0xffffffffu, mbar_wait(&o_done[last % G::VS], (last / G::VS) & 1));
    fence_after();
    xch[g * kRows + r] = make_float2(m, l);
    // Each group has waited for its own accumulator's last product; below it reads the other's too, which these
    // fences order behind the other group's wait.
    fence_before();
    asm volatile("bar.sync 1, 256;" ::: "memory");
    fence_after();
    if (!ok) {
      if (lane == 0) report(a.status, CDB_OPS_TIMEOUT);
    } else {
      // Join the groups; warps of group g write columns g HD/2 .. of the partial.
      float2 e0 = xch[r], e1 = xch[kRows + r];
      const float r0 = Q8 ? unit_sum(e0.x, e0.y) : 1.f, r1 = Q8 ? unit_sum(e1.x, e1.y) : 1.f;
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
        if (nb > 1) tmem_ld32(t0 + HD + c0, w);
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = v[e] * (f0 * r0) + (nb > 1 ? w[e] * (f1 * r1) : 0.f);
        if (live) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4*>(po + c0 + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
      }
      if (live && g == 0) A.part_ml[pi] = make_float2(mj, e0.y * f0 + e1.y * f1);
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 9) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(G::TMEM_COLS));
  }
  // This kernel follows the one for the rows' own keys and shares no data with
  // it, so it starts as soon as every CTA of that one has started, which is
  // after its own wait for whatever came before.  Waiting here makes the end of
  // this grid the end of both, which is what the join waits for.
  pdl_wait();
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
  if (Q8 ? !tmap_u8_2d(&tk, c.pool, HD, rows, HD, HD, 16, 0) : !tmap_bf16_octets(&tk, c.pool, HD, rows)) return cudaErrorInvalidValue;
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
