// The paged-cache operators of include/cdb_ops.h: the cache write (query / key
// norm, rotation, e4m3 or bf16 store) and decode attention over the cache with
// grouped heads.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "../../include/cdb.h"
#include "cache_ops.h"
#include "common.cuh"
#include "kernels.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace cdb {

// The slot of a row, -1 for one that the cache does not have.
__device__ __forceinline__ int row_slot(const cdb_paged_cache& c, int base, int depth) {
  const long long s = (long long)base + depth;
  return s >= 0 && s < c.n_kv_slots ? (int)s : -1;
}

// ---------------------------------------------------------------------------
// Cache write.
//
// A streaming kernel: every element of qkv is read once and written once, so
// HBM bounds it.  Persistent CTAs, three per SM: a producer warp looks up 32
// rows at a time (sequence, position, block) and copies each row, or a part of
// at most 24 KB of it, and its line of the rotation table into a three-stage
// ring with bulk copies, so that lookups and loads run two rows ahead of the
// arithmetic (one CTA per row, loading for itself, reached 3.8 TB/s where this
// reaches 5.4, 8192 rows of 16 heads fp32 to e4m3).  Eight warps do the
// arithmetic: groups of GW lanes take one head at a time, 8 elements per lane,
// four of the rotation's lower half and their four partners of the upper one
// (or, behind rot_dim, 8 in a row), so a rotation stays in the lane and the
// sums of the norm and the maximum of the quantisation are shuffles inside the
// group.
// ---------------------------------------------------------------------------
namespace cw {

constexpr int kConsumers = 256;
constexpr int kThreads = kConsumers + 32;
constexpr int kStages = 3;
constexpr int kData = 24 * 1024;  // bytes of a row part
constexpr int kTable = 512;       // bytes of a table line (128 elements)

// What the producer found out about a stage's row.
struct Meta {
  int row, h0, heads, in_page;  // in_page: position in the page, -1: nothing to do
  long long cell;               // cached heads before this position's block and slot
};
struct Stage {
  alignas(16) uint8_t data[kData];
  float2 table[kTable / 8];
  Meta meta;
};
struct Shared {
  Stage stage[kStages];
  uint64_t full[kStages], empty[kStages];
};

template <int HD>
struct Geo {
  static constexpr int GW = HD / 8 <= 4 ? 4 : HD / 8 <= 8 ? 8 : 16;  // lanes of a group (hd 96: 12 of 16 work)
  static constexpr int NG = kConsumers / GW;
};

// Four elements as fp32.
__device__ __forceinline__ void load4(const float* p, float* v) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* v) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(x.x << 16), v[1] = __uint_as_float(x.x & 0xFFFF0000u);
  v[2] = __uint_as_float(x.y << 16), v[3] = __uint_as_float(x.y & 0xFFFF0000u);
}
__device__ __forceinline__ uint2 pack4(const float* v) {
  return make_uint2(tc::pack_bf16(v[0], v[1]), tc::pack_bf16(v[2], v[3]));
}
// Eight e4m3 codes of v / (s + sl), inv the reciprocal of s, sl what rounding the
// scale to s left.  The quotients are corrected by their remainders, to the nearest
// fp32 number (P. Markstein, Computation of elementary functions on the IBM RISC
// System/6000 processor, IBM J. Res. Dev. 34, 1990; the scale's rest is added to its
// remainder).  One that thereby lands halfway between two (normal) codes, the 20th
// last bit set and none behind it, takes the side its remainder points to, so that
// no value is rounded twice: of 34 million codes (8192 rows of 16 heads) some 28
// differ from those of the formula in 64 bits, nearly all of them keys by norm and
// rotation, where 40 would: 50 us, 47 without.  (Norm and rotation with their
// roundings carried along took 70 and left as many.)
__device__ __forceinline__ uint2 code8(const float* v, float s, float sl, float inv) {
  float q[8];
  uint32_t off = ~0u;  // 0 if one is halfway
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    q[e] = v[e] * inv;
    const float r = fmaf(-q[e], sl, fmaf(-q[e], s, v[e]));
    q[e] = fmaf(r, inv, q[e]);  // an infinite scale gives NaN codes: its products are NaN with any code
    off = min(off, (__float_as_uint(q[e]) ^ 0x80000u) & 0xFFFFFu);
  }
  if (off == 0u) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float left = fmaf(-q[e], sl, fmaf(-q[e], s, v[e]));
      const uint32_t t = __float_as_uint(q[e]);
      // Away from zero if the remainder has the quotient's sign.  A border (5 bits) times the largest magnitude
      // differs from 448 v by 2^-34 of it or not at all; what is left of sl's rounding is below 2^-48.
      if (fabsf(left) > 0x1p-40f * fabsf(v[e]) && fabsf(left) < INFINITY && !(t & 0x7FFFFu))
        q[e] = __uint_as_float((t - ((__float_as_uint(left) ^ t) >> 31)) | 1u);
    }
  }
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = __nv_cvt_float2_to_fp8x2(make_float2(q[2 * e], q[2 * e + 1]), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// unit_heads: heads of a part; parts: parts of a row.
template <typename T, int HD, bool Q8>
__global__ void __launch_bounds__(kThreads, 3)
    k_cache_write(const __grid_constant__ cdb_cache_write_args a, int unit_heads, int parts) {
  using G = Geo<HD>;
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& S = *reinterpret_cast<Shared*>(raw);
  const cdb_paged_cache& c = a.cache;
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&S.full[i], 1);
      tc::mbar_init(&S.empty[i], kConsumers / 32);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const int H = a.n_heads, Hk = c.n_kv_heads, total = H + 2 * Hk;
  const long long units = (long long)a.rows * parts;
  const int n = (int)((units - blockIdx.x + gridDim.x - 1) / gridDim.x);  // of this CTA; >= 1

  if (tid >= kConsumers) {
    // ---------------- producer ----------------
    bool ok = true;
    int issued = 0, in_page = -1, row_l = 0, pos_l = 0;
    long long cell_l = 0;
    for (int i = 0; i < n; ++i) {
      if ((i & 31) == 0) {  // this lane looks up unit i + lane
        in_page = -1;
        const long long u = blockIdx.x + (long long)(i + lane) * gridDim.x;
        if (u < units) {
          row_l = (int)(u / parts);
          const int seq = a.seq[row_l];
          if (seq >= 0) {
            pos_l = a.pos[row_l];
            const int slot = row_slot(c, a.slot_base, a.depth ? a.depth[row_l] : 0);
            if (seq >= c.n_seqs || pos_l < 0 || pos_l >= c.max_blocks * 16 || (a.rope && pos_l >= a.rope_positions)) {
              report(a.status, CDB_OPS_BAD_ROW);
            } else {
              const int blk = c.block_table[(size_t)seq * c.max_blocks + (pos_l >> 4)];
              if (blk < 0 || blk >= c.kv_blocks) {
                report(a.status, CDB_OPS_BAD_BLOCK);
              } else if (slot < 0) {
                report(a.status, CDB_OPS_BAD_SLOT);
              } else {
                cell_l = ((long long)blk * c.n_kv_slots + slot) * 2 * Hk;
                in_page = pos_l & 15;
              }
            }
          }
        }
      }
      const int s = i % kStages;
      const int row = __shfl_sync(0xffffffffu, row_l, i & 31), pos = __shfl_sync(0xffffffffu, pos_l, i & 31);
      const int where = __shfl_sync(0xffffffffu, in_page, i & 31);
      const long long cell = __shfl_sync(0xffffffffu, cell_l, i & 31);
      if (i >= kStages && !(ok = __all_sync(0xffffffffu, tc::mbar_wait(&S.empty[s], ((i / kStages) - 1) & 1)))) break;
      const int part = (int)((blockIdx.x + (long long)i * gridDim.x) % parts);
      const int h0 = part * unit_heads, heads = min(unit_heads, total - h0);
      if (tc::elect_one()) {
        Stage& st = S.stage[s];
        st.meta = Meta{row, h0, heads, where, cell};
        const uint32_t bytes = (uint32_t)heads * HD * sizeof(T), line = a.rope ? (uint32_t)a.rot_dim * 4 : 0u;
        tc::mbar_arrive_tx(&S.full[s], where >= 0 ? bytes + line : 0u);
        if (where >= 0) {
          tc::bulk_1d(tc::su32(st.data), reinterpret_cast<const T*>(a.qkv) + (size_t)row * a.ldqkv + (size_t)h0 * HD, bytes,
                      &S.full[s]);
          if (line) tc::bulk_1d(tc::su32(st.table), a.rope + (size_t)pos * a.rot_dim, line, &S.full[s]);
        }
      }
      __syncwarp();
      issued = i + 1;
    }
    if (!ok && lane == 0) report(a.status, CDB_OPS_TIMEOUT);
    // Copies in flight land before the CTA may leave (at once when the consumers took every stage).
    for (int i = max(0, issued - kStages); i < issued; ++i) tc::mbar_wait(&S.full[i % kStages], (i / kStages) & 1);
    return;
  }

  // ---------------- arithmetic ----------------
  const int g = tid / G::GW, l = tid % G::GW;
  const bool on = l * 8 < HD;
  // Groups of a warp may be at different kinds of heads: shuffles name their group's lanes only.
  const uint32_t peers = (0xffffffffu >> (32 - G::GW)) << (lane / G::GW * G::GW);
  // This lane's elements e0..e0+3 and e1..e1+3: partners of the rotation, or 8 in a row.
  const int rl = a.rope ? a.rot_dim / 8 : 0;
  const bool turned = l < rl;
  const int e0 = turned ? 4 * l : 8 * l, e1 = turned ? a.rot_dim / 2 + 4 * l : 8 * l + 4;
  float wq[8] = {}, wk[8] = {};
  if (a.q_gain && on) {
    load4(a.q_gain + e0, wq), load4(a.q_gain + e1, wq + 4);
    load4(a.k_gain + e0, wk), load4(a.k_gain + e1, wk + 4);
  }
  bool ok = true;
  for (int i = 0; i < n; ++i) {
    const int s = i % kStages;
    if (!(ok = __all_sync(0xffffffffu, tc::mbar_wait(&S.full[s], (i / kStages) & 1)))) break;
    const Stage& st = S.stage[s];
    const Meta meta = st.meta;
    if (meta.in_page >= 0) {
      float2 cs[4];
      if (turned) {
#pragma unroll
        for (int e = 0; e < 4; ++e) cs[e] = st.table[e0 + e];
      }
      const T* src = reinterpret_cast<const T*>(st.data);
      for (int r = g; r < meta.heads; r += G::NG) {
        const int h = meta.h0 + r;
        float v[8] = {};  // zeros in the idle lanes of a 96-element head
        if (on) load4(src + r * HD + e0, v), load4(src + r * HD + e1, v + 4);
        if (h < H + Hk) {
          if (a.q_gain) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
#pragma unroll
            for (int o = G::GW / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(peers, ss, o, G::GW);
            const float f = rsqrtf(ss * (1.f / HD) + a.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = v[e] * f * (h < H ? wq[e] : wk[e]);
          }
          if (turned) {
#pragma unroll
            for (int e = 0; e < 4; ++e) rope_pair(v[e], v[e + 4], cs[e], v[e], v[e + 4]);
          }
        }
        if (h < H) {
          if (on) {
            __nv_bfloat16* q = reinterpret_cast<__nv_bfloat16*>(a.q) + (size_t)meta.row * a.ldq + (size_t)h * HD;
            *reinterpret_cast<uint2*>(q + e0) = pack4(v);
            *reinterpret_cast<uint2*>(q + e1) = pack4(v + 4);
          }
          continue;
        }
        const size_t at = (size_t)(meta.cell + (h - H)) * 16 + meta.in_page;  // K heads, then V heads
        if constexpr (Q8) {
          // Scale of this (position, head): the largest magnitude maps to 448; the
          // floor keeps the scale and its reciprocal normal numbers.
          float m = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[e]));
#pragma unroll
          for (int o = G::GW / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(peers, m, o, G::GW));
          const float f = fmaxf(__fdiv_rn(m, 448.f), 0x1p-126f);
          const float inv = __frcp_rn(f), fl = f > 0x1p-126f ? fmaf(-448.f, f, m) * (1.f / 448.f) : 0.f;
          uint8_t* dst = reinterpret_cast<uint8_t*>(c.pool) + at * HD;
          if (on) {
            const uint2 w = code8(v, f, fl, inv);
            *reinterpret_cast<uint32_t*>(dst + e0) = w.x;
            *reinterpret_cast<uint32_t*>(dst + e1) = w.y;
          }
          if (l == 0) c.scales[at] = f;
        } else if (on) {
          __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(c.pool) + at * HD;
          *reinterpret_cast<uint2*>(dst + e0) = pack4(v);
          *reinterpret_cast<uint2*>(dst + e1) = pack4(v + 4);
        }
      }
    }
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&S.empty[s]);
  }
  if (!ok && lane == 0) report(a.status, CDB_OPS_TIMEOUT);
}

template <typename T, int HD, bool Q8>
cudaError_t launch_as(cudaStream_t s, const cdb_cache_write_args& a) {
  static int sms[kMaxDevices] = {};
  const int dev = current_device();
  if (!sms[dev]) {
    int n = 0;
    cudaError_t e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k_cache_write<T, HD, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
    if (e != cudaSuccess) return e;
    sms[dev] = n;
  }
  const int total = a.n_heads + 2 * a.cache.n_kv_heads, most = kData / (HD * (int)sizeof(T));
  const int parts = (total + most - 1) / most, unit_heads = (total + parts - 1) / parts;
  const long long units = (long long)a.rows * parts;
  count_launch();
  return launch_pdl(k_cache_write<T, HD, Q8>, dim3((unsigned)std::min(units, 3ll * sms[dev])), dim3(kThreads), sizeof(Shared), s,
                    a, unit_heads, parts);
}

template <typename T, int HD>
cudaError_t launch(cudaStream_t s, const cdb_cache_write_args& a) {
  return a.cache.dtype == CDB_E4M3 ? launch_as<T, HD, true>(s, a) : launch_as<T, HD, false>(s, a);
}

}  // namespace cw

cudaError_t launch_cache_write(cudaStream_t s, const cdb_cache_write_args& a) {
  if (a.rows <= 0) return cudaSuccess;
  const bool f = a.dtype == CDB_FP32;
  switch (a.cache.head_dim) {
    case 32: return f ? cw::launch<float, 32>(s, a) : cw::launch<__nv_bfloat16, 32>(s, a);
    case 64: return f ? cw::launch<float, 64>(s, a) : cw::launch<__nv_bfloat16, 64>(s, a);
    case 96: return f ? cw::launch<float, 96>(s, a) : cw::launch<__nv_bfloat16, 96>(s, a);
    case 128: return f ? cw::launch<float, 128>(s, a) : cw::launch<__nv_bfloat16, 128>(s, a);
    default: return cudaErrorInvalidValue;
  }
}

// ---------------------------------------------------------------------------
// Decode attention, grouped heads, bf16 or e4m3 cache.
//
// One query token per row: every cached key of a row is read once per KV head,
// so HBM bounds it (128 rows of 17 to 8192 keys, 32/8 heads, bf16: 310 to 330 us, 6.4
// TB/s and more; 64 rows of 128 to 1280 keys, 16 heads, e4m3: 35 us, 5.4 TB/s).  A CTA takes `split` keys of one row and up to four KV
// heads: a producer warp moves 16-key pages of those heads (16 * heads rows of
// one rectangular tile for K, one for V, and the scales) with TMA into a ring,
// four consumer warps each take one (KV head, run of keys).  A warp computes
// S^T = K Q^T and O^T = V^T P^T with m16n8k16 MMAs: keys (then output columns)
// fill the 16 rows, the up to 8 query heads of the KV head the 8 columns, so no
// row of the larger operand is padding; P^T is turned into the second product's
// layout by one 8x8 transpose (movmatrix) per 8 keys.
// Weights enter as 16-bit numbers, high and low part: with up to four query
// heads the low parts sit in the columns 4..7, which costs nothing, else they
// take a second product.
// K and V fragments are read as whole 16-byte pieces of the page rows (any
// order of the summed index is fine as long as both operands use it; the order
// of the output columns is undone at the end); the pairs of keys that the MMA
// wants side by side are made with byte permutes, for e4m3 before the codes are
// widened to fp16 (exactly).  Codes are not scaled: a key's scale multiplies
// its score, a value's scale its weight.  e4m3 weights are taken relative to the
// largest weight times scale seen so far, not to the largest of either: a loud
// value that has no weight and a sink whose value is near zero leave the others
// their bits.  The sum of a key's two fp16 parts is within 2^-22 of its weight
// times scale, or 2^-33 of the row's largest.
// Partials (maximum, sum, unnormalised output) of the splits are joined in
// split order by k_join; a row that fits one split is written directly.
// The grid has every split of max_ctx for every row: a CTA without keys leaves
// after reading its row's place, but takes its turn on an SM (128 rows of 1000
// keys, 32/8 heads, bf16: 82 us with max_ctx 1024, 126 with 32768, 252 with 131072).
// ---------------------------------------------------------------------------
namespace da {

constexpr int kWarps = 4;  // consumer warps

template <int HD, bool Q8>
struct Geo {
  static constexpr int ES = Q8 ? 1 : 2;
  static constexpr int RB = HD * ES;                                             // bytes of a key row
  static constexpr int SB = RB % 128 == 0 ? 128 : RB % 64 == 0 ? 64 : RB;        // bytes of a tile row (slice)
  static constexpr int SW = SB == 128 ? 128 : SB == 64 ? 64 : 0;                 // swizzle span
  static constexpr int NX = RB / SB;                                             // slices of a key row
  static constexpr int KB = Q8 ? 32 : 16;                                        // keys of a warp per stage
  static constexpr int PG = kWarps * KB / 16;                                    // (page, head) cells of a stage
  static constexpr int CELL = 16 * RB;                                           // K (or V) bytes of a cell
  static constexpr int KREG = PG * CELL;                                         // K (or V) bytes of a stage
  static constexpr int SCALES = Q8 ? 2 * PG * 64 : 0;
  static constexpr int STAGE = (2 * KREG + SCALES + 1023) / 1024 * 1024;
  static constexpr int NS = 72 * 1024 / STAGE < 4 ? 72 * 1024 / STAGE : 4;       // stages: three CTAs per SM
  static constexpr size_t SMEM = 1024 + (size_t)NS * STAGE + NS * 2 * 8 + NS * 4;
  static constexpr int NT = HD / 16;                                             // 16-element tiles of the output
  static constexpr int KS = HD / 16;                                             // 16-element steps of q . k
  static constexpr int TE = SB / (4 * ES);    // elements of a slice row that one of 4 lanes takes from K
  static constexpr int VE = SB / (8 * ES);    // elements of a slice row that one of 8 lanes takes from V
  // First of the 4 elements that lane t takes in step s.
  __host__ __device__ static constexpr int k_elem(int t, int s) {
    return (4 * s / TE) * (SB / ES) + t * TE + (4 * s) % TE;
  }
  // The i-th of the HD / 8 elements that lane group g takes from V; row g of output tile j is element
  // 2j, row g + 8 element 2j + 1.  Four elements i..i+3 (i a multiple of 4) are adjacent.
  __host__ __device__ static constexpr int v_elem(int g, int i) { return (i / VE) * (SB / ES) + g * VE + i % VE; }
};

using namespace tc;

template <bool Q8>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  if constexpr (Q8) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}
template <bool Q8>
__device__ __forceinline__ float2 unpack(uint32_t w) {
  if constexpr (Q8) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
// D[16x8] += A[16x16] . B[16x8], fp32 accumulate; operands fp16 (Q8) or bf16.
template <bool Q8>
__device__ __forceinline__ void mma(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (Q8)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// N bytes (4, 8, 12 or 16) of shared memory into words.
template <int N>
__device__ __forceinline__ void lds(uint32_t addr, uint32_t* w) {
  if constexpr (N == 16)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
  else if constexpr (N == 8)
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[i]) : "r"(addr + 4 * i));
  }
}

// Partials of a row of L keys.
__device__ __forceinline__ int row_parts(int L, int first, int split) {
  return L <= first ? 0 : (L - first + split - 1) / split;
}

struct Args {
  cdb_attention_args a;
  int hpc, wph, split, qblocks, group, nhg;
  int first;        // keys below belong to the shared prefix
  int chunks;       // partials of the shared prefix, before a row's own
  int parts;        // partials a row can have
  float* part_o;    // [row][query head][parts][HD]
  float2* part_ml;  // [row][query head][parts]: maximum (log2), sum
};

// Shared offset of byte b of tile row r.
template <int SB, int SW>
__device__ __forceinline__ uint32_t swz(int r, int b) {
  if constexpr (SW == 128) return (uint32_t)(r * 128 + (b ^ ((r & 7) << 4)));
  else if constexpr (SW == 64) return (uint32_t)(r * 64 + (b ^ (((r >> 1) & 3) << 4)));
  else return (uint32_t)(r * SB + b);
}

// 8x8 transpose of 16-bit elements across the warp (lane 4r + t holds row r, columns 2t, 2t + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// WIDE: more than four query heads per KV head (up to 8 here).
template <int HD, bool Q8, bool WIDE>
__global__ void __launch_bounds__((kWarps + 1) * 32, 3)
    k_decode(const __grid_constant__ CUtensorMap tm, const __grid_constant__ Args A) {
  using G = Geo<HD, Q8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + (size_t)G::NS * G::STAGE);
  uint64_t* empty = full + G::NS;
  uint32_t* masks = reinterpret_cast<uint32_t*>(empty + G::NS);  // which pages of the stage arrived
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const cdb_attention_args& a = A.a;
  const cdb_paged_cache& c = a.cache;
  // Last splits first: they are the partly filled ones and, of the longest rows, the ones a launch in
  // ascending order would end with (64 rows of 128 to 1280 keys, e4m3: 38.7 us ascending, 35.4 so).
  const int row = blockIdx.x / A.nhg, hg = blockIdx.x % A.nhg, sp = gridDim.y - 1 - blockIdx.y;
  const int qb = hg % A.qblocks, k0 = hg / A.qblocks * A.hpc;  // first KV head
  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tm) : "memory");
    for (int i = 0; i < G::NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const int seq = a.seq[row], pos = a.pos[row], depth = a.depth ? a.depth[row] : 0;  // one latency for all
  if (seq < 0) return;  // padding
  const int slot = row_slot(c, a.slot_base, depth);
  if (seq >= c.n_seqs || pos >= a.max_ctx || slot < 0) {
    if (threadIdx.x == 0 && sp == 0 && hg == 0) report(a.status, slot < 0 ? CDB_OPS_BAD_SLOT : CDB_OPS_BAD_ROW);
    return;
  }
  const int L = pos + 1;
  const int lo = A.first + sp * A.split, hi = min(L, lo + A.split);
  // A row without keys gets its zeros here, unless k_join writes every row.
  if (lo >= L && (A.chunks > 0 || sp > 0 || L > 0)) return;
  const int pps = A.wph * (G::KB / 16);  // pages of one stage (per head)
  const int npg = max(0, (hi - lo + 15) >> 4), nst = (npg + pps - 1) / pps;

  if (warp == kWarps) {
    // ---------------- producer ----------------
    // The split's pages (at most 32), one per lane.
    const int blk = lane < npg ? c.block_table[(size_t)seq * c.max_blocks + (lo >> 4) + lane] : -1;
    const bool have = blk >= 0 && blk < c.kv_blocks;
    if (lane < npg && !have) report(a.status, CDB_OPS_BAD_BLOCK);
    const uint32_t pages = __ballot_sync(0xffffffffu, have);
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
    const int heads = min(A.hpc, c.n_kv_heads - k0);
    bool fail = false;
    int issued = 0;
    for (int st = 0; st < nst; ++st) {
      const int s = st % G::NS;
      const uint32_t mask = (pages >> (st * pps)) & ((1u << pps) - 1u);
      if (st >= G::NS && !__all_sync(0xffffffffu, mbar_wait(&empty[s], ((st / G::NS) - 1) & 1))) {
        fail = true;
        break;
      }
      const uint32_t cell = (uint32_t)A.hpc * G::CELL;  // one page of the CTA's heads, K or V
      const uint32_t stage = su32(smem + (size_t)s * G::STAGE);
      if (elect_one()) {
        masks[s] = mask;
        mbar_arrive_tx(&full[s], (uint32_t)__popc(mask) * (2 * cell + (Q8 ? 2u * heads * 64 : 0u)));
      }
      __syncwarp();
      for (int i = 0; i < pps; ++i) {
        const int b = __shfl_sync(0xffffffffu, blk, st * pps + i);
        if (!((mask >> i) & 1u)) continue;
        if (elect_one()) {
          // Rows of head k0's page at this block and slot; V follows n_kv_heads pages later.
          const long long head0 = ((long long)b * c.n_kv_slots + slot) * 2 * c.n_kv_heads + k0;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const int y = (int)((head0 + kv * c.n_kv_heads) * 16);
#pragma unroll
            for (int x = 0; x < G::NX; ++x)
              tma_2d(stage + i * cell + kv * G::KREG + x * (A.hpc * 16 * G::SB), &tm, &full[s], x * G::SB, y, pol);
            if constexpr (Q8)
              bulk_1d(stage + 2 * G::KREG + (kv * G::PG + i * A.hpc) * 64, c.scales + (head0 + kv * c.n_kv_heads) * 16,
                      (uint32_t)heads * 64, &full[s]);
          }
        }
        __syncwarp();
      }
      issued = st + 1;
    }
    if (fail && lane == 0) report(a.status, CDB_OPS_TIMEOUT);
    // Copies in flight land before the CTA may leave (at once when the consumers took every stage).
    for (int st = max(0, issued - G::NS); st < issued; ++st) mbar_wait(&full[st % G::NS], (st / G::NS) & 1);
    return;
  }

  // ---------------- consumers ----------------
  const int hh = warp % A.hpc, sub = warp / A.hpc;  // KV head of the CTA, run of keys of the stage
  const int g = lane >> 2, t = lane & 3;
  const int kh = k0 + hh;
  const int nq = min(8, A.group - qb * 8);
  const bool live = kh < c.n_kv_heads;
  const int q0 = kh * A.group + qb * 8;  // first query head
  // q as B fragments: column g is query head q0 + g (narrow: columns 4..7 repeat 0..3).
  uint32_t qf[G::KS][2];
  float mul[2];  // factor of the scores of columns 2t, 2t + 1 (log2 domain)
  {
    uint2 raw[G::KS];
    const int qi = WIDE ? g : g & 3;
    const bool have = live && qi < nq;
    const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) + (size_t)row * a.ldq + (size_t)(q0 + qi) * HD;
#pragma unroll
    for (int s = 0; s < G::KS; ++s)
      raw[s] = have ? *reinterpret_cast<const uint2*>(q + G::k_elem(t, s)) : make_uint2(0u, 0u);
    float f = a.scale * 1.4426950408889634f;
    if constexpr (Q8) {
      // fp16 copy of q, scaled by a power of two so that its largest element is in [1, 2).
      float mx = 0.f;
#pragma unroll
      for (int s = 0; s < G::KS; ++s) {
        const float2 x = unpack<false>(raw[s].x), y = unpack<false>(raw[s].y);
        mx = fmaxf(mx, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y))));
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // 2^-e and 2^e for mx = 2^e f; 1 for zero, tiny, infinite or NaN maxima.
      const uint32_t eb = __float_as_uint(mx) & 0x7F800000u;
      const bool norm = eb > 0x00800000u && eb < 0x7E000000u;
      const float down = norm ? __uint_as_float(0x7F000000u - eb) : 1.f, up = norm ? __uint_as_float(eb) : 1.f;
#pragma unroll
      for (int s = 0; s < G::KS; ++s) {
        const float2 x = unpack<false>(raw[s].x), y = unpack<false>(raw[s].y);
        qf[s][0] = pack<true>(x.x * down, x.y * down);
        qf[s][1] = pack<true>(y.x * down, y.y * down);
      }
      f *= up;
    } else {
#pragma unroll
      for (int s = 0; s < G::KS; ++s) qf[s][0] = raw[s].x, qf[s][1] = raw[s].y;
    }
    mul[0] = __shfl_sync(0xffffffffu, f, 8 * t);
    mul[1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
  }
  float o[G::NT][4];
#pragma unroll
  for (int j = 0; j < G::NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  // Columns 2t, 2t + 1: the reference that o and l are relative to (log2, the same in the 8 lanes of a column; bf16:
  // the maximum score, within 8; e4m3: the maximum of score + log2(value scale), see below), this lane's share of the sum.
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  constexpr int PW = G::KB / 16;           // pages of a warp per stage
  constexpr uint32_t kAll = PW == 1 ? 0xFFFFu : 0xffffffffu;
  bool ok = true;
  for (int st = 0; st < nst; ++st) {
    const int s = st % G::NS;
    if (!(ok = __all_sync(0xffffffffu, mbar_wait(&full[s], (st / G::NS) & 1)))) break;
    const uint32_t base = su32(smem + (size_t)s * G::STAGE);
    const uint32_t arrived = masks[s];
    const int key0 = lo + (st * pps + sub * PW) * 16;  // this warp's first key of the stage
    // Bit per key: within the split and in a page that arrived.
    uint32_t valid = key0 >= hi ? 0u : hi - key0 >= 32 ? 0xffffffffu : (1u << (hi - key0)) - 1u;
#pragma unroll
    for (int p = 0; p < PW; ++p)
      if (!((arrived >> (sub * PW + p)) & 1u)) valid &= ~(0xFFFFu << (16 * p));
    valid &= kAll;
    if (valid) {
      float sc[PW][4], vs[PW][2];  // keys g (0, 1), g + 8 (2, 3) of columns 2t, 2t + 1; value scales of g, g + 8
#pragma unroll
      for (int p = 0; p < PW; ++p) {
        const uint32_t page = base + (uint32_t)((sub * PW + p) * A.hpc) * G::CELL;
        sc[p][0] = sc[p][1] = sc[p][2] = sc[p][3] = 0.f;
#pragma unroll
        for (int x = 0; x < G::NX; ++x) {
          constexpr int TB = G::SB / 4;  // bytes of a slice row this lane takes
          constexpr int LD = TB % 16 == 0 ? 16 : 8;
          uint32_t w0[TB / 4], w1[TB / 4];
#pragma unroll
          for (int i = 0; i < TB; i += LD) {
            lds<LD>(page + x * (A.hpc * 16 * G::SB) + swz<G::SB, G::SW>(hh * 16 + g, t * TB + i), w0 + i / 4);
            lds<LD>(page + x * (A.hpc * 16 * G::SB) + swz<G::SB, G::SW>(hh * 16 + 8 + g, t * TB + i), w1 + i / 4);
          }
          if constexpr (Q8) {
#pragma unroll
            for (int i = 0; i < TB / 4; ++i) {
              const int s2 = x * (TB / 4) + i;
              mma<true>(sc[p], widen(w0[i]), widen(w1[i]), widen_hi(w0[i]), widen_hi(w1[i]), qf[s2][0], qf[s2][1]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < TB / 8; ++i) {
              const int s2 = x * (TB / 8) + i;
              mma<false>(sc[p], w0[2 * i], w1[2 * i], w0[2 * i + 1], w1[2 * i + 1], qf[s2][0], qf[s2][1]);
            }
          }
        }
        if constexpr (Q8) {
          const uint32_t sa = base + 2 * G::KREG + ((sub * PW + p) * A.hpc + hh) * 64 + g * 4;
          uint32_t w[4];
          lds<4>(sa, w);
          lds<4>(sa + 32, w + 1);
          lds<4>(sa + G::PG * 64, w + 2);
          lds<4>(sa + G::PG * 64 + 32, w + 3);
          vs[p][0] = __uint_as_float(w[2]), vs[p][1] = __uint_as_float(w[3]);
          sc[p][0] *= __uint_as_float(w[0]), sc[p][1] *= __uint_as_float(w[0]);
          sc[p][2] *= __uint_as_float(w[1]), sc[p][3] *= __uint_as_float(w[1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[p][e] *= mul[e & 1];
      }
      if (valid != kAll) {
#pragma unroll
        for (int p = 0; p < PW; ++p)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (!((valid >> (16 * p + 8 * e + g)) & 1u)) sc[p][2 * e] = sc[p][2 * e + 1] = -INFINITY, vs[p][e] = 0.f;
      }
      float mx[2] = {fmaxf(sc[0][0], sc[0][2]), fmaxf(sc[0][1], sc[0][3])};
#pragma unroll
      for (int p = 1; p < PW; ++p) {
        mx[0] = max3(mx[0], sc[p][0], sc[p][2]);
        mx[1] = max3(mx[1], sc[p][1], sc[p][3]);
      }
      float mm[2];
      auto move = [&](const float* to) {  // to the references `to`
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          f[e] = m[e] == -INFINITY ? 0.f : ex2(m[e] - to[e]);
          l[e] *= f[e];
          m[e] = to[e];
        }
#pragma unroll
        for (int j = 0; j < G::NT; ++j) {
          o[j][0] *= f[0], o[j][1] *= f[1];
          o[j][2] *= f[0], o[j][3] *= f[1];
        }
      };
      auto offsets = [&] { mm[0] = m[0] == -INFINITY ? 0.f : m[0], mm[1] = m[1] == -INFINITY ? 0.f : m[1]; };
      float w[PW][4], sum[2];  // e4m3: weights times value scales; the sums of the weights
      if constexpr (Q8) {
        // Weights times scales stay below 2^15.  Where one passes that, or at a column's first keys, the reference
        // goes to the largest one / 2^8, so that the smallest step of fp16, 2^-24, is 2^-32 of it.  A weight itself,
        // that of a zero value say, may be as far above the reference as 2^97.
        float top[2];
        auto weigh = [&] {
          offsets();
          top[0] = top[1] = sum[0] = sum[1] = 0.f;
#pragma unroll
          for (int p = 0; p < PW; ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = ex2(sc[p][e] - mm[e & 1]);
              sum[e & 1] += x;
              w[p][e] = x * vs[p][e >> 1];
              top[e & 1] = fmaxf(top[e & 1], fabsf(w[p][e]));
            }
        };
        weigh();
        if (__any_sync(0xffffffffu, fmaxf(top[0], top[1]) > 0x1p15f || fmaxf(sum[0], sum[1]) > 0x1p100f ||
                                        fminf(m[0], m[1]) == -INFINITY)) {
          float to[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = mx[e] - 90.f;
#pragma unroll
            for (int p = 0; p < PW; ++p)
              t = max3(t, sc[p][e] + (__log2f(fabsf(vs[p][0])) - 8.f), sc[p][2 + e] + (__log2f(fabsf(vs[p][1])) - 8.f));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
            to[e] = t > m[e] + 7.f ? t : m[e];
          }
          move(to);
          weigh();
        }
        l[0] += sum[0], l[1] += sum[1];
      } else {
        // The reference maximum moves only when a score passes it by 2^8: most stages rescale nothing.
        if (__any_sync(0xffffffffu, mx[0] > m[0] + 8.f || mx[1] > m[1] + 8.f)) {
          float to[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], d));
            to[e] = mx[e] > m[e] + 8.f ? mx[e] : m[e];
          }
          move(to);
        }
        offsets();
      }
      uint32_t bh[PW][2], bl[PW][2];  // weights of keys 0..7, 8..15 of the page as B fragments
#pragma unroll
      for (int p = 0; p < PW; ++p)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float p0, p1;
          if constexpr (Q8) {
            p0 = w[p][2 * e], p1 = w[p][2 * e + 1];
          } else {
            p0 = ex2(sc[p][2 * e] - mm[0]), p1 = ex2(sc[p][2 * e + 1] - mm[1]);
            l[0] += p0, l[1] += p1;
          }
          const uint32_t high = pack<Q8>(p0, p1);
          const float2 back = unpack<Q8>(high);
          const uint32_t low = pack<Q8>(p0 - back.x, p1 - back.y);
          if constexpr (WIDE) {
            bh[p][e] = transpose8(high);
            bl[p][e] = transpose8(low);
          } else {
            bh[p][e] = transpose8(t < 2 ? high : low);
          }
        }
      // O^T += V^T P^T: lanes (g, t) hold keys 2t, 2t+1, 2t+8, 2t+9 of elements v_elem(g, .).
#pragma unroll
      for (int p = 0; p < PW; ++p) {
        const uint32_t page = base + G::KREG + (uint32_t)((sub * PW + p) * A.hpc) * G::CELL;
        const uint32_t vb = valid >> (16 * p);
        auto product = [&](float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
          mma<Q8>(d, a0, a1, a2, a3, bh[p][0], bh[p][1]);
          if constexpr (WIDE) mma<Q8>(d, a0, a1, a2, a3, bl[p][0], bl[p][1]);
        };
#pragma unroll
        for (int x = 0; x < G::NX; ++x) {
          constexpr int VB = G::SB / 8;  // bytes of a slice row this lane takes
          uint32_t w[4][VB / 4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = 2 * t + (i & 1) + (i >> 1) * 8;
            lds<VB>(page + x * (A.hpc * 16 * G::SB) + swz<G::SB, G::SW>(hh * 16 + key, g * VB), w[i]);
            if (valid != kAll && !((vb >> key) & 1u)) {  // no weight, but the row may hold NaN
#pragma unroll
              for (int e = 0; e < VB / 4; ++e) w[i][e] = 0u;
            }
          }
#pragma unroll
          for (int e = 0; e < VB / 4; ++e) {
            if constexpr (Q8) {  // 4 elements per word
              const uint32_t a01 = __byte_perm(w[0][e], w[1][e], 0x5140), a23 = __byte_perm(w[0][e], w[1][e], 0x7362);
              const uint32_t b01 = __byte_perm(w[2][e], w[3][e], 0x5140), b23 = __byte_perm(w[2][e], w[3][e], 0x7362);
              const int j = (x * G::VE + e * 4) / 2;
              product(o[j], widen(a01), widen_hi(a01), widen(b01), widen_hi(b01));
              product(o[j + 1], widen(a23), widen_hi(a23), widen(b23), widen_hi(b23));
            } else {  // 2 elements per word
              product(o[(x * G::VE + e * 2) / 2], __byte_perm(w[0][e], w[1][e], 0x5410), __byte_perm(w[0][e], w[1][e], 0x7632),
                      __byte_perm(w[2][e], w[3][e], 0x5410), __byte_perm(w[2][e], w[3][e], 0x7632));
            }
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
  }
  if (!ok && lane == 0) report(a.status, CDB_OPS_TIMEOUT);  // what follows is undefined, but in bounds
  // Sums over the keys; high and low weight parts of a narrow group added.
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], d);
  if constexpr (!WIDE) {
#pragma unroll
    for (int j = 0; j < G::NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] += __shfl_xor_sync(0xffffffffu, o[j][e], 2);
  }
  // e4m3: sums may lie far from 1.  With the power of two in them taken into the reference, partials are joined by
  // what their rows weigh; fin is the factor for o.
  float fin[2] = {1.f, 1.f};
  if constexpr (Q8) {
#pragma unroll
    for (int e = 0; e < 2; ++e) fin[e] = unit_sum(m[e], l[e]);
  }
  if (A.wph > 1) {
    // Below four KV heads: the warps of a head add up, in order, in the ring's memory (no copy is in flight once
    // every warp is through its stages).
    constexpr int N = G::NT * 4;
    static_assert(kWarps * (N + 4) * 128 <= G::NS * G::STAGE, "exchange");
    asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
    float* x = reinterpret_cast<float*>(smem) + lane;
    if (sub > 0) {
      float* w = x + warp * (N + 4) * 32;
#pragma unroll
      for (int i = 0; i < N; ++i) w[i * 32] = o[i / 4][i % 4] * fin[i % 2];
#pragma unroll
      for (int e = 0; e < 2; ++e) w[(N + e) * 32] = m[e], w[(N + 2 + e) * 32] = l[e];
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
    if (sub > 0) return;
    for (int s = 1; s < A.wph; ++s) {
      const float* w = x + (s * A.hpc + hh) * (N + 4) * 32;
      float f0[2], f1[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float ms = w[(N + e) * 32], mj = fmaxf(m[e], ms);
        f0[e] = m[e] == -INFINITY ? 0.f : ex2(m[e] - mj);
        f1[e] = ms == -INFINITY ? 0.f : ex2(ms - mj);
        m[e] = mj;
        l[e] = l[e] * f0[e] + w[(N + 2 + e) * 32] * f1[e];
        f0[e] *= fin[e];
      }
#pragma unroll
      for (int i = 0; i < N; ++i) o[i / 4][i % 4] = o[i / 4][i % 4] * f0[i % 2] + w[i * 32] * f1[i % 2];
      fin[0] = fin[1] = 1.f;
    }
  }
  if (!live) return;
  const bool direct = A.chunks == 0 && row_parts(L, A.first, A.split) <= 1;
#pragma unroll
  for (int e = 0; e < 2; ++e) {  // query heads q0 + 2t, q0 + 2t + 1
    const int qi = 2 * t + e;
    if (qi >= nq || (!WIDE && t >= 2)) continue;
    if (direct) {
      const float inv = l[e] > 0.f ? fin[e] / l[e] : l[e] == 0.f ? 0.f : l[e];  // no keys: zeros; NaN stays
      __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.out) + (size_t)row * a.ldo + (size_t)(q0 + qi) * HD;
#pragma unroll
      for (int i = 0; i < HD / 8; i += 4)
        *reinterpret_cast<uint2*>(dst + G::v_elem(g, i)) =
            make_uint2(pack<false>(o[i / 2][e] * inv, o[i / 2][2 + e] * inv),
                       pack<false>(o[i / 2 + 1][e] * inv, o[i / 2 + 1][2 + e] * inv));
    } else {
      const size_t pi = ((size_t)row * a.n_heads + q0 + qi) * A.parts + A.chunks + sp;
      float* po = A.part_o + pi * HD;
#pragma unroll
      for (int i = 0; i < HD / 8; i += 4)
        *reinterpret_cast<float4*>(po + G::v_elem(g, i)) =
            make_float4(o[i / 2][e] * fin[e], o[i / 2][2 + e] * fin[e], o[i / 2 + 1][e] * fin[e], o[i / 2 + 1][2 + e] * fin[e]);
      if (g == 0) A.part_ml[pi] = make_float2(m[e], l[e]);
    }
  }
}

// Join a row's partials: lane j owns columns 4j..4j+3.  Up to kAhead partials
// are one warp's work, in order; of more, warp w of four takes w, w + 4, ...,
// and the four sums are added in order (few rows of long contexts have more
// partials than warps: 4 rows of 32/8 heads over 8000 e4m3 keys, the whole call, 23 us
// with one warp each, 18 so).  Which of the two goes by
// the row's own partials.  TEAM: four warps per (row, query head), else one.
constexpr int kAhead = 8;

template <int HD, bool TEAM>
__global__ void __launch_bounds__(128) k_join(const __grid_constant__ Args A) {
  // Before the wait: only what the caller gave.  The attention kernels let this
  // one start after their own wait, so earlier kernels' writes are visible.
  const cdb_attention_args& a = A.a;
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5, item = TEAM ? blockIdx.x : blockIdx.x * 4 + warp;
  const int row = item / a.n_heads, h = item % a.n_heads;
  const bool in = row < a.rows;
  const int seq = in ? a.seq[row] : -1, pos = in ? a.pos[row] : -1;
  const int slot = row_slot(a.cache, a.slot_base, in && a.depth ? a.depth[row] : 0);
  const bool live = seq >= 0 && seq < a.cache.n_seqs && pos < a.max_ctx && slot >= 0;
  if (A.chunks > 0 && h == 0 && live && (!TEAM || warp == 0)) {  // does the row name the prefix's blocks?
    int base = -1;
    for (int r0 = 0; base < 0; r0 += 32) {  // ends: this row has a sequence
      const int s = r0 + lane < a.rows ? a.seq[r0 + lane] : -1;
      const uint32_t has = __ballot_sync(0xffffffffu, s >= 0 && s < a.cache.n_seqs);
      if (has) base = __shfl_sync(0xffffffffu, s, __ffs(has) - 1);
    }
    const int* t0 = a.cache.block_table + (size_t)base * a.cache.max_blocks;
    const int* t1 = a.cache.block_table + (size_t)seq * a.cache.max_blocks;
    int differ = 0;
    const int pages = min(A.first, max(pos, -1) + 16) / 16;
#pragma unroll 8
    for (int p = lane; p < pages; p += 32) differ |= t0[p] ^ t1[p];
    if (differ) report(a.status, CDB_OPS_NOT_SHARED);
  }
  pdl_wait();
  pdl_trigger();
  if (!live) return;
  const int L = pos + 1;
  const int parts = A.chunks + row_parts(L, A.first, A.split);
  if (A.chunks == 0 && parts <= 1) return;  // written by the attention kernel
  const size_t pi = ((size_t)row * a.n_heads + h) * A.parts;
  const bool cols = 4 * lane < HD;
  const float* po = A.part_o + pi * HD + 4 * lane;
  const bool team = TEAM && parts > kAhead;
  if (TEAM && !team && warp > 0) return;
  const int step = team ? 4 : 1, k0 = team ? warp : 0;  // this warp's partials: k0, k0 + step, ...
  // The first ones are in flight while the weights are worked out.
  float4 x[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    x[k] = cols && k0 + k * step < parts ? *reinterpret_cast<const float4*>(po + (size_t)(k0 + k * step) * HD)
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY;
  for (int s = lane; s < parts; s += 32) m = fmaxf(m, A.part_ml[pi + s].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  auto add = [&](const float4& p, float wk) {
    if (wk != 0.f) v.x = fmaf(p.x, wk, v.x), v.y = fmaf(p.y, wk, v.y), v.z = fmaf(p.z, wk, v.z), v.w = fmaf(p.w, wk, v.w);
  };
  const int mine = (parts - k0 + step - 1) / step;
  for (int s0 = 0; s0 < mine; s0 += 32) {  // 32 of this warp's partials at a time, a weight per lane
    const int s = s0 + lane, n = min(32, mine - s0);
    const float2 ml = s < mine ? A.part_ml[pi + k0 + s * step] : make_float2(-INFINITY, 0.f);
    const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - m), ls = ml.y * w;
    int k1 = 0;
    if (s0 == 0) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, k);  // 0 behind the last partial
        l += __shfl_sync(0xffffffffu, ls, k);
        add(x[k], wk);
      }
      k1 = kAhead;
    }
#pragma unroll 4
    for (int k = k1; k < n; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      l += __shfl_sync(0xffffffffu, ls, k);
      if (cols) add(*reinterpret_cast<const float4*>(po + (size_t)(k0 + (s0 + k) * step) * HD), wk);
    }
  }
  if constexpr (TEAM) {
    if (team) {  // uniform in the block
      __shared__ float4 sv[3][32];
      __shared__ float sl[3];
      if (warp > 0) {
        sv[warp - 1][lane] = v;
        if (lane == 0) sl[warp - 1] = l;
      }
      __syncthreads();
      if (warp > 0) return;
#pragma unroll
      for (int w = 0; w < 3; ++w) {
        const float4 o = sv[w][lane];
        v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        l += sl[w];
      }
    }
  }
  if (!cols) return;
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // no keys: zeros; NaN stays
  uint2 r;
  r.x = pack<false>(v.x * inv, v.y * inv);
  r.y = pack<false>(v.z * inv, v.w * inv);
  *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + (size_t)row * a.ldo + (size_t)h * HD + 4 * lane) = r;
}

template <int HD, bool Q8, bool WIDE>
cudaError_t launch_as(cudaStream_t s, const Args& A) {
  using G = Geo<HD, Q8>;
  const cdb_paged_cache& c = A.a.cache;
  CUtensorMap tm;
  const uint64_t rows = (uint64_t)c.kv_blocks * c.n_kv_slots * 2 * c.n_kv_heads * 16;
  if (!tmap_u8_2d(&tm, c.pool, G::RB, rows, G::RB, G::SB, A.hpc * 16, G::SW)) return cudaErrorInvalidValue;
  static bool set[kMaxDevices] = {};
  const int dev = current_device();
  if (!set[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(k_decode<HD, Q8, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)G::SMEM);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  const int splits = std::max(1, (A.a.max_ctx - A.first + A.split - 1) / A.split);
  count_launch();
  return launch_pdl(k_decode<HD, Q8, WIDE>, dim3((unsigned)A.a.rows * A.nhg, splits), dim3((kWarps + 1) * 32), G::SMEM, s, tm,
                    A);
}

template <int HD, bool Q8>
cudaError_t launch(cudaStream_t s, const Args& A, const SharedPlan& sh) {
  cudaError_t e = A.group > 4 ? launch_as<HD, Q8, true>(s, A) : launch_as<HD, Q8, false>(s, A);
  // The prefix after the rows' own keys: its CTAs move in as the others drain.
  if (e == cudaSuccess && A.chunks > 0) e = launch_shared_prefix(s, A.a, sh, A.parts, A.part_o, A.part_ml);
  if (e != cudaSuccess || (A.chunks == 0 && A.parts <= 1)) return e;
  count_launch();
  const long long items = (long long)A.a.rows * A.a.n_heads;
  if (A.parts > kAhead) return launch_pdl(k_join<HD, true>, dim3((unsigned)items), dim3(128), 0, s, A);
  return launch_pdl(k_join<HD, false>, dim3((unsigned)((items + 3) / 4)), dim3(128), 0, s, A);
}

}  // namespace da

// Keys of a CTA: 128 per warp and head, 256 from four query heads per KV head
// on, whose partials would else weigh more than 3% of the keys read (a partial
// is head_dim + 2 floats per query head).  Below four KV heads the CTA's warps
// share a head, take runs of its keys and make one partial of them (123 rows of
// 3 to 14 keys, 14/2 heads of 64: 5.5 us with a partial per warp and a join, 3.6
// so; 128 rows of 100 to 8000, 8/1 heads, bf16: 54 and 50).  512 keys for one KV
// head (1024: the latter 52 us, one row of 8000 keys 16 for 11), 512 for two (256:
// 64 rows of 128 to 4096, 16/2 heads, bf16, 30 us for 27).  Nothing here looks at the batch, so
// a row's bits do not depend on it.
static AttnPlan attention_plan(int n_heads, int n_kv_heads, int max_ctx, int first) {
  AttnPlan p;
  const int group = n_heads / n_kv_heads;
  p.hpc = n_kv_heads >= 4 ? 4 : n_kv_heads >= 2 ? 2 : 1;
  p.warps_per_head = da::kWarps / p.hpc;
  p.qblocks = (group + 7) / 8;
  p.split = p.warps_per_head == 4 ? 512 : (group >= 4 ? 256 : 128) * p.warps_per_head;
  // At most 512: k_decode holds a split's 16-token pages in one warp.
  p.own_parts = (max_ctx - first + p.split - 1) / p.split;
  return p;
}

// How a shared prefix is cut: tiles of up to 128 query rows, and as many chunks
// of keys as give every SM one CTA (a chunk has at least four blocks of keys,
// so that its setup and partials stay small beside it).
constexpr int kSms = 152;
static SharedPlan shared_plan(int rows, int n_heads, int n_kv_heads, int head_dim, int shared_len) {
  SharedPlan p = {0, 0, 0};
  const int group = n_heads / n_kv_heads;
  if (shared_len <= 0 || rows < 2 || group > 128 || (head_dim != 64 && head_dim != 128)) return p;
  p.tile_rows = 128 / group;
  const long long tiles = (long long)n_kv_heads * ((rows + p.tile_rows - 1) / p.tile_rows);
  if (tiles > 65535) return SharedPlan{0, 0, 0};
  const int blocks = (shared_len + 63) / 64;
  const int want = (int)std::max(1ll, std::min((long long)(blocks + 3) / 4, kSms / std::min(tiles, (long long)kSms)));
  p.chunk = (blocks + want - 1) / want * 64;
  p.chunks = (shared_len + p.chunk - 1) / p.chunk;
  return p;
}

size_t attention_workspace(int rows, int n_heads, int n_kv_heads, int head_dim, int max_ctx, int shared_len) {
  const SharedPlan sh = shared_plan(rows, n_heads, n_kv_heads, head_dim, shared_len);
  const AttnPlan p = attention_plan(n_heads, n_kv_heads, max_ctx, sh.chunks ? shared_len : 0);
  size_t cells = (size_t)rows * n_heads * (sh.chunks + p.own_parts);
  // Any prefix, up to this many rows: chunks is 1, or chunks * tiles <= kSms with at most 128 query rows per tile.
  if (shared_len < 0) cells += std::max((size_t)rows * n_heads, (size_t)kSms * 128);
  return (cells * (head_dim + 2) * 4 + 511) / 256 * 256;
}

cudaError_t launch_decode_attention(cudaStream_t s, const cdb_attention_args& a) {
  if (a.rows <= 0) return cudaSuccess;
  const SharedPlan sh = shared_plan(a.rows, a.n_heads, a.cache.n_kv_heads, a.cache.head_dim, a.shared_len);
  const int first = sh.chunks ? a.shared_len : 0;
  const AttnPlan p = attention_plan(a.n_heads, a.cache.n_kv_heads, a.max_ctx, first);
  da::Args A;
  A.a = a;
  A.hpc = p.hpc;
  A.wph = p.warps_per_head;
  A.split = p.split;
  A.qblocks = p.qblocks;
  A.group = a.n_heads / a.cache.n_kv_heads;
  A.nhg = (a.cache.n_kv_heads + p.hpc - 1) / p.hpc * p.qblocks;
  A.first = first;
  A.chunks = sh.chunks;
  A.parts = sh.chunks + p.own_parts;
  const size_t cells = (size_t)a.rows * a.n_heads * A.parts;
  A.part_o = static_cast<float*>(a.workspace);
  A.part_ml = reinterpret_cast<float2*>(A.part_o + cells * a.cache.head_dim);
  const bool q8 = a.cache.dtype == CDB_E4M3;
  switch (a.cache.head_dim) {
    case 32: return q8 ? da::launch<32, true>(s, A, sh) : da::launch<32, false>(s, A, sh);
    case 64: return q8 ? da::launch<64, true>(s, A, sh) : da::launch<64, false>(s, A, sh);
    case 96: return q8 ? da::launch<96, true>(s, A, sh) : da::launch<96, false>(s, A, sh);
    case 128: return q8 ? da::launch<128, true>(s, A, sh) : da::launch<128, false>(s, A, sh);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace cdb
