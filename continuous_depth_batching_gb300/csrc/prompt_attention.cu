// Attention of packed prompts and of drafted tokens over the paged cache
// (cdb_prompt_attention, cdb_draft_attention of include/cdb_ops.h) on the
// 5th-generation tensor cores: bf16 or e4m3 cache, head_dim 32, 64, 96 or 128.
//
// The query rows of a tile are tokens times the query heads of one KV head, 128
// rows of a matrix product with the keys (so grouped heads read K and V once and
// a tile's rows lie close together: with four heads per KV head, 32 tokens of a
// causal prompt, hence little work above the diagonal).  An item is a stretch
// of a request's rows, up to two tiles of them, for one KV head, and a range of its
// keys, walked in blocks of 128; one CTA takes one item.  Two softmax groups
// of 128 threads, a thread per query row, work in turn:
//   two tiles   each group has a tile of its own and takes every block, so that a
//               block of keys is read once for 256 rows;
//   one tile    the groups take even and odd blocks of the same rows, and are joined
//               at the end.
// Either way the tensor cores work for one group while the other is in its
// exponentials.
//   warps 0-7    softmax: a thread reads the 128 scores of its row from TMEM, masks
//                them, and writes the weights over them in 16 bits, the A operand of
//                the second product.  bf16 weights are two numbers, what the first
//                leaves in the second (within 2^-17, a product each); e4m3: one
//                fp16 number of weight times value scale, relative to the row's largest (2^-11;
//                two numbers would take outputs from 1.660e-3 off to the 1.653e-3 of their bf16
//                rounding, a batch of drafts from 150 to 207 us, chunks behind cached tokens
//                from 147 to 208);
//   warp 9       issues S = Q K^T (128 x 128) and O += P V.  The next scores of a group
//                follow its product with V in the tensor core's queue, which keeps order,
//                so they may overwrite the weights, and their commit covers both;
//   warps 8, 11  copy K and V pages by TMA, and scales; bf16: then warp 11 looks the blocks that
//                some rows do not see through (below);
//   warps 12-15  e4m3: widen V's codes to fp16 in the MMA's swizzled layout.  K's codes are an
//                operand as they are: q becomes the sum of an e4m3 and an e5m2 number, exactly but for elements
//                far below a row's largest, and the scores of both are added up.
// A weight of 0 times an infinite or NaN value is NaN, so in blocks that not all
// rows see, V rows with such an element are set to zero in shared memory before the
// product, and rows that see them take a NaN weight; V rows behind the sequence's
// end, which may hold anything, are set to zero too.
// What bounds it.  A long bf16 prompt: the tensor cores, which compute three products of 512 cycles for a job (one
// for the scores, two for weights in two parts), together with the waits and commits of the warp that feeds them
// (8192 tokens of 32/8 heads: 555 us, 1.0 PFLOP/s of causal products; of 547 before, the products alone took 472 and
// softmax alone 444; pipe 63% active).  Drafts over long bf16 caches: HBM (32 drafts of 16 tokens
// behind 16000: 4.8 of 6.7 TB/s for the call, 5.3 over the growth from 4000 tokens).  e4m3: the chain from scores to
// weights to the next scores, in which a key's scales are read from shared memory by every thread (the same drafts: 2.2
// TB/s, 2.4 over the growth).  Short calls: setup, one chain of loads and the join.
// Every mbarrier wait is bounded; on expiry the kernel reports CDB_OPS_TIMEOUT,
// lets its copies and MMAs finish (bounded), frees TMEM and returns.
#include <algorithm>
#include <climits>

#include "../../include/cdb.h"
#include "common.cuh"
#include "kernels.cuh"
#include "row_ops.h"
#include "tc.cuh"
#include "tmap.h"

namespace cdb {
namespace pa {

using namespace tc;

constexpr int kRows = 128;   // query rows of a tile
constexpr int kKeys = 128;   // keys of a block: eight pages
constexpr int kSms = 152;
// Items (times KV heads) that cutting keys aims at.  One for each SM: setup, q and the end of an item do not overlap
// with another (32 drafts over 500 to 8000 e4m3 keys 162 us, chunks behind cached tokens 154; three for each SM 195 and
// 183, one and a half or two 177 to 180 for the drafts).
constexpr int kItems = kSms;
constexpr int kMinBlocks = 2;  // blocks of a cut item, at least (8 nodes behind 1000 tokens: 15.9 us, with four 20.8)
// Items without cutting, from which on no call cuts: SMs are busy then.  It depends on the lengths: equal ones prefer
// half as many (of 32/8 heads: 2500 tokens 85 us for 89, 3300 122 for 131, 4096 173 for 177, five chunks of 600 behind 1500
// 143 for 151), uneven ones do not (five chunks of 100 to 1100 behind up to 3000, bf16 133 for 121, e4m3 151 for 147; 44
// e4m3 drafts 278 for 263), and of twice as many 20 uneven chunks take 202 for 225, but 6000 tokens 336 for 325.
constexpr int kCutBelow = 4 * kSms;

template <int HD, bool Q8>
struct Geo {
  static_assert(HD % 32 == 0 && HD <= 128, "head dim");
  static constexpr int NX = (HD + 63) / 64;       // 128-byte slices of a 16-bit row
  static constexpr int SLICE = 128 * 128;         // one slice of 128 rows
  static constexpr int TILE = NX * SLICE;         // V block in 16 bits
  // bf16: Q tile and K block as V.  e4m3: K as it comes, a slice of up to 128 codes a row; Q in two parts like it.
  static constexpr int QT = Q8 ? 2 * SLICE : TILE, KB = Q8 ? SLICE : TILE;
  static constexpr int KS = NX == 2 || Q8 ? 3 : 4;   // K blocks in flight (bf16: of drafts over long caches 549 us with 2, 494 with 3)
  // V blocks in flight; bf16, with one tile: one more where the second Q tile would be (32 drafts behind 16000 tokens of 32/8
  // heads: 466 us without, 440 with; e4m3: no change, 1% less for prompts).
  static constexpr int VS = NX == 2 ? 2 : 4, VX = NX == 2 && !Q8 ? 1 : 0;
  // e4m3: V as it comes, a unit of 32 keys for each converter warp.
  static constexpr int UNIT = 32 * HD;
  static constexpr int NU = NX == 2 ? 2 : 3;      // units of a warp in flight
  static constexpr int NT = 8;                    // blocks whose end is told apart: more than a ring's slots and three
  static constexpr int NSC = 4;                   // blocks whose scales are kept
  static constexpr int SCN = 3 * kKeys + 4;       // scales of K, of V, the latter's logarithms, the largest of those by quarters
  static constexpr int OFF_K = 2 * QT;
  static constexpr int OFF_V = OFF_K + KS * KB;
  static constexpr int OFF_U = OFF_V + VS * TILE;
  static constexpr int OFF_SC = OFF_U + (Q8 ? 4 * NU * UNIT : 0);
  static constexpr int OFF_BAD = OFF_SC + (Q8 ? NSC * SCN * 4 : 0);  // [VS] keys whose value is not finite: bits (bf16), bytes (e4m3)
  // float2 [2][kRows], with one tile: the last K slot, which is not in use when a group has finished, or has nothing to do
  static constexpr int OFF_XCH = OFF_K + (KS - 1) * KB;
  static constexpr int OFF_UP = OFF_BAD + (VS + VX) * (Q8 ? kKeys : 16);
  static constexpr int OFF_BAR = OFF_UP + (Q8 ? 2 * kRows * 4 : 0);
  static constexpr int NBAR = 2 + KS + 2 * (VS + VX) + NT + 2 + 2 + 2 + 2 + 2 * 4 * NU + NSC;
  static constexpr size_t SMEM = 1024 + OFF_BAR + NBAR * 8 + 16;
  static constexpr int THREADS = Q8 ? 512 : 384;
  static constexpr int S_COL = 256;               // [2][128] scores, then weights
  static constexpr int O_COL = 0;                 // [2][128], HD of them used
  static_assert(SMEM + 512 <= 232448, "shared memory, static too");
};

struct Args {
  cdb_prompt_attention_args a;
  int group;    // query heads per KV head
  int tokens;   // of a tile: tokens * group <= 128
  int cut;      // items (per KV head) that cutting keys may add; 0: no request is cut
  int tiles;    // upper bound of double tiles
  float* part_o;   // [item][KV head][256][HD]
  float2* part_ml; // [item][KV head][256]
  int4* info;      // [tiles]: request, first token, first item, chunks
};

struct Item {
  int request, seq, row0, count, len;  // of the request
  int t0;                              // first token
  int chunk, chunks, cb;               // chunk of `chunks`, blocks of a chunk
  int tile;                            // of all double tiles, -1: this item is not there
};

__device__ __forceinline__ int div_up(int a, int b) { return (a + b - 1) / b; }

// The request's double tiles, its blocks of keys; false: it is not there.  count < 0: row_start descends.  Where it does
// not, requests that are there have rows of their own, hence A.tiles double tiles at most, all of them together.
__device__ __forceinline__ bool look(const Args& A, int i, Item& it, bool tell) {
  const cdb_prompt_attention_args& a = A.a;
  const int r0 = a.row_start[i], r1 = a.row_start[i + 1], len = a.lens[i], seq = a.seq ? a.seq[i] : i;
  it.request = i, it.seq = seq, it.row0 = r0, it.count = r1 < r0 ? -1 : r1 - r0, it.len = len;
  if (r1 < r0 && tell) report(a.status, CDB_OPS_BAD_ROW);
  if (seq < 0 || r1 == r0) return false;
  const bool ok = seq < a.cache.n_seqs && r0 >= 0 && r1 > r0 && r1 <= a.rows && len >= 0 && len <= a.max_ctx &&
                  (!a.visible || r1 - r0 <= 64 * a.mask_words);
  if (!ok && tell) report(a.status, CDB_OPS_BAD_ROW);
  return ok;
}

// Which item this CTA takes, found by all its threads: requests in order, of each
// request its cut ranges of keys, of those its double tiles, the last (most keys) first.
// A request's keys are cut into equal ranges of at most `cb` blocks, such that kItems items would
// hold all of the call's.
// Up to 32 requests: every warp by itself, without a barrier; where keys are cut, requests of
// longer ranges come first, so that the last CTAs to run are short.  Beyond: all warps, in the caller's order (drafts over
// 500 to 8000 e4m3 keys: 32 requests 152 us, 33 214).
__device__ __forceinline__ Item find_item_warp(const Args& A, int y) {
  const cdb_prompt_attention_args& a = A.a;
  const int lane = threadIdx.x & 31, step = 2 * A.tokens;
  const bool tell = blockIdx.x == 0 && y == 0 && threadIdx.x < 32;
  Item it = {};
  const bool there = lane < a.requests && look(A, lane, it, tell);
  const bool on = !__any_sync(0xffffffffu, it.count < 0) && there;
  const int nt = on ? div_up(it.count, step) : 0, blocks = max(1, div_up(it.len, kKeys));
  int cb = INT_MAX / kKeys;
  if (A.cut) {
    const int work = __reduce_add_sync(0xffffffffu, on ? nt * blocks : 0);  // cutting calls have few tiles
    cb = max(kMinBlocks, div_up(work, A.cut));
  }
  const int nc = on ? div_up(blocks, cb) : 0, range = nc ? div_up(blocks, nc) : 0;
  const int own = nt * nc;
  int xi = own, xt = nt;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int p = __shfl_up_sync(0xffffffffu, xi, o), q = __shfl_up_sync(0xffffffffu, xt, o);
    if (lane >= o) xi += p, xt += q;
  }
  const int tiles = __shfl_sync(0xffffffffu, xt, 31);
  xi -= own, xt -= nt;
  if (A.cut && a.requests > 1) {
    const int key = range * 32 + 31 - lane;  // by range, then by request
    xi = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int other = __shfl_sync(0xffffffffu, key, j), n = __shfl_sync(0xffffffffu, own, j);
      xi += other > key ? n : 0;
    }
  }
  const uint32_t mine = __ballot_sync(0xffffffffu, on && y >= xi && y < xi + nt * nc);
  if (A.cut && tell) {  // for the join
    if (on)
      for (int k = 0; k < nt; ++k) A.info[xt + k] = make_int4(lane, k * step, xi + nt - 1 - k, nc | (nt << 16));
    for (int t = tiles + lane; t < A.tiles; t += 32) A.info[t] = make_int4(0, 0, 0, 0);
  }
  const int from = mine ? __ffs(mine) - 1 : 0;
  const int k = y - xi, tile = nt ? nt - 1 - k % nt : 0;
  it.t0 = tile * step;
  it.chunk = nt ? k / nt : 0, it.chunks = nc, it.cb = A.cut ? range : cb;
  it.tile = xt + tile;
  int* f = reinterpret_cast<int*>(&it);
#pragma unroll
  for (int e = 0; e < (int)(sizeof(Item) / 4); ++e) f[e] = __shfl_sync(0xffffffffu, f[e], from);
  if (!mine) it.tile = -1;
  return it;
}

template <int THREADS>
__device__ __forceinline__ Item find_item(const Args& A, int y) {
  if (A.a.requests <= 32) return find_item_warp(A, y);
  __shared__ int sh[THREADS / 32][2];
  __shared__ long long work_s[THREADS / 32];
  __shared__ Item found;
  const cdb_prompt_attention_args& a = A.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, step = 2 * A.tokens;
  const bool tell = blockIdx.x == 0 && y == 0;
  Item it;
  int cb = INT_MAX / kKeys, falls = 0;
  if (A.cut) {
    long long work = 0;  // blocks of keys, once for each double tile
    for (int i = tid; i < a.requests; i += THREADS) {
      if (look(A, i, it, false)) work += (long long)div_up(it.count, step) * max(1, div_up(it.len, kKeys));
      falls |= it.count < 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) work += __shfl_xor_sync(0xffffffffu, work, o);
    if (lane == 0) work_s[warp] = work;
    falls = __syncthreads_or(falls);  // nothing is cut, or noted for the join, that may not fit the workspace
    work = 0;
    for (int w = 0; w < THREADS / 32; ++w) work += work_s[w];
    cb = (int)max((long long)kMinBlocks, (work + A.cut - 1) / A.cut);
  }
  if (tid == 0) found.tile = -1;
  int items = 0, tiles = 0;  // of the requests before this round
  for (int i0 = 0; i0 < a.requests; i0 += THREADS) {
    const int i = i0 + tid;
    const bool on = i < a.requests && look(A, i, it, tell) && !falls;
    const int nt = on ? div_up(it.count, step) : 0, nc = on ? max(1, div_up(div_up(it.len, kKeys), cb)) : 0;
    int xi = nt * nc, xt = nt;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int p = __shfl_up_sync(0xffffffffu, xi, o), q = __shfl_up_sync(0xffffffffu, xt, o);
      if (lane >= o) xi += p, xt += q;
    }
    if (lane == 31) sh[warp][0] = xi, sh[warp][1] = xt;
    __syncthreads();
    int all_i = 0, all_t = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w == warp) xi += items + all_i - nt * nc, xt += tiles + all_t - nt;
      all_i += sh[w][0], all_t += sh[w][1];
    }
    items += all_i, tiles += all_t;
    if (on && y >= xi && y < xi + nt * nc) {
      const int k = y - xi, tile = nt - 1 - k % nt;
      it.t0 = tile * step;
      it.chunk = k / nt, it.chunks = nc, it.cb = A.cut ? max(1, div_up(div_up(it.len, kKeys), nc)) : cb;
      it.tile = xt + tile;
      found = it;
    }
    if (A.cut && tell && on)  // for the join
      for (int k = 0; k < nt; ++k) A.info[xt + k] = make_int4(i, k * step, xi + nt - 1 - k, nc | (nt << 16));
    __syncthreads();
  }
  if (A.cut && tell)
    for (int t = tiles + tid; t < A.tiles; t += THREADS) A.info[t] = make_int4(0, 0, 0, 0);
  __syncthreads();
  return found;
}

// Two times two bf16 numbers times f as e4m3 codes, and what these leave of them as e5m2 codes.  Of the eight bits of a
// number the first takes four, which leaves at most half of its last step: 0 to 8 sixteenths of it, exact in e5m2's three
// bits.  e5m2, because its steps go down to 2^-16 where e4m3's end at 2^-9: with one channel of q 1000 times as loud as
// the others (and 4000 keys), outputs are 1.66e-3 off, which is their bf16 rounding; with the rest in e4m3 too 5.6e-3.
__device__ __forceinline__ void split_q(uint32_t a, uint32_t b, float f, uint32_t& one, uint32_t& rest) {
  asm("{\n .reg .b16 l, h;\n .reg .b32 x, y, u, v;\n .reg .f32 e, f;\n"
      " shl.b32 u, %2, 16;\n and.b32 v, %2, 0xFFFF0000;\n mul.f32 e, u, %4;\n mul.f32 f, v, %4;\n cvt.rn.f16x2.f32 x, f, e;\n"
      " shl.b32 u, %3, 16;\n and.b32 v, %3, 0xFFFF0000;\n mul.f32 e, u, %4;\n mul.f32 f, v, %4;\n cvt.rn.f16x2.f32 y, f, e;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 l, x;\n cvt.rn.satfinite.e4m3x2.f16x2 h, y;\n mov.b32 %0, {l, h};\n"
      " cvt.rn.f16x2.e4m3x2 u, l;\n cvt.rn.f16x2.e4m3x2 v, h;\n sub.rn.f16x2 x, x, u;\n sub.rn.f16x2 y, y, v;\n"
      " cvt.rn.satfinite.e5m2x2.f16x2 l, x;\n cvt.rn.satfinite.e5m2x2.f16x2 h, y;\n mov.b32 %1, {l, h};\n}\n"
      : "=&r"(one), "=r"(rest)
      : "r"(a), "r"(b), "f"(f));
}
// The largest magnitude of eight bf16 numbers, as bits (NaN: above infinity).
__device__ __forceinline__ uint32_t largest_bf16(uint4 w) {
  uint32_t m = 0;
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) m = max(m, max(v[e] << 16 & 0x7FFF0000u, v[e] & 0x7FFF0000u));
  return m >> 16;
}

// 32 keys from position s on that a row sees, as bits.  Prompt: positions up to
// lim.  Draft: those before `lim`, and behind them the row's mask.
__device__ __forceinline__ uint32_t seen(int s, int lim, const uint32_t* mask, int nodes) {
  if (!mask) return lim < s ? 0u : lim - s >= 31 ? ~0u : (2u << (lim - s)) - 1;
  const int u = s - lim;  // node of the first bit
  uint32_t w = u <= -32 ? ~0u : u < 0 ? (1u << -u) - 1 : 0u;
  if (u > -32 && u < nodes) {
    const int at = max(u, 0) / 32, off = max(u, 0) % 32, words = div_up(nodes, 32);
    uint32_t b = __funnelshift_r(mask[at], at + 1 < words ? mask[at + 1] : 0u, off);
    const int left = nodes - max(u, 0);
    if (left < 32) b &= (1u << left) - 1;
    w |= u < 0 ? b << -u : b;
  }
  return w;
}

// The products of one job, each issued as one piece: one lane is elected inside, and descriptors
// are made from 32-bit words by additions of constants.
#define CDB_SS(off, acc)                                                                         \
  " add.u32 x, %1, " off ";\n mov.b64 da, {x, %3};\n add.u32 x, %2, " off ";\n mov.b64 db, {x, %3};\n" \
  " @q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, " acc ";\n"
#define CDB_SS_BEGIN                                                                  \
  "{\n .reg .pred q, f, t;\n .reg .b32 x;\n .reg .b64 da, db;\n setp.ne.b32 t, 1, 0;\n setp.ne.b32 f, 0, 0;\n" \
  " elect.sync _|q, 0xffffffff;\n"
// S[tmem] = Q K^T; q, k: lower words of the descriptors, whose upper words are the same.
template <int STEPS>
__device__ __forceinline__ void issue_scores(uint32_t d, uint32_t q, uint32_t k, uint32_t upper, uint32_t id) {
  static_assert(STEPS == 2 || STEPS == 4 || STEPS == 6 || STEPS == 8, "head dim");
  if constexpr (STEPS == 2)
    asm volatile(CDB_SS_BEGIN CDB_SS("0", "f") CDB_SS("2", "t") "}\n" ::"r"(d), "r"(q), "r"(k), "r"(upper), "r"(id) : "memory");
  if constexpr (STEPS == 4)
    asm volatile(CDB_SS_BEGIN CDB_SS("0", "f") CDB_SS("2", "t") CDB_SS("4", "t") CDB_SS("6", "t") "}\n" ::"r"(d), "r"(q), "r"(k),
                 "r"(upper), "r"(id)
                 : "memory");
  if constexpr (STEPS == 6)
    asm volatile(CDB_SS_BEGIN CDB_SS("0", "f") CDB_SS("2", "t") CDB_SS("4", "t") CDB_SS("6", "t") CDB_SS("1024", "t")
                     CDB_SS("1026", "t") "}\n" ::"r"(d),
                 "r"(q), "r"(k), "r"(upper), "r"(id)
                 : "memory");
  if constexpr (STEPS == 8)
    asm volatile(CDB_SS_BEGIN CDB_SS("0", "f") CDB_SS("2", "t") CDB_SS("4", "t") CDB_SS("6", "t") CDB_SS("1024", "t")
                     CDB_SS("1026", "t") CDB_SS("1028", "t") CDB_SS("1030", "t") "}\n" ::"r"(d),
                 "r"(q), "r"(k), "r"(upper), "r"(id)
                 : "memory");
}
// The same of codes, 32 elements a step; Q is the sum of two tiles, of e4m3 (id) and of e5m2 (id5) codes.
#define CDB_S8(qoff, koff, id, acc)                                                                \
  " add.u32 x, %1, " qoff ";\n mov.b64 da, {x, %3};\n add.u32 x, %2, " koff ";\n mov.b64 db, {x, %3};\n" \
  " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, " id ", " acc ";\n"
#define CDB_S8_ONE(off, acc) CDB_S8(off, off, "%4", acc)
#define CDB_S8_REST(qoff, koff) CDB_S8(qoff, koff, "%5", "t")
template <int STEPS>
__device__ __forceinline__ void issue_scores_8(uint32_t d, uint32_t q, uint32_t k, uint32_t upper, uint32_t id, uint32_t id5) {
  static_assert(STEPS >= 1 && STEPS <= 4, "head dim");
  if constexpr (STEPS == 1)
    asm volatile(CDB_SS_BEGIN CDB_S8_ONE("0", "f") CDB_S8_REST("1024", "0") "}\n" ::"r"(d), "r"(q), "r"(k), "r"(upper), "r"(id),
                 "r"(id5)
                 : "memory");
  if constexpr (STEPS == 2)
    asm volatile(CDB_SS_BEGIN CDB_S8_ONE("0", "f") CDB_S8_ONE("2", "t") CDB_S8_REST("1024", "0") CDB_S8_REST("1026", "2")
                     "}\n" ::"r"(d),
                 "r"(q), "r"(k), "r"(upper), "r"(id), "r"(id5)
                 : "memory");
  if constexpr (STEPS == 3)
    asm volatile(CDB_SS_BEGIN CDB_S8_ONE("0", "f") CDB_S8_ONE("2", "t") CDB_S8_ONE("4", "t") CDB_S8_REST("1024", "0")
                     CDB_S8_REST("1026", "2") CDB_S8_REST("1028", "4") "}\n" ::"r"(d),
                 "r"(q), "r"(k), "r"(upper), "r"(id), "r"(id5)
                 : "memory");
  if constexpr (STEPS == 4)
    asm volatile(CDB_SS_BEGIN CDB_S8_ONE("0", "f") CDB_S8_ONE("2", "t") CDB_S8_ONE("4", "t") CDB_S8_ONE("6", "t")
                     CDB_S8_REST("1024", "0") CDB_S8_REST("1026", "2") CDB_S8_REST("1028", "4") CDB_S8_REST("1030", "6")
                         "}\n" ::"r"(d),
                 "r"(q), "r"(k), "r"(upper), "r"(id), "r"(id5)
                 : "memory");
}
// Instruction descriptor, kind::f8f6f4: fp32 accumulator, A e4m3 or e5m2, B e4m3, both K-major.
__host__ __device__ constexpr uint32_t idesc_8(bool a_e5m2, int M, int N) {
  return (1u << 4) | ((uint32_t)a_e5m2 << 7) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// O[tmem] (+)= P[tmem] V over up to eight pages of 16 keys.
#define CDB_TS(n, a, off, acc)                                                              \
  " setp.gt.s32 s, %5, " n ";\n and.pred s, s, q;\n add.u32 x, %1, " a ";\n add.u32 y, %2, " off ";\n mov.b64 db, {y, %3};\n" \
  " @s tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %4, " acc ";\n"
__device__ __forceinline__ void issue_values(uint32_t d, uint32_t p, uint32_t v, uint32_t upper, uint32_t id, int pages,
                                             bool add) {
  asm volatile(
      "{\n .reg .pred q, f, t, s;\n .reg .b32 x, y;\n .reg .b64 db;\n setp.ne.b32 t, 1, 0;\n setp.ne.b32 f, %6, 0;\n"
      " elect.sync _|q, 0xffffffff;\n" CDB_TS("0", "0", "0", "f") CDB_TS("1", "8", "128", "t") CDB_TS("2", "16", "256", "t")
          CDB_TS("3", "24", "384", "t") CDB_TS("4", "32", "512", "t") CDB_TS("5", "40", "640", "t")
              CDB_TS("6", "48", "768", "t") CDB_TS("7", "56", "896", "t") "}\n" ::"r"(d),
      "r"(p), "r"(v), "r"(upper), "r"(id), "r"(pages), "r"((int)add)
      : "memory");
}

template <int HD, bool Q8>
__global__ void __launch_bounds__(Geo<HD, Q8>::THREADS, 1)
    k_prompt(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ Args A) {
  using G = Geo<HD, Q8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float2* xch = reinterpret_cast<float2*>(smem + G::OFF_XCH);
  uint32_t* bad_keys = reinterpret_cast<uint32_t*>(smem + G::OFF_BAD);
  uint8_t* bad_bytes = smem + G::OFF_BAD;
  float* q_up = reinterpret_cast<float*>(smem + G::OFF_UP);  // e4m3: what a row of q was divided by
  uint64_t* q_ready = reinterpret_cast<uint64_t*>(smem + G::OFF_BAR);  // [2]
  uint64_t* k_full = q_ready + 2;
  uint64_t* v_full = k_full + G::KS;
  uint64_t* v_clean = v_full + G::VS + G::VX;    // blocks that were looked through
  uint64_t* taken = v_clean + G::VS + G::VX;     // V of this block, and K of the next, are free
  uint64_t* s_full = taken + G::NT;      // [2] by group
  uint64_t* p_full = s_full + 2;
  uint64_t* o_final = p_full + 2;
  uint64_t* done = o_final + 2;
  uint64_t* k_first = done + 1;          // K of the groups' first blocks is free
  constexpr int kUnits = 4 * G::NU;
  uint64_t* u_full = k_first + 1;        // [slots][4]
  uint64_t* u_empty = u_full + kUnits;
  uint64_t* sc_full = u_empty + kUnits;  // [NSC]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sc_full + G::NSC);

  const cdb_prompt_attention_args& a = A.a;
  const cdb_paged_cache& c = a.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kh = blockIdx.x;
  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmk) : "memory");
    for (int g = 0; g < 2; ++g) {
      mbar_init(&s_full[g], 1);
      mbar_init(&o_final[g], 1);
    }
    for (int s = 0; s < G::KS; ++s) {
      mbar_init(&k_full[s], 1);
    }
    for (int s = 0; s < G::VS + G::VX; ++s) {
      mbar_init(&v_full[s], Q8 ? 4 : 1);
      mbar_init(&v_clean[s], 1);
    }
    mbar_init(done, 1);
    mbar_init(k_first, 1);
    for (int s = 0; s < G::NT; ++s) mbar_init(&taken[s], 1);
    for (int s = 0; s < G::NSC; ++s) mbar_init(&sc_full[s], 4);
    for (int s = 0; s < kUnits; ++s) {
      mbar_init(&u_full[s], 1);
      mbar_init(&u_empty[s], 1);
    }
  }
  pdl_wait();
  pdl_trigger();
  const Item it = find_item<G::THREADS>(A, blockIdx.y);
  if (it.tile < 0) return;
  const int tt = A.tokens;
  const int n_tok = min(2 * tt, it.count - it.t0);      // tokens of this item
  const bool two = n_tok > tt;
  // Warps of a group that have rows; the others' lanes of the products hold what they may.
  auto live_warps = [&](int g) { return div_up(min(tt, two && g ? n_tok - tt : n_tok) * A.group, 32); };
  if (threadIdx.x == 0) {
    for (int g = 0; g < 2; ++g) {
      mbar_init(&q_ready[g], live_warps(g));
      mbar_init(&p_full[g], live_warps(g));
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(tmem_slot)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;

  const int before = it.len - it.count;                 // position of the request's first token; < 0: that many see nothing
  // Keys that a tile's rows may see, all of them together: the end of the last.
  auto end_of = [&](int last_token) { return a.visible ? it.len : min(it.len, max(0, before + last_token + 1)); };
  const int b_lo = it.chunk * it.cb;                    // first block of the range (cb is bounded: no overflow with chunk 0)
  auto blocks_to = [&](int keys) { return max(0, min(div_up(keys, kKeys) - b_lo, it.cb)); };
  const int end = end_of(it.t0 + n_tok - 1);
  const int nb = blocks_to(end);                        // blocks of the item
  const int nb0 = two ? blocks_to(end_of(it.t0 + tt - 1)) : nb;  // of the first tile
  // Blocks from this one on are not seen whole by every row: they are looked through.
  const int whole = max(0, a.visible ? before : before + it.t0 + 1) / kKeys - b_lo;
  const int first_part = max(0, min(nb, whole));

  auto wait_taken = [&](int b) { return mbar_wait(&taken[b % G::NT], (b / G::NT) & 1); };
  // K of block j may be written: the scores of the block that its slot held were issued with the job of the same group
  // before, a block earlier with two tiles, two with one.
  auto wait_k = [&](int j) {
    const int gone = j - G::KS - (two ? 1 : 2);
    return gone < 0 ? mbar_wait(k_first, 0) : wait_taken(gone);
  };

  auto unit_at = [&](int s, int w) { return smem + G::OFF_U + (s * 4 + w) * G::UNIT; };
  // V's ring: slots, a block's slot and turn, and where a slot is.
  const int slots_v = two ? G::VS : G::VS + G::VX;
  auto v_slot = [&](int b) { return two || !G::VX ? b % G::VS : b % (G::VS + G::VX); };
  auto v_turn = [&](int b) { return (two || !G::VX ? b / G::VS : b / (G::VS + G::VX)) & 1; };
  auto v_at = [&](int s) { return s < G::VS ? G::OFF_V + s * G::TILE : G::QT; };

  static_assert(!Q8 || 256 * 176 + 256 * 80 <= 512 * 128, "registers of the launch");
  static_assert(Q8 || 256 * 208 + 128 * 72 <= 384 * 168, "registers of the launch");
  if (warp >= 8) {
    if constexpr (Q8) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 9) {
      // ---------------- products ----------------
      // Jobs by block and group.  The tensor cores' queue holds some 400 cycles of work; what the waits, commits and sums
      // of a job take its warp beyond that, they stand still.  So a job has one wait (lane 1 for the weights, lane 2 for
      // the next keys, the others for the values), one commit for the scores and one for a block's K and V, and few sums.
      // (A product with V that starts on the first 64 weights: 565 us for 552, 8192 tokens of 32/8 heads.)
      constexpr uint32_t idS = Q8 ? idesc_8(false, kRows, kKeys) : idesc_16(true, kRows, kKeys, false);
      constexpr uint32_t idO = idesc_16(!Q8, kRows, HD, true);
      const uint32_t q = (uint32_t)desc_k(su32(smem), 1024), k = (uint32_t)desc_k(su32(smem + G::OFF_K), 1024);
      const uint32_t v = (uint32_t)desc_mn(su32(smem + G::OFF_V), G::SLICE, 1024);
      const uint32_t up_k = (uint32_t)(desc_k(0, 1024) >> 32), up_v = (uint32_t)(desc_mn(0, G::SLICE, 1024) >> 32);
      auto scores = [&](int slot, int g) {
        const uint32_t d = tmem + G::S_COL + g * kKeys, qa = q + (two ? g : 0) * (G::QT / 16), ka = k + slot * (G::KB / 16);
        if constexpr (Q8) issue_scores_8<HD / 32>(d, qa, ka, up_k, idS, idesc_8(true, kRows, kKeys));
        else issue_scores<HD / 16>(d, qa, ka, up_k, idS);
      };
      bool ok = true;
      for (int g = 0; ok && g < 2; ++g) {
        const int b = two ? 0 : g;
        if (b >= (two && g == 0 ? nb0 : nb)) continue;
        ok = __all_sync(0xffffffffu, mbar_wait(lane == 1 ? &q_ready[two ? g : 0] : &k_full[b % G::KS], 0));
        if (!ok) break;
        fence_after();
        scores(b % G::KS, g);
        if (elect_one()) commit(&s_full[g]);
        __syncwarp();
      }
      if (ok && elect_one()) commit(k_first);
      __syncwarp();
      const int far = two ? 1 : 2;                                   // a group's next block
      const int tail = div_up(end - (b_lo + nb - 1) * kKeys, 16);  // pages of the last one
      const uint32_t bars = su32(q_ready);
      auto bar_at = [&](const uint64_t* first, int i) { return bars + (uint32_t)((const char*)first - (const char*)q_ready) + i * 8; };
      for (int n = 0; ok && n * far < nb; ++n) {
        // (bf16: 577 us for 552, 8192 tokens of 32/8 heads, if the groups share this code; e4m3: 206 for 192, a batch of
        // drafts, if they do not.)
#pragma unroll Q8 ? 1 : 2
        for (int g = 0; g < 2; ++g) {
          const int b = two ? n : 2 * n + g, last = two && g == 0 ? nb0 : nb;  // blocks of this group end at `last`
          if (!ok || b >= last) continue;
          const bool more = b + far < last;
          const int sv = v_slot(b), sk = (b + far) % G::KS;
          uint32_t bar = bar_at(v_full, sv);
          int phase = v_turn(b);
          // v_clean completes a phase for each block looked through that came to this slot.
          if (!Q8 && b >= first_part) bar = bar_at(v_clean, sv), phase = v_turn(b - first_part);
          if (lane == 1) bar = bar_at(p_full, g), phase = n;
          if (lane == 2 && more) bar = bar_at(k_full, sk), phase = (b + far) / G::KS;
          ok = __all_sync(0xffffffffu, wait_at(bar, phase & 1));
          if (!ok) continue;
          fence_after();
          const uint32_t vb = v + (uint32_t)((v_at(sv) - G::OFF_V) / 16);
          const uint32_t d = tmem + G::O_COL + g * kRows, p = tmem + G::S_COL + g * kKeys;
          const int pages = b == nb - 1 ? tail : 8;
          issue_values(d, p, vb, up_v, idO, pages, n > 0);
          if constexpr (!Q8) issue_values(d, p + 64, vb, up_v, idO, pages, true);
          if (more) scores(sk, g);
          if (elect_one()) {
            commit(more ? &s_full[g] : &o_final[g]);
            if (!two || g == 1) commit(&taken[b % G::NT]);
          }
          __syncwarp();
        }
      }
      if (!ok && lane == 0) report(a.status, CDB_OPS_TIMEOUT);
      if (elect_one()) commit(done);  // every MMA issued above completes before TMEM is released
      __syncwarp();
      mbar_wait(done, 0);
    } else if (warp == 8 || warp == 11) {
      const int kv = warp == 8 ? 0 : 1;
      const int* bt = c.block_table + (size_t)it.seq * c.max_blocks;
      const int npg = div_up(end, 16);  // pages with keys
      bool ok = true;
      int issued = 0;
      auto block_at = [&](int pg) {
        int blk = pg < npg ? bt[pg] : -1;
        if (pg < npg && (blk < 0 || blk >= c.kv_blocks)) report(a.status, CDB_OPS_BAD_BLOCK), blk = -1;
        return blk;
      };
      // Key rows before this head's page of a block (V follows n_kv_heads pages after K).
      auto row_of = [&](int blk, int v) { return ((((long long)blk * c.n_kv_slots + a.slot) * 2 + v) * c.n_kv_heads + kh) * 16; };
      if constexpr (Q8) {
        // Warp 8: K's codes, as the bf16 ones; warp 11: V's codes.  Lane l has a page of a block.
        uint64_t pol;  // a sequence's keys are read again by its other tiles
        asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
        auto mine = [&](int j) { return lane < 8 && j < nb ? block_at((b_lo + j) * 8 + lane) : -1; };
        int blk = mine(0), s = 0, turn = 0;
        for (int j = 0; j < nb; ++j) {
          const int blk_next = mine(j + 1);  // on its way during this one
          const uint32_t there = __ballot_sync(0xffffffffu, blk >= 0);
          const long long r = row_of(max(blk, 0), kv);
          if (!kv) {
            if (j >= G::KS && !(ok = __all_sync(0xffffffffu, wait_k(j)))) break;
            if (elect_one()) mbar_arrive_tx(&k_full[s], (uint32_t)__popc(there) * (16 * 128));
            __syncwarp();
            if (blk >= 0) tma_2d(su32(smem + G::OFF_K + s * G::KB) + lane * 2048, &tmk, &k_full[s], 0, (int)r, pol);
            if (++s == G::KS) s = 0;
          } else {
            // The converters of the units have done with what was there.
            if (j >= G::NU && !(ok = __all_sync(0xffffffffu, mbar_wait(&u_empty[s * 4 + (lane & 3)], turn ^ 1)))) break;
            if (lane < 4) mbar_arrive_tx(&u_full[s * 4 + lane], (uint32_t)__popc((there >> (2 * lane)) & 3) * (16 * HD));
            __syncwarp();
            if (blk >= 0)
              bulk_1d(su32(unit_at(s, lane / 2)) + (lane & 1) * 16 * HD, static_cast<const uint8_t*>(c.pool) + r * HD, 16 * HD,
                      &u_full[s * 4 + lane / 2]);
            if (++s == G::NU) s = 0, turn ^= 1;
          }
          __syncwarp();
          issued = j + 1;
          blk = blk_next;
        }
        if (!ok && lane == 0) report(a.status, CDB_OPS_TIMEOUT);
        // Copies in flight land before the CTA may leave (at once when everything was used).
        const int slots = kv ? G::NU : G::KS;
        for (int j = max(0, issued - slots); j < issued; ++j)
          mbar_wait(kv ? &u_full[j % slots * 4 + (lane & 3)] : &k_full[j % slots], (j / slots) & 1);
      } else {
        const int slots = kv ? slots_v : G::KS;
        uint64_t* full = kv ? v_full : k_full;
        uint64_t pol;  // a sequence's keys are read again by its other tiles
        asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
        // The blocks that some rows do not see: rows behind the end and rows with a value that is not finite
        // become zeros; the latter are noted.
        auto clean = [&](int b) {
          const int s = v_slot(b), left = min(kKeys, end - (b_lo + b) * kKeys);
          if (!__all_sync(0xffffffffu, mbar_wait(&v_full[s], v_turn(b)))) return false;
          uint8_t* v = smem + v_at(s);
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            const int r = i * 32 + lane;
            uint32_t top = 0;
            if (r < left) {
#pragma unroll
              for (int x = 0; x < HD / 8; ++x) {
                const uint4 w = *reinterpret_cast<const uint4*>(v + (x / 8) * G::SLICE + r * 128 + (((x % 8) ^ (r & 7)) << 4));
                // an exponent of all ones carries into the sign's place
                top |= (((w.x & 0x7F807F80u) + 0x00800080u) | ((w.y & 0x7F807F80u) + 0x00800080u) |
                        ((w.z & 0x7F807F80u) + 0x00800080u) | ((w.w & 0x7F807F80u) + 0x00800080u));
              }
            }
            const bool bad = (top & 0x80008000u) != 0;
            if (bad || r >= left) {
#pragma unroll
              for (int x = 0; x < G::NX * 8; ++x)
                *reinterpret_cast<uint4*>(v + (x / 8) * G::SLICE + r * 128 + (x % 8) * 16) = make_uint4(0, 0, 0, 0);
            }
            const uint32_t bits = __ballot_sync(0xffffffffu, bad);
            if (lane == 0) bad_keys[s * 4 + i] = bits;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_clean[s]);
          return true;
        };
        int cleaned = kv ? first_part : nb;
        for (int j = 0; j < nb; ++j) {
          const int s = j % slots;
          const uint32_t to = su32(smem + (kv ? v_at(s) : G::OFF_K + s * G::TILE));
          const int blk = lane < 8 ? block_at((b_lo + j) * 8 + lane) : -1;
          const uint32_t there = __ballot_sync(0xffffffffu, blk >= 0);
          // A slot to be filled again may hold a block that waits to be looked through.
          while (cleaned < nb && cleaned <= j - slots && ok) ok = clean(cleaned++);
          if (!ok) break;
          if (j >= slots && !(ok = __all_sync(0xffffffffu, kv ? wait_taken(j - slots) : wait_k(j)))) break;
          if (elect_one()) mbar_arrive_tx(&full[s], (uint32_t)__popc(there) * (G::NX * 16 * 128));
          __syncwarp();
          for (int i = 0; i < 8; ++i) {
            const int bi = __shfl_sync(0xffffffffu, blk, i);
            if (bi >= 0 && elect_one()) {
              const int y = (int)row_of(bi, kv);
#pragma unroll
              for (int x = 0; x < G::NX; ++x)
                tma_2d(to + x * G::SLICE + i * 2048, &tmk, &full[s], x * 128, y, pol);
            }
            __syncwarp();
          }
          issued = j + 1;
        }
        while (cleaned < nb && ok) ok = clean(cleaned++);
        if (!ok && lane == 0) report(a.status, CDB_OPS_TIMEOUT);
        for (int j = max(0, issued - slots); j < issued; ++j) mbar_wait(&full[j % slots], (j / slots) & 1);
      }
    } else if (Q8 && warp >= 12) {
      // ---------------- code converters ----------------
      // V to fp16, 32 keys of a block for each warp: 16 codes to 32 bytes at a time; lanes of the upper half of a row
      // store their second piece first, so that the stores of eight lanes meet every bank once.
      const int w = warp - 12;
      constexpr int C = HD / 16, CL = HD == 96 ? 8 : C;  // of a row: pieces, lanes
      constexpr int B = CL < 4 ? CL : 4;                 // passes whose loads are on their way together
      // The scales of this lane's key go ahead of the codes, two blocks, so that scores need not wait for V; they are
      // on their way for a block before that.
      const int* bt = c.block_table + (size_t)it.seq * c.max_blocks;
      const int npg = div_up(end, 16);
      auto pool_block = [&](int b) {
        const int pg = (b_lo + b) * 8 + w * 2 + lane / 16, blk = b < nb && pg < npg ? bt[pg] : -1;
        return blk < c.kv_blocks ? blk : -1;  // reported by the producers
      };
      float k_scale = 0.f, v_scale = 0.f;
      auto fetch = [&](int blk) {
        const long long at = (((long long)max(blk, 0) * c.n_kv_slots + a.slot) * 2 * c.n_kv_heads + kh) * 16 + lane % 16;
        k_scale = blk >= 0 ? c.scales[at] : 0.f;
        v_scale = blk >= 0 ? c.scales[at + c.n_kv_heads * 16] : 0.f;
      };
      uint32_t bad_scales[3] = {0, 0, 0};  // keys of blocks b, b + 1 and b + 2 whose value scale is not finite
      auto put = [&](int b) {
        float* sc = reinterpret_cast<float*>(smem + G::OFF_SC) + (b % G::NSC) * G::SCN;
        const bool bad = b >= first_part && !(fabsf(v_scale) < INFINITY);
        // Keys behind the end, and in blocks looked through those whose scale is not finite, take no part.
        const float fv = bad || lane >= end - (b_lo + b) * kKeys - w * 32 ? 0.f : v_scale;
        sc[w * 32 + lane] = k_scale;
        sc[kKeys + w * 32 + lane] = fv;
        sc[2 * kKeys + w * 32 + lane] = __log2f(fabsf(fv));
        const uint32_t fm = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(fv)));
        if (lane == 0) sc[3 * kKeys + w] = fmaxf(__log2f(__uint_as_float(fm)), -82.f);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_full[b % G::NSC]);
        return __ballot_sync(0xffffffffu, bad);
      };
      const int first_ids = pool_block(0), second_ids = pool_block(1), third_ids = pool_block(2);
      fetch(first_ids);
      bad_scales[0] = put(0);
      fetch(second_ids);
      if (nb > 1) bad_scales[1] = put(1);
      fetch(third_ids);
      int ahead = pool_block(3), s = 0, turn = 0;
      bool ok = true;
      for (int b = 0; b < nb; ++b) {
        const int slot = v_slot(b);
        // Lane 1 waits for the slot, lane 2 for the place of the scales two blocks on, the others for the codes.
        if (!(ok = __all_sync(0xffffffffu, lane == 1 && b >= slots_v      ? wait_taken(b - slots_v)
                                           : lane == 2 && b + 2 >= G::NSC ? wait_taken(b + 2 - G::NSC)
                                                                          : mbar_wait(&u_full[s * 4 + w], turn))))
          break;
        if (b + 2 < nb) {
          bad_scales[2] = put(b + 2);
          fetch(ahead);
          ahead = pool_block(b + 4);
        }
        const uint8_t* raw = unit_at(s, w);
        uint8_t* to = smem + v_at(slot);
        const int left = end - (b_lo + b) * kKeys - w * 32;  // keys of this unit that are there
        const bool part = b >= first_part;
        const int x = lane % CL;
#pragma unroll 1
        for (int i0 = 0; i0 < CL; i0 += B) {
          uint4 v[B];
#pragma unroll
          for (int i = 0; i < B; ++i) {
            const int key = (i0 + i) * (32 / CL) + lane / CL;
            v[i] = make_uint4(0, 0, 0, 0);
            if (x < C && key < left) v[i] = *reinterpret_cast<const uint4*>(raw + key * HD + x * 16);
          }
          if (part) {
#pragma unroll
            for (int i = 0; i < B; ++i) {
              // A code of NaN has all seven lower bits.  Every element of a key that holds one, or whose scale is not
              // finite, becomes 0.
              const int key = (i0 + i) * (32 / CL) + lane / CL;
              const uint32_t f = ((v[i].x & 0x7F7F7F7Fu) + 0x01010101u) | ((v[i].y & 0x7F7F7F7Fu) + 0x01010101u) |
                                 ((v[i].z & 0x7F7F7F7Fu) + 0x01010101u) | ((v[i].w & 0x7F7F7F7Fu) + 0x01010101u);
              const uint32_t found = __ballot_sync(0xffffffffu, (f & 0x80808080u) != 0);
              const bool bad = key < left && (((found >> (lane / CL * CL)) & ((1u << CL) - 1)) || ((bad_scales[0] >> key) & 1));
              if (bad) v[i] = make_uint4(0, 0, 0, 0);
              if (x == 0) bad_bytes[slot * kKeys + w * 32 + key] = bad;
            }
          }
#pragma unroll
          for (int i = 0; i < B; ++i) {
            if (x < C) {
              const int r = w * 32 + (i0 + i) * (32 / CL) + lane / CL;
              uint8_t* d = to + (x / 4) * G::SLICE + r * 128;
              const uint4 lo = make_uint4(widen(v[i].x), widen_hi(v[i].x), widen(v[i].y), widen_hi(v[i].y));
              const uint4 hi = make_uint4(widen(v[i].z), widen_hi(v[i].z), widen(v[i].w), widen_hi(v[i].w));
              const int c0 = (x % 4) * 2, sw = r & 7;
              const bool swap = x >= 4;
              *reinterpret_cast<uint4*>(d + (((c0 + swap) ^ sw) << 4)) = swap ? hi : lo;
              *reinterpret_cast<uint4*>(d + (((c0 + !swap) ^ sw) << 4)) = swap ? lo : hi;
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&u_empty[s * 4 + w]);
          mbar_arrive(&v_full[slot]);
        }
        if (++s == G::NU) s = 0, turn ^= 1;
        bad_scales[0] = bad_scales[1], bad_scales[1] = bad_scales[2];
      }
      if (!ok && lane == 0) report(a.status, CDB_OPS_TIMEOUT);
    }
  } else {
    if constexpr (Q8) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ---------------- softmax groups ----------------
    const int q4 = warp & 3, g = warp >> 2;
    const bool works = q4 < live_warps(g);
    const int r = q4 * 32 + lane;
    const int tile = two ? g : 0;
    const int tk = it.t0 + tile * tt + r / A.group;  // token of this row
    const int head = kh * A.group + r % A.group;
    const bool live = r < tt * A.group && tk < it.count;
    const long long row = it.row0 + (live ? tk : 0);
    // Prompt: the last key of this row.  Draft: the first key of the request's rows, which the mask is for.
    const int lim = a.visible ? before : live ? before + tk : -1;
    const int nodes = live ? it.count : 0;
    const uint32_t* mask = a.visible ? reinterpret_cast<const uint32_t*>(a.visible + row * a.mask_words) : nullptr;
    const bool turn_round = a.scale < 0.f;  // a negative factor turns the scores around first
    float scale = fabsf(a.scale) * 1.4426950408889634f;
    constexpr float kTau = 8.f;  // rescale O only when the row maximum grows by more than 2^8
    const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
    const uint32_t to = trow + G::O_COL + g * kRows, ts = trow + G::S_COL + g * kKeys;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    {
      // This warp's rows of q into the tile, swizzled; with one tile the first group does it.  Lanes that follow one
      // another take pieces of 16 bytes that do, P of a row (a thread for a row: 1.5 us more for each item).
      constexpr int P = HD / 8, L = HD == 96 ? 16 : P, R = 32 / L;  // pieces, lanes of a row, rows at a time
      uint8_t* dst = smem + tile * G::QT;
      const int x = lane % L, rows_here = min(tt * A.group, (it.count - it.t0 - tile * tt) * A.group) - q4 * 32;
      if (works && (two || g == 0)) {
        // Token and head of this lane's row, R rows further in each pass.
        const int step_t = R / A.group, step_h = R - step_t * A.group;
        int rr = lane / L, t = (q4 * 32 + rr) / A.group, h = q4 * 32 + rr - t * A.group, loaded = rr;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + (long long)(it.row0 + it.t0 + tile * tt) * a.ldq +
                                   (size_t)kh * A.group * HD + x * 8;
        auto load_q = [&] {
          const uint4 v = x < P && loaded < rows_here ? *reinterpret_cast<const uint4*>(src + (long long)t * a.ldq + (size_t)h * HD)
                                                      : make_uint4(0, 0, 0, 0);
          t += step_t, h += step_h, loaded += R;
          if (h >= A.group) h -= A.group, ++t;
          return v;
        };
        if constexpr (!Q8) {
          uint4 piece[L];
#pragma unroll
          for (int i = 0; i < L; ++i) piece[i] = load_q();
#pragma unroll
          for (int i = 0; i < L; ++i) {
            const int row_t = q4 * 32 + rr + i * R;  // of the tile
            if (x < P)
              st_shared_v4(su32(dst + (x / 8) * G::SLICE + row_t * 128 + (((x % 8) ^ (row_t & 7)) << 4)), piece[i].x, piece[i].y,
                           piece[i].z, piece[i].w);
          }
        } else {
          // e4m3: each row times a power of two, which takes its largest element into [128, 256), in two parts, what
          // the first leaves in the second.  Elements from 2^-6 on, 2^-14 of the largest, are exact; of smaller ones the
          // first part leaves up to 2^-10, and of that the second up to 2^-14, 2^-21 of the largest.  A short loop:
          // its instructions are fetched once for every item (unrolled: 5 us more).
          constexpr int B = L < 4 ? L : 4;
          uint4 piece[B];
#pragma unroll
          for (int i = 0; i < B; ++i) piece[i] = load_q();
#pragma unroll 1
          for (int i0 = 0; i0 * R < rows_here && i0 < L; i0 += B) {
            uint4 later[B];
#pragma unroll
            for (int i = 0; i < B; ++i) later[i] = load_q();
#pragma unroll
            for (int i = 0; i < B; ++i, rr += R) {
              const int row_t = q4 * 32 + rr;
              uint32_t top = largest_bf16(piece[i]);
#pragma unroll
              for (int o = 1; o < L; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
              const uint32_t eb = (top & 0x7F80u) << 16;
              float down = 1.f, its_up = 1.f;
              if (eb == 0x7F800000u) {
                down = NAN;  // infinite or NaN; the conversion would make an infinite element a finite one
              } else if (eb >= 0x04000000u) {  // else zero or below 2^-119
                down = __uint_as_float(0x82800000u - eb);
                its_up = __uint_as_float(eb - 0x03800000u);
              }
              if (x == 0) q_up[tile * kRows + row_t] = its_up;
              uint32_t one[2], rest[2];
              split_q(piece[i].x, piece[i].y, down, one[0], rest[0]);
              split_q(piece[i].z, piece[i].w, down, one[1], rest[1]);
              if (x < P) {
                const uint32_t at = su32(dst + row_t * 128) + (((x / 2) ^ (row_t & 7)) << 4) + (x & 1) * 8;
                asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(one[0]), "r"(one[1]) : "memory");
                asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at + G::SLICE), "r"(rest[0]), "r"(rest[1]) : "memory");
              }
            }
#pragma unroll
            for (int i = 0; i < B; ++i) piece[i] = later[i];
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_ready[tile]);
      }
      float up = 1.f;
      if (Q8 && works) {
        ok = __all_sync(0xffffffffu, mbar_wait(&q_ready[tile], 0));  // the first group's
        if (live) up = q_up[tile * kRows + r];
      }
      scale = fmaxf(scale * up, 1e-37f);  // not 0: a masked score stays -inf
    }
    int n = 0;  // jobs of this group so far
    const int n_jobs = two ? (g ? nb : nb0) : (nb + 1 - g) / 2;
    for (; works && ok && n < n_jobs; ++n) {
      const int b = two ? n : 2 * n + g;
      const int k0 = (b_lo + b) * kKeys;
      float sv[128];
      auto load = [&] {
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&s_full[g], n & 1)))) return;
        fence_after();
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32_ahead(ts + i * 32, sv + i * 32);
        tmem_arrived();
#pragma unroll
        for (int i = 0; i < 4; ++i) pin32(sv + i * 32);
        if (turn_round) {
#pragma unroll
          for (int k = 0; k < 128; ++k) sv[k] = -sv[k];
        }
      };
      // Scores that the row does not see become -inf; those of keys whose value is not finite NaN.
      auto mask_out = [&] {
        if (b < first_part) return true;
        const int slot = v_slot(b);
        const bool there = Q8 ? mbar_wait(&v_full[slot], v_turn(b)) : mbar_wait(&v_clean[slot], v_turn(b - first_part));
        if (!(ok = __all_sync(0xffffffffu, there))) return false;
        // Four keys of a lane are looked at at once; hardly ever is one bad.
        const bool some = Q8 && __any_sync(0xffffffffu, bad_keys[slot * (kKeys / 4) + lane] != 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = seen(k0 + i * 32, lim, mask, nodes);
          const uint32_t bits = !Q8 ? bad_keys[slot * 4 + i]
                                : some ? __ballot_sync(0xffffffffu, bad_bytes[slot * kKeys + i * 32 + lane] != 0) : 0u;
          const uint32_t bad = bits & w;
          if (!__all_sync(0xffffffffu, w == ~0u)) {
#pragma unroll
            for (int k = 0; k < 32; ++k) sv[i * 32 + k] = (w >> k) & 1 ? sv[i * 32 + k] : -INFINITY;
          }
          if (__any_sync(0xffffffffu, bad != 0)) {
#pragma unroll
            for (int k = 0; k < 32; ++k) sv[i * 32 + k] = (bad >> k) & 1 ? NAN : sv[i * 32 + k];
          }
        }
        return true;
      };
      auto greatest = [&] {
        float x4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 128; k += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) x4[e] = max3(x4[e], sv[k + 2 * e], sv[k + 2 * e + 1]);
        return fmaxf(fmaxf(x4[0], x4[1]), fmaxf(x4[2], x4[3])) * scale;
      };
      // Moves the row to the reference `to_m`; O holds the group's earlier blocks, whose products the commit of these
      // scores covers, against the old one.
      auto move = [&](float to_m) {
        const float f = m == -INFINITY ? 0.f : ex2(m - to_m);
        l *= f;
        m = to_m;
        if (n == 0) return;
#pragma unroll 1
        for (int c0 = 0; c0 < HD; c0 += 16) {
          float v[16];
          tmem_ld16(to + c0, v);
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] *= f;
          tmem_st16(to + c0, reinterpret_cast<const uint32_t*>(v));
        }
      };
      if constexpr (Q8) {
        const uint32_t scales = su32(smem + G::OFF_SC + (b % G::NSC) * G::SCN * 4);
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sc_full[b % G::NSC], (b / G::NSC) & 1)))) break;
        load();
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const float4 f = ld_shared_v4(scales + k * 16);
          unpair(mul2(pair(sv[4 * k], sv[4 * k + 1]), pair(f.x, f.y)), sv[4 * k], sv[4 * k + 1]);
          unpair(mul2(pair(sv[4 * k + 2], sv[4 * k + 3]), pair(f.z, f.w)), sv[4 * k + 2], sv[4 * k + 3]);
        }
        if (!mask_out()) break;
        // No weight times scale may pass 2^15 (fp16 ends at 2^16), no weight 2^97.  The largest score with the largest
        // scale (2^-82 if that is less) bounds them; only where that passes is the largest product looked for.
        const float4 vm = ld_shared_v4(scales + 3 * kKeys * 4);
        const float mx = greatest();
        if (__any_sync(0xffffffffu, mx + fmaxf(fmaxf(vm.x, vm.y), fmaxf(vm.z, vm.w)) > m + 15.f)) {
          float t4[4] = {mx - 82.f, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float4 f = ld_shared_v4(scales + 2 * kKeys * 4 + k * 16);
            t4[k % 4] = max3(t4[k % 4], fmaf(sv[4 * k], scale, f.x), fmaf(sv[4 * k + 1], scale, f.y));
            t4[k % 4] = max3(t4[k % 4], fmaf(sv[4 * k + 2], scale, f.z), fmaf(sv[4 * k + 3], scale, f.w));
          }
          float tm = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) - 8.f;
          tm = tm > m + 7.f ? tm : m;
          if (__any_sync(0xffffffffu, tm != m)) move(tm);
        }
        const float mm = m == -INFINITY ? 0.f : m;
        const uint64_t s2 = pair(scale, scale), m2 = pair(-mm, -mm);
        uint64_t l2[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const int k = i * 32 + 2 * e;
            float x0, x1, x2, x3;
            unpair(fma2(pair(sv[k], sv[k + 1]), s2, m2), x0, x1);
            unpair(fma2(pair(sv[k + 2], sv[k + 3]), s2, m2), x2, x3);
            x0 = ex2(x0), x1 = ex2(x1), x2 = ex2(x2), x3 = ex2(x3);
            l2[0] = add2(l2[0], pair(x0, x1));
            l2[1] = add2(l2[1], pair(x2, x3));
            const float4 f = ld_shared_v4(scales + (kKeys + k) * 4);
            unpair(mul2(pair(f.x, f.y), pair(x0, x1)), x0, x1);
            unpair(mul2(pair(f.z, f.w), pair(x2, x3)), x2, x3);
            p[e] = pack_f16(x0, x1);
            p[e + 1] = pack_f16(x2, x3);
          }
          tmem_st16(ts + i * 16, p);
        }
        float la, lb, lc, ld;
        unpair(l2[0], la, lb);
        unpair(l2[1], lc, ld);
        l += (la + lb) + (lc + ld);
      } else {
        load();
        if (!ok || !mask_out()) break;
        const float mx = greatest();
        const float mnew = mx > m + kTau ? mx : m;
        if (__any_sync(0xffffffffu, mnew != m)) move(mnew);
        const float mm = m == -INFINITY ? 0.f : m;
        const uint64_t s2 = pair(scale, scale), m2 = pair(-mm, -mm);
        uint64_t l2[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t p[16], low[16];
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const int k = i * 32 + 2 * e;
            float x0, x1, x2, x3;
            unpair(fma2(pair(sv[k], sv[k + 1]), s2, m2), x0, x1);
            unpair(fma2(pair(sv[k + 2], sv[k + 3]), s2, m2), x2, x3);
            x0 = ex2(x0), x1 = ex2(x1), x2 = ex2(x2), x3 = ex2(x3);
            l2[0] = add2(l2[0], pair(x0, x1));
            l2[1] = add2(l2[1], pair(x2, x3));
            p[e] = pack_bf16(x0, x1);
            p[e + 1] = pack_bf16(x2, x3);
            low[e] = bf16_rest(x0, x1, p[e]);
            low[e + 1] = bf16_rest(x2, x3, p[e + 1]);
          }
          tmem_st16(ts + i * 16, p);
          tmem_st16(ts + 64 + i * 16, low);
        }
        float la, lb, lc, ld;
        unpair(l2[0], la, lb);
        unpair(l2[1], lc, ld);
        l += (la + lb) + (lc + ld);
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[g]);
    }
    if (ok && n > 0) ok = __all_sync(0xffffffffu, mbar_wait(&o_final[g], 0));
    if (!works) ok = false;
    if (works && !ok && lane == 0) report(a.status, CDB_OPS_TIMEOUT);
    fence_after();
    const size_t pi = (((size_t)blockIdx.y * c.n_kv_heads + kh) * 256) + tile * kRows + r;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row * a.ldo + (size_t)head * HD;
    auto store = [&](int c0, float* v, float f) {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] *= f;
      if (!live) {
      } else if (it.chunks > 1) {
        float* po = A.part_o + pi * HD + c0;
#pragma unroll
        for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4*>(po + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
      } else {
#pragma unroll
        for (int e = 0; e < 16; e += 8)
          *reinterpret_cast<uint4*>(out + c0 + e) = make_uint4(pack_bf16(v[e], v[e + 1]), pack_bf16(v[e + 2], v[e + 3]),
                                                               pack_bf16(v[e + 4], v[e + 5]), pack_bf16(v[e + 6], v[e + 7]));
      }
    };
    if (two) {
      if (ok) {
        const float r1 = Q8 ? unit_sum(m, l) : 1.f;
        const float f = it.chunks > 1 ? r1 : l == 0.f ? 0.f : r1 / l;
#pragma unroll 1
        for (int c0 = 0; c0 < HD; c0 += 16) {
          float v[16];
          if (n > 0) {
            tmem_ld16(to + c0, v);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0.f;
          }
          store(c0, v, f);
        }
        if (it.chunks > 1) A.part_ml[pi] = make_float2(m, l);
      }
    } else {
      // The groups' halves: each has waited for its own accumulator's last product, and reads the other's too, which
      // these fences order behind the other group's wait.
      if (works) xch[g * kRows + r] = make_float2(m, l);
      fence_before();
      asm volatile("bar.sync 1, 256;" ::: "memory");
      fence_after();
      if (ok) {
        float2 e0 = xch[r], e1 = xch[kRows + r];
        const float r0 = Q8 ? unit_sum(e0.x, e0.y) : 1.f, r1 = Q8 ? unit_sum(e1.x, e1.y) : 1.f;
        const float mj = fmaxf(e0.x, e1.x);
        const float f0 = e0.x == -INFINITY ? 0.f : ex2(e0.x - mj), f1 = e1.x == -INFINITY ? 0.f : ex2(e1.x - mj);
        const float lj = e0.y * f0 + e1.y * f1;
        const float f = it.chunks > 1 ? 1.f : lj == 0.f ? 0.f : 1.f / lj;
        const uint32_t t0 = trow + G::O_COL;
#pragma unroll 1
        for (int c0 = g * 16; c0 < HD; c0 += 32) {
          float v[16], w[16];
          if (nb > 0) tmem_ld16(t0 + c0, v);
          if (nb > 1) tmem_ld16(t0 + kRows + c0, w);
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = (nb > 0 ? v[e] * (f0 * r0) : 0.f) + (nb > 1 ? w[e] * (f1 * r1) : 0.f);
          store(c0, v, f);
        }
        if (it.chunks > 1 && g == 0) A.part_ml[pi] = make_float2(mj, lj);
      }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 9) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

// Adds up the ranges of keys of the requests that were cut.  A warp takes a token's row of one head at a time; a double
// tile and KV head has kJoin CTAs of 8 warps.  Latency bounds it, and CTAs without anything to add up (whole call, a
// batch of drafts / chunks behind cached tokens: 161 / 155 us with 32 CTAs, a row for each warp, 156 / 148 with 16, 169 /
// 144 with 8).
constexpr int kJoin = 16;
template <int HD>
__global__ void __launch_bounds__(256) k_prompt_join(const __grid_constant__ Args A) {
  pdl_wait();
  pdl_trigger();
  const int4 info = A.info[blockIdx.x];
  const int chunks = info.w & 0xFFFF, nt = info.w >> 16;
  if (chunks < 2) return;
  const cdb_prompt_attention_args& a = A.a;
  const int lane = threadIdx.x & 31, kh = blockIdx.y;
  const int row0 = a.row_start[info.x], count = a.row_start[info.x + 1] - row0;
  constexpr int E = HD / 32;
  const size_t step = (size_t)nt * a.cache.n_kv_heads * 256;
  for (int w = blockIdx.z * 8 + (threadIdx.x >> 5); w < 2 * kRows; w += 8 * kJoin) {
    const int tile = w / kRows, r = w % kRows, tk = info.y + tile * A.tokens + r / A.group;
    if (r >= A.tokens * A.group || tk >= count) continue;
    const size_t p0 = ((size_t)info.z * a.cache.n_kv_heads + kh) * 256 + w;
    float mj = -INFINITY;
    for (int k = lane; k < chunks; k += 32) mj = fmaxf(mj, A.part_ml[p0 + k * step].x);
#pragma unroll
    for (int o = 16; o > 0; o /= 2) mj = fmaxf(mj, __shfl_xor_sync(0xffffffffu, mj, o));
    float l = 0.f, v[E] = {};
#pragma unroll 4
    for (int k = 0; k < chunks; ++k) {
      const float2 ml = A.part_ml[p0 + k * step];
      const float f = ml.x == -INFINITY ? 0.f : tc::ex2(ml.x - mj);
      const float* po = A.part_o + (p0 + k * step) * HD + lane * E;
      l = fmaf(ml.y, f, l);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = fmaf(po[e], f, v[e]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (size_t)(row0 + tk) * a.ldo + (size_t)(kh * A.group + r % A.group) * HD + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] = __float2bfloat16_rn(v[e] * inv);
  }
}

struct Plan {
  int group, tokens, tiles, cut;
  size_t o_bytes, ml_bytes, info_bytes;
};

Plan plan(int rows, int requests, int n_heads, int n_kv_heads, int head_dim, int max_ctx) {
  Plan p = {};
  p.group = n_heads / n_kv_heads;
  p.tokens = kRows / p.group;
  // sum of ceil(count / (2 tokens)) over requests that have rows
  p.tiles = (int)std::min<long long>(rows, rows / (2 * p.tokens) + requests);
  // Cut only where a call may leave SMs without work for long: few items, and enough keys to cut.
  const long long items = (long long)p.tiles * n_kv_heads;
  const bool may = max_ctx > kMinBlocks * kKeys && items < kCutBelow;
  p.cut = may ? (kItems + n_kv_heads - 1) / n_kv_heads : 0;
  const size_t cells = may ? (size_t)(p.tiles + p.cut) * n_kv_heads * 256 : 0;
  p.o_bytes = cells * head_dim * 4;
  p.ml_bytes = cells * 8;
  p.info_bytes = may ? ((size_t)p.tiles * 16 + 255) / 256 * 256 : 0;
  return p;
}

template <int HD, bool Q8>
cudaError_t launch(cudaStream_t s, const Args& A) {
  using G = Geo<HD, Q8>;
  const cdb_paged_cache& c = A.a.cache;
  CUtensorMap tk = {};
  const uint64_t rows = (uint64_t)c.kv_blocks * c.n_kv_slots * 2 * c.n_kv_heads * 16;
  // A page is a box of 16 rows of 128 bytes; what a row has less is filled with zeros.
  constexpr int kRow = HD * (Q8 ? 1 : 2);
  if (!tmap_u8_2d(&tk, c.pool, kRow, rows, kRow, 128, 16, 128)) return cudaErrorInvalidValue;
  static bool set[kMaxDevices] = {};
  const int dev = current_device();
  if (!set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(k_prompt<HD, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)G::SMEM);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  count_launch();
  cudaError_t e = launch_pdl(k_prompt<HD, Q8>, dim3(c.n_kv_heads, A.tiles + A.cut), dim3(G::THREADS), G::SMEM, s, tk, A);
  if (e != cudaSuccess || !A.cut) return e;
  count_launch();
  return launch_pdl(k_prompt_join<HD>, dim3(A.tiles, c.n_kv_heads, kJoin), dim3(256), 0, s, A);
}

}  // namespace pa

size_t prompt_attention_workspace(int rows, int requests, int n_heads, int n_kv_heads, int head_dim, int max_ctx) {
  // Smaller calls may cut where this one does not: the most tiles that a call that cuts has.
  const pa::Plan p = pa::plan(rows, requests, n_heads, n_kv_heads, head_dim, max_ctx);
  if (max_ctx <= pa::kMinBlocks * pa::kKeys) return 256;
  const size_t tiles = std::min(p.tiles, (pa::kCutBelow - 1) / n_kv_heads);
  const size_t cells = (tiles * n_kv_heads + pa::kItems + n_kv_heads) * 256;
  return cells * (head_dim * 4 + 8) + tiles * 16 + 512;
}

cudaError_t launch_prompt_attention(cudaStream_t s, const cdb_prompt_attention_args& a) {
  const pa::Plan p = pa::plan(a.rows, a.requests, a.n_heads, a.cache.n_kv_heads, a.cache.head_dim, a.max_ctx);
  pa::Args A;
  A.a = a;
  A.group = p.group;
  A.tokens = p.tokens;
  A.cut = p.cut;
  A.tiles = p.tiles;
  A.info = static_cast<int4*>(a.workspace);
  A.part_o = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + p.info_bytes);
  A.part_ml = reinterpret_cast<float2*>(reinterpret_cast<char*>(A.part_o) + p.o_bytes);
  const bool q8 = a.cache.dtype == CDB_E4M3;
  switch (a.cache.head_dim) {
    case 32: return q8 ? pa::launch<32, true>(s, A) : pa::launch<32, false>(s, A);
    case 64: return q8 ? pa::launch<64, true>(s, A) : pa::launch<64, false>(s, A);
    case 96: return q8 ? pa::launch<96, true>(s, A) : pa::launch<96, false>(s, A);
    case 128: return q8 ? pa::launch<128, true>(s, A) : pa::launch<128, false>(s, A);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace cdb
