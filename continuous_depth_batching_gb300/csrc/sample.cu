// Sampling with temperature, top-k, top-p and min-p from given uniform numbers
// (include/cdb_ops.h has the definition).
//
// One thread-block cluster per row, each CTA holding a contiguous slice of the
// logits in shared memory, so the row is read from HBM once.  Every decision
// is a comparison of masses, and a mass is a sum of 64-bit fixed-point weights
// (unit 2^-44 of the row's largest weight): integer sums do not depend on the
// order, so the result does not depend on the cluster size or on other rows.
// A weight is exp((x - m) / T) to about 2^-36 (weight()): with 2^-24, an error
// of plain fp32, the running sum over a large vocabulary is off by enough that
// one draw in some ten thousand would cross a border.
//
// Thresholds (top-k by count, top-p by mass) come from a radix search without
// sorting: a first histogram over 1024 equal steps of m - x, then histograms
// over the ordered bit patterns of the chosen bin, until the bin holds exactly
// what is needed or a single value.  Each CTA adds up its slice in its own
// shared memory, all CTAs of the cluster then read one another's histograms
// (distributed shared memory) and find the same bin; two histogram buffers
// leave one cluster barrier per step.
#include <cooperative_groups.h>

#include <algorithm>

#include "../../include/cdb.h"
#include "../../include/cdb_ops.h"
#include "common.cuh"
#include "kernels.cuh"
#include "sample.h"

namespace cg = cooperative_groups;

namespace cdb {
namespace smp {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;       // two per thread
constexpr int kMaxCluster = 8;
constexpr int kUnit = 44;         // fixed-point weights: 2^kUnit is weight 1
constexpr int kTab = 64;          // 2^(j/64), j = 0..63

// 2^(j/64) in units of 2^-44, rounded.
__constant__ unsigned long long kExp2[kTab] = {
    17592186044416ull, 17783752390528ull, 17977404757381ull, 18173165860252ull,
    18371058661769ull, 18571106374610ull, 18773332464219ull, 18977760651566ull,
    19184414915921ull, 19393319497675ull, 19604498901178ull, 19817977897613ull,
    20033781527906ull, 20251935105661ull, 20472464220127ull, 20695394739203ull,
    20920752812471ull, 21148564874263ull, 21378857646762ull, 21611658143136ull,
    21846993670708ull, 22084891834158ull, 22325380538761ull, 22568487993661ull,
    22814242715178ull, 23062673530157ull, 23313809579344ull, 23567680320808ull,
    23824315533396ull, 24083745320225ull, 24346000112214ull, 24611110671650ull,
    24879108095804ull, 25150023820570ull, 25423889624159ull, 25700737630824ull,
    25980600314626ull, 26263510503246ull, 26549501381838ull, 26838606496915ull,
    27130859760289ull, 27426295453047ull, 27724948229574ull, 28026853121614ull,
    28332045542385ull, 28640561290725ull, 28952436555301ull, 29267707918846ull,
    29586412362452ull, 29908587269910ull, 30234270432094ull, 30563500051394ull,
    30896314746195ull, 31232753555409ull, 31572855943056ull, 31916661802889ull,
    32264211463077ull, 32615545690931ull, 32970705697691ull, 33329733143360ull,
    33692670141585ull, 34059559264602ull, 34430443548229ull, 34805366496913ull,
};

// What each CTA tells the others (one record per CTA, written remotely).
struct Note {
  float mx, mn;  // largest logit, smallest above -inf
  int first;     // lowest index of mx
  int pad;
};
struct Tail {
  unsigned long long mass;  // kept mass strictly above the threshold value
  unsigned int ties;        // entries equal to the threshold value
  unsigned int pad;
};

struct Shared {
  unsigned int hist[2][4][kBins];  // count, then the low, middle and high 16 bits of the masses
  uint2 tab[kTab];                 // 2^(j/64) * 2^44 (low, high words)
  int tab30[kTab];                 // 2^(j/64) * 2^30
  Note note[kMaxCluster];
  Tail tail[kMaxCluster];
  unsigned long long wm[kWarps];   // per-warp values of the scans
  unsigned int wc[kWarps];
  unsigned long long found_m;
  unsigned int found_c, found_bin, found_n;
  unsigned int lo, hi;
  float fmx[kWarps], fmn[kWarps];
  int fi[kWarps];
  int token;
};

// Ordered bit pattern of a float (never NaN); bf16 values use its upper half.
__device__ __forceinline__ unsigned int order_bits(float x) {
  const unsigned int b = __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float from_order(unsigned int k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// exp((x - m) c) 2^kUnit as an integer, c = ch + cl = 1 / T.  d = x - m as an
// exact sum of two floats (Knuth's two-sum), y = d c to about 2^-46 of its
// value; y = t ln2/64 + r with t an integer (Cody and Waite's two-part
// constant) and |r| < 0.0055; exp(r) - 1 = r + r^2/2 + r^3/6 + r^4/24 (the next
// term is below 2^-44) in units of 2^-36, times 2^(j/64) from the table,
// shifted by the integer part.  About 45 fp32 and integer instructions: fp64
// ones run at 1/64 of the fp32 rate here.
struct Weigher {
  float m, ch, cl;
  const uint2* tab;
  const int* tab30;
  __device__ __forceinline__ unsigned long long operator()(float x) const {
    const float d = __fsub_rn(x, m);
    if (d == 0.f) return 1ull << kUnit;
    const float db = __fsub_rn(d, x);
    const float dl = __fadd_rn(__fsub_rn(x, __fsub_rn(d, db)), __fsub_rn(-m, db));
    const float p = __fmul_rn(d, ch);
    if (!(p > -31.5f)) return 0;
    const float pl = __fmaf_rn(d, ch, -p) + __fmaf_rn(d, cl, dl * ch);
    constexpr float kMagic = 12582912.f;                   // 1.5 * 2^23: the sum's low bits are the rounded integer
    constexpr float kInv = 92.332482616893657f;            // 64 / ln 2
    constexpr float kC1 = 2839.f / 262144.f;               // ln2/64 to 12 bits: t C1 is exact (|t| < 2^12)
    constexpr float kC2 = 4.9915913977005e-07f;            // ln2/64 - kC1
    const float tm = __fmaf_rn(p, kInv, kMagic);
    const int t = __float_as_int(tm) - 0x4B400000;
    const float tf = __fsub_rn(tm, kMagic);
    const float r1 = __fmaf_rn(-tf, kC1, p);               // exact
    const float u2 = __fmul_rn(tf, kC2);
    const float rh = __fsub_rn(r1, u2);
    const float rb = __fsub_rn(rh, r1);
    const float re = __fadd_rn(__fsub_rn(r1, __fsub_rn(rh, rb)), __fsub_rn(-u2, rb));
    const float rl = re - __fmaf_rn(tf, kC2, -u2) + pl;    // r = rh + rl
    const float q = rh * rh * (0.5f + rh * (0.16666667f + rh * 0.041666668f));
    constexpr float k36 = 68719476736.f;                   // 2^36
    const int is = __float2int_rn(rh * k36) + (__float_as_int(__fmaf_rn(rl + rh * rl + q, k36, kMagic)) - 0x4B400000);
    const int j = t & (kTab - 1), n = -(t >> 6);
    const uint2 tv = tab[j];
    // 2^30 * 2^36 units to 2^-44 units: a shift by 22.
    const long long w = (long long)(((unsigned long long)tv.y << 32) | tv.x) + (((long long)tab30[j] * is) >> 22);
    return n > 45 ? 0ull : (unsigned long long)w >> n;
  }
};

__device__ __forceinline__ unsigned long long shfl_up64(unsigned long long v, int o) {
  return __shfl_up_sync(0xffffffffu, v, o);
}

// floor(f * s) for a float f in [0, 1) and s < 2^63, exactly.
__device__ __forceinline__ unsigned long long mul_floor(float f, unsigned long long s) {
  if (!(f > 0.f)) return 0;
  int e;
  const unsigned long long mant = (unsigned long long)(frexpf(f, &e) * 16777216.f);  // f = mant 2^(e-24)
  const int sh = 24 - e;                                                             // >= 24
  const unsigned long long lo = mant * s, hi = __umul64hi(mant, s);
  if (sh >= 128) return 0;
  if (sh >= 64) return hi >> (sh - 64);
  return (lo >> sh) | (hi << (64 - sh));
}
// ceil(f * s).
__device__ __forceinline__ unsigned long long mul_ceil(float f, unsigned long long s) {
  if (!(f > 0.f)) return 0;
  int e;
  const unsigned long long mant = (unsigned long long)(frexpf(f, &e) * 16777216.f);
  const int sh = 24 - e;
  const unsigned long long lo = mant * s, hi = __umul64hi(mant, s);
  unsigned long long q, rem;
  if (sh >= 128) return 1;
  if (sh >= 64) {
    q = hi >> (sh - 64);
    rem = lo | (sh > 64 ? hi << (128 - sh) : 0ull);
  } else {
    q = (lo >> sh) | (hi << (64 - sh));
    rem = lo << (64 - sh);
  }
  return q + (rem != 0);
}

// Which tokens stay: key > t, or key == t and among the first r of those.
struct Keep {
  unsigned int t, r;
};

template <typename T>
struct Row {
  static constexpr int kDrop = sizeof(T) == 2 ? 16 : 0;  // low key bits that a bf16 logit never uses
  Shared& S;
  const float* xs;  // this CTA's slice
  int n;            // its length
  int rank, nc;
  int buf = 0;
  float m;

  __device__ __forceinline__ unsigned int key(float x) const { return order_bits(x) >> kDrop; }

  // Sum of the cluster's histograms in buffer b, two bins per thread, then the
  // first bin whose running count (BY_MASS: mass) reaches `need`; the values
  // before it and in it go to S.found_*.  Every CTA finds the same.
  template <bool BY_MASS>
  __device__ __forceinline__ void find_bin(cg::cluster_group& cl, int b, unsigned long long need) {
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    unsigned int c[2] = {0, 0};
    unsigned long long v[2] = {0, 0};
    for (int i = 0; i < nc; ++i) {
      const Shared* o = cl.map_shared_rank(&S, i);
      const uint2 a = *reinterpret_cast<const uint2*>(&o->hist[b][0][2 * tid]);
      c[0] += a.x;
      c[1] += a.y;
      if constexpr (BY_MASS) {
        const uint2 l0 = *reinterpret_cast<const uint2*>(&o->hist[b][1][2 * tid]);
        const uint2 l1 = *reinterpret_cast<const uint2*>(&o->hist[b][2][2 * tid]);
        const uint2 l2 = *reinterpret_cast<const uint2*>(&o->hist[b][3][2 * tid]);
        v[0] += l0.x + ((unsigned long long)l1.x << 16) + ((unsigned long long)l2.x << 32);
        v[1] += l0.y + ((unsigned long long)l1.y << 16) + ((unsigned long long)l2.y << 32);
      }
    }
    if constexpr (!BY_MASS) v[0] = c[0], v[1] = c[1];
    unsigned long long s = v[0] + v[1], inc = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long up = shfl_up64(inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) S.wm[w] = inc;
    __syncthreads();
    unsigned long long before = inc - s;
    for (int i = 0; i < w; ++i) before += S.wm[i];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (before < need && before + v[e] >= need) {
        S.found_bin = 2 * tid + e;
        S.found_m = before;
        S.found_n = c[e];
      }
      before += v[e];
    }
    __syncthreads();
  }

  __device__ __forceinline__ void add(int b, int bin, unsigned long long wt, bool by_mass) {
    atomicAdd(&S.hist[b][0][bin], 1u);
    if (by_mass) {
      if (const unsigned int v = (unsigned int)wt & 0xFFFFu) atomicAdd(&S.hist[b][1][bin], v);
      if (const unsigned int v = (unsigned int)(wt >> 16) & 0xFFFFu) atomicAdd(&S.hist[b][2][bin], v);
      if (const unsigned int v = (unsigned int)(wt >> 32)) atomicAdd(&S.hist[b][3][bin], v);
    }
  }
  __device__ __forceinline__ void clear(int b, bool by_mass) {
    for (int i = threadIdx.x; i < (by_mass ? 4 : 1) * kBins; i += kThreads) S.hist[b][0][i] = 0;
  }

  // The threshold of the tokens above `base` (an earlier threshold; its ties
  // are not among them): by count the `need` largest, by mass the shortest
  // prefix with mass >= need.  need must be reachable.
  template <bool BY_MASS>
  __device__ Keep search(cg::cluster_group& cl, unsigned int base, unsigned long long need, float step, const Weigher& wt) {
    const int tid = threadIdx.x;
    const float top = m;
    auto coarse = [&](float x) { return min(kBins - 1, (int)((top - x) * step)); };
    // 1024 equal steps below the maximum; the last one holds everything further down.
    int b = buf;
    clear(b, BY_MASS);
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const float x = xs[i];
      if (x == -INFINITY || key(x) <= base) continue;
      unsigned long long w = 0;
      if constexpr (BY_MASS) {
        w = wt(x);
        if (w == 0) continue;
      }
      add(b, coarse(x), w, BY_MASS);
    }
    cl.sync();
    find_bin<BY_MASS>(cl, b, need);
    buf ^= 1;
    const int cb = (int)S.found_bin;
    need -= S.found_m;
    unsigned int cnt = S.found_n;
    // The keys of that step: coarse() falls as the key grows, so its bounds come by bisection.
    if (tid < 64 && (tid & 31) == 0) {
      // warp 0: smallest key with coarse <= cb; warp 1: smallest key with coarse <= cb - 1 (then minus 1).
      const int want = cb - (tid >> 5);
      unsigned int lo = order_bits(-3.402823466e38f) >> kDrop, hi = key(top) + 1;  // answer in [lo, hi]
      while (lo < hi) {
        const unsigned int mid = lo + ((hi - lo) >> 1);
        if (coarse(from_order((mid << kDrop) | (kDrop && !(mid & 0x8000u) ? 0xFFFFu : 0u))) <= want) hi = mid;
        else lo = mid + 1;
      }
      if (tid == 0) S.lo = lo;
      else S.hi = lo - 1;
    }
    __syncthreads();
    unsigned int lo = max(S.lo, base + 1), hi = S.hi;
    while (true) {
      if (BY_MASS ? cnt == 1 : need == cnt) return Keep{lo - 1, 0};  // the whole bin stays
      if (lo == hi) break;
      const unsigned int range = hi - lo;
      const int shift = max(0, 32 - __clz(range) - 10);  // (range >> shift) < kBins
      b = buf;
      clear(b, BY_MASS);
      __syncthreads();
      for (int i = tid; i < n; i += kThreads) {
        const float x = xs[i];
        if (x == -INFINITY) continue;
        const unsigned int k = key(x);
        if (k < lo || k > hi) continue;
        unsigned long long w = 0;
        if constexpr (BY_MASS) {
          w = wt(x);
          if (w == 0) continue;
        }
        add(b, (int)((hi - k) >> shift), w, BY_MASS);
      }
      cl.sync();
      find_bin<BY_MASS>(cl, b, need);
      buf ^= 1;
      need -= S.found_m;
      cnt = S.found_n;
      const unsigned int bin = S.found_bin;
      const unsigned int nh = hi - (bin << shift), width = (1u << shift) - 1;
      lo = nh - lo > width ? nh - width : lo;
      hi = nh;
      __syncthreads();  // S.found_* are read before the next step writes them
    }
    if constexpr (!BY_MASS) return Keep{lo, (unsigned int)need};
    const unsigned long long each = wt(from_order((lo << kDrop) | (kDrop && !(lo & 0x8000u) ? 0xFFFFu : 0u)));
    return Keep{lo, (unsigned int)((need + each - 1) / each)};
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
    k_sample(SampleRows a, int slice) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& S = *reinterpret_cast<Shared*>(raw);
  float* xs = reinterpret_cast<float*>(raw + sizeof(Shared));
  cg::cluster_group cl = cg::this_cluster();
  const int nc = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int row = blockIdx.x / nc;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cl.barrier_arrive();  // waited for before the first access to another CTA's shared memory
  if (tid < kTab) {
    const unsigned long long f = kExp2[tid];
    S.tab[tid] = make_uint2((unsigned int)f, (unsigned int)(f >> 32));
    S.tab30[tid] = (int)((f + (1u << 13)) >> 14);
  }
  pdl_wait();
  pdl_trigger();

  // The row's settings (uniform over the cluster).
  size_t out = row;
  float T_ = 0.f, u = 0.f, tp = 1.f, mp = 0.f;
  int tk = 0;
  if (a.slot) {  // engine rows: settings by sequence slot, numbers and tokens by (slot, token)
    const int sl = a.slot[row], t = a.t[row];
    const SampleParams P = a.params[sl];
    out = (size_t)sl * a.cap + t;
    if (!P.on || a.forced[out] >= 0) {
      cl.barrier_wait();
      return;
    }
    T_ = P.temperature, tk = P.top_k, tp = P.top_p, mp = P.min_p, u = a.u[out];
  } else {
    T_ = a.temperature[row], u = a.u[row];
    if (a.top_k) tk = a.top_k[row];
    if (a.top_p) tp = a.top_p[row];
    if (a.min_p) mp = a.min_p[row];
  }
  const int lo = min(a.vocab, rank * slice), n = min(a.vocab, lo + slice) - lo;
  const T* src = reinterpret_cast<const T*>(a.logits) + (size_t)row * a.ld + lo;

  // One read of the row: NaN counts as -inf, -0 as 0 (so that equal logits have equal keys).
  float mx = -INFINITY, mn = INFINITY;
  int fi = 0x7FFFFFFF;
  auto take = [&](int i, float x) {
    x = x != x ? -INFINITY : x + 0.f;
    xs[i] = x;
    if (x > mx) mx = x, fi = lo + i;
    if (x > -INFINITY) mn = fminf(mn, x);
  };
  constexpr int E = Chunk<T>::N;
  if ((reinterpret_cast<uintptr_t>(src) & 15) == 0) {
    const int nv = n / E;
#pragma unroll 4
    for (int i = tid; i < nv; i += kThreads) {
      float v[E];
      Chunk<T>::load(src + (size_t)i * E, v);
#pragma unroll
      for (int e = 0; e < E; ++e) take(i * E + e, v[e]);
    }
    for (int i = nv * E + tid; i < n; i += kThreads) take(i, to_f(src[i]));
  } else {
    for (int i = tid; i < n; i += kThreads) take(i, to_f(src[i]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, mx, o);
    const int oi = __shfl_xor_sync(0xffffffffu, fi, o);
    if (om > mx || (om == mx && oi < fi)) mx = om, fi = oi;
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
  }
  if (lane == 0) S.fmx[warp] = mx, S.fmn[warp] = mn, S.fi[warp] = fi;
  if (tid == 0) S.token = -1;
  cl.barrier_wait();
  __syncthreads();
  if (tid < nc) {  // thread i tells CTA i
    for (int w = 0; w < kWarps; ++w) {
      if (S.fmx[w] > mx || (S.fmx[w] == mx && S.fi[w] < fi)) mx = S.fmx[w], fi = S.fi[w];
      mn = fminf(mn, S.fmn[w]);
    }
    cl.map_shared_rank(&S, tid)->note[rank] = Note{mx, mn, fi, 0};
  }
  cl.sync();
  mx = -INFINITY, mn = INFINITY, fi = 0x7FFFFFFF;
  for (int i = 0; i < nc; ++i) {
    const Note o = S.note[i];
    if (o.mx > mx || (o.mx == mx && o.first < fi)) mx = o.mx, fi = o.first;
    mn = fminf(mn, o.mn);
  }
  const bool greedy = !(T_ > 0.f);
  if (mx == -INFINITY || greedy) {
    if (rank == 0 && tid == 0) {
      a.token[out] = mx == -INFINITY ? a.empty_token : fi;
      if (a.logprob) a.logprob[out] = mx == -INFINITY ? -INFINITY : 0.f;
    }
    return;
  }
  if (mx == INFINITY) {  // the +inf entries share the mass
    for (int i = tid; i < n; i += kThreads) xs[i] = xs[i] == INFINITY ? 0.f : -INFINITY;
    mx = mn = 0.f;
    __syncthreads();
  }
  // 1 / T in two parts.
  const float Tc = fmaxf(T_, 1.17549435e-38f);
  Weigher wt;
  wt.m = mx;
  wt.ch = __frcp_rn(Tc);
  wt.cl = __fmaf_rn(-Tc, wt.ch, 1.f) * wt.ch;
  wt.tab = S.tab;
  wt.tab30 = S.tab30;
  Row<T> R{S, xs, n, rank, nc};
  R.m = mx;

  Keep keep{0, 0};
  if (tk > 0 && tk < a.vocab) {
    // Fewer than top_k tokens above -inf: all stay.
    unsigned int have = 0;
    for (int i = tid; i < n; i += kThreads) have += xs[i] != -INFINITY;
    have = __reduce_add_sync(0xffffffffu, have);
    if (lane == 0) S.wc[warp] = have;
    __syncthreads();
    if (tid < nc) {
      unsigned int s = 0;
      for (int w = 0; w < kWarps; ++w) s += S.wc[w];
      cl.map_shared_rank(&S, tid)->tail[rank].ties = s;
    }
    cl.sync();
    unsigned int all = 0;
    for (int i = 0; i < nc; ++i) all += S.tail[i].ties;
    const float span = mx - mn;
    if ((unsigned int)tk < all)
      keep = R.template search<false>(cl, 0u, (unsigned long long)tk, span > 0.f ? (float)kBins / span : 0.f, wt);
    else
      cl.sync();  // S.tail is free for the sums below
  }
  // Mass of what is above the threshold, and of its kept ties.
  const unsigned int drop_fill = (Row<T>::kDrop && !(keep.t & 0x8000u)) ? 0xFFFFu : 0u;
  unsigned long long tie_w = keep.r ? wt(from_order((keep.t << Row<T>::kDrop) | drop_fill)) : 0ull;
  if (tp < 1.f) {
    unsigned long long s = 0;
    for (int i = tid; i < n; i += kThreads) {
      const float x = xs[i];
      if (x > -INFINITY && R.key(x) > keep.t) s += wt(x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) S.wm[warp] = s;
    __syncthreads();
    if (tid < nc) {
      s = 0;
      for (int w = 0; w < kWarps; ++w) s += S.wm[w];
      cl.map_shared_rank(&S, tid)->tail[rank].mass = s;
    }
    cl.sync();
    unsigned long long above = 0;
    for (int i = 0; i < nc; ++i) above += S.tail[i].mass;
    unsigned long long need = mul_ceil(tp, above + tie_w * keep.r);
    if (need == 0) need = 1;
    cl.sync();  // every CTA has read S.tail
    if (need <= above)
      keep = R.template search<true>(cl, keep.t, need, (float)kBins / 31.5f * wt.ch, wt);
    else
      keep.r = min(keep.r, (unsigned int)((need - above + tie_w - 1) / tie_w));
    const unsigned int fill = (Row<T>::kDrop && !(keep.t & 0x8000u)) ? 0xFFFFu : 0u;
    tie_w = keep.r ? wt(from_order((keep.t << Row<T>::kDrop) | fill)) : 0ull;
  }
  unsigned long long floor_w = 1;  // smallest weight that stays
  if (mp > 0.f) {
    floor_w = mp >= 1.f ? 1ull << kUnit : mul_ceil(mp, 1ull << kUnit);
    if (tie_w < floor_w) keep.r = 0;
  }

  // With u = 0 the first kept token wins however small its mass: weights that
  // the fixed-point unit rounds to none count as one unit there.
  const bool zero_u = !(u > 0.f) && floor_w == 1;
  auto kept_weight = [&](float x) {
    const unsigned long long w = wt(x);
    if (w >= floor_w) return w;
    return zero_u && (x - mx) * wt.ch > -700.f ? 1ull : 0ull;
  };

  // Kept mass of each warp's segment of the slice, in index order.
  const int seg = ((n + kWarps * 32 - 1) / (kWarps * 32)) * 32;
  const int s0 = min(n, warp * seg), s1 = min(n, s0 + seg);
  unsigned long long sum = 0;
  unsigned int ties = 0;
  for (int i = s0 + lane; i < s1; i += 32) {
    const float x = xs[i];
    if (x == -INFINITY) continue;
    const unsigned int k = R.key(x);
    if (k > keep.t) {
      sum += kept_weight(x);
    } else if (k == keep.t) {
      ++ties;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  ties = __reduce_add_sync(0xffffffffu, ties);
  __syncthreads();
  if (lane == 0) S.wm[warp] = sum, S.wc[warp] = ties;
  __syncthreads();
  if (tid < nc) {
    unsigned long long s = 0;
    unsigned int t = 0;
    for (int w = 0; w < kWarps; ++w) s += S.wm[w], t += S.wc[w];
    cl.map_shared_rank(&S, tid)->tail[rank] = Tail{s, t, 0};
  }
  cl.sync();
  // Ties and mass before this CTA and in total; a CTA's ties count while fewer than keep.r came before.
  unsigned long long total = 0, mine0 = 0;
  unsigned int tied = 0, mytied0 = 0;
  for (int i = 0; i < nc; ++i) {
    if (i == rank) mine0 = total, mytied0 = tied;
    total += S.tail[i].mass + tie_w * min(S.tail[i].ties, keep.r - min(keep.r, tied));
    tied += S.tail[i].ties;
  }
  const float uc = u > 0.f ? fminf(u, 0.99999994f) : 0.f;
  const unsigned long long goal = mul_floor(uc, total);  // the token's running mass is the first above goal
  // The segment (warp w of this CTA) whose running mass passes goal.
  unsigned long long before = mine0;
  unsigned int tb = mytied0;
  int hit = -1;
  for (int w = 0; w < kWarps; ++w) {
    const unsigned long long here = S.wm[w] + tie_w * min(S.wc[w], keep.r - min(keep.r, tb));
    if (before <= goal && goal < before + here) {
      hit = w;
      break;
    }
    before += here;
    tb += S.wc[w];
  }
  if (hit >= 0) {  // uniform in this CTA; no other CTA of the cluster has it
    // The segment again, cut into one run of 32-entry chunks per warp.
    __syncthreads();  // S.wm and S.wc are read
    const int g0 = min(n, hit * seg), g1 = min(n, g0 + seg);
    const int sub = ((g1 - g0 + kWarps * 32 - 1) / (kWarps * 32)) * 32;
    const int a0 = min(g1, g0 + warp * sub), a1 = min(g1, a0 + sub);
    unsigned long long s = 0;
    unsigned int tt = 0;
    for (int i = a0 + lane; i < a1; i += 32) {
      const float x = xs[i];
      if (x == -INFINITY) continue;
      const unsigned int k = R.key(x);
      if (k > keep.t) {
        s += kept_weight(x);
      } else if (k == keep.t) {
        ++tt;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    tt = __reduce_add_sync(0xffffffffu, tt);
    if (lane == 0) S.wm[warp] = s, S.wc[warp] = tt;
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
      before += S.wm[w] + tie_w * min(S.wc[w], keep.r - min(keep.r, tb));
      tb += S.wc[w];
    }
    const unsigned long long end = before + S.wm[warp] + tie_w * min(S.wc[warp], keep.r - min(keep.r, tb));
    if (before <= goal && goal < end) {
      for (int i0 = a0; i0 < a1; i0 += 32) {  // in index order, 32 entries at a time
        const int i = i0 + lane;
        const float x = i < a1 ? xs[i] : -INFINITY;
        const unsigned int k = x > -INFINITY ? R.key(x) : 0u;
        const bool tie = x > -INFINITY && k == keep.t;
        const unsigned int tm = __ballot_sync(0xffffffffu, tie);
        unsigned long long w = 0;
        if (tie) {
          if (tb + __popc(tm & ((1u << lane) - 1u)) < keep.r) w = tie_w;
        } else if (x > -INFINITY && k > keep.t) {
          w = kept_weight(x);
        }
        unsigned long long inc = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long up = shfl_up64(inc, o);
          if (lane >= o) inc += up;
        }
        const unsigned int past = __ballot_sync(0xffffffffu, before + inc > goal);
        if (past) {
          if (lane == __ffs(past) - 1) {
            a.token[out] = lo + i;
            if (a.logprob) {
              const float sum_hi = (float)total;  // total = 2^44 (hi + lo), at least 2^44
              const float sum_lo = (float)(long long)(total - (unsigned long long)sum_hi);
              const float d = x - mx;
              a.logprob[out] = fmaf(d, wt.ch, d * wt.cl) - (logf(sum_hi * 0x1p-44f) + sum_lo / sum_hi);
            }
          }
          break;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
        tb += __popc(tm);
      }
    }
  }
}

}  // namespace smp

// Cluster size: CTAs hold their slice beside 34 KB of tables, two CTAs per SM
// up to a 64 KB slice; small batches spread a row over more CTAs as long as
// all of them are resident at once.  The result does not depend on it.
template <typename T>
static cudaError_t sample_t(cudaStream_t s, const SampleRows& a) {
  constexpr int kTwoPerSm = 16384, kMost = 45056;  // slice entries for two CTAs per SM, for one
  static int sms[kMaxDevices] = {};
  const int dev = current_device();
  if (!sms[dev]) {
    int n = 0;
    cudaError_t e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(smp::k_sample<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(sizeof(smp::Shared) + (size_t)kMost * 4));
    if (e != cudaSuccess) return e;
    sms[dev] = n;
  }
  int nc = 1;
  while (nc < smp::kMaxCluster && a.vocab > nc * kTwoPerSm) nc *= 2;
  while (nc < smp::kMaxCluster && (long long)a.rows * nc * 2 <= 2ll * sms[dev] && a.vocab >= 2 * nc * 2048) nc *= 2;
  const int slice = (((a.vocab + nc - 1) / nc) + 31) / 32 * 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.rows * nc);
  cfg.blockDim = dim3(smp::kThreads);
  cfg.dynamicSmemBytes = sizeof(smp::Shared) + (size_t)slice * 4;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = nc;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  count_launch();
  return cudaLaunchKernelEx(&cfg, smp::k_sample<T>, a, slice);
}

cudaError_t launch_sample(cudaStream_t s, const SampleRows& a, bool bf16) {
  if (a.rows <= 0) return cudaSuccess;
  return bf16 ? sample_t<__nv_bfloat16>(s, a) : sample_t<float>(s, a);
}

}  // namespace cdb
