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
// Thresholds come from a radix search without sorting: a histogram over 1024
// equal steps of m - x, then histograms over the ordered bit patterns of the
// chosen bin, until the bin holds exactly what is needed or a single value.
// top_k counts, after the maxima of single threads have ruled out most of the
// row.  top_p guesses its bin from counts and mean offsets and adds up the exact mass
// above and in it, so each logit's exact weight is computed once; of bf16 rows in
// one or two CTAs it counts every value by itself, and weighs values, not logits.  Each CTA
// works on its slice in its own shared memory, all CTAs of the cluster then
// read one another's histograms or sums (distributed shared memory) and come to
// the same decision; two histogram buffers leave one cluster barrier per step.
// What bounds it: the instructions of the weights (about 50 for each logit that
// has mass), shared atomics (some 20 cycles a warp) and, with few rows, the
// barriers.  512 rows of 65536 bf16 logits (9.9 us of HBM traffic): argmax 22 us,
// temperature alone 98, top_k 76, top_p 157, min_p 60; 64 rows of 49152 fp32: 5,
// 16, 19, 30, 10; one row: 3.4, 8, 13, 18, 7.
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
constexpr int kList = 128;        // entries that are ranked one against another
constexpr int kUnit = 44;         // fixed-point weights: 2^kUnit is weight 1
constexpr int kTab = 64;          // 2^(-j/64), j = 0..63

// 2^(-j/64) in units of 2^-44, rounded.
__constant__ unsigned long long kExp2[kTab] = {
    17592186044416ull, 17402683248456ull, 17215221774115ull, 17029779632301ull,
    16846335070792ull, 16664866571680ull, 16485352848846ull, 16307772845465ull,
    16132105731538ull, 15958330901445ull, 15786427971528ull, 15616376777705ull,
    15448157373097ull, 15281750025697ull, 15117135216047ull, 14954293634955ull,
    14793206181226ull, 14633853959423ull, 14476218277651ull, 14320280645363ull,
    14166022771192ull, 14013426560807ull, 13862474114787ull, 13713147726524ull,
    13565429880144ull, 13419303248457ull, 13274750690919ull, 13131755251623ull,
    12990300157313ull, 12850368815412ull, 12711944812080ull, 12575011910285ull,
    12439554047902ull, 12305555335825ull, 12173000056107ull, 12041872660113ull,
    11912157766698ull, 11783840160404ull, 11656904789672ull, 11531336765078ull,
    11407121357589ull, 11284243996830ull, 11162690269381ull, 11042445917079ull,
    10923496835354ull, 10805829071568ull, 10689428823381ull, 10574282437131ull,
    10460376406236ull, 10347697369602ull, 10236232110063ull, 10125967552830ull,
    10016890763953ull, 9908988948806ull, 9802249450589ull, 9696659748838ull,
    9592207457961ull, 9488880325783ull, 9386666232110ull, 9285553187305ull,
    9185529330885ull, 9086582930126ull, 8988702378691ull, 8891876195264ull,
};

// What each CTA tells the others (one record per CTA, written remotely).
struct Note {
  float mx, mn;  // largest logit, smallest above -inf of the threads' largest
  int first;     // lowest index of mx
  int pad;
};
struct Tail {
  unsigned long long mass, in, below;  // kept mass above the threshold value; top_p: mass above the bin, in it, below it
  unsigned int ties, cnt;       // entries equal to the threshold value; top_p: entries of the bin
  float mn;                     // largest(): smallest logit above -inf
};

// Entries in place of a histogram: one CTA's, or the cluster's.
struct List {
  unsigned long long w[kList];
  unsigned int key[kList];
};

struct alignas(16) Shared {
  unsigned int hist[2][4][kBins];  // count, then the low, middle and high 16 bits of the masses
  uint4 tab[kTab];                 // 2^(-j/64): in units of 2^-44 (low, high word), in units of 2^-30
  Note note[kMaxCluster];
  Tail tail[2][kMaxCluster];  // in turn
  unsigned long long wm[kWarps], wi[kWarps], wb[kWarps];  // per-warp values of the scans and sums
  unsigned int wc[kWarps], wn[kWarps];
  unsigned long long found_m;
  unsigned int found_bin, found_n;
  unsigned int lo, hi;
  unsigned int list_n;  // entries of this CTA's list
  unsigned int small[4];  // by_value: mass of the values too small for a bin, 16 bits at a time
  float fmx[kWarps], fmn[kWarps];
  int fi[kWarps];
};

// Ordered bit pattern of a float (never NaN); bf16 values use its upper half.
__device__ __forceinline__ unsigned int order_bits(float x) {
  const unsigned int b = __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float from_order(unsigned int k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// exp((x - m) c) 2^kUnit as an integer, c = ch + cl = 1 / T, x <= m.  d = x - m
// as an exact sum of two floats (Knuth's two-sum), y = d c = p + pl to about
// 2^-46 of its value; y = r - t ln2/64 with t an integer and |r| < 0.0055
// (Cody and Waite's constants: t C1 and t C2 are exact products).  exp(r) - 1 =
// r + r^2/2 + r^3/6 + r^4/24 (the next term is below 2^-44) is an integer in
// units of 2^-38; times 2^(-j/64) from the table, shifted by the integer part.
// 45 fp32 and integer instructions: fp64 ones run at 1/64 of the fp32 rate.
struct Weigher {
  float m, ch, cl;
  const uint4* tab;
  __device__ __forceinline__ unsigned long long operator()(float x) const {
    const float d = __fsub_rn(x, m);
    const float db = __fsub_rn(d, x);
    const float dl = __fadd_rn(__fsub_rn(x, __fsub_rn(d, db)), __fsub_rn(-m, db));
    const float p = __fmul_rn(d, ch);
    const float pl = __fmaf_rn(dl, ch, __fmaf_rn(d, cl, __fmaf_rn(d, ch, -p)));
    constexpr float kMagic = 12582912.f;         // 1.5 * 2^23: the sum's low bits are the rounded integer
    constexpr float kInv = 92.332482616893657f;  // 64 / ln 2
    constexpr float kC1 = 2839.f / 262144.f;     // ln2/64 = C1 + C2 + C3: 12 bits, 12 bits, the rest
    constexpr float kC2 = 2144.f / 4294967296.f;
    constexpr float kC3 = -2.9760223437e-11f;
    constexpr float k37 = 137438953472.f, k38 = 2.f * k37;  // 2^37, 2^38
    const float tm = __fmaf_rn(p, -kInv, kMagic);
    const unsigned int t = __float_as_uint(tm) - 0x4B400000u;
    const float tf = __fsub_rn(tm, kMagic);
    const float r1 = __fmaf_rn(tf, kC1, p);      // exact
    const float rr = __fmaf_rn(tf, kC2, r1);
    const float low = __fmaf_rn(tf, kC3, pl);
    const float q = rr * rr * __fmaf_rn(rr, __fmaf_rn(rr, 0.041666668f, 0.16666667f), 0.5f);
    const float s = __fmaf_rn(rr, low, low) + q;
    const int is = __float2int_rn(r1 * k38) + __float2int_rn(tf * (kC2 * k38)) +
                   2 * (__float_as_int(__fmaf_rn(s, k37, kMagic)) - 0x4B400000);
    const uint4 e = tab[t & (kTab - 1)];
    // 2^30 * 2^38 / 2^32 = 2^36 units, times 2^8.
    const unsigned long long w = (unsigned long long)((long long)__mulhi((int)e.z, is) * 256 +
                                                      (long long)(((unsigned long long)e.y << 32) | e.x));
    return p > -31.5f ? w >> (t >> 6) : 0ull;
  }
};

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

// 16 bytes of logits as stored: 4 fp32 or 8 bf16.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4, kDrop = 0;  // kDrop: low key bits that a logit of this type never uses
  float4 v;
  __device__ __forceinline__ float get(int i) const { return reinterpret_cast<const float*>(&v)[i]; }
  __device__ __forceinline__ void set(int i, float x) { reinterpret_cast<float*>(&v)[i] = x; }
  // NaN to -inf, -0 to 0; the largest.
  __device__ __forceinline__ float clean() {
    float* x = reinterpret_cast<float*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = fmaxf(x[i], -INFINITY) + 0.f;
    return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8, kDrop = 16;
  uint4 v;
  __device__ __forceinline__ float get(int i) const {
    const unsigned int w = reinterpret_cast<const unsigned int*>(&v)[i >> 1];
    return __uint_as_float((i & 1) ? w & 0xFFFF0000u : w << 16);
  }
  __device__ __forceinline__ void set(int i, float x) {
    unsigned int& w = reinterpret_cast<unsigned int*>(&v)[i >> 1];
    w = (i & 1) ? (w & 0xFFFFu) | __float_as_uint(x) : (w & 0xFFFF0000u) | (__float_as_uint(x) >> 16);
  }
  __device__ __forceinline__ float clean() {
    __nv_bfloat162* x = reinterpret_cast<__nv_bfloat162*>(&v);
    const __nv_bfloat162 low = __floats2bfloat162_rn(-INFINITY, -INFINITY), zero = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __hadd2(__hmax2(x[i], low), zero);
    const __nv_bfloat162 t = __hmax2(__hmax2(x[0], x[1]), __hmax2(x[2], x[3]));
    return fmaxf(__low2float(t), __high2float(t));
  }
};

// Bins of a histogram by value: bf16 has 128 values per sign and power of two, so
// 15 powers of two have 3840 of them, in falling order 0..1919 for positive and
// 1921..3840 for negative ones; those of smaller magnitude share bin 1920.
struct ValueBins {
  static constexpr int kSide = 15 * 128, kSmall = kSide, kAll = 4096;  // eight per thread
  int low;  // smallest magnitude (15 bits) with a bin
  __device__ __forceinline__ int bin(unsigned int bits) const {  // < 0 or >= kAll: none
    const int d = (int)(bits & 0x7FFFu) - low;
    if (d < 0) return kSmall;
    return (bits & 0x8000u) ? (d < kSide ? kSmall + 1 + d : kAll) : kSide - 1 - d;
  }
  __device__ __forceinline__ unsigned int key(int b) const {  // b != kSmall
    return b < kSide ? 0x8000u + low + (kSide - 1 - b) : 0x7FFFu - (low + b - kSmall - 1);
  }
};

// The cluster's view of one row; every member function is called by all
// threads of all its CTAs.
template <typename T>
struct Row {
  static constexpr int E = Vec<T>::N, kDrop = Vec<T>::kDrop;
  Shared& S;
  cg::cluster_group& cl;
  const Vec<T>* xs;  // this CTA's slice, filled up with -inf to nv vectors
  int nv, rank, nc;
  float m;           // largest logit
  float own_max;     // largest logit this thread loaded
  int buf = 0;       // histogram buffer of the next step
  int tbuf = 0;      // tails of the next step

  // Barrier of the cluster; the shared memory of its CTA i.
  __device__ __forceinline__ void sync() const {
    if (nc > 1) cl.sync();
    else __syncthreads();
  }
  __device__ __forceinline__ Shared* peer(int i) const { return i == rank ? &S : cl.map_shared_rank(&S, i); }

  static __device__ __forceinline__ unsigned int key(float x) { return order_bits(x) >> kDrop; }
  static __device__ __forceinline__ float value(unsigned int k) {  // of a key
    return from_order((k << kDrop) | (kDrop && !(k & 0x8000u) ? 0xFFFFu : 0u));
  }
  // The largest logit with a key <= k, for comparisons of logits against a border between keys.  No logit has the
  // key of -0, but a border may: as a value it equals 0, whose key lies above it.
  static __device__ __forceinline__ float at_most(unsigned int k) { return value(k == (0x7FFFFFFFu >> kDrop) ? k - 1 : k); }

  // Every logit of the slice, in no particular order.  One vector a turn here and
  // below: with two, fetching the longer code takes more than it saves (8 rows of
  // 151936 bf16 logits, top_k and top_p: 33 us with two, 26 with one).
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll 1
    for (int i = threadIdx.x; i < nv; i += kThreads) {
      const Vec<T> v = xs[i];
#pragma unroll
      for (int e = 0; e < E; ++e) f(v.get(e));
    }
  }
  // Vectors [v0, v1) by one warp.
  template <typename F>
  __device__ __forceinline__ void each_of(int v0, int v1, F f) const {
#pragma unroll 1
    for (int i = v0 + (threadIdx.x & 31); i < v1; i += 32) {
      const Vec<T> v = xs[i];
#pragma unroll
      for (int e = 0; e < E; ++e) f(v.get(e));
    }
  }

  __device__ __forceinline__ void clear(int b, int arrays) {
    for (int i = threadIdx.x; i < arrays * kBins; i += kThreads) S.hist[b][0][i] = 0;
  }
  __device__ __forceinline__ void add_mass(int b, int bin, unsigned long long wt) {
    atomicAdd(&S.hist[b][0][bin], 1u);
    if (const unsigned int v = (unsigned int)wt & 0xFFFFu) atomicAdd(&S.hist[b][1][bin], v);
    if (const unsigned int v = (unsigned int)(wt >> 16) & 0xFFFFu) atomicAdd(&S.hist[b][2][bin], v);
    if (const unsigned int v = (unsigned int)(wt >> 32)) atomicAdd(&S.hist[b][3][bin], v);
  }

  // First of the 1024 bins (two per thread, v of each and its count c) whose
  // running sum reaches `need`; the sum before it and its count go to S.found_*.
  template <typename V>
  __device__ __forceinline__ void find(const V* v, const unsigned int* c, V need) {
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    V* part = reinterpret_cast<V*>(S.wm);
    V inc = v[0] + v[1];
    const V mine = inc;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const V up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) part[w] = inc;
    if (tid == 0) S.found_bin = kBins;  // none
    __syncthreads();
    V before = inc - mine;
#pragma unroll
    for (int i = 0; i < kWarps - 1; ++i) before += i < w ? part[i] : V(0);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (before < need && before + v[e] >= need) {
        S.found_bin = 2 * tid + e;
        S.found_m = (unsigned long long)before;
        S.found_n = c[e];
      }
      before += v[e];
    }
    __syncthreads();
  }
  // The cluster's histograms in buffer b, added up.
  template <bool BY_MASS>
  __device__ __forceinline__ void find_bin(int b, unsigned long long need) {
    const int tid = threadIdx.x;
    unsigned int c[2] = {0, 0};
    unsigned long long v[2] = {0, 0};
#pragma unroll (BY_MASS ? 2 : 4)  // reads of another CTA's memory in flight
    for (int i = 0; i < nc; ++i) {
      const Shared* o = peer(i);
      const uint2 a = *reinterpret_cast<const uint2*>(&o->hist[b][0][2 * tid]);
      c[0] += a.x, c[1] += a.y;
      if constexpr (BY_MASS) {
        const uint2 l0 = *reinterpret_cast<const uint2*>(&o->hist[b][1][2 * tid]);
        const uint2 l1 = *reinterpret_cast<const uint2*>(&o->hist[b][2][2 * tid]);
        const uint2 l2 = *reinterpret_cast<const uint2*>(&o->hist[b][3][2 * tid]);
        v[0] += l0.x + ((unsigned long long)l1.x << 16) + ((unsigned long long)l2.x << 32);
        v[1] += l0.y + ((unsigned long long)l1.y << 16) + ((unsigned long long)l2.y << 32);
      }
    }
    if constexpr (!BY_MASS) v[0] = c[0], v[1] = c[1];
    find<unsigned long long>(v, c, need);
  }

  // The keys with coarse(value) == bin into S.lo, S.hi: coarse() falls as the key grows, so its bounds come
  // by bisection, 32 keys at a time (warp 0: the smallest key with coarse <= bin, warp 1: with coarse <= bin - 1).
  template <typename F>
  __device__ __forceinline__ void bin_keys(int bin, F coarse) {
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid < 64) {
      const int want = bin - (tid >> 5);
      unsigned int lo = key(-3.402823466e38f), hi = key(m) + 1;  // answer in [lo, hi]
      while (lo < hi) {
        const unsigned int step = (hi - lo) / 32 + 1, mid = lo + lane * step;
        const bool below = mid >= hi || coarse(value(mid)) <= want;  // the answer is not above mid
        const unsigned int first = __ffs(__ballot_sync(0xffffffffu, below)) - 1;  // 32 if none
        const unsigned int l = lo;
        if (first == 0) {
          hi = lo;
        } else {
          lo = l + (first > 32 ? 31 : first - 1) * step + 1;
          if (first <= 31) hi = min(hi, l + first * step);
        }
      }
      if (lane == 0) {
        if (tid == 0) S.lo = lo;
        else S.hi = lo - 1;
      }
    }
    __syncthreads();
  }

  // refine() for at most kList entries: they are gathered, and each is ranked
  // against all by a thread of its own.
  template <bool BY_MASS>
  __device__ __forceinline__ Keep rank_few(unsigned int lo, unsigned int hi, unsigned long long need, const Weigher& wt) {
    const int tid = threadIdx.x;
    List& own = *reinterpret_cast<List*>(S.hist[buf]);
    List& all = *reinterpret_cast<List*>(S.hist[buf ^ 1]);
    if (tid == 0) S.list_n = 0;
    __syncthreads();
    const float xlo = value(lo), xhi = at_most(hi);
    each([&](float x) {
      if (x < xlo || x > xhi) return;
      const unsigned long long w = BY_MASS ? wt(x) : 1ull;
      if (w == 0) return;
      const unsigned int at = atomicAdd(&S.list_n, 1u);
      if (at < kList) own.key[at] = key(x), own.w[at] = w;
    });
    sync();
    unsigned int n[kMaxCluster], total = 0;
#pragma unroll
    for (int i = 0; i < kMaxCluster; ++i) n[i] = i < nc ? peer(i)->list_n : 0;
    int from = 0;
    unsigned int first = 0;  // the list that holds entry tid, and the entries before it
#pragma unroll
    for (int i = 0; i < kMaxCluster; ++i) {
      if ((unsigned int)tid >= total && n[i]) from = i, first = total;
      total += n[i];
    }
    total = min(total, (unsigned int)kList);
    unsigned int k = 0;
    unsigned long long w = 0;
    if ((unsigned int)tid < total) {
      const List* l = reinterpret_cast<const List*>(peer(from)->hist[buf]);
      k = l->key[tid - first], w = l->w[tid - first];
      all.key[tid] = k, all.w[tid] = w;
    }
    buf ^= 1;
    __syncthreads();
    if ((unsigned int)tid < total) {
      unsigned long long above = 0, equal = 0;
#pragma unroll 4
      for (unsigned int j = 0; j < total; ++j) {
        const unsigned int kj = all.key[j];
        const unsigned long long wj = all.w[j];
        above += kj > k ? wj : 0ull;
        equal += kj == k ? wj : 0ull;
      }
      if (above < need && need <= above + equal) {  // every entry of this key says the same
        S.lo = k;
        S.found_n = (unsigned int)((need - above + w - 1) / w);
      }
    }
    __syncthreads();
    return Keep{S.lo, S.found_n};
  }

  // Threshold inside the keys lo..hi, which hold cnt entries: by count the
  // `need` largest stay, by mass the shortest prefix with mass >= need.
  template <bool BY_MASS>
  __device__ __forceinline__ Keep refine(unsigned int lo, unsigned int hi, unsigned int cnt, unsigned long long need, const Weigher& wt) {
    while (true) {
      if (BY_MASS ? cnt == 1 : need == cnt) return Keep{lo - 1, 0};  // all of them stay
      if (lo == hi) break;
      const int shift = max(0, 32 - __clz(hi - lo) - 10);  // ((hi - lo) >> shift) < kBins
      // Few entries, and one histogram would not settle it (fp32, 64 rows of 49152 logits, top_p: 34 us so, 39
      // with histograms alone; where one does, as mostly with bf16, it is the quicker by 2%).
      if (cnt <= kList && shift > 0) return rank_few<BY_MASS>(lo, hi, need, wt);
      const int b = buf;
      clear(b, BY_MASS ? 4 : 1);
      __syncthreads();
      const float xlo = value(lo), xhi = at_most(hi);
      each([&](float x) {
        if (x < xlo || x > xhi) return;
        const int bin = (int)((hi - key(x)) >> shift);
        if constexpr (BY_MASS) {
          if (const unsigned long long w = wt(x)) add_mass(b, bin, w);
        } else {
          atomicAdd(&S.hist[b][0][bin], 1u);
        }
      });
      sync();
      find_bin<BY_MASS>(b, need);
      buf ^= 1;
      need -= S.found_m;
      cnt = S.found_n;
      const unsigned int width = (1u << shift) - 1, nh = hi - (S.found_bin << shift);
      lo = nh - lo > width ? nh - width : lo;
      hi = nh;
      __syncthreads();  // S.found_* are read before the next step writes them
    }
    if constexpr (!BY_MASS) return Keep{lo, (unsigned int)need};
    const unsigned long long each_w = wt(value(lo));
    return Keep{lo, (unsigned int)((need + each_w - 1) / each_w)};
  }

  // bf16: the threshold of top_p among the logits that `keep` leaves, from one
  // histogram with a bin per value, whose masses are counts times weights.  `zero`:
  // logits at or below it have no mass.  False, and nothing done, where a threshold
  // is among the values that share a bin or have none.  kept: the number that stay.
  __device__ __forceinline__ bool by_value(float tp, float zero, const Weigher& wt, Keep& keep, unsigned int& kept) {
    const int tid = threadIdx.x, lane = tid & 31, b = buf;
    const float far = fmaxf(fabsf(m), fabsf(zero));  // no larger magnitude needs a bin
    if (!(far < INFINITY)) return false;
    const ValueBins vb{max((int)(__float_as_uint(far) >> 23) - 14, 1) << 7};
    const int last = keep.r ? vb.bin(__float_as_uint(value(keep.t)) >> 16) : -1;  // bin of top_k's ties
    if (last == ValueBins::kSmall) return false;
    const float least = fmaxf(zero, at_most(keep.t));
    clear(b, 4);
    if (tid < 4) S.small[tid] = 0;
    __syncthreads();
    unsigned int* hist = S.hist[b][0];
    each([&](float x) {
      if (!(x > least)) return;
      const int c = vb.bin(__float_as_uint(x) >> 16);
      if (c >= ValueBins::kAll) return;
      atomicAdd(&hist[c], 1u);
      if (c == ValueBins::kSmall) {
        const unsigned long long w = wt(x);
        atomicAdd(&S.small[0], (unsigned int)w & 0xFFFFu);
        atomicAdd(&S.small[1], (unsigned int)(w >> 16) & 0xFFFFu);
        atomicAdd(&S.small[2], (unsigned int)(w >> 32));
      }
    });
    sync();
    unsigned int c[8] = {};
#pragma unroll 4
    for (int i = 0; i < nc; ++i) {
      const Shared* o = peer(i);
      const uint4 x = *reinterpret_cast<const uint4*>(&o->hist[b][0][8 * tid]), y = *reinterpret_cast<const uint4*>(&o->hist[b][0][8 * tid + 4]);
      c[0] += x.x, c[1] += x.y, c[2] += x.z, c[3] += x.w, c[4] += y.x, c[5] += y.y, c[6] += y.z, c[7] += y.w;
    }
    buf ^= 1;
    unsigned long long small = 0;
    if (tid == ValueBins::kSmall / 8) {
      for (int i = 0; i < nc; ++i) {
        const unsigned int* o = peer(i)->small;
        small += o[0] + ((unsigned long long)o[1] << 16) + ((unsigned long long)o[2] << 32);
      }
    }
    unsigned long long v[8], inc = 0;  // masses
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int bin = 8 * tid + e;
      if (bin == last) c[e] = keep.r;
      v[e] = c[e] == 0 ? 0ull : bin == ValueBins::kSmall ? small : wt(value(vb.key(bin))) * c[e];
      inc += v[e];
    }
    const unsigned long long mine = inc;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) S.wm[tid >> 5] = inc;
    if (tid == 0) S.found_bin = ValueBins::kAll;
    __syncthreads();
    unsigned long long before = inc - mine, total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i == tid >> 5) before += total;
      total += S.wm[i];
    }
    const unsigned long long goal = max(mul_ceil(tp, total), 1ull);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (before < goal && goal <= before + v[e]) S.found_bin = 8 * tid + e, S.found_n = c[e], S.found_m = before;
      before += v[e];
    }
    __syncthreads();
    const int at = (int)S.found_bin;
    if (at == ValueBins::kAll || at == ValueBins::kSmall) return false;
    const unsigned int k = vb.key(at);
    const unsigned long long w = wt(value(k));
    const unsigned int r = (unsigned int)((goal - S.found_m + w - 1) / w);
    keep = r == S.found_n && at != last ? Keep{k - 1, 0} : Keep{k, r};
    unsigned int n = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) n += 8 * tid + e <= at ? c[e] : 0;
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) S.wn[tid >> 5] = n;
    __syncthreads();
    kept = 0;
    for (int i = 0; i < kWarps; ++i) kept += S.wn[i];
    return true;
  }

  // Sums that each CTA tells the others (the values of all warps, added up); the
  // returned records stay until the call after the next.  BIN: top_p's sums.
  template <bool BIN>
  __device__ __forceinline__ const Tail* tell(unsigned long long mass, unsigned long long in, unsigned long long below,
                                              unsigned int ties, unsigned int cnt) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mass += __shfl_xor_sync(0xffffffffu, mass, o);
      if constexpr (BIN) {
        in += __shfl_xor_sync(0xffffffffu, in, o);
        below += __shfl_xor_sync(0xffffffffu, below, o);
      }
    }
    if constexpr (BIN) cnt = __reduce_add_sync(0xffffffffu, cnt);
    else ties = __reduce_add_sync(0xffffffffu, ties);
    __syncthreads();  // S.wm and its neighbours are free
    if (lane == 0) {
      S.wm[warp] = mass;
      if constexpr (BIN) S.wi[warp] = in, S.wb[warp] = below, S.wn[warp] = cnt;
      else S.wc[warp] = ties;
    }
    __syncthreads();
    if (tid < nc) {
      Tail t = {};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        t.mass += S.wm[w];
        if constexpr (BIN) t.in += S.wi[w], t.below += S.wb[w], t.cnt += S.wn[w];
        else t.ties += S.wc[w];
      }
      peer(tid)->tail[tbuf][rank] = t;
    }
    sync();
    const Tail* r = S.tail[tbuf];
    tbuf ^= 1;
    return r;
  }

  // The threshold of the `need` largest logits; all of them, where there are no more above -inf.
  __device__ __forceinline__ Keep largest(unsigned int need, float lowest_own, const Weigher& wt) {
    const float top = m;
    // The `need` largest of the threads' own maxima are as many logits, so the
    // wanted ones lie no lower: a histogram of one value per thread rules out
    // most of the row, and the next one meets few entries.
    float step = 0.f, least = -INFINITY;
    int bound = kBins;
    auto coarse = [&](float x) { return min(kBins - 1, (int)((top - x) * step)); };
    if (need <= (unsigned int)(nc * kThreads) / 2) {
      step = (float)kBins / (top - lowest_own);  // infinite where all are equal: the maximum in bin 0, the rest in the last
      const int b = buf;
      clear(b, 1);
      __syncthreads();
      if (own_max > -INFINITY) atomicAdd(&S.hist[b][0][coarse(own_max)], 1u);
      sync();
      find_bin<false>(b, need);
      buf ^= 1;
      bound = (int)S.found_bin;
      if (bound < kBins - 1) least = top - (float)(bound + 1) * (top - lowest_own) * (1.00001f / kBins) - 1e-6f * fabsf(top);
    }
    if (bound == kBins) {  // more are wanted: the range and the number of all logits
      float mn = INFINITY;
      unsigned int have = 0;
      each([&](float x) {
        if (x == -INFINITY) return;
        mn = fminf(mn, x);
        ++have;
      });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      have = __reduce_add_sync(0xffffffffu, have);
      const int tid = threadIdx.x;
      __syncthreads();
      if ((tid & 31) == 0) S.fmn[tid >> 5] = mn, S.wc[tid >> 5] = have;
      __syncthreads();
      if (tid < nc) {
        have = 0;
        for (int w = 0; w < kWarps; ++w) mn = fminf(mn, S.fmn[w]), have += S.wc[w];
        Tail& t = peer(tid)->tail[tbuf][rank];
        t.ties = have;
        t.mn = mn;
      }
      sync();
      have = 0;
      for (int i = 0; i < nc; ++i) mn = fminf(mn, S.tail[tbuf][i].mn), have += S.tail[tbuf][i].ties;
      tbuf ^= 1;
      if (need >= have) return Keep{0, 0};
      step = top > mn ? (float)kBins / (top - mn) : 0.f;
      bound = kBins - 1;
    }
    const int b = buf;
    clear(b, 1);
    __syncthreads();
    each([&](float x) {
      if (x == -INFINITY || x < least) return;
      const int c = coarse(x);
      if (c <= bound) atomicAdd(&S.hist[b][0][c], 1u);
    });
    sync();
    find_bin<false>(b, need);
    buf ^= 1;
    const int bin = (int)S.found_bin;
    const unsigned long long rest = need - S.found_m;
    const unsigned int cnt = S.found_n;
    bin_keys(bin, coarse);
    return refine<false>(S.lo, S.hi, cnt, rest, wt);
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
    k_sample(SampleRows a, int slice) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& S = *reinterpret_cast<Shared*>(raw);
  Vec<T>* xs = reinterpret_cast<Vec<T>*>(raw + sizeof(Shared));
  using R_ = Row<T>;
  constexpr int E = R_::E;
  cg::cluster_group cl = cg::this_cluster();
  const int nc = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int row = blockIdx.x / nc;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (nc > 1) cl.barrier_arrive();  // waited for before the first access to another CTA's shared memory
  if (tid < kTab) {
    const unsigned long long f = kExp2[tid];
    S.tab[tid] = make_uint4((unsigned int)f, (unsigned int)(f >> 32), (unsigned int)((f + (1u << 13)) >> 14), 0u);
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
      if (nc > 1) cl.barrier_wait();
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

  const int nv = (n + 32 * E - 1) / (32 * E) * 32;  // whole warps of vectors, the last ones filled up with -inf
  R_ R{S, cl, xs, nv, rank, nc};

  // One read of the row: NaN counts as -inf, -0 as 0 (so that equal logits have equal keys).
  float mx = -INFINITY;
  int fi = 0x7FFFFFFF;
  const bool wide = (reinterpret_cast<uintptr_t>(src) & 15) == 0;
#pragma unroll 4
  for (int i = tid; i < nv; i += kThreads) {
    Vec<T> v;
    if (wide && (i + 1) * E <= n) {
      v.v = *reinterpret_cast<const decltype(v.v)*>(src + (size_t)i * E);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) v.set(e, i * E + e < n ? to_f(src[i * E + e]) : -INFINITY);
    }
    const float top = v.clean();
    if (top > mx) {
      mx = top;
#pragma unroll
      for (int e = E - 1; e >= 0; --e)
        if (v.get(e) == top) fi = lo + i * E + e;
    }
    xs[i] = v;
  }
  float mn = mx > -INFINITY ? mx : INFINITY;
  const float own_max = mx;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, mx, o);
    const int oi = __shfl_xor_sync(0xffffffffu, fi, o);
    if (om > mx || (om == mx && oi < fi)) mx = om, fi = oi;
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
  }
  if (lane == 0) S.fmx[warp] = mx, S.fmn[warp] = mn, S.fi[warp] = fi;
  if (nc > 1) cl.barrier_wait();
  __syncthreads();
  if (tid < nc) {  // thread i tells CTA i
    for (int w = 0; w < kWarps; ++w) {
      if (S.fmx[w] > mx || (S.fmx[w] == mx && S.fi[w] < fi)) mx = S.fmx[w], fi = S.fi[w];
      mn = fminf(mn, S.fmn[w]);
    }
    R.peer(tid)->note[rank] = Note{mx, mn, fi, 0};
  }
  R.sync();
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
  R.own_max = own_max;
  if (mx == INFINITY) {  // the +inf entries share the mass
    for (int i = tid; i < nv; i += kThreads) {
      Vec<T> v = xs[i];
#pragma unroll
      for (int e = 0; e < E; ++e) v.set(e, v.get(e) == INFINITY ? 0.f : -INFINITY);
      xs[i] = v;
    }
    R.own_max = own_max == INFINITY ? 0.f : -INFINITY;
    mx = mn = 0.f;
    __syncthreads();
  }
  R.m = mx;
  // 1 / T in two parts.
  const float Tc = fminf(fmaxf(T_, 0x1p-126f), 0x1p126f);
  Weigher wt;
  wt.m = mx;
  wt.ch = __frcp_rn(Tc);
  wt.cl = __fmaf_rn(-Tc, wt.ch, 1.f) * wt.ch;
  wt.tab = S.tab;
  unsigned long long floor_w = 1;  // smallest weight that stays
  if (mp > 0.f) floor_w = mp >= 1.f ? 1ull << kUnit : mul_ceil(mp, 1ull << kUnit);
  // Logits at or below `cut` weigh nothing, or less than min_p allows: a
  // comparison instead of a weight (with a margin for its own rounding).
  float cut = mx - 31.75f * Tc;
  if (mp > 0.f) cut = fmaxf(cut, mx + (mp < 1.f ? logf(mp) * 1.0001f - 1e-4f : -1e-4f) * Tc);
  cut -= 1e-6f * fabsf(mx);

  Keep keep{0, 0};
  if (tk > 0 && tk < a.vocab) keep = R.largest((unsigned int)tk, mn, wt);
  const float zero = mx - 31.75f * Tc - 1e-6f * fabsf(mx);  // logits below it have no mass
  bool guess = tp < 1.f;
  unsigned int kept = 0;  // logits that stay, where by_value() counted them
  if constexpr (R_::kDrop == 16) {
    // The histogram of all CTAs is 16 KB a CTA to each of them: up to two CTAs it is the quicker (512 rows of
    // 65536 logits, top_p 165 us against 215, behind top_k 122 against 131, when added), with eight the slower by half.
    if (guess && nc <= 2) guess = !R.by_value(tp, zero, wt, keep, kept);
  }
  // This warp's segment of the slice: the sums below go by it.
  const int seg = (nv / 32 + kWarps - 1) / kWarps * 32;
  const int s0 = min(nv, warp * seg), s1 = min(nv, s0 + seg);
  // Where most logits have a weight, weights without a branch around them overlap.
  const bool dense = keep.t == 0 && !(mp > 1e-4f);
  unsigned long long tie_w = keep.r ? wt(R.value(keep.t)) : 0ull;
  unsigned long long sum = 0;             // this lane's kept mass above keys `counted`
  float counted = INFINITY;               // logits above it are in `sum` already
  if (guess) {
    // A first guess of the bin, 1024 equal steps of the logits that have mass,
    // from each bin's count and mean offset (its mass to 1e-4), in one word: 16 bits
    // of count, 16 of the offsets' sum in 32nds (rounded up or down by lane, so that the
    // roundings cancel; a bin of more than 2000 logits may get its mean wrong).  Then the exact mass above it, in it and
    // below decides.
    const float step = (float)kBins / 31.5f * wt.ch;
    auto coarse = [&](float x) { return min(kBins - 1, (int)((mx - x) * step)); };
    const float least = fmaxf(zero, R.at_most(keep.t));  // above it is what top_k keeps whole and has mass
    const float dither = ((float)(lane * 13 % 32) + 0.5f) / 32.f;
    const int b = R.buf;
    R.clear(b, 1);
    __syncthreads();
    R.each([&](float x) {
      if (!(x > least)) return;
      const float y = (mx - x) * step;
      const int c = min(kBins - 1, (int)y);
      atomicAdd(&S.hist[b][0][c], 1u + ((unsigned int)fmaf(y - (float)c, 32.f, dither) << 16));
    });
    R.sync();
    unsigned int hc[2] = {0, 0}, ho[2] = {0, 0};
#pragma unroll 4
    for (int i = 0; i < nc; ++i) {
      const Shared* o = R.peer(i);
      const uint2 x = *reinterpret_cast<const uint2*>(&o->hist[b][0][2 * tid]);
      hc[0] += x.x & 0xFFFFu, hc[1] += x.y & 0xFFFFu, ho[0] += x.x >> 16, ho[1] += x.y >> 16;
    }
    R.buf ^= 1;
    float fv[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float mean = hc[e] ? (float)ho[e] / (32.f * (float)hc[e]) : 0.f;
      fv[e] = (float)hc[e] * exp2f(-((float)(2 * tid + e) + mean) * (31.5f * 1.4426950408889634f / kBins));
    }
    float ft = fv[0] + fv[1];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ft += __shfl_xor_sync(0xffffffffu, ft, o);
    if (lane == 0) S.fmx[warp] = ft;
    __syncthreads();
    ft = 0.f;
    for (int w = 0; w < kWarps; ++w) ft += S.fmx[w];
    const float with_ties = ft + (float)tie_w * 0x1p-44f * (float)keep.r;
    R.template find<float>(fv, hc, fmaxf(fminf(tp * with_ties, 0.999998f * ft), 1e-30f));
    int bin = min((int)S.found_bin, kBins - 1);
    bool moved = false;
    while (true) {
      unsigned long long above = 0, in = 0, below = 0;
      unsigned int cnt = 0;
      auto put = [&](float x, unsigned long long w) {
        const int c = coarse(x);
        above += c < bin ? w : 0ull;
        in += c == bin ? w : 0ull;
        below += c > bin ? w : 0ull;
        cnt += c == bin && w != 0;
      };
      if (dense) {
        R.each_of(s0, s1, [&](float x) {
          const unsigned long long w = wt(x);
          put(x, x > least ? w : 0ull);
        });
      } else {
        R.each_of(s0, s1, [&](float x) {
          if (x > least) put(x, wt(x));
        });
      }
      const Tail* tail = R.template tell<true>(above, in, below, 0, cnt);
      unsigned long long A = 0, B = 0, C = 0;
      cnt = 0;
      for (int i = 0; i < nc; ++i) A += tail[i].mass, B += tail[i].in, C += tail[i].below, cnt += tail[i].cnt;
      unsigned long long need = mul_ceil(tp, A + B + C + tie_w * keep.r);
      if (need == 0) need = 1;
      if (need > A + B + C) {  // into the ties of top_k
        keep.r = min(keep.r, (unsigned int)((need - (A + B + C) + tie_w - 1) / tie_w));
        sum = above + in + below;
        counted = R.at_most(keep.t);
        break;
      }
      if (need > A && need <= A + B) {
        R.bin_keys(bin, coarse);
        const unsigned int hi = S.hi;
        keep = R.template refine<true>(max(S.lo, keep.t + 1), hi, cnt, need - A, wt);
        sum = above;
        counted = R.at_most(hi);
        break;
      }
      // Off (a border within the guess's rounding): most often by one bin, else the bin from exact masses.
      const int next = need <= A ? bin - 1 : bin + 1;
      if (!moved && next >= 0 && next < kBins) {
        moved = true;
        bin = next;
        continue;
      }
      const int h = R.buf;
      R.clear(h, 4);
      __syncthreads();
      R.each([&](float x) {
        if (!(x > least)) return;
        if (const unsigned long long w = wt(x)) R.add_mass(h, coarse(x), w);
      });
      R.sync();
      R.template find_bin<true>(h, need);
      R.buf ^= 1;
      bin = min((int)S.found_bin, kBins - 1);
    }
    tie_w = keep.r ? wt(R.value(keep.t)) : 0ull;
  }
  // With u = 0 the first kept token wins however small its mass: weights that
  // the fixed-point unit rounds to none count as one unit there.
  const bool zero_u = !(u > 0.f) && floor_w == 1;
  if (zero_u) sum = 0, counted = INFINITY, cut = -INFINITY;
  // min_p may lie below the unit too: its logarithm.
  const float lowest = mp > 0.f ? logf(mp) : -INFINITY;
  auto kept_weight = [&](float x) {
    const unsigned long long w = wt(x);
    if (w >= floor_w) return w;
    const float z = (x - mx) * wt.ch;
    return zero_u && z > -700.f && z >= lowest ? 1ull : 0ull;
  };
  if (zero_u && keep.r) tie_w = kept_weight(R.value(keep.t));
  if (mp > 0.f) {
    sum = 0, counted = INFINITY;  // some of it may fall below the floor
    if (tie_w < floor_w) keep.r = 0;
  }

  // Kept mass of each warp's segment, in index order from warp to warp.
  // The threshold as a value; a tie of it counts only if some of them stay.
  const float at = R.at_most(keep.t), least = fmaxf(cut, at), tie_x = keep.r ? at : NAN;
  unsigned int ties = 0;
  if ((dense || kept > (unsigned int)a.vocab / 32) && counted == INFINITY && !zero_u) {  // many stay
    if (keep.r) R.each_of(s0, s1, [&](float x) { ties += x == tie_x; });
    R.each_of(s0, s1, [&](float x) {
      const unsigned long long w = wt(x);
      sum += x > least && w >= floor_w ? w : 0ull;
    });
  } else {
    R.each_of(s0, s1, [&](float x) {
      ties += x == tie_x;
      if (x > least && x <= counted) sum += kept_weight(x);
    });
  }
  const Tail* tail = R.template tell<false>(sum, 0, 0, ties, 0);
  // Ties and mass before this CTA and in total; a CTA's ties count while fewer than keep.r came before.
  unsigned long long total = 0, mine0 = 0;
  unsigned int tied = 0, mytied0 = 0;
  for (int i = 0; i < nc; ++i) {
    if (i == rank) mine0 = total, mytied0 = tied;
    total += tail[i].mass + tie_w * min(tail[i].ties, keep.r - min(keep.r, tied));
    tied += tail[i].ties;
  }
  const float uc = u > 0.f ? fminf(u, 0.99999994f) : 0.f;
  const unsigned long long goal = mul_floor(uc, total);  // the token's running mass is the first above goal
  // Lane w of every warp: the mass and the ties before S.wm[w], S.wc[w], and what the former and its ties weigh.
  unsigned long long before, here;
  unsigned int tb;
  auto running = [&](unsigned long long mass0, unsigned int ties0) {
    const unsigned int tc = lane < kWarps ? S.wc[lane] : 0;
    unsigned int ti = tc;
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) {
      const unsigned int up = __shfl_up_sync(0xffffffffu, ti, o);
      if (lane >= o) ti += up;
    }
    tb = ties0 + ti - tc;
    here = lane < kWarps ? S.wm[lane] + tie_w * min(tc, keep.r - min(keep.r, tb)) : 0;
    unsigned long long inc = here;
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) {
      const unsigned long long up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    before = mass0 + inc - here;
  };
  // The segment (warp `hit` of this CTA) whose running mass passes goal.
  running(mine0, mytied0);
  const int hit = __ffs(__ballot_sync(0xffffffffu, lane < kWarps && before <= goal && goal < before + here)) - 1;
  if (hit >= 0) {  // uniform in this CTA; no other CTA of the cluster has it
    const unsigned long long before0 = __shfl_sync(0xffffffffu, before, hit);
    const unsigned int tb0 = __shfl_sync(0xffffffffu, tb, hit);
    // The segment again, cut into one run of vectors per warp.
    __syncthreads();  // S.wm and S.wc are read
    const int g0 = min(nv, hit * seg), g1 = min(nv, g0 + seg);
    const int sub = (g1 - g0 + kWarps - 1) / kWarps;
    const int a0 = min(g1, g0 + warp * sub), a1 = min(g1, a0 + sub);
    unsigned long long s = 0;
    unsigned int tt = 0;
    R.each_of(a0, a1, [&](float x) {
      tt += x == tie_x;
      if (x > least) s += kept_weight(x);
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    tt = __reduce_add_sync(0xffffffffu, tt);
    if (lane == 0) S.wm[warp] = s, S.wc[warp] = tt;
    __syncthreads();
    running(before0, tb0);
    before = __shfl_sync(0xffffffffu, before, warp);
    here = __shfl_sync(0xffffffffu, here, warp);
    tb = __shfl_sync(0xffffffffu, tb, warp);
    if (before <= goal && goal < before + here) {
      for (int i0 = a0 * E; i0 < a1 * E; i0 += 32) {  // in index order, 32 entries at a time
        const int i = i0 + lane;
        const float x = i < a1 * E ? xs[i / E].get(i % E) : -INFINITY;
        const bool tie = x == tie_x;
        const unsigned int tm = __ballot_sync(0xffffffffu, tie);
        unsigned long long w = 0;
        if (tie) {
          if (tb + __popc(tm & ((1u << lane) - 1u)) < keep.r) w = tie_w;
        } else if (x > least) {
          w = kept_weight(x);
        }
        unsigned long long inc = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long up = __shfl_up_sync(0xffffffffu, inc, o);
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
// up to a slice of 72 KB; small batches spread a row over more CTAs as long as
// all of them are resident at once.  The result does not depend on it.
template <typename T>
static cudaError_t sample_t(cudaStream_t s, const SampleRows& a) {
  constexpr int kTwoPerSm = 72 * 1024 / sizeof(T), kStep = 32 * 16 / sizeof(T);  // entries of such a slice; of a warp's vectors
  constexpr int kMost = 176 * 1024;  // bytes of the largest slice
  static int sms[kMaxDevices] = {};
  const int dev = current_device();
  if (!sms[dev]) {
    int n = 0;
    cudaError_t e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(smp::k_sample<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(sizeof(smp::Shared) + kMost));
    if (e != cudaSuccess) return e;
    sms[dev] = n;
  }
  int nc = 1;
  while (nc < smp::kMaxCluster && a.vocab > nc * kTwoPerSm) nc *= 2;
  while (nc < smp::kMaxCluster && (long long)a.rows * nc * 2 <= 2ll * sms[dev] && a.vocab >= 2 * nc * 2048) nc *= 2;
  const int slice = (((a.vocab + nc - 1) / nc) + kStep - 1) / kStep * kStep;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.rows * nc);
  cfg.blockDim = dim3(smp::kThreads);
  cfg.dynamicSmemBytes = sizeof(smp::Shared) + (size_t)slice * sizeof(T);
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
