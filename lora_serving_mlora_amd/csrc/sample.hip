// Sampling of one token a row from its logits: temperature, top-k, top-p and
// min-p of each row's own, and a given random number.
//
// Weights are w = 2^((l - max) log2(e) / T) in 64 bits, rounded to whole
// multiples of 2^-42, so that sums of them are integers and come out the same
// in any order.  Tokens stand in the order of falling logits, lower index
// first; what top-k, top-p and min-p keep is a beginning of that order, and
// the token drawn is the one at which the running weight passes u times the
// weight kept.  So all that is asked of the order is where its running count
// or weight reaches a given number, and nothing but a few hundred tokens near
// those places is ever put in order:
//   1. the largest logit (one pass over the row);
//   2. a histogram of the weights over 4096 equal ranges of logits (a pass;
//      the exponentials and the LDS atomics bound it);
//   3. the ranges in which the running numbers can reach what they are asked
//      for are known then: their tokens go to a list (a pass), which is put in
//      order by counting, and the exact places are read off its running sums.
// A small top-k needs no histogram: the list holds the tokens down to the
// range of the k-th largest of the threads' own largest logits.
// Where too many tokens share a range (ties, narrow clusters), `reach` parts
// it again and again instead, at two passes a part.
#include "sample.h"

namespace mlora {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBins = 4096, kPer = kBins / kThreads, kCap = 1024;
constexpr int kFrac = 42;  // a weight of 1 is 2^42: 2^20 of them stay below 2^63
constexpr int kSmallK = 512;  // largest top-k that is looked for among the threads' maxima
constexpr float kNone = -__builtin_huge_valf();

constexpr int kValues = 1 << 16;     // bf16 values
constexpr int kValueVocab = 16384;  // smallest vocabulary whose bf16 values are counted

struct Bins {
  __attribute__((aligned(16))) u64 mass[kBins + 2];  // histogram, then the weight before each range
  __attribute__((aligned(16))) uint32_t count[kBins + 4];
};
struct Red {  // of a running sum over the workgroup
  u64 m[kWaves];
  uint32_t c[kWaves];
};
// V: room for counts of every bf16 value, 16 bits each: word w holds that of
// the bits w in its lower half and of w with the sign in its upper one
template <bool V>
struct SharedOf {
  union {
    Bins bins;
    __attribute__((aligned(16))) uint32_t words[V ? kValues / 2 : 4];
  };
  u64 key[kCap], skey[kCap];  // listed tokens (order and index), the same in order
  uint32_t rank[kCap];
  Red red[3];
  float redf[2][kWaves];
  u64 got[4];  // what one thread found for all
  int bin[6];
  uint32_t n_list;
};

// f(i, x) for every piece of the row that falls to this thread: x[e] is logit
// i + e of 16 bytes of them, NaN where there is none (the ends of the row come
// one at a time).  U pieces are loaded at once.
template <int U, class T, class F>
__device__ __forceinline__ void for_row(const T* __restrict__ row, int V, F f) {
  constexpr int E = 16 / sizeof(T);
  const int tid = threadIdx.x;
  const int head = min(V, (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(T)));
  const int body = (V - head) / E, tail = head + body * E;
  const uint4* p = reinterpret_cast<const uint4*>(row + head);
  float x[E];
  if (head + V - tail > 0) {
    const int i = tid < head ? tid : tail + tid - head;
#pragma unroll
    for (int e = 1; e < E; ++e) x[e] = __builtin_nanf("");
    if (i < V) {
      if constexpr (sizeof(T) == 2)
        x[0] = bf2f(row[i]);
      else
        x[0] = row[i];
      f(i, x);
    }
  }
  auto piece = [&](int v, const uint4& y) {
    const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if constexpr (sizeof(T) == 2)
        x[e] = (e & 1) ? hi_bf(w[e >> 1]) : lo_bf(w[e >> 1]);
      else
        x[e] = __uint_as_float(w[e]);
    }
    f(head + v * E, x);
  };
  for (int v = tid; v < body; v += U * kThreads) {
    uint4 y[U];
#pragma unroll
    for (int k = 0; k < U; ++k) y[k] = p[min(v + k * kThreads, body - 1)];
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (v + k * kThreads < body) piece(v + k * kThreads, y[k]);
  }
}

struct Row {
  double mx, scale;  // largest logit; log2(e) / T
  float fit, fit0;   // a logit's place in the histogram: fit0 - fit * logit
  float least;       // below mx; the weight is 0 from here down
  bool top;          // the largest is +infinity: those stand at 0, all else at -infinity
  // A logit as it is compared: NaN counts as -infinity.
  __device__ __forceinline__ float clean(float x) const {
    x = fmaxf(x, kNone);
    if (top) x = x == -kNone ? 0.f : kNone;
    return x;
  }
};

// Weight of a logit, in multiples of 2^-42.  ANY: of any clean logit; else of
// one that is not below r.least.
template <bool ANY = false>
__device__ __forceinline__ u64 weight(const Row& r, float x) {
  double d = ((double)x - r.mx) * r.scale;
  if (ANY) d = fmax(d, -64.0);  // also for the NaN of -infinity * 0
  const double t = d + 6755399441055744.0;  // 1.5 * 2^52: the nearest whole number in the low word
  const double f = d - (t - 6755399441055744.0);
  // 2^f, |f| <= 1/2: relative error 8e-14, 1 at f = 0 (minimax fit)
  double p = 9.16811938851594e-08;
  p = fma(p, f, 1.3255182784592006e-06);
  p = fma(p, f, 1.5258493063907014e-05);
  p = fma(p, f, 0.0001540345603665657);
  p = fma(p, f, 0.0013333547331461978);
  p = fma(p, f, 0.009618129159172244);
  p = fma(p, f, 0.055504108739712246);
  p = fma(p, f, 0.24022650695813708);
  p = fma(p, f, 0.6931471805585505);
  p = fma(p, f, 1.0);
  p = __hiloint2double(__double2hiint(p) + (__double2loint(t) << 20), __double2loint(p));
  // in a sum with 2^10 the last place is 2^-42: rounded to nearest
  return (u64)__double_as_longlong(p + 1024.0) & 0xfffffffffffffull;
}

// place of a logit in the histogram, and its range there: they fall with the
// logit, never the other way (every step is monotone)
__device__ __forceinline__ float place_of(const Row& r, float x) { return fmaf(x, -r.fit, r.fit0); }
__device__ __forceinline__ int range_of(const Row& r, float x) {
  return (int)__builtin_amdgcn_fmed3f(place_of(r, x), 0.f, (float)(kBins - 1));
}

// floats as whole numbers that rise with them
__device__ __forceinline__ uint32_t rising(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_rising(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ float next_up(float x) { return from_rising(rising(x) + 1); }
__device__ __forceinline__ float next_down(float x) { return from_rising(rising(x) - 1); }

// The temperature, or for one far below a last place of the largest logit the
// 64th part of that: a logit a place or more down has no weight either way, and
// the exponents stay within reach of `weight` (-44.7 - 2.2 * 64).
__device__ __forceinline__ float warm(float mx, float temp) { return fmaxf(temp, (mx - next_down(mx)) * 0.015625f); }

// A logit below the largest from which on, down, every weight is 0: 31 nats
// down (44.7 powers of two).  The difference is rounded, to `mx` itself where
// 31 temperatures are less than half its last place, so the float below it is
// taken: that lies below `mx` and not above the exact difference.
__device__ __forceinline__ float least_of(float mx, float temp) { return next_down(mx - 31.f * fminf(temp, 1e30f)); }

// place of a token in the order, rising: falling logits, then rising indices
__device__ __forceinline__ u64 order_key(float x, int i) {
  return ((u64)~rising(x + 0.f) << 32) | (uint32_t)i;  // -0 and 0 are alike
}

// the logit of a key
__device__ __forceinline__ float key_logit(u64 key) { return from_rising(~(uint32_t)(key >> 32)); }

// v of the lane that the DPP pattern names, 0 where there is none
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ u64 dpp(u64 v) {
  return (u64)dpp<CTRL, ROWS>((uint32_t)(v >> 32)) << 32 | dpp<CTRL, ROWS>((uint32_t)v);
}
template <class N>
__device__ __forceinline__ N row_scan(N v) {  // inclusive, in rows of 16 lanes
  v += dpp<0x111, 0xf>(v);
  v += dpp<0x112, 0xf>(v);
  v += dpp<0x114, 0xf>(v);
  v += dpp<0x118, 0xf>(v);
  return v;
}
template <class N>
__device__ __forceinline__ N wave_scan(N v) {
  v = row_scan(v);
  v += dpp<0x142, 0xa>(v);  // the row before's last lane
  v += dpp<0x143, 0xc>(v);  // lane 31
  return v;
}
__device__ __forceinline__ uint32_t lane_value(uint32_t v, int l) { return (uint32_t)__builtin_amdgcn_readlane((int)v, l); }
__device__ __forceinline__ u64 lane_value(u64 v, int l) {
  return (u64)lane_value((uint32_t)(v >> 32), l) << 32 | lane_value((uint32_t)v, l);
}
// inclusive running sums of m and c over the workgroup's threads, in place;
// the totals.  One barrier: `red` is free again after the next one.
__device__ __forceinline__ void block_scan(u64& m, uint32_t& c, Red& red, u64& mall, uint32_t& call) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  m = wave_scan(m);
  c = wave_scan(c);
  if (lane == 63) {
    red.m[wave] = m;
    red.c[wave] = c;
  }
  __syncthreads();
  static_assert(kWaves == 16, "a row of lanes holds the waves' sums");
  const u64 wm = row_scan(red.m[lane & 15]);
  const uint32_t wc = row_scan(red.c[lane & 15]);
  mall = lane_value(wm, 15);
  call = lane_value(wc, 15);
  if (wave > 0) {
    m += lane_value(wm, wave - 1);
    c += lane_value(wc, wave - 1);
  }
}

template <class S>
__device__ __forceinline__ void clear_bins(S& sh) {
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    sh.bins.mass[i * kThreads + threadIdx.x] = 0;
    sh.bins.count[i * kThreads + threadIdx.x] = 0;
  }
  __syncthreads();
}

// This thread's ranges kPer * tid .. of the histogram: the running weight and
// count before each (and after the last), also left in place of the histogram.
struct Ends {
  u64 m[kPer + 1];
  uint32_t c[kPer + 1];
};
template <class S>
__device__ __forceinline__ Ends scan_bins(S& sh, u64& mass, uint32_t& count) {
  static_assert(kPer == 4, "vector loads of a thread's ranges");
  const int t = threadIdx.x * kPer;
  const ulonglong2 m01 = *reinterpret_cast<const ulonglong2*>(&sh.bins.mass[t]);
  const ulonglong2 m23 = *reinterpret_cast<const ulonglong2*>(&sh.bins.mass[t + 2]);
  const uint4 c = *reinterpret_cast<const uint4*>(&sh.bins.count[t]);
  u64 m = m01.x + m01.y + m23.x + m23.y;
  uint32_t n = c.x + c.y + c.z + c.w;
  const u64 own = m;
  const uint32_t nown = n;
  block_scan(m, n, sh.red[0], mass, count);
  Ends e;
  e.m[0] = m - own;
  e.m[1] = e.m[0] + m01.x;
  e.m[2] = e.m[1] + m01.y;
  e.m[3] = e.m[2] + m23.x;
  e.m[4] = m;
  e.c[0] = n - nown;
  e.c[1] = e.c[0] + c.x;
  e.c[2] = e.c[1] + c.y;
  e.c[3] = e.c[2] + c.z;
  e.c[4] = n;
  *reinterpret_cast<ulonglong2*>(&sh.bins.mass[t]) = make_ulonglong2(e.m[0], e.m[1]);
  *reinterpret_cast<ulonglong2*>(&sh.bins.mass[t + 2]) = make_ulonglong2(e.m[2], e.m[3]);
  *reinterpret_cast<uint4*>(&sh.bins.count[t]) = make_uint4(e.c[0], e.c[1], e.c[2], e.c[3]);
  if (threadIdx.x == kThreads - 1) {
    sh.bins.mass[kBins] = m;
    sh.bins.count[kBins] = n;
  }
  __syncthreads();
  return e;
}
// the range in which the running weight reaches `aim` (1 .. the total), to *bin
__device__ __forceinline__ void find_mass(const Ends& e, u64 aim, int* bin) {
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (e.m[i] < aim && aim <= e.m[i + 1]) *bin = threadIdx.x * kPer + i;
}
__device__ __forceinline__ void find_count(const Ends& e, uint32_t aim, int* bin) {
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (e.c[i] < aim && aim <= e.c[i + 1]) *bin = threadIdx.x * kPer + i;
}

// the histogram of the row; returns this thread's weight of the tokens with at
// least `least`
template <class S, class T>
__device__ __forceinline__ u64 histogram(S& sh, const Row& r, const T* __restrict__ row, int V, u64 least,
                                         bool counts) {
  u64 strong = 0;
  for_row<2>(row, V, [&](int, const float (&xs)[16 / sizeof(T)]) {
#pragma unroll
    for (int e = 0; e < (int)(16 / sizeof(T)); ++e) {
      const float x = fmaxf(xs[e], r.least);
      const u64 w = weight(r, x);
      const int b = range_of(r, x);
      if (x > r.least) {
        atomicAdd(&sh.bins.mass[b], w);
        if (counts) atomicAdd(&sh.bins.count[b], 1u);
      }
      if (least != 0 && w >= least) strong += w;
      if (e & 1) __builtin_amdgcn_sched_barrier(0);  // keeps the next logits' work out of the registers
    }
  });
  return strong;
}

// Lists the tokens whose places in the histogram lie in one of N intervals
// (lo inside, hi outside): their keys, in any order; all are counted, the
// first kCap of them held.
struct Interval {
  float lo, hi;
};
template <int N, class S, class T>
__device__ __forceinline__ void list_in(S& sh, const Row& r, const T* __restrict__ row, int V,
                                        const Interval (&iv)[3]) {
  constexpr int E = 16 / sizeof(T);
  // a logit below which none is in an interval (the place is off by two
  // roundings at most), so that most pieces take a look at their largest only
  float far = iv[0].hi;
  if (N > 1) far = fmaxf(far, iv[1].hi);
  if (N > 2) far = fmaxf(far, iv[2].hi);
  const float from = (float)r.mx - (far / r.fit * 1.000001f + fabsf((float)r.mx) * 1e-6f);
  for_row<4>(row, V, [&](int i, const float (&xs)[E]) {
    float top = xs[0];
#pragma unroll
    for (int e = 1; e < E; ++e) top = fmaxf(top, xs[e]);
    if (top < from) return;
    uint32_t hit = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float t = place_of(r, xs[e]);  // NaN is in none
      bool in = t >= iv[0].lo && t < iv[0].hi;
      if (N > 1) in = in || (t >= iv[1].lo && t < iv[1].hi);
      if (N > 2) in = in || (t >= iv[2].lo && t < iv[2].hi);
      hit |= in ? 1u << e : 0u;
    }
    while (hit) {
      const int e = __builtin_ctz(hit);
      hit &= hit - 1;
      float x = xs[0];
#pragma unroll
      for (int j = 1; j < E; ++j) x = e == j ? xs[j] : x;
      const uint32_t p = atomicAdd(&sh.n_list, 1u);
      if (p < kCap) sh.key[p] = order_key(x, i + e);
    }
  });
  __syncthreads();
}
template <class S, class T>
__device__ __forceinline__ void list_tokens(S& sh, const Row& r, const T* __restrict__ row, int V, int n,
                                            const Interval (&iv)[3]) {
  if (n == 1)
    list_in<1>(sh, r, row, V, iv);
  else if (n == 2)
    list_in<2>(sh, r, row, V, iv);
  else
    list_in<3>(sh, r, row, V, iv);
}

// Puts the n listed tokens in order (skey).  A list that is the beginning of
// the order has its places between 0 and `far`: a long one is dealt to 1024
// equal ranges and compared within them (242 rows of 1002: 10.2 us, all
// compared with all 34); a short one is not worth the barriers.
constexpr int kShortList = 128;
template <class S>
__device__ __forceinline__ void rank_by_ranges(S& sh, const Row& r, int n, float far) {
  const int tid = threadIdx.x;
  uint32_t* start = sh.bins.count;
  start[tid] = 0;
  __syncthreads();
  const u64 key = tid < n ? sh.key[tid] : 0;
  int b = 0;
  uint32_t slot = 0;
  if (tid < n) {
    const float p = place_of(r, key_logit(key)) * ((float)kThreads / far);
    b = (int)__builtin_amdgcn_fmed3f(p, 0.f, (float)(kThreads - 1));
    slot = atomicAdd(&start[b], 1u);
  }
  __syncthreads();
  const uint32_t size = start[tid];
  uint32_t c = size, all;
  u64 none = 0, nothing;
  block_scan(none, c, sh.red[2], nothing, all);
  start[tid] = c - size;
  if (tid == kThreads - 1) start[kThreads] = c;
  __syncthreads();
  uint32_t lo = 0, hi = 0;
  if (tid < n) {
    lo = start[b];
    hi = start[b + 1];
    sh.key[lo + slot] = key;
  }
  __syncthreads();
  uint32_t rank = lo;
#pragma unroll 4
  for (uint32_t j = lo; j < hi; ++j) rank += sh.key[j] < key ? 1u : 0u;
  if (tid < n) sh.skey[rank] = key;
  __syncthreads();
}
template <class S>
__device__ __forceinline__ void rank_by_all(S& sh, int n) {
  const int tid = threadIdx.x;
  sh.rank[tid] = 0;
  __syncthreads();
  // the rank is the number of smaller keys, counted by all threads
  const int np = (n + 63) & ~63, parts = kThreads / np, i = tid % np, part = tid / np;
  if (i < n && part < parts) {
    const u64 k = sh.key[i];
    uint32_t before = 0;
#pragma unroll 8
    for (int j = part; j < n; j += parts) before += sh.key[j] < k ? 1u : 0u;
    if (parts == 1)
      sh.rank[i] = before;
    else
      atomicAdd(&sh.rank[i], before);
  }
  __syncthreads();
  if (tid < n) sh.skey[sh.rank[tid]] = sh.key[tid];
  __syncthreads();
}

// Puts the n listed tokens in order (skey) and returns, to thread i, the
// running weight up to and with token i, in *c its running count and in *own
// its weight, all from the beginning of the order: what lies between the
// listed ranges is taken from the histogram (`ranged`; else the list is the
// beginning).  far: see above, 0 where the places are not known.
template <class S>
__device__ __forceinline__ u64 order_list(S& sh, const Row& r, int n, bool ranged, float far, uint32_t* c, u64* own) {
  const int tid = threadIdx.x;
  if (far > 0.f && n > kShortList)
    rank_by_ranges(sh, r, n, far);
  else
    rank_by_all(sh, n);
  u64 m = 0, w = 0;
  uint32_t k = 0;
  if (tid < n) {
    const float x = key_logit(sh.skey[tid]);
    w = weight<true>(r, x);
    m = w;
    k = 1;
    if (ranged) {
      const int b = range_of(r, x), pb = tid > 0 ? range_of(r, key_logit(sh.skey[tid - 1])) : -1;
      if (b != pb) {  // the first of its range: what lies since the range listed before
        m += sh.bins.mass[b] - sh.bins.mass[pb + 1];
        k += sh.bins.count[b] - sh.bins.count[pb + 1];
      }
    }
  }
  u64 mall;
  uint32_t call;
  *own = w;
  block_scan(m, k, sh.red[1], mall, call);
  *c = k;
  return m;
}

// ceil(p * mass), at least 1, p below 1
__device__ __forceinline__ u64 part_up(float p, u64 mass) {
  if (!(p > 0.f)) return 1;
  const u64 q = (u64)((double)p * 18446744073709551616.0);
  const u64 a = __umul64hi(q, mass) + (q * mass != 0 ? 1 : 0);
  return a > 0 ? a : 1;
}
// floor(u * mass) + 1, at most mass
__device__ __forceinline__ u64 part_past(float u, u64 mass) {
  if (!(u > 0.f)) return 1;
  return __umul64hi((u64)((double)fminf(u, 0.99999994f) * 18446744073709551616.0), mass) + 1;
}

// The token at which the running count or weight of the order first reaches
// `aim`, in whatever passes it takes: its index in *token, the weight up to
// and with it as the result.  For ranges with more tokens than the list holds.
template <class S, class T>
__device__ __forceinline__ u64 reach(S& sh, const Row& r, const T* __restrict__ row, int V, u64 aim,
                                     bool by_count, int* token) {
  constexpr int E = 16 / sizeof(T);
  u64 m0 = 0, c0 = 0;      // before the tokens looked at
  u64 lo = 0, hi = ~0ull;  // their keys lie from lo to hi
  int bin = -1;            // their range (-1: any)
  bool first = true;
  while (true) {
    int shift = 0;  // the histogram's ranges are of 2^shift keys, but the first one's
    if (!first) {
      // the least and the largest key that there are
      u64 a = ~0ull, b = 0;
      for_row<1>(row, V, [&](int i, const float (&xs)[E]) {
#pragma unroll 1
        for (int e = 0; e < E; ++e) {
          const float x = r.clean(xs[e]);
          const u64 k = order_key(x, i + e);
          if (k < lo || k > hi || range_of(r, x) != bin || weight<true>(r, x) == 0) continue;
          a = min(a, k);
          b = max(b, k);
        }
      });
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) {
        a = min(a, (u64)__shfl_xor((long long)a, d, 64));
        b = max(b, (u64)__shfl_xor((long long)b, d, 64));
      }
      __syncthreads();
      if ((threadIdx.x & 63) == 0) {
        sh.key[threadIdx.x >> 6] = a;
        sh.skey[threadIdx.x >> 6] = b;
      }
      __syncthreads();
      lo = sh.key[0];
      hi = sh.skey[0];
      for (int i = 1; i < kWaves; ++i) {
        lo = min(lo, sh.key[i]);
        hi = max(hi, sh.skey[i]);
      }
      while (((hi - lo) >> shift) >= kBins) ++shift;
    }
    clear_bins(sh);
    for_row<1>(row, V, [&](int i, const float (&xs)[E]) {
#pragma unroll 1
      for (int e = 0; e < E; ++e) {
        const float x = r.clean(xs[e]);
        const u64 w = weight<true>(r, x);
        if (w == 0) continue;
        const int b = range_of(r, x);
        int at = b;
        if (!first) {
          const u64 k = order_key(x, i + e);
          if (b != bin || k < lo || k > hi) continue;
          at = (int)((k - lo) >> shift);
        }
        atomicAdd(&sh.bins.mass[at], w);
        atomicAdd(&sh.bins.count[at], 1u);
      }
    });
    __syncthreads();
    u64 mall;
    uint32_t call;
    const Ends e = scan_bins(sh, mall, call);
    if (by_count)
      find_count(e, (uint32_t)(aim - c0), &sh.bin[0]);
    else
      find_mass(e, aim - m0, &sh.bin[0]);
    __syncthreads();
    const int at = sh.bin[0];
    const uint32_t size = sh.bins.count[at + 1] - sh.bins.count[at];
    m0 += sh.bins.mass[at];
    c0 += sh.bins.count[at];
    if (first) {
      bin = at;
    } else {
      lo += (u64)at << shift;
      hi = min(hi, lo + ((1ull << shift) - 1));
    }
    first = false;
    if (size <= kCap) break;
  }
  if (threadIdx.x == 0) sh.n_list = 0;
  __syncthreads();
  for_row<1>(row, V, [&](int i, const float (&xs)[E]) {
#pragma unroll 1
    for (int e = 0; e < E; ++e) {
      const float x = r.clean(xs[e]);
      const u64 k = order_key(x, i + e);
      if (range_of(r, x) != bin || k < lo || k > hi || weight<true>(r, x) == 0) continue;
      sh.key[atomicAdd(&sh.n_list, 1u)] = k;
    }
  });
  __syncthreads();
  const int n = (int)sh.n_list;
  uint32_t c;
  u64 w;
  const u64 m = order_list(sh, r, n, false, 0.f, &c, &w);
  if ((int)threadIdx.x < n) {
    const u64 left = aim - (by_count ? c0 : m0);
    if (by_count ? left == c : m - w < left && left <= m) {
      sh.got[0] = m0 + m;
      sh.got[1] = sh.skey[threadIdx.x] & 0xffffffffu;
    }
  }
  __syncthreads();
  *token = (int)sh.got[1];
  const u64 got = sh.got[0];
  __syncthreads();
  return got;
}

// --- counts of every bf16 value ---------------------------------------------
// Values in falling order: place 0 .. 32767 those without the sign, from bits
// 0x7fff down, then those with it, from 0x8000 (-0, the same value as the one
// before) up.  The ends are NaN.
constexpr int kPlus0 = 32767, kMinus0 = 32768, kPlusInf = 0x7fff - 0x7f80;
__device__ __forceinline__ float value_at(int place) {
  return bf2f(place <= kPlus0 ? (uint32_t)(kPlus0 - place) : (uint32_t)place);
}
template <class S>
__device__ __forceinline__ uint32_t count_at(const S& sh, int place) {
  return place <= kPlus0 ? sh.words[kPlus0 - place] & 0xffffu : sh.words[place - kMinus0] >> 16;
}
constexpr int kGroup = kValues / kThreads;  // places of a group: a lane each, and a thread's share of the running sums
static_assert(kGroup == 64, "a lane a place");

// The place at which the running count or weight reaches `aim`, given the
// running numbers before (c0, m0) and with (c1, m1) each thread's group of
// places: the thread names its group, the first wave looks at the places side
// by side.  The place in *place, how many of its tokens are needed in *nth, the
// running weight with them as the result.
template <class S>
__device__ __forceinline__ u64 reach_value(S& sh, const Row& r, u64 aim, bool by_count, u64 m0, u64 m1, uint32_t c0,
                                           uint32_t c1, int* place, uint32_t* nth) {
  const int tid = threadIdx.x;
  if (by_count ? c0 < aim && aim <= c1 : m0 < aim && aim <= m1) {
    sh.bin[0] = tid;
    sh.got[0] = m0;
    sh.got[1] = c0;
  }
  __syncthreads();
  if (tid < 64) {
    const int at = sh.bin[0] * kGroup + tid;
    const float x = value_at(at);
    const bool has = at >= kPlusInf && x > r.least;  // no NaN
    const uint32_t n = has ? count_at(sh, at) : 0;
    const u64 w = has ? weight(r, x) : 0;
    const u64 m = wave_scan((u64)n * w) + sh.got[0], mb = m - n * w;
    const uint32_t c = wave_scan(n) + (uint32_t)sh.got[1], cb = c - n;
    if (by_count ? cb < aim && aim <= c : mb < aim && aim <= m) {
      const uint32_t need = by_count ? (uint32_t)aim - cb : (uint32_t)((aim - mb + w - 1) / w);
      sh.bin[1] = at;
      sh.bin[2] = (int)need;
      sh.got[2] = mb + need * w;
    }
  }
  __syncthreads();
  *place = sh.bin[1];
  *nth = (uint32_t)sh.bin[2];
  return sh.got[2];
}

// A row of bf16 logits by the counts of their values: one pass counts, then
// all is settled among the values but for the index of the token drawn, which
// another pass finds.  False (nothing drawn) where a count overran its 16
// bits, the numbers are past those of any model, or more tokens than the list
// holds share the value drawn.
template <class S>
__device__ __forceinline__ bool sample_values(S& sh, const uint16_t* __restrict__ row, int V, float temp, int top_k,
                                              float top_p, float min_p, float u, int32_t* out) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  constexpr int kClear = kValues / 2 / 4 / kThreads;
  uint4* words = reinterpret_cast<uint4*>(sh.words);
#pragma unroll
  for (int i = 0; i < kClear; ++i) words[i * kThreads + tid] = make_uint4(0u, 0u, 0u, 0u);
  u64* group_mass = sh.key;
  uint32_t* group_count = sh.rank;
  group_mass[tid] = 0;
  group_count[tid] = 0;
  if (tid == 0) sh.n_list = 0;
  __syncthreads();
  float mx = kNone;
  for_row<4>(row, V, [&](int, const float (&xs)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t b = __float_as_uint(xs[e]);
      mx = fmaxf(mx, xs[e]);
      atomicAdd(&sh.words[(b >> 16) & 0x7fffu], (b >> 31) ? 0x10000u : 1u);
    }
  });
  __syncthreads();
  // the largest logit; all counts together tell whether one overran (the
  // pieces at the ends of the row count a NaN for each logit that they lack)
  uint32_t sum = 0, all_held;
  u64 none = 0, nothing;
#pragma unroll
  for (int i = 0; i < kClear; ++i) {
    const uint4 w = words[i * kThreads + tid];
    sum = __builtin_amdgcn_sad_u16(w.x, 0, sum);
    sum = __builtin_amdgcn_sad_u16(w.y, 0, sum);
    sum = __builtin_amdgcn_sad_u16(w.z, 0, sum);
    sum = __builtin_amdgcn_sad_u16(w.w, 0, sum);
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d, 64));
  if (lane == 0) sh.redf[0][wave] = mx;
  block_scan(none, sum, sh.red[0], nothing, all_held);
#pragma unroll
  for (int w = 0; w < kWaves; ++w) mx = fmaxf(mx, sh.redf[0][w]);
  const int head = min(V, (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / 2));
  if (all_held != (uint32_t)(V + 7 * (head + (V - head) % 8))) return false;
  if (mx == kNone) {  // nothing to draw from
    if (tid == 0) *out = -1;
    return true;
  }
  float x = mx;
  uint32_t nth = 1;
  int place = -1;
  if (temp > 0.f) {
    if (!(fabsf(mx) <= 1e30f && temp >= 1e-20f && temp <= 1e20f)) return false;
    temp = warm(mx, temp);
    Row r;
    r.mx = mx;
    r.scale = 1.4426950408889634074 / (double)temp;
    r.least = least_of(mx, temp);
    r.top = false;
    r.fit = r.fit0 = 0.f;
    const u64 least = min_p > 0.f ? (u64)ceil((double)fminf(min_p, 1.f) * (double)(1ull << kFrac)) : 0ull;
    // weight and count of the groups that hold the largest logit down to r.least
    auto group_of = [](float v) {
      const uint32_t b = __float_as_uint(v) >> 16;
      return (int)((b & 0x8000u) ? b : kPlus0 - b) / kGroup;
    };
    const int last = group_of(r.least);
    u64 strong = 0;
    int g = group_of(mx) + wave;
    uint32_t next = count_at(sh, min(g, last) * kGroup + lane);
    for (; g <= last; g += kWaves) {
      uint32_t n = next;
      next = count_at(sh, min(g + kWaves, last) * kGroup + lane);
      if (__ballot(n != 0) == 0) continue;  // most are empty
      const int at = g * kGroup + lane;
      const float v = value_at(at);
      if (at < kPlusInf || !(v > r.least)) n = 0;
      const u64 w = n != 0 ? weight(r, v) : 0;
      const u64 m = wave_scan(n * w);
      if (w >= least) strong += n * w;
      if (lane == 63) group_mass[g] = m;
      if (top_k > 0) {
        const uint32_t c = wave_scan(n);
        if (lane == 63) group_count[g] = c;
      }
    }
    __syncthreads();
    const u64 m = group_mass[tid];
    const uint32_t n = group_count[tid];
    u64 m1 = m, all, kept;
    uint32_t c1 = n, live, zero = 0;
    block_scan(m1, c1, sh.red[1], all, live);
    if (least != 0) {
      block_scan(strong, zero, sh.red[2], kept, zero);
    } else {
      kept = all;
    }
    const u64 m0 = m1 - m;
    const uint32_t c0 = c1 - n;
    u64 mass = all;
    if (top_k > 0 && (uint32_t)top_k < live)
      mass = reach_value(sh, r, (u64)top_k, true, m0, m1, c0, c1, &place, &nth);
    if (top_p < 1.f) mass = reach_value(sh, r, part_up(top_p, mass), false, m0, m1, c0, c1, &place, &nth);
    reach_value(sh, r, part_past(u, min(mass, kept)), false, m0, m1, c0, c1, &place, &nth);
    x = value_at(place);
  }
  // the nth token of that value (0: of either sign, those without it first)
  const uint32_t b = __float_as_uint(x) >> 16;
  uint32_t same;
  if ((b & 0x7fffu) == 0) {
    const uint32_t n0 = count_at(sh, kPlus0);
    same = n0 + count_at(sh, kMinus0);
    if (place == kMinus0) nth += n0;
  } else {
    same = count_at(sh, (b & 0x8000u) ? (int)b : kPlus0 - (int)b);
  }
  if (same > kCap) return false;
  uint32_t* list = sh.rank;  // the groups' counts are not needed any more
  for_row<4>(row, V, [&](int i, const float (&xs)[8]) {
    uint32_t hit = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) hit |= xs[e] == x ? 1u << e : 0u;
    while (hit) {
      const int e = __builtin_ctz(hit);
      hit &= hit - 1;
      list[atomicAdd(&sh.n_list, 1u)] = (uint32_t)(i + e);
    }
  });
  __syncthreads();
  if (tid < (int)same) {
    const uint32_t i = list[tid];
    uint32_t before = 0;
#pragma unroll 4
    for (uint32_t j = 0; j < same; ++j) before += list[j] < i ? 1u : 0u;
    if (before == nth - 1) *out = (int32_t)i;
  }
  return true;
}

template <class T>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs a) {
  __shared__ SharedOf<sizeof(T) == 2> sh;
  constexpr int E = 16 / sizeof(T);
  const int row_i = blockIdx.x, V = a.V, tid = threadIdx.x;
  const T* row = static_cast<const T*>(a.logits) + row_i * a.stride;
  float temp = a.temperature ? a.temperature[row_i] : 1.f;
  const int top_k = a.top_k ? a.top_k[row_i] : 0;
  const float top_p = a.top_p ? a.top_p[row_i] : 1.f;
  const float min_p = a.min_p ? a.min_p[row_i] : 0.f;
  const float u = a.u[row_i];

  if constexpr (sizeof(T) == 2) {
    if (V >= kValueVocab && !(temp > 0.f && top_k > 0 && top_k <= kSmallK)) {
      if (sample_values(sh, row, V, temp, top_k, top_p, min_p, u, a.out + row_i)) return;
      __syncthreads();
    }
  }

  // the largest and the smallest logit (fmax and fmin pass over NaN)
  float mx = kNone, mn = -kNone;
  for_row<4>(row, V, [&](int, const float (&xs)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      mx = fmaxf(mx, xs[e]);
      mn = fminf(mn, xs[e]);
    }
  });
  const float mine = mx;
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    mx = fmaxf(mx, __shfl_xor(mx, d, 64));
    mn = fminf(mn, __shfl_xor(mn, d, 64));
  }
  if ((tid & 63) == 0) {
    sh.redf[0][tid >> 6] = mx;
    sh.redf[1][tid >> 6] = mn;
  }
  if (tid == 0) sh.n_list = 0;
  sh.rank[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    mx = fmaxf(mx, sh.redf[0][w]);
    mn = fminf(mn, sh.redf[1][w]);
  }
  if (mx == kNone) {  // nothing to draw from
    if (tid == 0) a.out[row_i] = -1;
    return;
  }
  if (!(temp > 0.f)) {  // the first of the largest
    int at = 0x7fffffff;
    for_row<4>(row, V, [&](int i, const float (&xs)[E]) {
#pragma unroll
      for (int e = E - 1; e >= 0; --e)
        if (xs[e] == mx) at = min(at, i + e);
    });
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) at = min(at, __shfl_xor(at, d, 64));
    if ((tid & 63) == 0) sh.red[0].c[tid >> 6] = (uint32_t)at;
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < kWaves; ++w) at = min(at, (int)sh.red[0].c[w]);
      a.out[row_i] = at;
    }
    return;
  }

  Row r;
  r.top = mx == -kNone;
  const u64 least = min_p > 0.f ? (u64)ceil((double)fminf(min_p, 1.f) * (double)(1ull << kFrac)) : 0ull;
  const bool limit_p = top_p < 1.f;
  // The ranges run over what has a weight, down to 30 nats or the smallest
  // logit.  Numbers past those of any model take the passes of `reach` alone.
  const bool plain = fabsf(mx) <= 1e30f && temp >= 1e-20f && temp <= 1e20f;
  if (plain) temp = warm(mx, temp);
  if (r.top) mx = mn = 0.f;
  r.mx = mx;
  r.scale = 1.4426950408889634074 / (double)temp;
  r.least = least_of(mx, temp);
  const float span = fminf(mx - mn, 30.f * temp);
  r.fit = span > 0.f ? fminf((float)kBins / span, 1e36f / fmaxf(fabsf(mx), 1.f)) : 0.f;
  r.fit0 = mx * r.fit;

  // the list: for a small vocabulary all that has a weight, for a small top-k
  // the tokens down to the least of the k largest of the threads' maxima, else,
  // and where those are more than it holds, the ranges in which the running
  // numbers get to where they have to
  Interval iv[3];
  const float end = next_up(place_of(r, r.least));
  iv[0] = {kNone, end};
  int n_iv = V <= kCap ? 1 : 0;
  if (plain && n_iv == 0 && top_k > 0 && top_k <= kSmallK) {
    // by a histogram of them over ranges four times as wide (the counts cleared above)
    const int b = mine != kNone ? range_of(r, mine) / kPer : -1;
    if (b >= 0) atomicAdd(&sh.rank[b], 1u);
    __syncthreads();
    const uint32_t own = sh.rank[tid];
    uint32_t c = own, call;
    u64 none = 0, nothing;
    block_scan(none, c, sh.red[0], nothing, call);
    if (c - own < (uint32_t)top_k && (uint32_t)top_k <= c) sh.bin[0] = tid;
    __syncthreads();
    if ((uint32_t)top_k <= call) {
      const int last = sh.bin[0];
      iv[0].hi = last < kThreads - 1 ? (float)((last + 1) * kPer) : end;
      n_iv = 1;
    }
  }
  bool ranged = n_iv == 0;
  u64 kept = ~0ull, all = 0;  // weight that min-p keeps; of all tokens
  uint32_t live = 0;          // tokens that may have a weight
  int n = kCap + 1;
  if (plain && !ranged) {
    list_tokens(sh, r, row, V, n_iv, iv);
    n = (int)sh.n_list;
    if (n > kCap) {
      __syncthreads();
      if (tid == 0) sh.n_list = 0;
      ranged = true;
      n_iv = 0;
    }
  }
  if (plain && ranged) {
    clear_bins(sh);
    u64 strong = histogram(sh, r, row, V, least, top_k > 0);
    uint32_t none = 0;
    __syncthreads();
    const Ends e = scan_bins(sh, all, live);
    if (least != 0) {
      u64 sum;
      block_scan(strong, none, sh.red[2], sum, none);
      kept = sum;
    }
    // the ranges in which each number is reached, from the first that it can
    // be to the last: top-k's, then with its weight between the ends of that
    // range top-p's, and so on
    u64 mlo = all, mhi = all;
    int pl = -1, ph = -1;
    auto add = [&](int l, int h) {
      if (l != pl || h != ph) iv[n_iv++] = {l > 0 ? (float)l : kNone, h < kBins - 1 ? (float)(h + 1) : end};
      pl = l;
      ph = h;
    };
    if (top_k > 0 && (uint32_t)top_k < live) {
      find_count(e, (uint32_t)top_k, &sh.bin[0]);
      __syncthreads();
      add(sh.bin[0], sh.bin[0]);
      mlo = sh.bins.mass[pl] + 1;
      mhi = sh.bins.mass[ph + 1];
    }
    if (limit_p) {
      find_mass(e, part_up(top_p, mlo), &sh.bin[2]);
      find_mass(e, part_up(top_p, mhi), &sh.bin[3]);
      __syncthreads();
      add(sh.bin[2], sh.bin[3]);
      mlo = sh.bins.mass[pl] + 1;
      mhi = sh.bins.mass[ph + 1];
    }
    find_mass(e, part_past(u, min(mlo, kept)), &sh.bin[4]);
    find_mass(e, part_past(u, min(mhi, kept)), &sh.bin[5]);
    __syncthreads();
    add(sh.bin[4], sh.bin[5]);
    list_tokens(sh, r, row, V, n_iv, iv);
    n = (int)sh.n_list;
  }
  if (n <= kCap) {
    uint32_t c;
    u64 w;
    const u64 m = order_list(sh, r, n, ranged, ranged ? 0.f : iv[0].hi, &c, &w);
    u64 mass = all;
    if (!ranged) {
      live = (uint32_t)n;
      if (tid == n - 1) sh.got[0] = m;
      // the last token that min-p keeps: weights fall along the order
      if (least > 0 && tid < n && w >= least && (tid == n - 1 || weight<true>(r, key_logit(sh.skey[tid + 1])) < least))
        sh.got[3] = m;
    }
    if (top_k > 0 && (uint32_t)top_k < live && tid < n && c == (uint32_t)top_k) sh.got[1] = m;
    __syncthreads();
    if (!ranged) {
      mass = sh.got[0];
      if (least > 0) kept = sh.got[3];
    }
    if (top_k > 0 && (uint32_t)top_k < live) mass = sh.got[1];
    if (limit_p) {
      const u64 aim = part_up(top_p, mass);
      if (m - w < aim && aim <= m) sh.got[2] = m;
      __syncthreads();
      mass = sh.got[2];
    }
    const u64 aim = part_past(u, min(mass, kept));
    if (m - w < aim && aim <= m) a.out[row_i] = (int32_t)(sh.skey[tid] & 0xffffffffu);
    return;
  }
  // too many tokens in a range, or numbers past those of any model: one number
  // after another
  u64 strong = 0;
  live = 0;
  all = 0;
  for_row<1>(row, V, [&](int, const float (&xs)[E]) {
#pragma unroll 1
    for (int e = 0; e < E; ++e) {
      const u64 w = weight<true>(r, r.clean(xs[e]));
      all += w;
      live += w != 0;
      if (w >= least) strong += w;
    }
  });
  u64 mass;
  uint32_t none = 0, tokens;
  __syncthreads();
  block_scan(all, live, sh.red[0], mass, tokens);
  block_scan(strong, none, sh.red[1], kept, none);
  int token = -1;
  for (int step = 0; step < 3; ++step) {
    u64 aim;
    if (step == 0) {
      if (!(top_k > 0 && (uint32_t)top_k < tokens)) continue;
      aim = (u64)top_k;
    } else if (step == 1) {
      if (!limit_p) continue;
      aim = part_up(top_p, mass);
    } else {
      aim = part_past(u, min(mass, kept));
    }
    mass = reach(sh, r, row, V, aim, step == 0, &token);
  }
  if (tid == 0) a.out[row_i] = token;
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, hipStream_t stream) {
  if (a.f32)
    MLORA_LAUNCH("sample", sample_kernel<float>, dim3(a.n), dim3(kThreads), 0, stream, a);
  else
    MLORA_LAUNCH("sample", sample_kernel<uint16_t>, dim3(a.n), dim3(kThreads), 0, stream, a);
  return launched();
}

}  // namespace mlora
