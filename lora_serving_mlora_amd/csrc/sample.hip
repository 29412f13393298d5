// Sampling of one token a row from its logits: temperature, top-k, top-p and
// min-p of each row's own, and a given random number.
//
// Weights are w = 2^((l - max) log2(e) / T) in 64 bits, rounded to whole
// multiples of 2^-42, so that sums of them are integers and come out the same
// in any order.  Tokens stand in the order of falling logits, lower index
// first; what top-k, top-p and min-p keep is a beginning of that order, and
// the token drawn is the one at which the running weight passes u times the
// weight kept.  So all that is asked of the order is where its running count
// or weight reaches a given number.  A histogram over the logits (count and
// weight of 2048 equal ranges from the largest down) finds the range, and the
// few tokens of that range are compared among themselves; nothing is sorted.
#include "sample.h"

namespace mlora {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBins = 2048, kCap = 2048;
constexpr int kFrac = 42;  // a weight of 1 is 2^42: 2^20 of them stay below 2^63
constexpr float kNone = -__builtin_huge_valf();

struct Shared {
  u64 mass[kBins];
  uint32_t count[kBins];
  u64 key[kCap];  // tokens of the range: order, index
  u64 w[kCap];
  u64 red[kWaves];
  uint32_t redc[kWaves];
  float redf[2][kWaves];
  int redi[kWaves];
  u64 res[4];  // what one thread found for all
  uint32_t n_list;
  int bin;
};

// bf16 or fp32 logits as floats: NaN counts as -infinity, -0 as 0
__device__ __forceinline__ float clean(float x) { return x == x ? x + 0.f : kNone; }

// f(index, logit) for every logit of the row that falls to this thread, in
// rising order of the index; 16-byte loads between the ends
template <class T, class F>
__device__ __forceinline__ void for_row(const T* __restrict__ row, int V, F f) {
  constexpr int E = 16 / sizeof(T);
  const int tid = threadIdx.x;
  const int head = min(V, (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(T)));
  const int body = (V - head) / E;
  auto one = [&](int i) {
    if constexpr (sizeof(T) == 2)
      f(i, clean(bf2f(row[i])));
    else
      f(i, clean(row[i]));
  };
  if (tid < head) one(tid);
  const uint4* p = reinterpret_cast<const uint4*>(row + head);
  constexpr int U = 4;
  for (int v0 = tid; v0 < body; v0 += U * kThreads) {
    uint4 x[U];
#pragma unroll
    for (int k = 0; k < U; ++k) x[k] = p[min(v0 + k * kThreads, body - 1)];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int v = v0 + k * kThreads;
      if (v < body) {
        const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
        for (int e = 0; e < E; ++e) {
          float l;
          if constexpr (sizeof(T) == 2)
            l = (e & 1) ? hi_bf(w[e >> 1]) : lo_bf(w[e >> 1]);
          else
            l = __uint_as_float(w[e]);
          f(head + v * E + e, clean(l));
        }
      }
    }
  }
  const int tail = head + body * E;
  if (tail + tid < V) one(tail + tid);
}

struct Row {
  float mx;        // largest logit
  double inv_l2;   // log2(e) / T
  float inv, fit;  // 1 / T, histogram ranges per nat
};

// weight of a logit, in multiples of 2^-42 (0 for -infinity)
__device__ __forceinline__ u64 weight(const Row& r, float x) {
  if (x == r.mx) return 1ull << kFrac;
  const double d = ((double)x - (double)r.mx) * r.inv_l2;  // <= 0, -infinity or NaN where x is -infinity
  if (!(d > -(kFrac + 1.0)) || x == kNone) return 0;
  const double n = __builtin_rint(d), f = (d - n) * 0.69314718055994530942;
  // e^f, |f| <= 0.347: the next term of the series is below 2^-52
  double p = 1.0 / 6227020800.0;
  p = fma(p, f, 1.0 / 479001600.0);
  p = fma(p, f, 1.0 / 39916800.0);
  p = fma(p, f, 1.0 / 3628800.0);
  p = fma(p, f, 1.0 / 362880.0);
  p = fma(p, f, 1.0 / 40320.0);
  p = fma(p, f, 1.0 / 5040.0);
  p = fma(p, f, 1.0 / 720.0);
  p = fma(p, f, 1.0 / 120.0);
  p = fma(p, f, 1.0 / 24.0);
  p = fma(p, f, 1.0 / 6.0);
  p = fma(p, f, 0.5);
  p = fma(p, f, 1.0);
  p = fma(p, f, 1.0);
  // adding 2^10 leaves the sum's last place at 2^-42: rounds to nearest
  const double v = ldexp(p, (int)n) + 1024.0;
  return (u64)__double_as_longlong(v) - (u64)__double_as_longlong(1024.0);
}

// histogram range of a logit with a weight: falls with the logit, never the
// other way (every step is monotone)
__device__ __forceinline__ int range_of(const Row& r, float x) {
  return x == r.mx ? 0 : (int)fminf((r.mx - x) * r.inv * r.fit, kBins - 1);
}

// place of a token in the order, rising: falling logits, then rising indices
__device__ __forceinline__ u64 order_key(float x, int i) {
  uint32_t b = __float_as_uint(x);
  b ^= (b >> 31) ? 0xffffffffu : 0x80000000u;
  return ((u64)~b << 32) | (uint32_t)i;
}
// inclusive running sum over the workgroup's threads; total in *all
template <class N>
__device__ __forceinline__ N block_scan(N v, N* red, N* all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    N o;
    if constexpr (sizeof(N) == 8)
      o = (N)__shfl_up((long long)v, d, 64);
    else
      o = (N)__shfl_up((int)v, d, 64);
    if (lane >= d) v += o;
  }
  __syncthreads();
  if (lane == 63) red[wave] = v;
  __syncthreads();
  N before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += red[w];
    total += red[w];
  }
  *all = total;
  return v + before;
}

// Where the running number of the histogram (its counts or its weights)
// first reaches `aim` (1 .. its total): that range in sh.bin, the count and
// weight before it in sh.res[0], sh.res[1].
__device__ __forceinline__ void find_bin(Shared& sh, u64 aim, bool by_count) {
  const int t = threadIdx.x;
  const u64 m0 = sh.mass[2 * t], m1 = sh.mass[2 * t + 1];
  const uint32_t c0 = sh.count[2 * t], c1 = sh.count[2 * t + 1];
  u64 mall;
  uint32_t call;
  const u64 m = block_scan(m0 + m1, sh.red, &mall) - (m0 + m1);
  const uint32_t c = block_scan(c0 + c1, sh.redc, &call) - (c0 + c1);
  const u64 b0 = by_count ? c : m, b1 = b0 + (by_count ? c0 : m0), b2 = b1 + (by_count ? c1 : m1);
  if (b0 < aim && aim <= b2) {
    const bool second = b1 < aim;
    sh.bin = 2 * t + (second ? 1 : 0);
    sh.res[0] = c + (second ? c0 : 0u);
    sh.res[1] = m + (second ? m0 : 0ull);
  }
  __syncthreads();
}

__device__ __forceinline__ void clear_bins(Shared& sh) {
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    sh.mass[i] = 0;
    sh.count[i] = 0;
  }
  __syncthreads();
}

// The token at which the running count or weight of the order first reaches
// `aim`, given the histogram of the whole row in sh: its index in *token, the
// weight up to and with it as the result.
template <class T>
__device__ u64 reach(Shared& sh, const Row& r, const T* __restrict__ row, int V, u64 aim, bool by_count, int* token) {
  find_bin(sh, aim, by_count);
  const int bin = sh.bin;
  u64 c0 = sh.res[0], m0 = sh.res[1];
  uint32_t size = sh.count[bin];
  u64 lo = 0, hi = ~0ull;  // order keys of the tokens looked at, both inside
  bool first = true;
  __syncthreads();
  while (size > kCap) {
    // too many for the list: their keys' own range in 2048 parts
    if (first) {
      u64 a = ~0ull, b = 0;
      for_row(row, V, [&](int i, float x) {
        if (weight(r, x) != 0 && range_of(r, x) == bin) {
          const u64 k = order_key(x, i);
          a = min(a, k);
          b = max(b, k);
        }
      });
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) {
        a = min(a, (u64)__shfl_xor((long long)a, d, 64));
        b = max(b, (u64)__shfl_xor((long long)b, d, 64));
      }
      if ((threadIdx.x & 63) == 0) {
        sh.key[threadIdx.x >> 6] = a;
        sh.w[threadIdx.x >> 6] = b;
      }
      __syncthreads();
      lo = sh.key[0];
      hi = sh.w[0];
      for (int i = 1; i < kWaves; ++i) {
        lo = min(lo, sh.key[i]);
        hi = max(hi, sh.w[i]);
      }
      first = false;
    }
    int shift = 0;
    while (((hi - lo) >> shift) >= kBins) ++shift;
    clear_bins(sh);
    for_row(row, V, [&](int i, float x) {
      const u64 k = order_key(x, i);
      if (k < lo || k > hi) return;
      const u64 w = weight(r, x);
      if (w == 0 || range_of(r, x) != bin) return;
      atomicAdd(&sh.mass[(k - lo) >> shift], w);
      atomicAdd(&sh.count[(k - lo) >> shift], 1u);
    });
    __syncthreads();
    find_bin(sh, aim - (by_count ? c0 : m0), by_count);
    c0 += sh.res[0];
    m0 += sh.res[1];
    size = sh.count[sh.bin];
    lo += (u64)sh.bin << shift;
    hi = min(hi, lo + ((1ull << shift) - 1));
    __syncthreads();
  }
  if (threadIdx.x == 0) sh.n_list = 0;
  __syncthreads();
  for_row(row, V, [&](int i, float x) {
    if (x == kNone || range_of(r, x) != bin) return;
    const u64 k = order_key(x, i);
    if (k < lo || k > hi) return;
    const u64 w = weight(r, x);
    if (w == 0) return;
    const uint32_t at = atomicAdd(&sh.n_list, 1u);
    sh.key[at] = k;
    sh.w[at] = w;
  });
  __syncthreads();
  const uint32_t n = sh.n_list;
  const u64 left = aim - (by_count ? c0 : m0);
  for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
    const u64 k = sh.key[i];
    u64 m = 0;
    uint32_t c = 0;
    for (uint32_t j = 0; j < n; ++j) {
      const bool before = sh.key[j] < k;
      m += before ? sh.w[j] : 0ull;
      c += before ? 1u : 0u;
    }
    const u64 b = by_count ? c : m, e = b + (by_count ? 1ull : sh.w[i]);
    if (b < left && left <= e) {
      sh.res[2] = m0 + m + sh.w[i];
      sh.res[3] = k & 0xffffffffu;
    }
  }
  __syncthreads();
  *token = (int)sh.res[3];
  const u64 got = sh.res[2];
  __syncthreads();
  return got;
}

// the histogram of the row; returns the weight of the tokens with at least `least`
template <class T>
__device__ u64 histogram(Shared& sh, const Row& r, const T* __restrict__ row, int V, u64 least) {
  clear_bins(sh);
  u64 strong = 0;
  for_row(row, V, [&](int, float x) {
    const u64 w = weight(r, x);
    if (w == 0) return;
    const int b = range_of(r, x);
    atomicAdd(&sh.mass[b], w);
    atomicAdd(&sh.count[b], 1u);
    if (w >= least) strong += w;
  });
  u64 all;
  block_scan(strong, sh.red, &all);
  __syncthreads();
  return all;
}

template <class T>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs a) {
  __shared__ Shared sh;
  const int row_i = blockIdx.x, V = a.V, tid = threadIdx.x;
  const T* row = static_cast<const T*>(a.logits) + row_i * a.stride;
  const float temp = a.temperature ? a.temperature[row_i] : 1.f;

  // the largest logit, the first token that has it, the smallest above -infinity
  float mx = kNone, mn = __builtin_huge_valf();
  int at = 0x7fffffff;
  for_row(row, V, [&](int i, float x) {
    if (x > mx) {
      mx = x;
      at = i;
    }
    if (x != kNone) mn = fminf(mn, x);
  });
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const float ox = __shfl_xor(mx, d, 64);
    const int oi = __shfl_xor(at, d, 64);
    if (ox > mx || (ox == mx && oi < at)) {
      mx = ox;
      at = oi;
    }
    mn = fminf(mn, __shfl_xor(mn, d, 64));
  }
  if ((tid & 63) == 0) {
    sh.redf[0][tid >> 6] = mx;
    sh.redf[1][tid >> 6] = mn;
    sh.redi[tid >> 6] = at;
  }
  __syncthreads();
  mx = sh.redf[0][0];
  mn = sh.redf[1][0];
  at = sh.redi[0];
  for (int w = 1; w < kWaves; ++w) {
    const float ox = sh.redf[0][w];
    if (ox > mx || (ox == mx && sh.redi[w] < at)) {
      mx = ox;
      at = sh.redi[w];
    }
    mn = fminf(mn, sh.redf[1][w]);
  }
  __syncthreads();
  if (mx == kNone || !(temp > 0.f)) {  // nothing to draw from, or the largest asked for
    if (tid == 0) a.out[row_i] = mx == kNone ? -1 : at;
    return;
  }

  Row r;
  r.mx = mx;
  r.inv_l2 = 1.4426950408889634074 / (double)temp;
  r.inv = 1.f / temp;
  // ranges over what has a weight: down to 30 nats, or to the smallest logit
  const float span = fminf((mx - mn) * r.inv, 30.f);
  r.fit = span > 0.f ? (float)kBins / span : 0.f;

  const float mp = a.min_p ? a.min_p[row_i] : 0.f;
  const u64 least = mp > 0.f ? (u64)ceil((double)fminf(mp, 1.f) * (double)(1ull << kFrac)) : 0ull;
  u64 kept = histogram(sh, r, row, V, least);  // by min-p
  u64 all;
  uint32_t live;
  block_scan(sh.mass[2 * tid] + sh.mass[2 * tid + 1], sh.red, &all);
  block_scan(sh.count[2 * tid] + sh.count[2 * tid + 1], sh.redc, &live);
  __syncthreads();

  // each filter keeps a beginning of the order, so the least of their weights is what all keep
  int token = at;
  u64 mass = all;
  const int k = a.top_k ? a.top_k[row_i] : 0;
  bool spoilt = false;  // the histogram was used for a smaller range
  auto find = [&](u64 aim, bool by_count) {
    if (spoilt) histogram(sh, r, row, V, 0);
    find_bin(sh, aim, by_count);
    spoilt = sh.count[sh.bin] > kCap;
    __syncthreads();
    return reach(sh, r, row, V, aim, by_count, &token);
  };
  if (k > 0 && (uint32_t)k < live) mass = find(k, true);
  const float tp = a.top_p ? a.top_p[row_i] : 1.f;
  if (tp < 1.f) {
    u64 aim = 1;
    if (tp > 0.f) {
      const u64 p = (u64)((double)tp * 18446744073709551616.0);
      aim = max(aim, __umul64hi(p, mass) + (p * mass != 0 ? 1 : 0));
    }
    mass = find(aim, false);
  }
  kept = min(kept, mass);
  const float u = a.u[row_i];
  u64 aim = 0;
  if (u > 0.f) aim = __umul64hi((u64)((double)fminf(u, 0.99999994f) * 18446744073709551616.0), kept);
  find(aim + 1, false);
  if (tid == 0) a.out[row_i] = token;
}

}  // namespace

size_t sample_work_bytes(int n, int V) { return 0; }

hipError_t launch_sample(const SampleArgs& a, void* work, hipStream_t stream) {
  if (a.f32)
    MLORA_LAUNCH("sample", sample_kernel<float>, dim3(a.n), dim3(kThreads), 0, stream, a);
  else
    MLORA_LAUNCH("sample", sample_kernel<uint16_t>, dim3(a.n), dim3(kThreads), 0, stream, a);
  return launched();
}

}  // namespace mlora
