// The norm of each query and key head and the rotation by the row's position,
// in one pass over the rows.
//
// y = x * w / sqrt(mean(x^2) + eps) over the channels of a head, then the
// pairs of the first `rot` channels turn by position * freq.  freq is held as
// a fraction of a revolution in 64-bit fixed point: the product with the
// position modulo 2^64 is then the fraction of a revolution without error, at
// any position, and 32 bits of it go through an octant's series in fp32.
// Bound by memory (each element read and written once) and, for few rows, by
// the latency of the loads that find a row's position; the rows' own loads go
// out before those.  A lane takes two runs of 8 channels (8 pairs), so a
// rotation never leaves the lane; dim / 16 lanes make a head, as many heads
// as fit a wave (8 prompts of 64 heads of 80 channels: 38.2 us with four pairs
// a lane and 16 lanes for the 10 that a head needs).
#include "kv.h"
#include "qk_rotary.h"

namespace mlora {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

// sin and cos of a fraction of a revolution u / 2^32
__device__ __forceinline__ void turn(uint32_t u, float& s, float& c) {
  const uint32_t k = (u + 0x20000000u) >> 30;  // nearest quarter
  const float a = (float)(int32_t)(u - (k << 30)) * (6.28318530717958647692f / 4294967296.f);  // |a| <= pi / 4
  const float z = a * a;
  float p = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
  p = fmaf(z, p, 8.3333333e-3f);
  p = fmaf(z, p, -1.6666667e-1f);
  const float sa = fmaf(a * z, p, a);
  float q = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
  q = fmaf(z, q, -1.3888889e-3f);
  q = fmaf(z, q, 4.1666667e-2f);
  q = fmaf(z, q, -0.5f);
  const float ca = fmaf(z, q, 1.f);
  s = (k & 1) ? ca : sa;
  c = (k & 1) ? sa : ca;
  if (k & 2) s = -s;
  if ((k + 1) & 2) c = -c;
}

// the sequence of a row: the last one that starts at or before it, found by
// the whole wave 64 places at a time; -1 for a row past the last sequence
__device__ __forceinline__ int sequence_of(const int32_t* __restrict__ row_off, int n_seq, int row) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = n_seq + 1;
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) / 64, at = lo + (lane + 1) * step;
    const bool before = at < hi && row_off[at] <= row;
    const int n = (int)__popcll(__ballot(before));
    lo += n * step;
    hi = min(hi, lo + step);
  }
  return lo < n_seq ? lo : -1;
}

// Two runs of C channels of a head, `a` and `b` elements from its start, as
// packed bf16.  VEC: a run is one aligned load.
template <int C>
struct Runs {
  uint32_t w[C];  // the first run's C / 2 words, then the second's
  __device__ __forceinline__ float operator[](int e) const { return (e & 1) ? hi_bf(w[e >> 1]) : lo_bf(w[e >> 1]); }
};
template <int C, bool VEC>
__device__ __forceinline__ Runs<C> load_runs(const uint16_t* __restrict__ p, int a, int b) {
  Runs<C> r;
  if constexpr (VEC && C == 8) {
    const uint4 x = *reinterpret_cast<const uint4*>(p + a), y = *reinterpret_cast<const uint4*>(p + b);
    r = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  } else if constexpr (VEC) {
    const uint2 x = *reinterpret_cast<const uint2*>(p + a), y = *reinterpret_cast<const uint2*>(p + b);
    r = {x.x, x.y, y.x, y.y};
  } else {
#pragma unroll
    for (int e = 0; e < C / 2; ++e) {
      r.w[e] = p[a + 2 * e] | (uint32_t)p[a + 2 * e + 1] << 16;
      r.w[C / 2 + e] = p[b + 2 * e] | (uint32_t)p[b + 2 * e + 1] << 16;
    }
  }
  return r;
}
template <int C, bool VEC>
__device__ __forceinline__ void store_runs(uint16_t* __restrict__ p, int a, int b, const float (&x)[2 * C]) {
  uint32_t w[C];
#pragma unroll
  for (int e = 0; e < C; ++e) w[e] = pack_bf2_hw(x[2 * e], x[2 * e + 1]);
  if constexpr (VEC && C == 8) {
    *reinterpret_cast<uint4*>(p + a) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(p + b) = make_uint4(w[4], w[5], w[6], w[7]);
  } else if constexpr (VEC) {
    *reinterpret_cast<uint2*>(p + a) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(p + b) = make_uint2(w[2], w[3]);
  } else {
#pragma unroll
    for (int e = 0; e < C / 2; ++e) {
      p[a + 2 * e] = (uint16_t)w[e];
      p[a + 2 * e + 1] = (uint16_t)(w[e] >> 16);
      p[b + 2 * e] = (uint16_t)w[C / 2 + e];
      p[b + 2 * e + 1] = (uint16_t)(w[C / 2 + e] >> 16);
    }
  }
}

// Sum over a head's g neighbouring lanes (u: this one's place, l0: the first):
// runs of 1, 2, 4, .. lanes from each on, round the head, of which those that
// g's bits name make the whole.
__device__ __forceinline__ float head_sum(float v, int g, int u, int l0) {
  float sum = 0.f;
  int off = 0;
  for (int n = 1; n <= g; n <<= 1) {
    if (g & n) {
      sum += off ? __shfl(v, l0 + (u + off < g ? u + off : u + off - g), 64) : v;
      off += n;
    }
    if (2 * n <= g) v += __shfl(v, l0 + (u + n < g ? u + n : u + n - g), 64);
  }
  return sum;
}

// A wave takes `iters` runs of `hw` heads of a row, the queries' heads first,
// then the keys'; g lanes a head (inv: 65536 / g rounded up).
template <int C, bool VEC>
__global__ __launch_bounds__(kThreads) void qk_rotary_kernel(QkRotary a, int g, int inv, int hw, int per_row, int iters) {
  const int lane = threadIdx.x & 63;
  const long wv = (long)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = (int)(wv / per_row);
  if (row >= a.n_rows) return;
  const int hl = (lane * inv) >> 16, l0 = hl * g, u = lane - l0;  // this lane's head and its place there
  const int h0 = (int)(wv % per_row) * iters * hw + hl;
  const int heads = a.side[0].heads + a.side[1].heads;
  // this lane's channels: a pair of runs of the two halves, or one run
  // (neighbouring pairs, and what is not rotated)
  const int half = a.rot / 2;
  const bool mine = hl < hw, rotated = u < a.rot / (2 * C);
  const int at = rotated && !a.interleaved ? C * u : 2 * C * u, bt = rotated && !a.interleaved ? half + C * u : at + C;

  auto load = [&](int h) {
    h = min(h, heads - 1);
    const bool key = h >= a.side[0].heads;
    const QkSide& s = a.side[key];
    return load_runs<C, VEC>(s.x + row * s.rs + (h - (key ? a.side[0].heads : 0)) * s.hs, at, bt);
  };
  Runs<C> next = load(h0), wq{}, wk{};
  if (a.side[0].w) wq = load_runs<C, VEC>(a.side[0].w, at, bt);
  if (a.side[1].w) wk = load_runs<C, VEC>(a.side[1].w, at, bt);
  uint64_t f[C];
#pragma unroll
  for (int e = 0; e < C; ++e) f[e] = rotated ? a.freq[C * u + e] : 0;

  const int seq = sequence_of(a.row_off, a.n_seq, row);
  if (seq < 0) return;  // past the last sequence: left alone
  KvView c{};
  c.row_off = a.row_off;
  c.kv_len = a.kv_len;
  c.n_rows = a.n_rows;
  const KvSeq sq = kv_seq(c, seq);
  if (row < sq.row0 || row >= sq.row0 + sq.m) return;
  const int pos = sq.n - sq.m + (row - sq.row0);
  float sn[C], cs[C];
#pragma unroll
  for (int e = 0; e < C; ++e) {
    turn((uint32_t)((f[e] * (uint64_t)(int64_t)pos) >> 32), sn[e], cs[e]);
    sn[e] *= a.factor;
    cs[e] *= a.factor;
  }

  for (int i = 0; i < iters; ++i) {
    const int h = h0 + i * hw;
    const Runs<C> in = next;
    if (i + 1 < iters) next = load(h + hw);
    const bool key = h >= a.side[0].heads;
    const QkSide& s = a.side[key];
    float x[2 * C];
#pragma unroll
    for (int e = 0; e < 2 * C; ++e) x[e] = in[e];
    if (a.side[0].w || a.side[1].w) {
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 2 * C; ++e) sum = fmaf(x[e], x[e], sum);
      sum = head_sum(sum, g, u, l0);
      if (s.w) {
        const float r = 1.f / sqrtf(sum / (float)a.D + a.eps);
#pragma unroll
        for (int e = 0; e < 2 * C; ++e) x[e] *= r * (key ? wk[e] : wq[e]);
      }
    }
    if (rotated) {
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < C; ++e) {
          const float l = x[2 * e], r = x[2 * e + 1];
          x[2 * e] = l * cs[e] - r * sn[e];
          x[2 * e + 1] = l * sn[e] + r * cs[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < C; ++e) {
          const float l = x[e], r = x[C + e];
          x[e] = l * cs[e] - r * sn[e];
          x[C + e] = l * sn[e] + r * cs[e];
        }
      }
    }
    if (mine && h < heads)
      store_runs<C, VEC>(s.y + row * s.ors + (h - (key ? a.side[0].heads : 0)) * s.ohs, at, bt, x);
  }
}

template <int C, bool VEC>
hipError_t launch(const QkRotary& a, hipStream_t st) {
  const int g = a.D / (2 * C), hw = 64 / g, inv = (65536 + g - 1) / g;
  const int runs = (a.side[0].heads + a.side[1].heads + hw - 1) / hw;
  // a run a wave up to 4096 of them, then more, so that the position and its
  // angles serve several (1571 rows of 36 heads of 256 channels 12.9 us, up to
  // 16384 of them 16.2)
  int iters = (int)((long)a.n_rows * runs / 4096);
  iters = iters < 1 ? 1 : (iters > runs ? runs : iters);
  const int per_row = (runs + iters - 1) / iters;
  const long waves = (long)a.n_rows * per_row;
  MLORA_LAUNCH("qk_norm_rotary", (qk_rotary_kernel<C, VEC>), dim3((unsigned)((waves + kWaves - 1) / kWaves)),
               dim3(kThreads), 0, st, a, g, inv, hw, per_row, iters);
  return launched();
}

}  // namespace

hipError_t launch_qk_rotary(const QkRotary& a, hipStream_t stream) {
  uintptr_t ends = 0;  // of all addresses and strides, in bytes
  for (const QkSide& s : a.side) {
    if (s.heads == 0) continue;
    ends |= reinterpret_cast<uintptr_t>(s.x) | reinterpret_cast<uintptr_t>(s.y) | reinterpret_cast<uintptr_t>(s.w) |
            (uintptr_t)(2 * (s.rs | s.hs | s.ors | s.ohs));
  }
  if (ends % 16 == 0 && a.rot % 16 == 0) return launch<8, true>(a, stream);
  if (ends % 8 == 0) return launch<4, true>(a, stream);
  return launch<4, false>(a, stream);
}

}  // namespace mlora
