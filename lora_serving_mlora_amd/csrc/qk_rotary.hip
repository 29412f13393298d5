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
// out before those.  A unit of 8 channels (four pairs) is a lane's share, so a
// rotation never leaves the lane; 2 .. 32 lanes make a head.
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

// 8 channels of a head: two runs of four, `a` and `b` elements from its start
template <bool VEC>
__device__ __forceinline__ void load_unit(const uint16_t* __restrict__ p, int a, int b, float (&x)[8]) {
  if (VEC) {
    const uint2 l = *reinterpret_cast<const uint2*>(p + a), h = *reinterpret_cast<const uint2*>(p + b);
    x[0] = lo_bf(l.x); x[1] = hi_bf(l.x); x[2] = lo_bf(l.y); x[3] = hi_bf(l.y);
    x[4] = lo_bf(h.x); x[5] = hi_bf(h.x); x[6] = lo_bf(h.y); x[7] = hi_bf(h.y);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = bf2f(p[a + e]);
      x[4 + e] = bf2f(p[b + e]);
    }
  }
}
template <bool VEC>
__device__ __forceinline__ void store_unit(uint16_t* __restrict__ p, int a, int b, const float (&x)[8]) {
  if (VEC) {
    *reinterpret_cast<uint2*>(p + a) = make_uint2(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]));
    *reinterpret_cast<uint2*>(p + b) = make_uint2(pack_bf2(x[4], x[5]), pack_bf2(x[6], x[7]));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      p[a + e] = (uint16_t)f2bf(x[e]);
      p[b + e] = (uint16_t)f2bf(x[4 + e]);
    }
  }
}

// L lanes a head; a wave takes `iters` runs of 64 / L heads of a row, the
// queries' heads first, then the keys'
template <int L, bool VEC>
__global__ __launch_bounds__(kThreads) void qk_rotary_kernel(QkRotary a, int per_row, int iters) {
  constexpr int HW = 64 / L;
  const int lane = threadIdx.x & 63;
  const long wv = (long)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = (int)(wv / per_row);
  if (row >= a.n_rows) return;
  const int h0 = (int)(wv % per_row) * iters * HW + lane / L;
  const int heads = a.side[0].heads + a.side[1].heads;
  // this lane's channels: a pair of runs of four of the two halves, or eight
  // neighbours (pairs of neighbours, and what is not rotated)
  const int u = lane % L, half = a.rot / 2;
  const bool mine = u < a.D / 8, rotated = mine && u < a.rot / 8;
  int at, bt;
  if (rotated && !a.interleaved) {
    at = 4 * u;
    bt = half + 4 * u;
  } else {
    at = 8 * (mine ? u : 0);
    bt = at + 4;
  }

  auto place = [&](int h, const uint16_t*& p) {
    const QkSide& s = a.side[h >= a.side[0].heads];
    p = s.x + row * s.rs + (h - (h >= a.side[0].heads ? a.side[0].heads : 0)) * s.hs;
  };
  float x[8], nx[8];
  const uint16_t* p;
  place(min(h0, heads - 1), p);
  load_unit<VEC>(p, at, bt, x);
  uint64_t f[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = rotated ? a.freq[4 * u + e] : 0;

  const int seq = sequence_of(a.row_off, a.n_seq, row);
  if (seq < 0) return;  // past the last sequence: left alone
  KvView c{};
  c.row_off = a.row_off;
  c.kv_len = a.kv_len;
  c.n_rows = a.n_rows;
  const KvSeq sq = kv_seq(c, seq);
  if (row < sq.row0 || row >= sq.row0 + sq.m) return;
  const int pos = sq.n - sq.m + (row - sq.row0);
  float sn[4], cs[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    turn((uint32_t)((f[e] * (uint64_t)(int64_t)pos) >> 32), sn[e], cs[e]);
    sn[e] *= a.factor;
    cs[e] *= a.factor;
  }

  for (int i = 0; i < iters; ++i) {
    const int h = h0 + i * HW;
    if (i + 1 < iters) {
      place(min(h + HW, heads - 1), p);
      load_unit<VEC>(p, at, bt, nx);
    }
    const QkSide& s = a.side[h >= a.side[0].heads];
    if (s.w) {
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
      if (!mine) sum = 0.f;
#pragma unroll
      for (int d = L / 2; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, 64);
      const float inv = 1.f / sqrtf(sum / (float)a.D + a.eps);
      float w[8];
      load_unit<VEC>(s.w, at, bt, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= inv * w[e];
    }
    if (rotated) {
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float l = x[2 * e], r = x[2 * e + 1];
          x[2 * e] = l * cs[e] - r * sn[e];
          x[2 * e + 1] = l * sn[e] + r * cs[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float l = x[e], r = x[4 + e];
          x[e] = l * cs[e] - r * sn[e];
          x[4 + e] = l * sn[e] + r * cs[e];
        }
      }
    }
    if (mine && h < heads)
      store_unit<VEC>(s.y + row * s.ors + (h - (h >= a.side[0].heads ? a.side[0].heads : 0)) * s.ohs, at, bt, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = nx[e];
  }
}

template <int L>
hipError_t launch(const QkRotary& a, bool vec, hipStream_t st) {
  constexpr int HW = 64 / L;
  const int runs = (a.side[0].heads + a.side[1].heads + HW - 1) / HW;
  // a run a wave while that fills the chip, then more, so that the position
  // and its angles serve several
  int iters = (int)((long)a.n_rows * runs / 16384);
  iters = iters < 1 ? 1 : (iters > runs ? runs : iters);
  const int per_row = (runs + iters - 1) / iters;
  const long waves = (long)a.n_rows * per_row;
  const dim3 g((unsigned)((waves + kWaves - 1) / kWaves)), b(kThreads);
  if (vec)
    MLORA_LAUNCH("qk_norm_rotary", (qk_rotary_kernel<L, true>), g, b, 0, st, a, per_row, iters);
  else
    MLORA_LAUNCH("qk_norm_rotary", (qk_rotary_kernel<L, false>), g, b, 0, st, a, per_row, iters);
  return launched();
}

}  // namespace

hipError_t launch_qk_rotary(const QkRotary& a, hipStream_t stream) {
  bool vec = true;  // 8-byte aligned runs of four everywhere
  for (const QkSide& s : a.side) {
    if (s.heads == 0) continue;
    vec = vec && ((reinterpret_cast<uintptr_t>(s.x) | reinterpret_cast<uintptr_t>(s.y) |
                   reinterpret_cast<uintptr_t>(s.w)) % 8 == 0) &&
          (s.rs | s.hs | s.ors | s.ohs) % 4 == 0;
  }
  if (a.D <= 16) return launch<2>(a, vec, stream);
  if (a.D <= 32) return launch<4>(a, vec, stream);
  if (a.D <= 64) return launch<8>(a, vec, stream);
  if (a.D <= 128) return launch<16>(a, vec, stream);
  return launch<32>(a, vec, stream);
}

}  // namespace mlora
