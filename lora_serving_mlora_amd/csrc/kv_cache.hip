// Writing new tokens into the paged 8-bit key/value cache, and reading them
// back.  Both are bound by memory traffic (2 bytes a channel on the bf16
// side, 1 on the cache's) and, for a decode step, by the latency of a launch
// with a few dependent loads (row_off -> table -> page):
//   one new token of 256 requests (8 heads of 128 channels) written in 4.7 us
//   (5.8 .. 6.3 us between a layer's projections), the 2265 tokens of the pages
//   read back in 8.7 us;
//   6451 tokens of 8 prompts written in 13 us (40 MB, 3.1 TB/s);
//   32768 tokens read back in 44 us from memory (201 MB, 4.6 TB/s; a plain copy
//   reaches 5.2) and 32 us from the last-level cache;
//   64 histories of 1 .. 1500 tokens, 80 channels, in 17 us (5.4 TB/s).
//
// A page of one head, keys or values, is written by the waves of one
// workgroup, so its scale is found and used without another launch, and no two
// workgroups write one page.  The sequence and page of a workgroup come from
// its index in closed form: sequence i's pages start at item row_off[i] / B +
// 2 i, which leaves it at least as many items as m rows touch pages, so the
// grid is known on the host although the lengths are not, and no prefix sum is
// needed.
#include <algorithm>
#include <type_traits>

#include "kv.h"

namespace mlora {
namespace {

constexpr int kThreads = 256;
constexpr int kReadGroups = 1792;  // workgroups of the read kernel that the card holds at once

struct Item {
  int seq, blk;    // sequence, index in it of the page or token block (blk < 0: nothing to do)
  int lo, hi;      // positions of its rows of this batch
  int row;         // row of position lo
  bool kept;       // it holds older tokens of the sequence
  int id;          // page of the pool, -1 if there is none
  int row0, before;  // the sequence's first item: its first row, and its rows at negative positions
};

// The same in every lane: scalar loads.  Items hold 2^li tokens, pages 2^c.lb.
// single: every sequence has one row at most, and item i is sequence i
__device__ __forceinline__ Item find_item(const KvView& c, int item, int li, bool single) {
  Item it{};
  it.blk = -1;
  const int lane = threadIdx.x & 63;
  if (single) {
    it.seq = item;
  } else {
    // the last sequence whose items start at or before this one: the starts
    // increase, so it is their count less one (the loads do not depend on
    // each other, unlike a bisection's)
    int count = 0;
    for (int i0 = 0; i0 < c.n_seq; i0 += 256) {
      int r[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + 64 * u + lane;
        r[u] = i < c.n_seq ? (c.row_off[i] >> li) + 2 * i : INT32_MAX;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) count += __popcll(__ballot(r[u] <= item));
    }
    if (count == 0) return it;
    it.seq = __builtin_amdgcn_readfirstlane(count - 1);
  }
  const KvSeq s = kv_seq_scalar(c, it.seq);
  const int start = single ? item : (kv_scalar(c.row_off + it.seq) >> li) + 2 * it.seq;
  const int first = s.n - s.m, a = first < 0 ? 0 : first;
  const int p = (a >> li) + item - start;
  it.row0 = s.row0;
  it.before = item == start ? min(s.m, max(0, -first)) : 0;
  if (s.m <= 0 || s.n <= a || item < start || p > (s.n - 1) >> li) return it;
  it.lo = max(a, p << li);
  it.hi = min(s.n, (p + 1) << li);
  it.row = s.row0 + it.lo - first;
  it.kept = it.lo > p << li;
  it.blk = p;
  it.id = kv_page_scalar(c, it.seq, (p << li) >> c.lb);
  return it;
}

// the number of items that covers every sequence's pages
inline int item_count(const KvView& c, int li, bool single) {
  return single ? c.n_seq : (c.n_rows >> li) + 2 * c.n_seq;
}

// Largest magnitude of bf16 pairs: as integers, which order as the values do,
// so one instruction takes a pair.  Not finite ones come out on top; a wave
// that met one (SLOW below) goes over its data again without them.
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2 larger2(u16x2 m, uint32_t w) {
  return __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w & 0x7fff7fffu));
}
__device__ __forceinline__ u16x2 larger2_finite(u16x2 m, uint32_t w) {
  const uint32_t a = w & 0x7fffu, b = (w >> 16) & 0x7fffu;
  return larger2(m, (a < 0x7f80u ? a : 0u) | (b < 0x7f80u ? b << 16 : 0u));
}
__device__ __forceinline__ uint32_t wave_max(u16x2 m) {
  uint32_t x = max(m[0], m[1]);
#pragma unroll
  for (int i = 32; i >= 1; i >>= 1) x = max(x, (uint32_t)__shfl_xor((int)x, i, 64));
  return x;
}
constexpr uint32_t kNotFinite = 0x7f80u;

// the least e with amax <= 448 * 2^e, from amax's bf16 bits: 448 = 1.75 * 2^8
__device__ __forceinline__ int scale_exp(uint32_t u) {
  const int e = (int)(u >> 7) - 127 - 8 + ((u & 0x7fu) > 0x60u ? 1 : 0);
  return u == 0 ? kKvExpMin : min(max(e, kKvExpMin), kKvExpMax);
}

__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// four values -> codes (inv = 2^-e).  The product with a power of two is exact
// (what it makes subnormal lies far below the smallest code), so the
// conversion is the only rounding: to nearest even.
// SLOW: also what is not finite, and what lies past 448 under the largest scale.
template <bool SLOW>
__device__ __forceinline__ float in_range(float x) {
  if constexpr (!SLOW) return x;
  return x - x == 0.f ? fminf(fmaxf(x, -448.f), 448.f) : __uint_as_float(0x7fc00000u);
}
template <bool SLOW>
__device__ __forceinline__ uint32_t to_codes4(float a, float b, float c, float d, float inv) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(in_range<SLOW>(a * inv), in_range<SLOW>(b * inv), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(in_range<SLOW>(c * inv), in_range<SLOW>(d * inv), lo, true);
}

// four codes of one scale to another: f = 2^(old - new)
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  const uint32_t a = kv_bf2<false>(w, f), b = kv_bf2<true>(w, f);
  return to_codes4<true>(lo_bf(a), hi_bf(a), lo_bf(b), hi_bf(b), 1.f);
}
__device__ __forceinline__ uint4 rescale16(uint4 w, float f) {
  return uint4{rescale4(w.x, f), rescale4(w.y, f), rescale4(w.z, f), rescale4(w.w, f)};
}

// exponent of a page's new scale, and what its older tokens take for it.  A
// scale outside the range, in pages that the caller filled, is brought into it.
struct Scale {
  int e;
  bool moved;  // older tokens have to be rounded to it
  float inv, again;
};
__device__ __forceinline__ Scale new_scale(uint32_t amax, bool kept, float was) {
  const int need = scale_exp(amax);
  const int old = (int)((__float_as_uint(was) >> 23) & 255u) - 127;
  const int e = kept ? min(max(old, need), kKvExpMax) : need;
  return {e, kept && e != old, exp2i(-e), exp2i(max(old - e, -126))};
}

// One new row of each sequence: a wave takes it for one head, keys or values,
// a lane 2 * NC channels (10.4 us by the kernel for pages, 4.7 us by this one:
// 256 rows, 8 heads).  What bounds it is the chain of dependent loads
// (kv_len -> table -> scale), so nothing else waits: the row is on its way
// before the table's entry is looked at.
template <bool VEC, int NC>
__global__ __launch_bounds__(kThreads) void kv_append_one_kernel(KvView c, const uint16_t* __restrict__ knew,
                                                                 const uint16_t* __restrict__ vnew, int64_t rs,
                                                                 int64_t hs) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int what = blockIdx.y * 4 + wave;
  if (what >= 2 * c.H) return;
  const Item it = find_item(c, blockIdx.x, c.lb, true);
  if (it.blk < 0) return;
  const int h = what >> 1, is_v = what & 1, D = c.D, t = it.lo & ((1 << c.lb) - 1);
  const uint16_t* src = (is_v ? vnew : knew) + (int64_t)it.row * rs + (int64_t)h * hs;
  uint32_t x[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int d = 2 * (lane + 64 * i);
    x[i] = 0;
    if (d < D)
      x[i] = VEC ? *reinterpret_cast<const uint32_t*>(src + d) : (uint32_t)src[d] | ((uint32_t)src[d + 1] << 16);
  }
  if (it.id < 0) return;
  const size_t ph = (size_t)it.id * c.H + h;
  float* scale = (is_v ? c.v_scale : c.k_scale) + ph;
  const float was = it.kept ? *scale : 0.f;
  u16x2 m{0, 0};
#pragma unroll
  for (int i = 0; i < NC; ++i) m = larger2(m, x[i]);
  uint32_t amax = wave_max(m);
  if (amax >= kNotFinite) {
    m = u16x2{0, 0};
#pragma unroll
    for (int i = 0; i < NC; ++i) m = larger2_finite(m, x[i]);
    amax = wave_max(m);
  }
  const Scale s = new_scale(amax, it.kept, was);
  if (lane == 0) *scale = exp2i(s.e);
  uint8_t* page = (is_v ? c.v : c.k) + ph * ((size_t)D << c.lb);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int d = 2 * (lane + 64 * i);
    if (d >= D) continue;
    const uint32_t code = to_codes4<true>(lo_bf(x[i]), hi_bf(x[i]), 0.f, 0.f, s.inv);
    if (!is_v) {
      if (s.moved)
        for (int j = 0; j < t; ++j) {
          uint16_t* w = reinterpret_cast<uint16_t*>(page + (size_t)j * D + d);
          *w = (uint16_t)rescale4(*w, s.again);
        }
      *reinterpret_cast<uint16_t*>(page + (size_t)t * D + d) = (uint16_t)code;
      continue;
    }
    if (s.moved)
      for (int b = 0; 16 * b < t; ++b) {
        uint4* w = reinterpret_cast<uint4*>(page + ((size_t)16 * b * D + d * kKvBlk));
        w[0] = rescale16(w[0], s.again), w[1] = rescale16(w[1], s.again);
      }
    uint8_t* dst = page + ((size_t)(t & ~15) * D + d * kKvBlk);
    if ((t & 15) == 0) {  // a block's first token: zeros after it
      reinterpret_cast<uint4*>(dst)[0] = uint4{code & 255u, 0, 0, 0};
      reinterpret_cast<uint4*>(dst)[1] = uint4{code >> 8, 0, 0, 0};
    } else {
      dst[t & 15] = (uint8_t)code;
      dst[kKvBlk + (t & 15)] = (uint8_t)(code >> 8);
    }
  }
}

// TEAM waves write one page of one head, keys or values, wave r of them its
// 16-token blocks r, r + TEAM, ...; with TEAM >= block / 16 a wave has one
// block, read once and held in registers while the page's largest magnitude is
// found.  A lane holds pieces of 8 channels of the keys, or
// NC channel pairs of the values with all 16 tokens: 2 x 16 contiguous bytes
// of the page, whose rows the wave reads 256 bytes at a time.
// VEC: rows are 16-byte aligned in every head.
template <bool VEC, int TEAM, int NC>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(KvView c, const uint16_t* __restrict__ knew,
                                                             const uint16_t* __restrict__ vnew, int64_t rs,
                                                             int64_t hs) {
  constexpr int NK = 4 * NC;  // pieces of a lane for the keys of 16 tokens
  __shared__ float red[kThreads / 64];
  const Item it = find_item(c, blockIdx.x, c.lb, false);
  if (it.blk < 0 || it.id < 0) return;  // the same for the whole workgroup
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int what = blockIdx.y * (4 / TEAM) + wave / TEAM, r = wave % TEAM;
  if (TEAM == 1 && what >= 2 * c.H) return;
  const bool on = what < 2 * c.H;
  const int h = on ? what >> 1 : 0, is_v = what & 1, D = c.D, B = 1 << c.lb;
  const size_t ph = (size_t)it.id * c.H + h;
  const int cnt = it.hi - it.lo, t0 = it.lo & (B - 1);  // rows, first one's place in the page
  const uint16_t* src = (is_v ? vnew : knew) + (int64_t)it.row * rs + (int64_t)h * hs;
  uint8_t* page = (is_v ? c.v : c.k) + ph * ((size_t)D << c.lb);
  float* scale = (is_v ? c.v_scale : c.k_scale) + ph;
  const float was = it.kept ? *scale : 0.f;
  const int b0 = t0 >> 4, b1 = on ? (t0 + cnt - 1) >> 4 : -1, units = D >> 3;

  uint4 kr[NK];          // piece lane + 64 i of the block's keys
  uint32_t vr[NC][16];   // channel pair lane + 64 i of its values, token j
  auto load = [&](int b) {
    if (!is_v) {
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const int at = lane + 64 * i, t = at / units, tok = 16 * b + t - t0;
        kr[i] = uint4{0, 0, 0, 0};
        if (t < 16 && tok >= 0 && tok < cnt) {
          const uint16_t* p = src + (int64_t)tok * rs + 8 * (at - t * units);
          if (VEC) {
            kr[i] = *reinterpret_cast<const uint4*>(p);
          } else {
            auto two = [&](int e) { return p[e] | (uint32_t)p[e + 1] << 16; };
            kr[i] = uint4{two(0), two(2), two(4), two(6)};
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int tok = 16 * b + j - t0;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int d = 2 * (lane + 64 * i);
          vr[i][j] = 0;
          if (tok >= 0 && tok < cnt && d < D) {
            const uint16_t* p = src + (int64_t)tok * rs + d;
            vr[i][j] = VEC ? *reinterpret_cast<const uint32_t*>(p) : (uint32_t)p[0] | ((uint32_t)p[1] << 16);
          }
        }
      }
    }
  };

  auto largest = [&](auto&& more) {
    u16x2 m{0, 0};
    if (!is_v) {
#pragma unroll
      for (int i = 0; i < NK; ++i) m = more(more(more(more(m, kr[i].x), kr[i].y), kr[i].z), kr[i].w);
    } else {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) m = more(m, vr[i][j]);
    }
    return wave_max(m);
  };
  uint32_t amax = 0;
  bool slow = false;
  for (int b = b0 + r; b <= b1; b += TEAM) {
    load(b);
    uint32_t x = largest(larger2);
    if (x >= kNotFinite) {
      slow = true;
      x = largest(larger2_finite);
    }
    amax = max(amax, x);
  }
  if constexpr (TEAM > 1) {
    if (lane == 0) red[wave] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TEAM; ++w) amax = max(amax, red[wave / TEAM * TEAM + w]);
  }
  const Scale s = new_scale(amax, it.kept, was);
  slow |= s.e == kKvExpMax;
  if (on && r == 0 && lane == 0) *scale = exp2i(s.e);

  if (s.moved && on) {
    // the older tokens to the new scale, what is also written below by the same
    // lane (bytes of tokens to come may change: they hold nothing)
    const int end = (t0 - 1) >> 4;
    for (int b = (b0 + r) % TEAM; b <= end; b += TEAM) {
      uint4* w = reinterpret_cast<uint4*>(page + (size_t)16 * b * D);
      if (is_v) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int d = 2 * (lane + 64 * i);
          if (d < D) w[d] = rescale16(w[d], s.again), w[d + 1] = rescale16(w[d + 1], s.again);
        }
      } else {
        for (int i = lane; i < min(16, t0 - 16 * b) * (D >> 4); i += 64) w[i] = rescale16(w[i], s.again);
      }
    }
  }
  auto store = [&](int b, auto is_slow) {
    constexpr bool SLOW = decltype(is_slow)::value;
    if (!is_v) {
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const int at = lane + 64 * i, t = at / units, tok = 16 * b + t - t0;
        if (t < 16 && tok >= 0 && tok < cnt) {
          const uint4 x = kr[i];
          *reinterpret_cast<uint2*>(page + (size_t)16 * b * D + 8 * at) =
              uint2{to_codes4<SLOW>(lo_bf(x.x), hi_bf(x.x), lo_bf(x.y), hi_bf(x.y), s.inv),
                    to_codes4<SLOW>(lo_bf(x.z), hi_bf(x.z), lo_bf(x.w), hi_bf(x.w), s.inv)};
        }
      }
      return;
    }
    const int lo = t0 - 16 * b, hi = t0 + cnt - 16 * b;  // new tokens of this block: lo <= j < hi
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int d = 2 * (lane + 64 * i);
      if (d >= D) continue;
      uint8_t* dst = page + ((size_t)16 * b * D + d * kKvBlk);
      uint32_t w[2][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t* x = &vr[i][4 * q];
        w[0][q] = to_codes4<SLOW>(lo_bf(x[0]), lo_bf(x[1]), lo_bf(x[2]), lo_bf(x[3]), s.inv);
        w[1][q] = to_codes4<SLOW>(hi_bf(x[0]), hi_bf(x[1]), hi_bf(x[2]), hi_bf(x[3]), s.inv);
      }
      if (lo <= 0) {  // no older tokens: whole pieces, zeros after the last token
        reinterpret_cast<uint4*>(dst)[0] = uint4{w[0][0], w[0][1], w[0][2], w[0][3]};
        reinterpret_cast<uint4*>(dst)[1] = uint4{w[1][0], w[1][1], w[1][2], w[1][3]};
      } else {
#pragma unroll
        for (int j = 1; j < 16; ++j)
          if (j >= lo && j < hi) {
            dst[j] = (uint8_t)(w[0][j >> 2] >> (8 * (j & 3)));
            dst[kKvBlk + j] = (uint8_t)(w[1][j >> 2] >> (8 * (j & 3)));
          }
      }
    }
  };
  for (int b = b0 + r; b <= b1; b += TEAM) {
    if (b0 + r + TEAM <= b1) load(b);
    if (slow)
      store(b, std::true_type{});
    else
      store(b, std::false_type{});
  }
}

// A workgroup reads 16 tokens, keys and values, of all heads or of a
// blockIdx.y-th part: unit i < H * D / 2 is a channel pair of the values (2 x
// 16 contiguous bytes; 64 lanes write 256 contiguous bytes of a row), the
// others are two 16-byte pieces of the keys.  Units run on over the heads,
// so no lane is idle whatever dim is.
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvView c, uint16_t* __restrict__ kout,
                                                           uint16_t* __restrict__ vout, bool single) {
  const Item it = find_item(c, blockIdx.x, 4, single);
  const int D = c.D, half = c.H * D >> 1;
  const int first = blockIdx.y * kThreads + threadIdx.x, step = gridDim.y * kThreads;
  for (int64_t i = first; i < (int64_t)it.before * 2 * half; i += step) {  // rows that are in no page
    kout[(int64_t)it.row0 * 2 * half + i] = 0x7fc0;
    vout[(int64_t)it.row0 * 2 * half + i] = 0x7fc0;
  }
  if (it.blk < 0) return;
  const bool none = it.id < 0;
  const int base = it.blk << 4, in_page = base & ((1 << c.lb) - 1);
  const int lo = it.lo - base, hi = it.hi - base;  // of the 16 tokens
  const size_t page = (size_t)(none ? 0 : it.id) * c.H;
  const int64_t row = (int64_t)(it.row - lo) * 2 * half;  // of token `base` (which may lie before the batch's rows)
  for (int i = first; i < 2 * half; i += step) {
    if (i < half) {
      const int h = i / (D >> 1), d = 2 * (i - h * (D >> 1));
      const float s = none ? 1.f : c.v_scale[page + h];
      const uint4* src = reinterpret_cast<const uint4*>(c.v + (((page + h) << c.lb) + in_page) * D + d * kKvBlk);
      uint4 x = src[0], y = src[1];
      if (none) x = y = uint4{0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu};
      const uint32_t wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
      uint16_t* dst = vout + row + 2 * i;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t a[2] = {kv_bf2<false>(wx[q], s), kv_bf2<true>(wx[q], s)};
        const uint32_t e[2] = {kv_bf2<false>(wy[q], s), kv_bf2<true>(wy[q], s)};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 4 * q + r;
          const uint32_t w =
              r & 1 ? (a[r >> 1] >> 16) | (e[r >> 1] & 0xffff0000u) : (a[r >> 1] & 0xffffu) | (e[r >> 1] << 16);
          if (j >= lo && j < hi) *reinterpret_cast<uint32_t*>(dst + (int64_t)j * 2 * half) = w;
        }
      }
    } else {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int at = i - half + n * half;  // of H * D pieces
        const int h = at / D, q = at - h * D, t = q / (D >> 4), u = q - t * (D >> 4);
        if (t < lo || t >= hi) continue;
        const float s = none ? 1.f : c.k_scale[page + h];
        uint4 w = reinterpret_cast<const uint4*>(c.k + (((page + h) << c.lb) + in_page) * D)[q];
        if (none) w = uint4{0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu};
        uint4* o = reinterpret_cast<uint4*>(kout + row + (int64_t)t * 2 * half + h * D + 16 * u);
        o[0] = uint4{kv_bf2<false>(w.x, s), kv_bf2<true>(w.x, s), kv_bf2<false>(w.y, s), kv_bf2<true>(w.y, s)};
        o[1] = uint4{kv_bf2<false>(w.z, s), kv_bf2<true>(w.z, s), kv_bf2<false>(w.w, s), kv_bf2<true>(w.w, s)};
      }
    }
  }
}

struct NewRows {
  const uint16_t *k, *v;
  int64_t rs, hs;
};

template <bool VEC, int NC>
void append(const KvView& c, const NewRows& x, hipStream_t stream) {
  auto go = [&](auto kernel, int items, int team) {
    MLORA_LAUNCH("kv_append", kernel, dim3(items, (2 * c.H * team + 3) / 4), dim3(kThreads), 0, stream, c, x.k, x.v,
                 x.rs, x.hs);
  };
  const int items = item_count(c, c.lb, false);
  if (c.max_new == 1)
    go(kv_append_one_kernel<VEC, NC>, c.n_seq, 1);
  else if (c.lb == 4)
    go(kv_append_kernel<VEC, 1, NC>, items, 1);
  else if (c.lb == 5)
    go(kv_append_kernel<VEC, 2, NC>, items, 2);
  else
    go(kv_append_kernel<VEC, 4, NC>, items, 4);
}

}  // namespace

hipError_t launch_kv_append(const KvView& c, const uint16_t* k, const uint16_t* v, int64_t rs, int64_t hs,
                            hipStream_t stream) {
  const bool vec = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15u) == 0 && rs % 8 == 0 &&
                   hs % 8 == 0;
  const NewRows x{k, v, rs, hs};
  if (vec)
    c.D <= 128 ? append<true, 1>(c, x, stream) : append<true, 2>(c, x, stream);
  else
    c.D <= 128 ? append<false, 1>(c, x, stream) : append<false, 2>(c, x, stream);
  return launched();
}

hipError_t launch_kv_read(const KvView& c, uint16_t* k, uint16_t* v, hipStream_t stream) {
  const bool single = c.max_new == 1;
  const int items = item_count(c, 4, single), full = std::max(1, c.H * c.D / kThreads);
  // A unit a thread where all workgroups run at once, and where there are many
  // rounds of them anyway (32768 tokens 36.4 us, 39.0 us with four units a
  // thread); in between as many as fill one round (pages of 256 requests 8.8 us,
  // 10.0 us with a unit a thread, 9.6 us with four).
  const int split = items > kReadGroups ? full : std::min(full, kReadGroups / items);
  MLORA_LAUNCH("kv_read", kv_read_kernel, dim3(items, split), dim3(kThreads), 0, stream, c, k, v, single);
  return launched();
}

}  // namespace mlora
