// Writing new tokens into the paged 8-bit key/value cache, and reading them
// back.  Both are bound by memory traffic (2 bytes a channel on the bf16
// side, 1 on the cache's) and, for a decode step, by the latency of a launch
// with a few dependent loads (row_off -> table -> page).
//
// One workgroup owns one page of one head, keys or values, so a page's scale
// is found and used without another launch, and no two workgroups write one
// page.  The sequence and page of a workgroup come from its index in closed
// form: sequence i's pages start at item row_off[i] / B + 2 i, which leaves it
// at least as many items as m rows touch pages, so the grid is known on the
// host although the lengths are not, and no prefix sum is needed.
#include "kv.h"

namespace mlora {
namespace {

constexpr int kThreads = 256;

struct Item {
  int seq, page;   // sequence, page's index in it (page < 0: nothing to do)
  int lo, hi;      // positions of the page's rows of this batch
  int row;         // row of position lo
  bool kept;       // the page holds older tokens of the sequence
  int id;          // page of the pool, -1 if there is none
  int row0, before;  // the sequence's first item: its first row, and its rows at negative positions
};

// single: every sequence has one row at most, and item i is sequence i
__device__ __forceinline__ Item find_item(const KvView& c, int item, bool single) {
  Item it{};
  it.page = -1;
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
        r[u] = i < c.n_seq ? (c.row_off[i] >> c.lb) + 2 * i : INT32_MAX;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) count += __popcll(__ballot(r[u] <= item));
    }
    if (count == 0) return it;
    it.seq = __builtin_amdgcn_readfirstlane(count - 1);
  }
  const KvSeq s = kv_seq(c, it.seq);
  const int start = single ? item : (c.row_off[it.seq] >> c.lb) + 2 * it.seq;
  const int first = s.n - s.m, a = first < 0 ? 0 : first;
  const int p = (a >> c.lb) + item - start;
  it.row0 = s.row0;
  it.before = item == start ? min(s.m, max(0, -first)) : 0;
  if (s.m <= 0 || s.n <= a || item < start || p > (s.n - 1) >> c.lb) return it;
  it.lo = max(a, p << c.lb);
  it.hi = min(s.n, (p + 1) << c.lb);
  it.row = s.row0 + it.lo - first;
  it.kept = it.lo > p << c.lb;
  it.page = p;
  it.id = kv_page(c, it.seq, p);
  return it;
}

// the number of items that covers every sequence's pages
inline int item_count(const KvView& c, bool single) {
  return single ? c.n_seq : (c.n_rows >> c.lb) + 2 * c.n_seq;
}

__device__ __forceinline__ float finite_abs(uint32_t b16) {
  const uint32_t a = b16 & 0x7fffu;
  return a >= 0x7f80u ? 0.f : bf2f(a);
}

// the least e with amax <= 448 * 2^e, from the bits: 448 = 1.75 * 2^8
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return u == 0 ? kKvExpMin : min(max(e, kKvExpMin), kKvExpMax);
}

__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// bf16 pair -> two codes in the low half (inv = 2^-e).  The product with a
// power of two is exact (what it makes subnormal lies far below the smallest
// code), so the conversion is the only rounding: to nearest even.
__device__ __forceinline__ uint32_t to_codes(float a, float b, float inv) {
  float x = a * inv, y = b * inv;
  x = x - x == 0.f ? fminf(fmaxf(x, -448.f), 448.f) : __uint_as_float(0x7fc00000u);
  y = y - y == 0.f ? fminf(fmaxf(y, -448.f), 448.f) : __uint_as_float(0x7fc00000u);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x, y, 0, false) & 0xffffu;
}

// four codes of one scale to another: f = 2^(old - new)
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  const uint32_t a = kv_bf2<false>(w, f), b = kv_bf2<true>(w, f);
  return to_codes(lo_bf(a), hi_bf(a), 1.f) | (to_codes(lo_bf(b), hi_bf(b), 1.f) << 16);
}

__device__ __forceinline__ float block_max(float x, float* red) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x = fmaxf(x, __shfl_xor(x, m, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  float y = red[0];
  for (int w = 1; w < (int)blockDim.x / 64; ++w) y = fmaxf(y, red[w]);
  return y;
}

// VEC: rows are 16-byte aligned in every head
template <bool VEC>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(KvView c, const uint16_t* __restrict__ knew,
                                                             const uint16_t* __restrict__ vnew, int64_t rs,
                                                             int64_t hs, bool single) {
  __shared__ float red[kThreads / 64];
  const Item it = find_item(c, blockIdx.x, single);
  if (it.page < 0 || it.id < 0) return;
  const int h = blockIdx.y, D = c.D, B = 1 << c.lb, tid = threadIdx.x, nt = blockDim.x;
  const size_t ph = (size_t)it.id * c.H + h;
  const int cnt = it.hi - it.lo, t0 = it.lo & (B - 1);  // rows, first one's place in the page
  const bool is_v = blockIdx.z != 0;
  const uint16_t* src = (is_v ? vnew : knew) + (size_t)it.row * rs + (size_t)h * hs;
  uint8_t* page = (is_v ? c.v : c.k) + ph * ((size_t)D << c.lb);
  float* scale = (is_v ? c.v_scale : c.k_scale) + ph;

  const int units = D >> 3;
  float amax = 0.f;
  for (int i = tid; i < cnt * units; i += nt) {
    const int t = i / units, u = i - t * units;
    const uint16_t* p = src + (size_t)t * rs + u * 8;
    if (VEC) {
      const uint4 w = *reinterpret_cast<const uint4*>(p);
      const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fmaxf(finite_abs(x[e] & 0xffffu), finite_abs(x[e] >> 16)));
    } else {
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, finite_abs(p[e]));
    }
  }
  const float was = it.kept ? *scale : 0.f;
  amax = block_max(amax, red);
  const int need = scale_exp(amax);
  const int old = min(max((int)((__float_as_uint(was) >> 23) & 255u) - 127, kKvExpMin), kKvExpMax);
  const int e = it.kept ? max(old, need) : need;
  const bool grown = it.kept && e > old;
  const float inv = exp2i(-e), again = exp2i(old - e < -126 ? -126 : old - e);
  if (tid == 0) *scale = exp2i(e);

  if (!is_v) {
    for (int i = tid; i < cnt * units; i += nt) {
      const int t = i / units, u = i - t * units;
      const uint16_t* p = src + (size_t)t * rs + u * 8;
      float x[8];
      load8<VEC>(p, 0, 8, x);
      uint2 w;
      w.x = to_codes(x[0], x[1], inv) | (to_codes(x[2], x[3], inv) << 16);
      w.y = to_codes(x[4], x[5], inv) | (to_codes(x[6], x[7], inv) << 16);
      *reinterpret_cast<uint2*>(page + (size_t)(t0 + t) * D + u * 8) = w;
    }
    if (grown)
      for (int i = tid; i < t0 * D / 4; i += nt) {
        uint32_t* w = reinterpret_cast<uint32_t*>(page) + i;
        *w = rescale4(*w, again);
      }
    return;
  }
  // values: a thread owns a channel pair of 16 tokens, 2 x 16 contiguous
  // bytes; it reads the rows (64 lanes: 256 bytes of a row) and puts the
  // tokens of each channel side by side
  const int pairs = D >> 1, b0 = grown ? 0 : t0 >> 4, b1 = (t0 + cnt - 1) >> 4;
  for (int i = tid; i < (b1 - b0 + 1) * pairs; i += nt) {
    const int b = b0 + i / pairs, d = 2 * (i % pairs);
    uint4* dst = reinterpret_cast<uint4*>(page + ((size_t)b * D + d) * kKvBlk);
    const int lo = t0 - 16 * b, hi = t0 + cnt - 16 * b;  // new tokens of this block: lo <= j < hi
    uint32_t w[2][4] = {};
    if (lo > 0) {  // it holds older tokens too
      const uint4 x = dst[0], y = dst[1];
      w[0][0] = x.x; w[0][1] = x.y; w[0][2] = x.z; w[0][3] = x.w;
      w[1][0] = y.x; w[1][1] = y.y; w[1][2] = y.z; w[1][3] = y.w;
      if (grown)
#pragma unroll
        for (int q = 0; q < 4; ++q) w[0][q] = rescale4(w[0][q], again), w[1][q] = rescale4(w[1][q], again);
    }
    uint32_t x[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      x[j] = 0;
      if (j >= lo && j < hi) {
        const uint16_t* p = src + (int64_t)(j - lo) * rs + d;
        x[j] = VEC ? *reinterpret_cast<const uint32_t*>(p) : (uint32_t)p[0] | ((uint32_t)p[1] << 16);
      }
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint32_t code = to_codes(lo_bf(x[j]), hi_bf(x[j]), inv);
      const int sh = 8 * (j & 3);
      if (j >= lo && j < hi) {
        w[0][j >> 2] = (w[0][j >> 2] & ~(255u << sh)) | ((code & 255u) << sh);
        w[1][j >> 2] = (w[1][j >> 2] & ~(255u << sh)) | ((code >> 8) << sh);
      }
    }
    dst[0] = uint4{w[0][0], w[0][1], w[0][2], w[0][3]};
    dst[1] = uint4{w[1][0], w[1][1], w[1][2], w[1][3]};
  }
}

__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvView c, uint16_t* __restrict__ kout,
                                                           uint16_t* __restrict__ vout, bool single) {
  const Item it = find_item(c, blockIdx.x, single);
  const int h = blockIdx.y, D = c.D, B = 1 << c.lb, tid = threadIdx.x, nt = blockDim.x;
  for (int i = tid; i < it.before * D; i += nt)  // rows that are in no page
    (blockIdx.z == 0 ? kout : vout)[((size_t)(it.row0 + i / D) * c.H + h) * D + i % D] = 0x7fc0;
  if (it.page < 0) return;
  const size_t ph = (size_t)(it.id < 0 ? 0 : it.id) * c.H + h;
  const int cnt = it.hi - it.lo, t0 = it.lo & (B - 1);
  const size_t orow = (size_t)c.H * D;
  if (blockIdx.z == 0) {
    const uint8_t* page = c.k + ph * ((size_t)D << c.lb) + (size_t)t0 * D;
    uint16_t* dst = kout + (size_t)it.row * orow + (size_t)h * D;
    const float s = it.id < 0 ? 1.f : c.k_scale[ph];
    const int units = D >> 4;
    for (int i = tid; i < cnt * units; i += nt) {
      const int t = i / units, u = i - t * units;
      uint4 w = *reinterpret_cast<const uint4*>(page + (size_t)i * 16);
      if (it.id < 0) w = uint4{0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu};
      uint4* o = reinterpret_cast<uint4*>(dst + (size_t)t * orow + u * 16);
      o[0] = uint4{kv_bf2<false>(w.x, s), kv_bf2<true>(w.x, s), kv_bf2<false>(w.y, s), kv_bf2<true>(w.y, s)};
      o[1] = uint4{kv_bf2<false>(w.z, s), kv_bf2<true>(w.z, s), kv_bf2<false>(w.w, s), kv_bf2<true>(w.w, s)};
    }
    return;
  }
  const uint8_t* page = c.v + ph * ((size_t)D << c.lb);
  uint16_t* dst = vout + (size_t)it.row * orow + (size_t)h * D;
  const float s = it.id < 0 ? 1.f : c.v_scale[ph];
  const int pairs = D >> 1, b0 = t0 >> 4, b1 = (t0 + cnt - 1) >> 4;
  for (int i = tid; i < (b1 - b0 + 1) * pairs; i += nt) {
    const int b = b0 + i / pairs, d = 2 * (i % pairs);
    const uint4* src = reinterpret_cast<const uint4*>(page + ((size_t)b * D + d) * kKvBlk);
    const uint4 x = src[0], y = src[1];
    const uint32_t wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
    const int lo = t0 - 16 * b, hi = t0 + cnt - 16 * b;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t a[2] = {kv_bf2<false>(wx[q], s), kv_bf2<true>(wx[q], s)};
      const uint32_t e[2] = {kv_bf2<false>(wy[q], s), kv_bf2<true>(wy[q], s)};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = 4 * q + r;
        uint32_t w = r & 1 ? (a[r >> 1] >> 16) | (e[r >> 1] & 0xffff0000u) : (a[r >> 1] & 0xffffu) | (e[r >> 1] << 16);
        if (it.id < 0) w = 0x7fc07fc0u;
        if (j >= lo && j < hi) *reinterpret_cast<uint32_t*>(dst + (int64_t)(j - lo) * orow + d) = w;
      }
    }
  }
}

}  // namespace

hipError_t launch_kv_append(const KvView& c, const uint16_t* k, const uint16_t* v, int64_t rs, int64_t hs,
                            hipStream_t stream) {
  const bool single = c.max_new == 1;
  const dim3 grid(item_count(c, single), c.H, 2);
  const bool vec = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15u) == 0 && rs % 8 == 0 &&
                   hs % 8 == 0;
  if (vec)
    MLORA_LAUNCH("kv_append", kv_append_kernel<true>, grid, dim3(kThreads), 0, stream, c, k, v, rs, hs, single);
  else
    MLORA_LAUNCH("kv_append", kv_append_kernel<false>, grid, dim3(kThreads), 0, stream, c, k, v, rs, hs, single);
  return launched();
}

hipError_t launch_kv_read(const KvView& c, uint16_t* k, uint16_t* v, hipStream_t stream) {
  const bool single = c.max_new == 1;
  MLORA_LAUNCH("kv_read", kv_read_kernel, dim3(item_count(c, single), c.H, 2), dim3(kThreads), 0, stream, c, k, v,
               single);
  return launched();
}

}  // namespace mlora
