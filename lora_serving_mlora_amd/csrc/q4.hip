// 4-bit weights: e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign) with a
// power-of-two scale for 32 channels of a row; their quantiser, the way back
// to bf16, and products of few rows with them.
#include "q4.h"
#include "row_kernels.h"

namespace mlora {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ bf16x8 as_bf16x8(uint4 v) { return __builtin_bit_cast(bf16x8, v); }

constexpr int kConvThreads = 256;

// ---------------------------------------------------------------------------
// quantiser: a thread takes 8 weights, four threads a group.  The least
// exponent e with amax <= 6 * 2^e is read off the bits of amax = 1.m * 2^x:
// 6 = 1.5 * 2^2, so e = x - 2 up to a fraction of one half and x - 1 above.
// The codes come from the conversion instruction, which rounds to nearest
// even and ends at 6.  Bound by memory (4096 -> 11008 and read back: 43.4 us at
// 5.3 TB/s; with the codes counted up by seven comparisons 49.3, bound by those).
// ---------------------------------------------------------------------------
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
// the other value of lanes 1 and 2 apart
template <int PERM>
__device__ __forceinline__ uint32_t quad(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, PERM, 0xf, 0xf, true);
}
__global__ __launch_bounds__(kConvThreads) void q4_quantize_kernel(const uint16_t* __restrict__ W,
                                                                   uint8_t* __restrict__ codes,
                                                                   uint8_t* __restrict__ scales, int64_t n8) {
  const int64_t stride = (int64_t)gridDim.x * kConvThreads;
  for (int64_t i = (int64_t)blockIdx.x * kConvThreads + threadIdx.x; i < n8; i += stride) {
    const uint4 v = reinterpret_cast<const uint4*>(W)[i];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t both = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) both = max_u16x2(both, w[j] & 0x7fff7fffu);
    // n8 is a multiple of 4: the four threads of a group are here together
    both = max_u16x2(both, quad<0xb1>(both));  // lanes 1 apart
    both = max_u16x2(both, quad<0x4e>(both));  // lanes 2 apart
    const uint32_t top = max(both & 0xffffu, both >> 16);
    uint32_t b = 255, code = 0;
    if (top < 0x7f80u) {
      const int e = (int)(top >> 7) - ((top & 127u) <= 64u ? 2 : 1);
      b = min(max(e, kQ4ExpMin), kQ4ExpMax);
      const float scale = q4_scale(b);
      code = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(code, __builtin_bit_cast(bf16x2, w[0]), scale, 0);
      code = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(code, __builtin_bit_cast(bf16x2, w[1]), scale, 1);
      code = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(code, __builtin_bit_cast(bf16x2, w[2]), scale, 2);
      code = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(code, __builtin_bit_cast(bf16x2, w[3]), scale, 3);
    }
    reinterpret_cast<uint32_t*>(codes)[i] = code;
    if ((i & 3) == 0) scales[i >> 2] = (uint8_t)b;
  }
}

// ---------------------------------------------------------------------------
// the way back: 8 codes a thread, 16-byte stores
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kConvThreads) void q4_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                     const uint8_t* __restrict__ scales,
                                                                     uint16_t* __restrict__ W, int64_t n8) {
  const int64_t stride = (int64_t)gridDim.x * kConvThreads;
  for (int64_t i = (int64_t)blockIdx.x * kConvThreads + threadIdx.x; i < n8; i += stride)
    reinterpret_cast<uint4*>(W)[i] = q4_bf8(reinterpret_cast<const uint32_t*>(codes)[i], q4_scale(scales[i >> 2]));
}

// The same into rows of Kp channels, and the M rows of X into such rows behind
// them: zeros past the K that there are.  A workgroup a row.
__global__ __launch_bounds__(kConvThreads) void q4_pad_kernel(Q4View w, const uint16_t* __restrict__ X,
                                                              uint16_t* __restrict__ Wp, uint16_t* __restrict__ Xp,
                                                              int K8, int Kp8) {
  const int r = (int)blockIdx.x;
  if (r < w.N) {
    const uint32_t* c = reinterpret_cast<const uint32_t*>(w.codes) + (size_t)r * K8;
    const uint8_t* s = w.scales + (size_t)r * (K8 / 4);
    uint4* o = reinterpret_cast<uint4*>(Wp) + (size_t)r * Kp8;
    for (int j = threadIdx.x; j < Kp8; j += kConvThreads)
      o[j] = j < K8 ? q4_bf8(c[j], q4_scale(s[j >> 2])) : make_uint4(0u, 0u, 0u, 0u);
  } else {
    const uint4* x = reinterpret_cast<const uint4*>(X) + (size_t)(r - w.N) * K8;
    uint4* o = reinterpret_cast<uint4*>(Xp) + (size_t)(r - w.N) * Kp8;
    for (int j = threadIdx.x; j < Kp8; j += kConvThreads) o[j] = j < K8 ? x[j] : make_uint4(0u, 0u, 0u, 0u);
  }
}

// ---------------------------------------------------------------------------
// Products of few rows, 64 to a workgroup.  What bounds them is the codes' way from memory,
// so each code is read once, by the lane whose operand it is: a lane takes
// the 16 bytes (32 channels, one group) of one column at a time, the 16
// columns of a group by the 4 lane groups' next groups of channels, and feeds
// them as four 16x16x32 products.  Which channel stands where in K is free as
// long as X agrees.  A workgroup has 16 * CG columns and a slice of K; its
// waves take shares of the slice and all of the columns each, so that no two
// of them need the same codes or the same part of X, and there is no barrier
// before the shares are summed through LDS in order.
// Codes and X come through LDS all the same, a wave's own: whole row pieces (64
// bytes of codes, 256 of X) whose 16-byte chunks are XOR-ed with the row, since
// the 16 rows of an operand would all hit the same banks otherwise; conflicts
// still take 38 to 44 % of the cycles in which LDS is read.  (Operands loaded from
// memory as they are have a row to a lane, which the address unit takes four
// times as long for: 61 rows of 11008 channels 23.5 us, X alone through LDS
// 18.8.)
// Codes and X run D steps of 128 channels ahead.  With the low-rank term the
// waves also compute T = Down x, once their share of the product is done.
// ---------------------------------------------------------------------------
constexpr int kStep = 128, kStepGroups = kStep / kQ4Group;

// a place that is the same for the whole wave: a scalar load (the pool's and
// the batch's tables, which do not change while a kernel runs)
template <class T>
__device__ __forceinline__ T scalar(const T* p) {
  typedef const T __attribute__((address_space(4))) * constant;
  return *(constant)(uintptr_t)p;
}

// s_waitcnt immediate for "vmcnt <= v" (expcnt and lgkmcnt not waited)
constexpr int vmcnt_imm(int v) { return (v & 15) | ((v >> 4) << 14) | (7 << 4) | (15 << 8); }

// The low-rank inner products T[sl][r][q] = Down[q] . x_r over slice sl of SK
// of the channels (the scale is left out), of up to 64 rows from X on; a lane
// holds the key and the rank of each (0: none).  An item is a slice of up to
// 16 rows of one adapter by 16 of its ranks, one wave's; the waves take the
// items in turn.  So rows that share an adapter share what is read of it (61
// rows of 11008 channels, three adapters of up to 64 ranks: the layer 29.2 us,
// when each row read its own 38.7).
__device__ __forceinline__ void shrink_items(const PoolView& pv, int proj, const uint16_t* __restrict__ X,
                                             int key, int rank, int worker, int workers, int SK,
                                             float* __restrict__ T, size_t slice) {
  const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
  const uint64_t served = __ballot(rank > 0);
  const int steps = pv.din / 32;
  for (int t = worker;; t += workers) {
    // the item's adapter: the first rows of each one's in turn
    int unit = t / SK, k0 = 0, n_ranks = 0, chunk = 0, block = 0;
    uint64_t left = served, rows = 0;
    while (left) {
      const int first = __builtin_ctzll(left);
      k0 = __builtin_amdgcn_readlane(key, first);
      n_ranks = __builtin_amdgcn_readlane(rank, first);
      rows = __ballot(key == k0) & left;
      const int blocks = (n_ranks + 15) / 16, units = (__popcll(rows) + 15) / 16 * blocks;
      if (unit < units) {
        chunk = unit / blocks, block = unit % blocks;
        break;
      }
      unit -= units;
      left &= ~rows;
    }
    if (!left) return;
    const int sl = t % SK, u0 = (int)((long)steps * sl / SK), u1 = (int)((long)steps * (sl + 1) / SK);
    // lanes r16 of every quarter hold row r16 of the chunk, or its first
    const int at = __popcll(rows & ((1ull << lane) - 1)) - 16 * chunk, n = min(__popcll(rows) - 16 * chunk, 16);
    int row = 0;
    {
      const bool mine = ((rows >> lane) & 1) != 0 && at >= 0 && at < 16;
      // (the others send to lanes that nothing is read from)
      row = __builtin_amdgcn_ds_permute((mine ? at : 16 + (lane & 31)) * 4, lane);
      row = __shfl(row, r16 < n ? r16 : 0, 64);
    }
    const int32_t* dpage = pv.down_page + ((size_t)k0 * pv.n_proj + proj) * pv.max_rank;
    const int page = dpage[min(16 * block + r16, n_ranks - 1)];
    const uint4* x = reinterpret_cast<const uint4*>(X + (size_t)row * pv.din) + q;
    const uint4* d = reinterpret_cast<const uint4*>(pv.down + (size_t)page * pv.din) + q;
    floatx4 acc = {0.f, 0.f, 0.f, 0.f};
    constexpr int U = 8;
    for (int u = u0; u < u1; u += U) {
      uint4 xa[U], da[U];
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const int v = min(u + e, u1 - 1);
        xa[e] = x[4 * v];
        da[e] = d[4 * v];
      }
#pragma unroll
      for (int e = 0; e < U; ++e) {
        if (u + e < u1)
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(xa[e]), as_bf16x8(da[e]), acc, 0, 0, 0);
      }
    }
    if (16 * block + r16 >= n_ranks) n_ranks = 0;  // a lane behind the last rank writes nothing
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int r = __shfl(row, q * 4 + v, 64);
      if (n_ranks > 0 && q * 4 + v < n) T[sl * slice + (size_t)r * pv.max_rank + 16 * block + r16] = acc[v];
    }
  }
}

// The body of q4_rows_kernel.  x0 .. x2: LDS for a step, a slot of every
// wave's (16 * MB rows of 256 bytes of X, 16 * CG of 64 bytes of codes); arrays
// of their own, so that the compiler knows that reads of one do not wait for
// what is on its way into another (the first D of them are used).
template <int MB, int CG, int NW, int D, bool LORA>
__device__ __forceinline__ void q4_rows_body(const Q4View& w, const uint16_t* __restrict__ Xall, int rows, int S,
                                             uint16_t* __restrict__ Y, float* __restrict__ part, const PoolView& pv,
                                             int proj, const int32_t* __restrict__ row_key, float* __restrict__ T,
                                             int SK, uint8_t* __restrict__ x0, uint8_t* __restrict__ x1,
                                             uint8_t* __restrict__ x2) {
  static_assert(CG <= 4 && D >= 2 && D <= 3, "the waves' sums fit in a slot; slots are named below");
  const int K = w.K, N = w.N, G = K / kQ4Group;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ncb = (N + 16 * CG - 1) / (16 * CG);
  const int cb = (int)blockIdx.x % ncb, kq = (int)blockIdx.x / ncb % S, m0 = (int)blockIdx.x / (ncb * S) * kQ4RowBlock;
  const int M = min(rows - m0, kQ4RowBlock);  // rows of this workgroup, from m0 on
  const uint16_t* X = Xall + (size_t)m0 * K;
  const int steps = (K + kStep - 1) / kStep;
  // this wave's steps [u0, u0 + mine) of the NW * S shares of K
  const int u0 = (int)((long)steps * (kq * NW + wave) / (NW * S));
  const int mine = (int)((long)steps * (kq * NW + wave + 1) / (NW * S)) - u0;
  const int r16 = lane & 15, q = lane >> 4;

  const int n0 = cb * 16 * CG, cols = min(16 * CG, N - n0);
  const uint8_t* wc = w.codes + (size_t)n0 * (K / 2);
  const uint8_t* ws = w.scales + (size_t)n0 * G;
  constexpr int kX = MB * 4096, kSlot = kX + CG * 1024;  // bytes of a wave
  uint32_t sb[D];                             // scale bytes of a step: lane l holds column l's four
  constexpr int kLoads = 4 * MB + CG + 1;     // of a step
  const int scol = min(lane, cols - 1), send = cols * G - 4;
  // one step's part of X (four rows an instruction), codes and scales.  Past
  // the end of a row X reads on (the next row, or zeros past the last) and the
  // last group is read again; both count for nothing below.  A step past this
  // wave's last makes the same loads of empty buffers, so that what is on its
  // way can be told by its number.
  auto fetch = [&](int u, uint8_t* slot, uint32_t& sv) {
    const bool any = u < mine;
    const __amdgpu_buffer_rsrc_t rx =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(X), (short)0, any ? M * K * 2 : 0, 0x00020000);
    const __amdgpu_buffer_rsrc_t rc =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(wc), (short)0, any ? cols * (K / 2) : 0, 0x00020000);
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(ws), (short)0, any ? cols * G : 0, 0x00020000);
    const int g0 = (u0 + u) * kStepGroups;
#pragma unroll
    for (int c = 0; c < CG; ++c) {
      const int row = 16 * c + (lane >> 2), g = min(g0 + ((lane ^ (lane >> 4)) & 3), G - 1);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rc, slot + wave * kSlot + kX + c * 1024, 16,
                                               min(row, cols - 1) * (K / 2) + g * 16, 0, 0, 0);
    }
    sv = __builtin_amdgcn_raw_buffer_load_b32(rs, min(scol * G + g0, send), 0, 0);
#pragma unroll
    for (int i = 0; i < 4 * MB; ++i) {
      const int row = 4 * i + q, r = min(row, M - 1);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, slot + wave * kSlot + i * 1024, 16,
                                               r * 2 * K + ((r16 ^ (row & 15)) << 4), (u0 + u) * kStep * 2, 0, 0);
    }
    asm volatile("" ::: "memory");
  };
  auto slot_of = [&](int d) { return d == 0 ? x0 : (d == 1 ? x1 : x2); };
  // (each row's adapter and rank, for later: loaded here, they are waited for
  // with the first steps)
  const int key = LORA && lane < M ? row_key[m0 + lane] : -1;
  asm volatile("" ::: "memory");
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(d, slot_of(d), sb[d]);
  asm volatile("" ::: "memory");
  const int rank = key >= 0 ? pv.rank[key] : 0;
  asm volatile("" ::: "memory");

  floatx4 acc[CG][MB];
#pragma unroll
  for (int c = 0; c < CG; ++c)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) acc[c][mb] = floatx4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](int u, const uint8_t* slot, uint32_t sv) {
    const uint8_t* xs = slot + wave * kSlot;
    uint4 xf[MB][4], code[CG];
    float scale[CG];
    const int g0 = (u0 + u) * kStepGroups;
#pragma unroll
    for (int c = 0; c < CG; ++c) {
      code[c] = *reinterpret_cast<const uint4*>(xs + kX + (16 * c + r16) * 64 + ((q ^ (r16 >> 2)) << 4));
      const int from = min(16 * c + r16, cols - 1);
      const uint32_t four = (uint32_t)__builtin_amdgcn_ds_bpermute(from * 4, (int)sv);
      scale[c] = q4_scale((four >> (8 * (q + max(from * G + g0 - send, 0)) & 31)) & 255u);
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        xf[mb][j] = *reinterpret_cast<const uint4*>(xs + (16 * mb + r16) * 256 + (((4 * q + j) ^ r16) << 4));
    if (g0 + kStepGroups > G) {  // the last step of a ragged K
      const bool in = g0 + q < G;
#pragma unroll
      for (int c = 0; c < CG; ++c) {
        code[c].x = in ? code[c].x : 0u;
        code[c].y = in ? code[c].y : 0u;
        code[c].z = in ? code[c].z : 0u;
        code[c].w = in ? code[c].w : 0u;
        scale[c] = in ? scale[c] : 1.f;
      }
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          xf[mb][j].x = in ? xf[mb][j].x : 0u;
          xf[mb][j].y = in ? xf[mb][j].y : 0u;
          xf[mb][j].z = in ? xf[mb][j].z : 0u;
          xf[mb][j].w = in ? xf[mb][j].w : 0u;
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int c = 0; c < CG; ++c) {
        const uint4 v = code[c];
        const uint4 f = q4_bf8(j == 0 ? v.x : (j == 1 ? v.y : (j == 2 ? v.z : v.w)), scale[c]);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
          acc[c][mb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(xf[mb][j]), as_bf16x8(f), acc[c][mb], 0, 0, 0);
      }
  };
  int i = 0;
  for (; i + D < mine; i += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      __builtin_amdgcn_s_waitcnt(vmcnt_imm((D - 1) * kLoads));  // this step has landed, those after it may not have
      asm volatile("" ::: "memory");
      multiply(i + d, slot_of(d), sb[d]);
      // the slot's reads are done before it is filled again
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(63) & ~(15 << 8));
      fetch(i + d + D, slot_of(d), sb[d]);
    }
  }
#pragma unroll
  for (int d = 0; d < D; ++d) {  // the last steps
    if (D - 1 - d == 2)
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(2 * kLoads));
    else if (D - 1 - d == 1)
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(kLoads));
    else
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    asm volatile("" ::: "memory");
    if (i + d < mine) multiply(i + d, slot_of(d), sb[d]);
  }

  if (LORA) {
    shrink_items(pv, proj, X, key, rank, (int)(blockIdx.x % (ncb * S)) + ncb * S * wave, ncb * S * NW, SK,
                 T + (size_t)m0 * pv.max_rank, (size_t)rows * pv.max_rank);
  }

  // the waves' shares of K, in order; a thread takes four rows of a column
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  floatx4* red = reinterpret_cast<floatx4*>(x0);  // [NW][CG][MB][64]
#pragma unroll
  for (int c = 0; c < CG; ++c)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) red[((wave * CG + c) * MB + mb) * 64 + lane] = acc[c][mb];
  __syncthreads();
  for (int e = wave; e < CG * MB; e += NW) {
    floatx4 sum = red[e * 64 + lane];
#pragma unroll
    for (int h = 1; h < NW; ++h) sum += red[(h * CG * MB + e) * 64 + lane];
    const int c = n0 + 16 * (e / MB) + r16;
    if (c >= N) continue;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int r = (e % MB) * 16 + q * 4 + v;
      if (r >= M) continue;
      if (part)
        part[((size_t)kq * rows + m0 + r) * N + c] = sum[v];
      else
        Y[(size_t)(m0 + r) * N + c] = (uint16_t)f2bf(sum[v]);
    }
  }
}

template <int MB, int CG, int NW, int D, bool LORA>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(NW / 4, 8))) void q4_rows_kernel(
    Q4View w, const uint16_t* __restrict__ X, int M, int S, uint16_t* __restrict__ Y, float* __restrict__ part,
    PoolView pv, int proj, const int32_t* __restrict__ row_key, float* __restrict__ T, int SK) {
  constexpr int kSlot = NW * (MB * 4096 + CG * 1024);
  __shared__ __attribute__((aligned(16))) uint8_t x0[kSlot], x1[kSlot], x2[D > 2 ? kSlot : 16];
  q4_rows_body<MB, CG, NW, D, LORA>(w, X, M, S, Y, part, pv, proj, row_key, T, SK, x0, x1, x2);
}

// Sums the S slices' partial products in order, adds the row's low-rank term
// (T's slices in order; the ranks 16 at a time to the waves in turn, each in
// order, then the waves' sums in order) and writes Y: a workgroup 512 columns of
// a row, eight side by side to a thread, loaded at once wherever they begin
// (rows of an odd N have no alignment; 1024 rows of 4100 columns, 16 ranks: 14
// us, a column at a time 48).  The last thread of a row takes the last eight
// and writes what is its own.  What takes the time is waiting, so a wave's next
// pages of Up are on their way while those before are added.  WIDE: N >= 8;
// else a column at a time.
struct __attribute__((packed, aligned(2))) Words4 { uint32_t v[4]; };
struct __attribute__((packed, aligned(4))) Floats8 { float v[8]; };
constexpr int kQ4FinishColumns = 8 * 64, kQ4FinishWaves = 4;
template <bool WIDE, bool LORA>
__global__ __launch_bounds__(64 * (LORA ? kQ4FinishWaves : 1)) void q4_finish_kernel(const float* __restrict__ part, int S,
                                                                     uint16_t* __restrict__ Y, int M, int N,
                                                                     PoolView pv, int proj,
                                                                     const int32_t* __restrict__ row_key,
                                                                     const float* __restrict__ T, int SK) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int r = (int)blockIdx.y, b0 = (int)blockIdx.x * kQ4FinishColumns;
  const int c0 = b0 + 8 * lane, at = WIDE ? min(c0, N - 8) : 0;  // this thread's columns, and the eight it loads
  const int key = LORA ? scalar(row_key + r) : -1;
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.f;
  const float* p = part + (size_t)r * N;
  const size_t stride = (size_t)M * N;
#pragma unroll 4
  for (int s = 0; s < (wave == 0 ? S : 0); ++s, p += stride) {
    if (WIDE) {
      const Floats8 f = *reinterpret_cast<const Floats8*>(p + at);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += f.v[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += p[min(e, N - 1)];
    }
  }
  float low[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) low[e] = 0.f;
  if (LORA && key >= 0) {
    const int rank = scalar(pv.rank + key);
    const float scale = scalar(pv.scale + key);
    const int32_t* upage = pv.up_page + ((size_t)key * pv.n_proj + proj) * pv.max_rank;
    constexpr int Q = 16;  // ranks of a round
    struct Round { Words4 u[Q]; };
    for (int q0 = 0; q0 < rank; q0 += 64) {
      const int n = min(rank - q0, 64), own = q0 + min(lane, n - 1);  // a rank a lane
      const int page = upage[own];
      float t = 0.f;
#pragma unroll 4
      for (int k = 0; k < SK; ++k) t += T[((size_t)k * M + r) * pv.max_rank + own];
      t *= scale;
      const auto load = [&](int j, Round& o) {
#pragma unroll
        for (int i = 0; i < Q; ++i) {
          const uint16_t* up = pv.up + (size_t)__builtin_amdgcn_readlane(page, min(j + i, n - 1)) * N;
          if (WIDE) {
            o.u[i] = *reinterpret_cast<const Words4*>(up + at);
          } else {
#pragma unroll
            for (int f = 0; f < 4; ++f) o.u[i].v[f] = up[min(2 * f, N - 1)] | (uint32_t)up[min(2 * f + 1, N - 1)] << 16;
          }
        }
      };
      const auto add = [&](int j, const Round& o) {
#pragma unroll
        for (int i = 0; i < Q; ++i) {
          if (j + i >= n) break;
          const float ti = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(t), j + i));
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            low[2 * f] = fmaf(ti, lo_bf(o.u[i].v[f]), low[2 * f]);
            low[2 * f + 1] = fmaf(ti, hi_bf(o.u[i].v[f]), low[2 * f + 1]);
          }
        }
      };
      Round a, b;
      const int step = Q * waves;
      if (Q * wave < n) load(Q * wave, a);
      for (int j = Q * wave; j < n; j += 2 * step) {
        if (j + step < n) load(j + step, b);
        add(j, a);
        if (j + 2 * step < n) load(j + 2 * step, a);
        if (j + step < n) add(j + step, b);
      }
    }
  }
  if (LORA) {
    __shared__ float other[kQ4FinishWaves - 1][8][64];
    if (wave > 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) other[wave - 1][e][lane] = low[e];
    }
    if (waves > 1) __syncthreads();
    if (wave > 0) return;
    for (int w = 1; w < waves; ++w)
#pragma unroll
      for (int e = 0; e < 8; ++e) low[e] += other[w - 1][e][lane];
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += low[e];
  }
  if (LORA && key == -2) {
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = __uint_as_float(0x7fc00000u);
  }
  uint16_t* y = Y + (size_t)r * N;
  if (WIDE && c0 + 8 <= N) {
    *reinterpret_cast<Words4*>(y + c0) = Words4{
        {pack_bf2(sum[0], sum[1]), pack_bf2(sum[2], sum[3]), pack_bf2(sum[4], sum[5]), pack_bf2(sum[6], sum[7])}};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (at + e >= c0 && at + e < N) y[at + e] = (uint16_t)f2bf(sum[e]);
  }
}

int conv_grid(int64_t n8) {
  const int64_t g = (n8 + kConvThreads - 1) / kConvThreads;
  return (int)(g < 8192 ? g : 8192);
}

struct RowsArgs {
  const Q4View& w;
  const uint16_t* X;
  int M;
  uint16_t* Y;
  float* part;
  PoolView pv;
  int proj;
  const int32_t* row_key;
  float* T;
};

template <int MB, int CG, int NW, int D, bool LORA>
hipError_t launch_rows(const RowsArgs& a, const Q4Plan& p, hipStream_t st) {
  const int ncb = (a.w.N + 16 * CG - 1) / (16 * CG);
  MLORA_LAUNCH(LORA ? "q4_rows+shrink" : "q4_rows", (q4_rows_kernel<MB, CG, NW, D, LORA>), dim3(ncb * p.S * q4_row_blocks(a.M)),
               dim3(64 * NW),
               0, st, a.w, a.X, a.M, p.S, a.Y, p.direct ? nullptr : a.part, a.pv, a.proj, a.row_key, a.T, p.SK);
  return launched();
}

template <bool LORA>
hipError_t launch_rows_form(const RowsArgs& a, const Q4Plan& p, hipStream_t st) {
  if (a.M <= 16) {
    if (p.cg == 1) return launch_rows<1, 1, 8, 2, LORA>(a, p, st);
    if (p.cg == 2) return launch_rows<1, 2, 8, 2, LORA>(a, p, st);
    if (p.cg == 3) return launch_rows<1, 3, 8, 2, LORA>(a, p, st);
    return launch_rows<1, 4, 8, 2, LORA>(a, p, st);
  }
  if (a.M <= 32) {
    if (p.cg == 1) return launch_rows<2, 1, 8, 2, LORA>(a, p, st);
    if (p.cg == 2) return launch_rows<2, 2, 4, 3, LORA>(a, p, st);
    if (p.cg == 3) return launch_rows<2, 3, 4, 3, LORA>(a, p, st);
    return launch_rows<2, 4, 4, 3, LORA>(a, p, st);
  }
  if (a.M <= 48) return launch_rows<3, 4, 4, 2, LORA>(a, p, st);
  return launch_rows<4, 4, 4, 2, LORA>(a, p, st);
}

}  // namespace

hipError_t launch_q4_quantize(const uint16_t* W, uint8_t* codes, uint8_t* scales, int64_t n, hipStream_t stream) {
  MLORA_LAUNCH("q4_quantize", q4_quantize_kernel, dim3(conv_grid(n / 8)), dim3(kConvThreads), 0, stream, W, codes,
               scales, n / 8);
  return launched();
}

hipError_t launch_q4_dequantize(const uint8_t* codes, const uint8_t* scales, uint16_t* W, int64_t n,
                                hipStream_t stream) {
  MLORA_LAUNCH("q4_dequantize", q4_dequantize_kernel, dim3(conv_grid(n / 8)), dim3(kConvThreads), 0, stream, codes,
               scales, W, n / 8);
  return launched();
}

bool q4_few_rows(int M, int K, int N) {
  // The bf16 products have a rate that these do not reach, but the weight has
  // to be made first, and a small product does not reach it either (4096
  // channels, three adapters of rank 16; as they are against bf16 first: 256
  // rows x 4096 27.3 and 38.5 us, 600 x 4096 61 and 68, 1500 x 2048 66 and 63,
  // without adapters 46 and 58, 400 x 11008 96 and 88, 1024 x 4096 88 and 67,
  // 4000 x 1000 92 and 75; 800 x 1024 of 1024 channels 17 and 30).  Where K is
  // not whole steps or N not whole vectors they are slower still (1024 x 4096,
  // K 4064: 83 and 238 us).
  if (K < kQ4MinDin) return false;
  if (M <= 256 || (long)M * N <= 3l << 20) return true;
  return (K % kStep != 0 || N % 8 != 0) && M <= 1024;
}

hipError_t launch_q4_pad(const Q4View& w, const uint16_t* X, int M, uint16_t* Wp, uint16_t* Xp, hipStream_t stream) {
  MLORA_LAUNCH("q4_pad", q4_pad_kernel, dim3(w.N + M), dim3(kConvThreads), 0, stream, w, X, Wp, Xp, w.K / 8,
               q4_padded(w.K) / 8);
  return launched();
}

Q4Plan q4_plan(int M, int K, int N, bool lora) {
  Q4Plan p{};
  const int steps = (K + kStep - 1) / kStep, groups = (N + 15) / 16;
  // Columns of a workgroup: as few groups of 16 as let one round of workgroups
  // (one a CU) cover the columns (11008 columns, 16 rows: three groups 9.2 us,
  // one 10.8, two 11.9, four 10.5); above 32 rows four, because X is read
  // again by every workgroup; two where a wave has few steps (4096 x 4096, one
  // row: 6.0 us, one group 6.6).
  p.cg = M > 32 ? 4 : (groups + 255) / 256;
  if (p.cg > 4) p.cg = 4;
  if (M <= 16 && p.cg == 1 && steps <= 32) p.cg = 2;
  // Slices of K where workgroups are few.  They cost a launch that sums them
  // (4 us), so without the low-rank term, which has that launch anyway, only
  // many rows or steps are sliced (61 rows of 11008 channels, 4096 columns:
  // four slices 20.4 us, one 48; one row of it: one slice 8.3 us, two 11.3).
  const int ncb = (groups + p.cg - 1) / p.cg * q4_row_blocks(M), waves = M > 32 ? 4 : 8;
  p.S = 1;
  if (M > 32 || lora || steps > 16 * waves) p.S = 256 / ncb;
  if (p.S > steps / waves) p.S = steps / waves;
  if (p.S > 16) p.S = 16;
  if (p.S < 1) p.S = 1;
  p.direct = p.S == 1 && !lora;
  // the low-rank inner product: slices of 512 channels or more
  p.SK = (K + 511) / 512;
  if (p.SK > kQ4TSlices) p.SK = kQ4TSlices;
  return p;
}

hipError_t launch_q4_rows(const Q4View& w, const uint16_t* X, int M, uint16_t* Y, float* part, const PoolView* pv,
                          int proj, const int32_t* row_key, float* T, hipStream_t stream) {
  const Q4Plan p = q4_plan(M, w.K, w.N, pv != nullptr);
  const RowsArgs a{w, X, M, Y, part, pv ? *pv : PoolView{}, proj, row_key, T};
  const hipError_t e = pv ? launch_rows_form<true>(a, p, stream) : launch_rows_form<false>(a, p, stream);
  if (e != hipSuccess || p.direct) return e;
  const bool wide = w.N >= 8;
  // several waves a workgroup while that leaves a CU 16 of them (61 rows of 4096
  // columns, ranks to 64: 6.1 us, one wave 8.7; 406 rows of 15769: 62 and 45)
  const int tiles = (w.N + kQ4FinishColumns - 1) / kQ4FinishColumns;
  int waves = pv ? (pv->max_rank + 15) / 16 : 1;
  const int room = (int)(4096 / ((long)tiles * M));
  waves = waves > kQ4FinishWaves ? kQ4FinishWaves : waves;
  waves = waves > room ? (room < 1 ? 1 : room) : waves;
  const dim3 g(tiles, M), b(64 * waves);
  if (pv) {
    if (wide)
      MLORA_LAUNCH("q4_finish", (q4_finish_kernel<true, true>), g, b, 0, stream, part, p.S, Y, M, w.N, a.pv, proj,
                   row_key, T, p.SK);
    else
      MLORA_LAUNCH("q4_finish", (q4_finish_kernel<false, true>), g, b, 0, stream, part, p.S, Y, M, w.N, a.pv, proj,
                   row_key, T, p.SK);
  } else {
    if (wide)
      MLORA_LAUNCH("q4_finish", (q4_finish_kernel<true, false>), g, b, 0, stream, part, p.S, Y, M, w.N, a.pv, proj,
                   row_key, T, p.SK);
    else
      MLORA_LAUNCH("q4_finish", (q4_finish_kernel<false, false>), g, b, 0, stream, part, p.S, Y, M, w.N, a.pv, proj,
                   row_key, T, p.SK);
  }
  return launched();
}

}  // namespace mlora
