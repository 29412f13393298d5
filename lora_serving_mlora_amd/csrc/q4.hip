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
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kConvThreads) void q4_quantize_kernel(const uint16_t* __restrict__ W,
                                                                   uint8_t* __restrict__ codes,
                                                                   uint8_t* __restrict__ scales, int64_t n8) {
  const int64_t stride = (int64_t)gridDim.x * kConvThreads;
  for (int64_t i = (int64_t)blockIdx.x * kConvThreads + threadIdx.x; i < n8; i += stride) {
    const uint4 v = reinterpret_cast<const uint4*>(W)[i];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) top = max(top, max(w[j] & 0x7fffu, (w[j] >> 16) & 0x7fffu));
    // n8 is a multiple of 4: the four threads of a group are here together
    top = max(top, (uint32_t)__shfl_xor((int)top, 1, 64));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2, 64));
    uint32_t b = 255, code = 0;
    if (top < 0x7f80u) {
      const int e = (int)(top >> 7) - ((top & 127u) <= 64u ? 2 : 1);
      b = min(max(e, kQ4ExpMin), kQ4ExpMax);
      const float inv = __uint_as_float((254u - b) << 23);  // 2^(127 - b), a normal number for b <= 252
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t x = (w[j >> 1] >> (16 * (j & 1))) & 0xffffu;
        const float a = bf2f(x & 0x7fffu) * inv;
        // halfway values go to the even code
        uint32_t c = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) + (a > 5.f);
        c |= (x >> 15) << 3;
        code |= c << (4 * j);
      }
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

// ---------------------------------------------------------------------------
// Products of up to 64 rows.  What bounds them is the codes' way from memory,
// so each code is read once, by the lane whose operand it is: a lane takes
// the 16 bytes (32 channels, one group) of one column at a time, the 16
// columns of a wave by the 4 lane groups' next groups of channels, and feeds
// them as four 16x16x32 products.  Which channel stands where in K is free as
// long as X agrees, so X is read from LDS in the same order.  8 waves: CG
// column groups of 16, 8 / CG shares of the slice of K (its 128-channel steps
// dealt in turn), summed through LDS in order.
// LDS: X slice [M][xs_stride] in 1 KiB blocks whose 16-byte chunks are
// XOR-swizzled by (row & 15), so that the 16 rows of a fragment hit 16
// different chunk positions.
// ---------------------------------------------------------------------------
constexpr int kRowsWaves = 8, kStep = 128, kRound = 4;
constexpr size_t kXsMax = 128 << 10;  // bytes of LDS for X

template <int MB, int CG, bool LORA>
__global__ __launch_bounds__(64 * kRowsWaves) void q4_rows_kernel(Q4View w, const uint16_t* __restrict__ X, int M,
                                                                  int S, int xs_stride, uint16_t* __restrict__ Y,
                                                                  float* __restrict__ part, PoolView pv, int proj,
                                                                  const int32_t* __restrict__ row_key,
                                                                  float* __restrict__ T, int n_shrink) {
  extern __shared__ __attribute__((aligned(16))) uint16_t xs[];
  constexpr int KH = kRowsWaves / CG;
  if (LORA && (int)blockIdx.x < n_shrink) {
    for (int k = blockIdx.x; k < M; k += n_shrink)
      shrink_row_body<true, kRowsWaves>(pv, proj, X, row_key, k, T, row_desc(T, M, pv.max_rank));
    return;
  }
  const int K = w.K, N = w.N, G = K / kQ4Group;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int cg = wave % CG, kh = wave / CG;
  const int ncb = (N + 16 * CG - 1) / (16 * CG);
  const int b = (int)blockIdx.x - (LORA ? n_shrink : 0);
  const int cb = b % ncb, kq = b / ncb;
  const int steps = (K + kStep - 1) / kStep;
  const int s0 = (int)((long)steps * kq / S), ns = (int)((long)steps * (kq + 1) / S) - s0;
  const int k0 = s0 * kStep, Kq = min(ns * kStep, K - k0);
  const int r16 = lane & 15, q = lane >> 4;

  // X slice -> LDS: instruction (row r, 1 KiB block bl); lane l fetches chunk
  // l ^ (r & 15) of the block into place l; nothing is fetched past the slice
  const __amdgpu_buffer_rsrc_t rx =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(X), (short)0, M * K * 2, 0x00020000);
  const int blocks = (Kq + 511) / 512;
  for (int i = wave; i < M * blocks; i += kRowsWaves) {
    const int r = i / blocks, bl = i % blocks;
    if (bl * 64 + (lane ^ (r & 15)) < Kq / 8)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, xs + (size_t)r * xs_stride + bl * 512, 16,
                                               (lane ^ (r & 15)) * 16, (r * K + k0 + bl * 512) * 2, 0, 0);
  }

  // the codes and scale bytes of kRound steps of this wave, from its step
  // kh + KH * i on; past the weight's end the last group is read again
  const int col = min(cb * 16 * CG + 16 * cg + r16, N - 1);
  const uint8_t* wc = w.codes + (size_t)col * (K / 2);
  const uint8_t* ws = w.scales + (size_t)col * G;
  uint4 code[kRound], code_n[kRound];
  uint32_t sb[kRound], sb_n[kRound];
  auto fetch = [&](int i, uint4 (&c)[kRound], uint32_t (&s)[kRound]) {
#pragma unroll
    for (int u = 0; u < kRound; ++u) {
      const int g = min((s0 + kh + KH * (i + u)) * (kStep / kQ4Group) + q, G - 1);
      c[u] = *reinterpret_cast<const uint4*>(wc + (size_t)g * 16);
      s[u] = ws[g];
    }
  };
  fetch(0, code, sb);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();

  floatx4 acc[MB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) acc[mb] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int mine = (ns - kh + KH - 1) / KH;  // steps of this wave
  for (int i = 0; i < mine; i += kRound) {
    if (i + kRound < mine) fetch(i + kRound, code_n, sb_n);
#pragma unroll
    for (int u = 0; u < kRound; ++u) {
      if (i + u < mine) {
        const int s = kh + KH * (i + u);
        const bool in = (s0 + s) * (kStep / kQ4Group) + q < G;  // false in the last step of a ragged K
        const float scale = in ? q4_scale(sb[u]) : 1.f;
        const uint32_t dw[4] = {code[u].x, code[u].y, code[u].z, code[u].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 f = q4_bf8(in ? dw[j] : 0u, scale);
          const int c = s * 16 + q * 4 + j;  // 16-byte chunk of the slice row
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) {
            const int r = min(mb * 16 + r16, M - 1);
            uint4 a = *reinterpret_cast<const uint4*>(xs + (size_t)r * xs_stride + (c >> 6) * 512 +
                                                      (((c & 63) ^ (r & 15)) << 3));
            if (!in) a = make_uint4(0u, 0u, 0u, 0u);
            acc[mb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(f), acc[mb], 0, 0, 0);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kRound; ++u) {
      code[u] = code_n[u];
      sb[u] = sb_n[u];
    }
  }

  // the shares of K, in order
  __syncthreads();
  floatx4* red = reinterpret_cast<floatx4*>(xs);  // [KH - 1][CG][MB][64]
  if (kh > 0) {
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) red[(((kh - 1) * CG + cg) * MB + mb) * 64 + lane] = acc[mb];
  }
  __syncthreads();
  if (kh > 0) return;
#pragma unroll
  for (int h = 0; h < KH - 1; ++h)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) acc[mb] += red[((h * CG + cg) * MB + mb) * 64 + lane];
  const int c = cb * 16 * CG + 16 * cg + r16;
  if (c >= N) return;
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int r = mb * 16 + q * 4 + v;
      if (r >= M) continue;
      if (part)
        part[((size_t)kq * M + r) * N + c] = acc[mb][v];
      else
        Y[(size_t)r * N + c] = (uint16_t)f2bf(acc[mb][v]);
    }
}

// Sums the S slices' partial products in order, adds the row's low-rank term
// and writes Y; 8 columns a thread.  VEC: N a multiple of 8, 16-byte aligned.
constexpr int kQ4FinishThreads = 64;
template <bool VEC, bool LORA>
__global__ __launch_bounds__(kQ4FinishThreads) void q4_finish_kernel(const float* __restrict__ part, int S,
                                                                     uint16_t* __restrict__ Y, int M, int N,
                                                                     PoolView pv, const float* __restrict__ T) {
  const int t = blockIdx.x * kQ4FinishThreads + threadIdx.x;
  const int per_row = (N + 7) / 8;
  if (t >= M * per_row) return;
  const int r = t / per_row, c0 = (t % per_row) * 8;
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.f;
  const float* p = part + (size_t)r * N + c0;
  const size_t stride = (size_t)M * N;
#pragma unroll 4
  for (int s = 0; s < S; ++s, p += stride) {
    if (VEC) {
      const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
      sum[0] += a.x; sum[1] += a.y; sum[2] += a.z; sum[3] += a.w;
      sum[4] += b.x; sum[5] += b.y; sum[6] += b.z; sum[7] += b.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c0 + e < N) sum[e] += p[e];
    }
  }
  if (LORA) {
    float y[8];
    lora_delta8_desc<VEC, false, 16>(pv, row_desc(const_cast<float*>(T), M, pv.max_rank), T, r, M, c0, N, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += y[e];
  }
  uint16_t* y = Y + (size_t)r * N + c0;
  if (VEC) {
    *reinterpret_cast<uint4*>(y) = make_uint4(pack_bf2(sum[0], sum[1]), pack_bf2(sum[2], sum[3]),
                                              pack_bf2(sum[4], sum[5]), pack_bf2(sum[6], sum[7]));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c0 + e < N) y[e] = (uint16_t)f2bf(sum[e]);
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

template <int MB, int CG, bool LORA>
hipError_t launch_rows(const RowsArgs& a, const Q4Plan& p, hipStream_t st) {
  const int n_shrink = LORA ? min((a.M + 7) / 8 * 8, 256) : 0;
  const int ncb = (a.w.N + 16 * CG - 1) / (16 * CG);
  const size_t red = (size_t)(kRowsWaves / CG - 1) * CG * MB * 64 * sizeof(floatx4);
  const size_t x = (size_t)a.M * p.xs_stride * 2;
  const size_t lds = x > red ? x : red;
  static LdsLimit limit;
  const hipError_t e = limit.ensure({(const void*)q4_rows_kernel<MB, CG, LORA>}, lds);
  if (e != hipSuccess) return e;
  MLORA_LAUNCH(LORA ? "q4_rows+shrink_rows" : "q4_rows", (q4_rows_kernel<MB, CG, LORA>), dim3(n_shrink + ncb * p.S),
               dim3(64 * kRowsWaves), lds, st, a.w, a.X, a.M, p.S, p.xs_stride, a.Y, p.direct ? nullptr : a.part, a.pv,
               a.proj, a.row_key, a.T, n_shrink);
  return launched();
}

template <int CG, bool LORA>
hipError_t launch_rows_mb(const RowsArgs& a, const Q4Plan& p, hipStream_t st) {
  if (a.M <= 16) return launch_rows<1, CG, LORA>(a, p, st);
  if (a.M <= 32) return launch_rows<2, CG, LORA>(a, p, st);
  if (a.M <= 48) return launch_rows<3, CG, LORA>(a, p, st);
  return launch_rows<4, CG, LORA>(a, p, st);
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

Q4Plan q4_plan(int M, int K, int N, bool lora) {
  Q4Plan p{};
  const int steps = (K + kStep - 1) / kStep;
  // the fewest slices whose X fits in LDS
  const int deepest = (int)(kXsMax / 2 / M) / 512 * 512 / kStep;
  int S = (steps + deepest - 1) / deepest;
  p.cg = !lora && M <= 16 ? 1 : 4;
  if (p.cg == 4) {
    const int ncb = (N + 63) / 64;
    while (ncb * S < 256 && steps / (S + 1) >= 2) ++S;
  }
  p.S = S;
  p.direct = S == 1 && !lora;
  p.xs_stride = ((steps + S - 1) / S * kStep + 511) / 512 * 512;
  return p;
}

hipError_t launch_q4_rows(const Q4View& w, const uint16_t* X, int M, uint16_t* Y, float* part, const PoolView* pv,
                          int proj, const int32_t* row_key, float* T, hipStream_t stream) {
  const Q4Plan p = q4_plan(M, w.K, w.N, pv != nullptr);
  const RowsArgs a{w, X, M, Y, part, pv ? *pv : PoolView{}, proj, row_key, T};
  hipError_t e;
  if (pv)
    e = launch_rows_mb<4, true>(a, p, stream);
  else
    e = p.cg == 1 ? launch_rows<1, 1, false>(a, p, stream) : launch_rows_mb<4, false>(a, p, stream);
  if (e != hipSuccess || p.direct) return e;
  const bool vec = w.N % 8 == 0 && reinterpret_cast<uintptr_t>(Y) % 16 == 0 &&
                   (!pv || reinterpret_cast<uintptr_t>(pv->up) % 16 == 0);
  const dim3 g((M * ((w.N + 7) / 8) + kQ4FinishThreads - 1) / kQ4FinishThreads), b(kQ4FinishThreads);
  if (pv) {
    if (vec)
      MLORA_LAUNCH("q4_finish", (q4_finish_kernel<true, true>), g, b, 0, stream, part, p.S, Y, M, w.N, *pv, T);
    else
      MLORA_LAUNCH("q4_finish", (q4_finish_kernel<false, true>), g, b, 0, stream, part, p.S, Y, M, w.N, *pv, T);
  } else {
    if (vec)
      MLORA_LAUNCH("q4_finish", (q4_finish_kernel<true, false>), g, b, 0, stream, part, p.S, Y, M, w.N, a.pv, T);
    else
      MLORA_LAUNCH("q4_finish", (q4_finish_kernel<false, false>), g, b, 0, stream, part, p.S, Y, M, w.N, a.pv, T);
  }
  return launched();
}

}  // namespace mlora
