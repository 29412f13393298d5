// Shared by the kernels of 4-bit weights: the view of a weight and the
// conversion of its codes to bf16.
#pragma once

#include "internal.h"

namespace mlora {

constexpr int kQ4Group = 32;                  // channels that share a scale
constexpr int kQ4ExpMin = 2, kQ4ExpMax = 252;  // scale bytes of finite weights

struct Q4View {
  const uint8_t* codes;   // [N][K/2], the lower half of a byte first
  const uint8_t* scales;  // [N][K/32]
  int32_t K, N;           // K a multiple of 32
};

// the scale that a byte stands for: 2^(b - 127) from 2 to 252, NaN else
__device__ __forceinline__ float q4_scale(uint32_t b) {
  return b - kQ4ExpMin <= (uint32_t)(kQ4ExpMax - kQ4ExpMin) ? __uint_as_float(b << 23) : __uint_as_float(0x7fc00000u);
}

// the two codes of byte B of w times the scale, as packed bf16: exact (a code
// has 2 significant bits and the scale's range leaves it a normal number)
template <int B>
__device__ __forceinline__ uint32_t q4_bf2(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, B));
}
// the eight codes of w
__device__ __forceinline__ uint4 q4_bf8(uint32_t w, float scale) {
  return make_uint4(q4_bf2<0>(w, scale), q4_bf2<1>(w, scale), q4_bf2<2>(w, scale), q4_bf2<3>(w, scale));
}

hipError_t launch_q4_quantize(const uint16_t* W, uint8_t* codes, uint8_t* scales, int64_t n, hipStream_t stream);
hipError_t launch_q4_dequantize(const uint8_t* codes, const uint8_t* scales, uint16_t* W, int64_t n,
                                hipStream_t stream);

// Products of few rows, and small ones, take the codes as they are, 64 rows to
// a workgroup; larger ones make the weight bf16 first and take the bf16 products.
constexpr int kQ4RowBlock = 64, kQ4MinDin = 128, kQ4TSlices = 16;
inline int q4_row_blocks(int M) { return (M + kQ4RowBlock - 1) / kQ4RowBlock; }
bool q4_few_rows(int M, int K, int N);
// For the bf16 products of more rows: the weight, and X, in rows of a multiple
// of 128 channels, zeros past K (the products are slow for other K: 2048 rows,
// K 4064: 103 us, padded 80; with the low-rank term 117 and 96).
__host__ __device__ constexpr int q4_padded(int K) { return (K + 127) / 128 * 128; }
hipError_t launch_q4_pad(const Q4View& w, const uint16_t* X, int M, uint16_t* Wp, uint16_t* Xp, hipStream_t stream);
// The form of a product of M rows: workgroups of 16 * cg columns, K in S
// slices.  Without the low-rank term and with one slice the product is
// written as it is; else partial products [S][M][N] go to scratch and a
// finish pass sums them.
struct Q4Plan {
  int cg, S;
  bool direct;
  int SK;  // slices of din of the low-rank inner product, at most kQ4TSlices
  size_t part_floats(int M, int N) const { return direct ? 0 : (size_t)S * M * N; }
};
Q4Plan q4_plan(int M, int K, int N, bool lora);
// Y = X W^T, with row_key also the low-rank term of each row: T its scratch,
// the plan's SK times [M][max_rank].
hipError_t launch_q4_rows(const Q4View& w, const uint16_t* X, int M, uint16_t* Y, float* part, const PoolView* pv,
                          int proj, const int32_t* row_key, float* T, hipStream_t stream);

}  // namespace mlora
