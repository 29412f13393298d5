// Shared by the key/value cache kernels: the view of one layer's pages and of
// a batch that they take, and the conversions between e4m3 codes and bf16.
#pragma once

#include "internal.h"

namespace mlora {

constexpr int kKvBlk = 16;  // tokens that are contiguous for one channel of the values
constexpr int kKvExpMin = -64, kKvExpMax = 119;  // exponents of a page's scale

struct KvView {
  uint8_t* k;       // [n_blocks][H][B][D]
  uint8_t* v;       // [n_blocks][H][B/16][D][16]
  float* k_scale;   // [n_blocks][H]
  float* v_scale;
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* row_off;
  int32_t n_seq, width, table_stride, n_rows, max_new;
  int32_t H, D, lb;  // key/value heads, channels, log2 of a page's tokens
  int32_t n_blocks;
};

// rows of sequence i, kept inside the batch whatever row_off holds
struct KvSeq {
  int32_t row0, m, n;  // first row, rows, tokens with the new ones
};
__device__ __forceinline__ int kv_clamp(int n) { return min(max(n, -(1 << 30)), 1 << 30); }
__device__ __forceinline__ KvSeq kv_seq(const KvView& c, int i) {
  KvSeq s;
  const int a = c.row_off[i], b = c.row_off[i + 1];
  s.n = kv_clamp(c.kv_len[i]);
  s.row0 = min(max(a, 0), c.n_rows);
  s.m = min(max(b, s.row0), c.n_rows) - s.row0;
  return s;
}

// a place that is the same for the whole wave: a scalar load (the batch's
// tables, which do not change while a kernel runs)
template <class T>
__device__ __forceinline__ T kv_scalar(const T* p) {
  typedef const T __attribute__((address_space(4))) * constant;
  return *(constant)(uintptr_t)p;
}
__device__ __forceinline__ KvSeq kv_seq_scalar(const KvView& c, int i) {
  KvSeq s;
  const int a = kv_scalar(c.row_off + i), b = kv_scalar(c.row_off + i + 1);
  s.n = kv_clamp(kv_scalar(c.kv_len + i));
  s.row0 = min(max(a, 0), c.n_rows);
  s.m = min(max(b, s.row0), c.n_rows) - s.row0;
  return s;
}

// page of sequence i's page-index p, -1 where it has none that exists
__device__ __forceinline__ int kv_page_scalar(const KvView& c, int i, int p) {
  int id = -1;
  if (p >= 0 && p < c.width) id = kv_scalar(c.table + (size_t)i * c.table_stride + p);
  return (unsigned)id < (unsigned)c.n_blocks ? id : -1;
}

typedef __bf16 kv_bf16x2 __attribute__((ext_vector_type(2)));

// two e4m3 codes (the low or high half of w) times 2^e (scale's exponent), as
// packed bf16: exact, because a code has 4 significant bits
template <bool HI>
__device__ __forceinline__ uint32_t kv_bf2(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, HI));
}

hipError_t launch_kv_append(const KvView& c, const uint16_t* k, const uint16_t* v, int64_t rs, int64_t hs,
                            hipStream_t stream);
hipError_t launch_kv_read(const KvView& c, uint16_t* k, uint16_t* v, hipStream_t stream);

struct KvAttn {
  const uint16_t* q;
  int64_t rs, hs;  // q's strides in elements
  uint16_t* out;   // [n_rows][G * H][D]
  float scale;
  int32_t G, causal, window;
  void* work;
};
bool kv_attention_dim(int dim);
size_t kv_work_bytes(const KvView& c, int heads);
hipError_t launch_kv_attention(const KvView& c, const KvAttn& a, hipStream_t stream);

}  // namespace mlora
