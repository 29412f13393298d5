// Host side of the queries' and keys' norm and rotation.
#pragma once

#include "internal.h"

namespace mlora {

struct QkSide {
  const uint16_t* x;
  uint16_t* y;
  int64_t rs, hs, ors, ohs;  // strides of rows and heads in elements, in and out
  const uint16_t* w;         // [D], NULL: no norm
  int32_t heads;
};
struct QkRotary {
  QkSide side[2];  // queries, keys (heads 0: none)
  const int32_t* kv_len;
  const int32_t* row_off;
  int32_t n_seq, n_rows, D, rot, interleaved;
  const uint64_t* freq;  // [rot / 2] revolutions per position * 2^64
  float factor, eps;
};
hipError_t launch_qk_rotary(const QkRotary& a, hipStream_t stream);

}  // namespace mlora
