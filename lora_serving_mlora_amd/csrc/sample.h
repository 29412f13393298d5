// Host side of the sampler.
#pragma once

#include "internal.h"

namespace mlora {

constexpr int kSampleMaxVocab = 1 << 20;

struct SampleArgs {
  const void* logits;
  int64_t stride;  // elements between rows
  int32_t n, V;
  bool f32;
  const float* u;
  const float* temperature;  // each [n] or NULL
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* out;
};
hipError_t launch_sample(const SampleArgs& a, hipStream_t stream);

}  // namespace mlora
