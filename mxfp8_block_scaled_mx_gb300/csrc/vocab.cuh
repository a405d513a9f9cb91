// vocab.cuh -- what the kernels of the vocabulary loss share: the softmax in powers
// of two, and labels.
#pragma once

#include <cstdint>

#include "kernels.h"

namespace mx {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ int64_t label_of(const VocabParams& p, int32_t row) {
  return p.labels_64 ? static_cast<const int64_t*>(p.labels)[row]
                     : static_cast<const int32_t*>(p.labels)[row];
}

__device__ __forceinline__ bool counts(const VocabParams& p, int64_t label) {
  return label != p.ignore_index && label >= 0 && label < p.vocab;
}

}  // namespace mx
