// vocab.cuh -- what the kernels of the vocabulary loss share: labels, and the runs of
// a logit's contraction.
#pragma once

#include <cstdint>

#include "kernels.h"
#include "softmax.cuh"

namespace mx {

__device__ __forceinline__ int64_t label_of(const VocabParams& p, int32_t row) {
  return p.labels_64 ? static_cast<const int64_t*>(p.labels)[row]
                     : static_cast<const int32_t*>(p.labels)[row];
}

__device__ __forceinline__ bool counts(const VocabParams& p, int64_t label) {
  return label != p.ignore_index && label >= 0 && label < p.vocab;
}

// The tensor core cuts its FP32 accumulator off where it adds to it, so a long
// contraction loses a little of every term in the same direction: over 4096
// elements 1.2e-6 of lse.  For the logits (of the losses and, so that these are the
// same, of dz) a contraction of more than kRunSteps steps of 64 elements is therefore taken
// in equal runs of at most that, each in an accumulator of its own, which the epilogue
// adds in FP32, rounded to nearest.
constexpr int32_t kRunSteps = 16;
struct Runs {
  int32_t count, steps;  // steps of all but the last
  __device__ __forceinline__ explicit Runs(int32_t all, bool split) {
    count = split ? (all + kRunSteps - 1) / kRunSteps : 1;
    steps = (all + count - 1) / count;
    count = (all + steps - 1) / steps;
  }
};

}  // namespace mx
