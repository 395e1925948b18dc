// Internal interface between the C ABI layer and the sampling kernel.
#pragma once

#include "common.cuh"

namespace specv {

struct SampleArgs {
  const void* logits;
  int64_t stride;  // elements between rows
  int rows, V, dtype;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* uniform;
  int32_t* out_tokens;
  float* out_prob;
  uint32_t* status;
};

constexpr int kSampleMaxVocab = 1 << 20;

cudaError_t sample_launch(const SampleArgs& a, cudaStream_t st, int* launches);

}  // namespace specv
