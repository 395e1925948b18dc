// Internal interface between the C ABI layer and the norm-and-rotation kernel.
#pragma once

#include "common.cuh"

namespace specv {

struct RopeArgs {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements between rows
  const void *q_weight, *k_weight;
  float eps;
  const int32_t* positions;
  const double* inv_freq;
  int rot_dim, interleaved, rows;
  void *q_out, *k_out;
  const int64_t* slots;
  void *k_cache, *v_cache;
  spec_dims d;
  void* ws;
};

cudaError_t qk_norm_rope_launch(const RopeArgs& a, const WsLayout& lay, cudaStream_t st,
                                int* launches);

}  // namespace specv
