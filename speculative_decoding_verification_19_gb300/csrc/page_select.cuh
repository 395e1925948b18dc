// Internal interface between the C ABI layer and the page-selection kernels.
#pragma once

#include "common.cuh"

namespace specv {

constexpr int kSelectMostPages = 1 << 30;  // places of a list (counts stay 32-bit)

struct BoundsArgs {
  const void* k_cache;
  const int32_t* block_table;
  const int32_t* from_lens;  // NULL: from the first page on
  const int32_t* ctx_lens;
  void* bounds;
  spec_dims d;
  uint32_t* status;
};
struct ScoreArgs {
  const void* q;
  const void* bounds;
  const int32_t* block_table;
  const int32_t* ctx_lens;
  float* scores;
  spec_dims d;
  uint32_t* status;
};
struct SelectArgs {
  const float* scores;
  const int32_t* ctx_lens;
  int n_pages, first, last;
  int32_t* pages;
  int32_t* counts;
  spec_dims d;
  uint32_t* status;
};

// Extrema that keep a NaN: a page whose sums hold one gets it as its score, and the
// selection says so.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

cudaError_t page_bounds_launch(const BoundsArgs& a, cudaStream_t st, int* launches);
cudaError_t page_score_launch(const ScoreArgs& a, cudaStream_t st, int* launches);
bool page_score_tc_ok(const spec_dims& d);
cudaError_t page_score_tc_launch(const ScoreArgs& a, cudaStream_t st, int* launches);
cudaError_t page_select_launch(const SelectArgs& a, cudaStream_t st, int* launches);

}  // namespace specv
