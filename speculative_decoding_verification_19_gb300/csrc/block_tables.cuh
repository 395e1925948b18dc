// Internal interface between the C ABI layer and the block-table kernel.
#pragma once

#include "common.cuh"

namespace specv {

// Most rows, and most block-table entries, of one call.
constexpr int kPagesMaxItems = 1 << 30;

struct PageArgs {
  const int32_t* ctx_lens;
  const int32_t* row_start;
  const int32_t* parent;
  int rows, window, sinks;
  int32_t* block_table;
  int32_t* span;
  int32_t* pool;
  int32_t* pool_state;
  int64_t* slots;
  int32_t* positions;
  int32_t* ok;
  spec_dims d;
  void* ws;
};

cudaError_t block_tables_launch(const PageArgs& a, const WsLayout& lay, cudaStream_t st,
                                int* launches);

}  // namespace specv
