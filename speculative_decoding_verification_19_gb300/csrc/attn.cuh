// Internal interface between the C ABI layer and the attention kernels.
#pragma once

#include "common.cuh"

namespace specv {

struct AttnArgs {
  const void* q;
  const void* k_new;
  const void* v_new;
  void* k_cache;
  void* v_cache;
  const int32_t* block_table;
  const int32_t* ctx_lens;
  const int32_t* parent;
  void* out;
  float* lse;
  spec_dims d;
  float scale;
  int window, sinks;  // window 0: every cached position is visible
  void* ws;
};

// What a sliding window and sinks leave of a request with ctx cached tokens:
// the first position of the window of its first new row (the others' windows
// start later), the first page of the window, the pages of the sinks.
__host__ __device__ __forceinline__ int win_first(int ctx, int window) {
  return ctx - window + 1 > 0 ? ctx - window + 1 : 0;
}
__host__ __device__ __forceinline__ bool win_page(int page, int ctx, int window, int sinks) {
  return page < ceil_div(sinks, kBlock) || page >= win_first(ctx, window) / kBlock;
}
// Key tiles of `keys` positions: the sinks' tiles come first, then the
// window's; tiles between them are skipped.  Tile j of the kept ones is tile
// j, or j + skip from the sinks' tiles on.
__host__ __device__ __forceinline__ int win_skip(int ctx, int window, int sinks, int keys) {
  const int s = win_first(ctx, window) / keys - ceil_div(sinks, keys);
  return s > 0 ? s : 0;
}

// CTAs of the persistent tensor-core kernel never exceed this (partials are
// sized for it).
constexpr int kMaxAttnCtas = 512;

// Floats per partial row of the tensor-core path: D outputs, the log2-sum-exp
// at index D, padded so every row starts on a 16-byte boundary.
__host__ __device__ constexpr int tc_part_stride(int D) { return D + 4; }

// Depth of new row n of a request, and the mask of its ancestors-or-self that
// are fewer than `window` positions above it or among the sinks (par: the
// request's checked topology, or NULL for a chain).
__device__ __forceinline__ void win_row_mask(const int32_t* par, int n, int ctx, int window,
                                             int sinks, ulonglong2* mask, int32_t* depth) {
  int at = n;
  if (par != nullptr) {
    at = 0;
    for (int k = n; k > 0 && at < kMaxNodes; k = par[k]) ++at;
  }
  unsigned long long lo = 0, hi = 0;
  for (int k = n, dk = at; k >= 0 && dk >= 0; k = par != nullptr ? par[k] : k - 1, --dk) {
    if (at - dk >= window && ctx + dk >= sinks) continue;
    if (k < 64) lo |= 1ull << k;
    else hi |= 1ull << (k - 64);
  }
  *mask = make_ulonglong2(lo, hi);
  *depth = at;
}

size_t attn_simt_smem_bytes(int R, int D);
size_t attn_tc_part_floats(const spec_dims& d);
cudaError_t kv_append_launch(const AttnArgs& a, const WsLayout& lay, cudaStream_t st, int* launches);
cudaError_t attn_launch_simt(const AttnArgs& a, const WsLayout& lay, cudaStream_t st, int* launches);
cudaError_t attn_launch_tc(const AttnArgs& a, const WsLayout& lay, cudaStream_t st, int* launches);

}  // namespace specv
