// Internal interface between the C ABI layer and the attention kernels.
#pragma once

#include "common.cuh"

namespace specv {

// A request as the attention kernels see it where they do not read the whole
// context.  They run on a view: ctx cached keys in blocks of a table of its own,
// then the M new rows, as if that were the request; only the append and the
// checks go by the request itself.
//   kViewPrefix  the first prefix_len positions are the batch's shared prefix
//                and read elsewhere: ctx is less by prefix_len, the table starts
//                prefix_len / 16 entries later
//   kViewWhole   the same requests where reading the prefix once is not worth a
//                pass of its own: ctx as it is, the request check writes a table
//                of the shared pages and the request's own
//   kViewPages   the selected whole pages of each KV head, then the pages from
//                the last (partial) one of the context on; the request check
//                writes a table of block ids for every KV head
enum { kViewNone = 0, kViewPrefix = 1, kViewWhole = 2, kViewPages = 3 };
struct AttnView {
  int mode;
  const int32_t* prefix_table;  // [prefix_len / 16]
  int prefix_len;
  const int32_t* pages;   // [B, Hkv, n_pages], ascending
  const int32_t* counts;  // [B]
  int n_pages;
  const int32_t* table;   // block of page p of the view: table[b * stride_b + h * stride_h + p]
  int64_t stride_b, stride_h;
  int entries;            // pages of a view at most
  int32_t* ctx;           // [B] cached keys of the views (CUDA cores)
};
// Cached keys of a request's view (the request itself has been checked).
__device__ __forceinline__ int view_ctx(const AttnView& v, int b, int ctx) {
  if (v.mode == kViewPrefix) return ctx - v.prefix_len;
  if (v.mode == kViewWhole) return ctx;
  return __ldcg(v.counts + b) * kBlock + ctx % kBlock;
}

// Places in the workspace of what a call on views keeps while it runs.  No two of
// them overlap; they may lie where calls without a view have split-KV partials.
struct ViewPlaces {
  size_t part;    // partials of the requests' own keys, and the ranges that they have room for
  int ranges;     // (CUDA cores)
  size_t ctx;     // [B] int32 cached keys of every view (CUDA cores)
  size_t table;   // [B, Hkv, <= max_blocks] int32 block ids (kViewWhole, kViewPages)
  size_t own;     // [B*Hkv, rows] f32 rows of a request's own keys (kViewPrefix, tensor cores)
  size_t pfx;     // f32 rows: partials of the prefix (kViewPrefix)
  size_t end;     // bytes of the workspace up to the last of them
};

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
  AttnView view;      // mode kViewNone: the requests themselves
  ViewPlaces at;      // of the view, if there is one
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

// Checks of a view that needs the whole CTA (the request's length has been
// checked): bit 0 a bad argument, bit 1 a bad block id among the pages that the
// view holds, for this thread's share.  `write`: the table of block ids is
// written (kViewWhole and kViewPages; entries that are no block id stay out of it).
__device__ __forceinline__ int view_check(const AttnView& v, const spec_dims& d, const int32_t* bt,
                                          int b, int ctx, bool write) {
  const int pages = (int)ceil_div64((int64_t)ctx + d.M, kBlock);
  int bad = 0;
  int32_t* table = const_cast<int32_t*>(v.table) + (int64_t)b * v.stride_b;
  if (v.mode != kViewPages) {
    if (ctx < v.prefix_len) return 1;
    const int pp = v.prefix_len / kBlock;
#pragma unroll 4
    for (int p = threadIdx.x; p < pages; p += blockDim.x) {
      const int id = __ldcg(p < pp ? v.prefix_table + p : bt + p);
      if (id < 0 || id >= d.num_blocks) bad |= 2;
      else if (write && v.mode == kViewWhole) table[p] = id;
    }
    return bad;
  }
  const int n = __ldcg(v.counts + b), full = ctx / kBlock;
  if (n < 0 || n > v.n_pages || n > full) return 1;
  const int len = n + pages - full;  // pages of the view: at most `pages`
  constexpr int kAtOnce = 4;  // chains of loads (list, block table) of a thread side by side
  for (int e0 = threadIdx.x; e0 < d.Hkv * len; e0 += kAtOnce * blockDim.x) {
    int p[kAtOnce], before[kAtOnce], id[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int e = e0 + u * blockDim.x, h = e / len, j = e - h * len;
      p[u] = full + j - n;
      before[u] = -1;
      if (j < n && h < d.Hkv) {
        const int32_t* list = v.pages + ((int64_t)b * d.Hkv + h) * v.n_pages + j;
        p[u] = __ldcg(list);
        if (j > 0) before[u] = __ldcg(list - 1);
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int e = e0 + u * blockDim.x, h = e / len, j = e - h * len;
      id[u] = 0;
      if (h >= d.Hkv) continue;
      if (j < n && (p[u] < 0 || p[u] >= full || before[u] >= p[u])) bad |= 1;
      else id[u] = __ldcg(bt + p[u]);
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int e = e0 + u * blockDim.x, h = e / len, j = e - h * len;
      if (h >= d.Hkv) continue;
      if (id[u] < 0 || id[u] >= d.num_blocks) bad |= 2;
      else if (write) table[h * v.stride_h + j] = id[u];
    }
  }
  return bad;
}

// One pass over the keys of a shared prefix, for all rows of the batch that
// read a KV head: rows b * R + i * group + g of the head, in tiles.  A partial
// is a slot of tile rows of tc_part_stride(D) floats: the normalised output,
// then the log2-sum-exp at index D.
struct PrefixPlan {
  int tile;        // rows of a tile
  int tiles;       // tiles of a KV head
  int key_tiles;   // key tiles of the prefix
  int ctas;        // CTAs that share all (head, tile, key tile) items evenly, in this order; a
                   // unit (head, tile) u has its partials in slots u + c of the CTAs c that ran
                   // some of it.  0: every unit has `splits` ranges of keys, in slots
                   // u * splits + s
  int splits;
};
// The CTA of plan p that runs item x.
__host__ __device__ __forceinline__ int prefix_cta(const PrefixPlan& p, int64_t items, int64_t x) {
  const int64_t n = (x + 1) * p.ctas - 1;
  return (n | items) >> 32 == 0 ? (int)((uint32_t)n / (uint32_t)items) : (int)(n / items);
}

// What the merge needs of the attention over a request's own keys.
struct OwnPart {
  const float* part;  // row r of split s of (request, head) pair: part[((pair * splits + s) * R + r) * stride]
  int splits, stride, split_keys;
  const int32_t* ctx;     // of the views
  const int32_t* ok;      // [B] nonzero: the request has passed its checks
};

// Views of the requests in ranges of keys, for prefix_simt_kernel's tiles.
struct ViewRanges {
  int64_t stride_b, stride_h;
  const int32_t* ctx;
  const int32_t* ok;
  const ulonglong2* anc;  // [B, M] ancestors-or-self
  int split_keys;
};
int view_range_unit(const spec_dims& d);  // ranges are whole numbers of it
int view_ctas();                          // CTAs of a wave
cudaError_t view_split_launch(const AttnArgs& a, const ViewRanges& own, int splits, float* part,
                              cudaStream_t st);

size_t attn_simt_smem_bytes(int R, int D);
// CTAs of the prefix kernel on tensor cores never exceed this (its partials are
// sized for it).
constexpr int kMaxPrefixCtas = 160;

size_t prefix_part_floats(const spec_dims& d);
size_t prefix_pass_floats(const spec_dims& d);
bool prefix_tc_ok(const spec_dims& d);
int view_ranges_most(const spec_dims& d, int mode, int max_splits);
size_t prefix_tc_part_floats(const spec_dims& d);
cudaError_t prefix_tc_launch(const AttnArgs& a, float* part, uint32_t* status, cudaStream_t st,
                             PrefixPlan* plan);
cudaError_t prefix_launch(const AttnArgs& a, const WsLayout& lay, cudaStream_t st, PrefixPlan* plan,
                          int* launches);
cudaError_t prefix_merge_launch(const AttnArgs& a, const PrefixPlan& plan, const OwnPart& own,
                                cudaStream_t st, int* launches);
size_t attn_tc_part_floats(const spec_dims& d);
cudaError_t kv_append_launch(const AttnArgs& a, const WsLayout& lay, cudaStream_t st, int* launches);
cudaError_t attn_launch_simt(const AttnArgs& a, const WsLayout& lay, cudaStream_t st, int* launches);
cudaError_t attn_launch_tc(const AttnArgs& a, const WsLayout& lay, cudaStream_t st, int* launches);

}  // namespace specv
