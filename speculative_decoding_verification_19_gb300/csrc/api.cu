// C ABI of the verify step: argument checks, workspace layout and launches.
// Every check that the host can make happens here, before anything is
// enqueued; the kernels only check what lives in device memory.
#include <math.h>
#include <string.h>

#include "attn.cuh"
#include "block_tables.cuh"
#include "common.cuh"
#include "kv_commit.cuh"
#include "philox.cuh"
#include "lm_head.cuh"
#include "page_select.cuh"
#include "qk_norm_rope.cuh"
#include "reject_sample.cuh"
#include "sample.cuh"

namespace specv {

static thread_local int32_t g_launches = 0;

static size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

static int attn_split_keys(const spec_dims& d) {
  // Aim for about eight CTAs per SM over the whole batch (152 SMs), with
  // ranges of 256..4096 keys in whole 32-key tiles.
  const int64_t max_keys = (int64_t)d.max_blocks * kBlock;
  int64_t s = (int64_t)d.B * d.Hkv * max_keys / 1216;
  s = (s + 31) / 32 * 32;
  if (s < 256) s = 256;
  if (s > 4096) s = 4096;
  return (int)s;
}

// Whether every request reads a shared prefix itself (its pages come from L2 after
// the first), rather than one pass over it for the batch with a merge after it.
// A pass of its own with its merge costs some 20 to 30 us more than reading nothing,
// the requests' reads grow with their number.  The figures are a GB300's (152 SMs);
// elsewhere either way gives the same results.
// Measured, us, requests / one pass (B, Hkv, group, M, prefix):
//   tensor cores: the requests' reads cost 82 us for 10^6 keys (heads of 128), the pass
//   24 us and 0.8 for 10^9 operations of whole units of 256 rows.  38 / 62 (64, 1, 4, 1,
//   4096), 42 / 51 (16, 8, 8, 5, 2048), 45 / 49 (64, 8, 8, 1, 512), 62 / 70 (2, 8, 4, 1,
//   32768), 64 / 62 (64, 1, 4, 9, 8192), 64 / 66 (8, 8, 8, 9, 8192), 55 / 44 (16, 8, 4, 1,
//   4096), 60 / 51 (64, 8, 4, 1, 1024), 81 / 60 (4, 8, 4, 1, 24576), 121 / 144 (1, 8, 4, 1,
//   131072)
//   CUDA cores: the requests' reads cost 2.75 us for 10^6 elements of keys and 0.15 for
//   10^6 products, the pass 21 or 29 us (heads of 64, 128) and 0.09 for 10^6 products
//   of whole tiles of 64 rows.  fp32, heads of 64: 21 / 29 (8, 8, 1,
//   1, 512), 40 / 39 (8, 8, 1, 1, 2048), 41 / 50 (4, 8, 1, 1, 4096), 69 / 81 (2, 8, 1, 1,
//   16384), 79 / 39 (64, 8, 1, 1, 512), 112 / 44 (26, 8, 1, 1, 2208); heads of 128: 38 / 52
//   (16, 2, 4, 1, 2048), 41 / 61 (4, 8, 4, 1, 2048), 46 / 57 (8, 8, 4, 5, 512), 74 / 69 (16, 8,
//   4, 5, 512), 77 / 48 (16, 8, 1, 1, 1024), 112 / 89 (4, 8, 4, 1, 8192), 147 / 55 (64, 8, 1, 1,
//   512)
//   bf16 heads of 64, the pass on tensor cores and the rest on CUDA cores, by keys and
//   keys times rows: 17 / 19 (4, 8, 4, 1, 512), 20 / 20 (8, 8, 1, 1, 512), 25 / 30 (1, 2, 4, 1,
//   4096), 27 / 22 (16, 8, 1, 1, 512), 39 / 24 (8, 8, 1, 1, 2048), 42 / 33 (4, 1, 8, 8, 512)
static bool prefix_in_requests(const spec_dims& d, int64_t prefix_len, bool tc) {
  const int64_t keys = (int64_t)d.B * d.Hkv * prefix_len;
  const int64_t rows = (int64_t)(d.Hq / d.Hkv) * d.M;
  if (tc) {
    const double units = 256.0 * (double)ceil_div64(d.B * rows, 256) * d.Hkv * prefix_len;
    return d.B == 1 || 82e-6 * (double)keys <= 24.0 + 0.8e-9 * 4.0 * d.D * units;
  }
  if (d.attn_impl != SPEC_ATTN_CUDA_CORES && prefix_tc_ok(d))
    return keys <= 40000 && keys * rows <= 100000;
  const double tiles = 64.0 * (double)ceil_div64(d.B * rows, 64) * d.Hkv * prefix_len;
  const double requests = d.D * 1e-6 * (2.75 * (double)keys + 0.15 * (double)(keys * rows));
  const double pass = (d.D == 64 ? 21.0 : 29.0) + d.D * 1e-6 * 0.09 * tiles;
  return d.B == 1 || requests <= pass;
}

// The tensor-core attention takes the shape: bf16 heads of 128, up to 128 rows per KV
// head, tiles of all pairs counted in 32 bits.
static bool attn_tc_ok(const spec_dims& d) {
  return d.kv_dtype == SPEC_BF16 && d.D == 128 && (int64_t)(d.Hq / d.Hkv) * d.M <= 128 &&
         (int64_t)d.B * d.Hkv * ceil_div64((int64_t)d.max_blocks * kBlock, 64) <
             ((int64_t)1 << 31);
}

// Positions, and a request's (KV head, page) pairs, of views stay 32-bit; KV heads are
// a grid's second extent.
static bool view_counts_ok(const spec_dims& d) {
  return (int64_t)d.max_blocks * kBlock <= INT32_MAX / 2 && d.Hkv <= 65535 &&
         (int64_t)d.max_blocks * d.Hkv <= INT32_MAX / 2;
}
// Dims whose calls on views are not refused (the others have no room for them, and
// sizes of these do not overflow).
static bool view_dims_ok(const spec_dims& d) {
  return d.B <= 65535 && d.Hkv >= 1 && d.Hq >= d.Hkv && d.Hq % d.Hkv == 0 &&
         (int64_t)(d.Hq / d.Hkv) * d.M <= kMaxNodes && (d.D == 64 || d.D == 128) &&
         d.max_blocks >= 1 && view_counts_ok(d);
}

// Where a call on views of this mode keeps what it needs (tc: on tensor cores).  The
// partials' region of the calls without views is laid out for the most that either
// path may take, so the rest of it mostly has room for everything; what it has no
// room for goes behind all else (`behind`).
static ViewPlaces view_places(const spec_dims& d, const WsLayout& L, int mode, bool tc,
                              size_t behind) {
  ViewPlaces v = {};
  size_t free = L.attn_off, end = L.attn_off + L.attn_bytes;
  auto take = [&](size_t bytes) {
    size_t& from = free + bytes <= end ? free : behind;
    const size_t o = from;
    from = align_up(from + bytes, 256);
    return o;
  };
  const size_t pairs = (size_t)d.B * d.Hkv;
  if (tc) {
    v.part = take(sizeof(float) * attn_tc_part_floats(d));
  } else {
    v.ranges = view_ranges_most(d, mode, L.max_splits);
    v.part = take(sizeof(float) * pairs * v.ranges * L.rows * (d.D + 1));
    v.ctx = take(sizeof(int32_t) * (size_t)d.B);
  }
  if (mode == kViewPrefix) {
    if (tc) v.own = take(sizeof(float) * pairs * L.rows * tc_part_stride(d.D));
    v.pfx = take(sizeof(float) * prefix_pass_floats(d));
  } else {
    v.table = take(sizeof(int32_t) * pairs * d.max_blocks);
  }
  v.end = behind;
  return v;
}

// Bytes of the workspace with these dims' views.
static size_t view_total(const spec_dims& d, const WsLayout& L) {
  const bool tc = d.attn_impl != SPEC_ATTN_CUDA_CORES && attn_tc_ok(d);
  size_t most = view_places(d, L, kViewPages, tc, L.plain).end;
  // a pass over the prefix, unless even the longest one is read by the requests (the
  // rule turns to the pass as a prefix grows, and never back)
  if (!prefix_in_requests(d, ((int64_t)d.max_blocks - 1) * kBlock, tc)) {
    const size_t end = view_places(d, L, kViewPrefix, tc, L.plain).end;
    if (end > most) most = end;
  }
  return most;
}

WsLayout workspace_layout(const spec_dims& d) {
  WsLayout L;
  memset(&L, 0, sizeof(L));
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  // the status word, and the counters that have to be zero between calls of
  // any dims: their places do not depend on dims
  L.status_off = take(256);
  L.tc_sync_off = L.status_off + 64;
  L.pg_sync_off = L.status_off + 128;
  L.attn_ok_off = take(sizeof(int32_t) * (size_t)d.B);
  L.tc_ntiles_off = take(sizeof(int32_t) * (size_t)d.B);
  L.tc_pre_off = take(sizeof(int64_t) * 2 * ((size_t)d.B + 1));
  L.tc_rq_off = take(16 * (size_t)d.B);
  L.tc_start_off = take(32 * ((size_t)kMaxAttnCtas + 1));
  L.tc_pair_off = take(sizeof(int32_t) * (size_t)d.B * (size_t)(d.Hkv > 0 ? d.Hkv : 0));
  L.tc_anc_off = take(2 * sizeof(uint64_t) * (size_t)d.B * d.M);
  L.win_depth_off = take(sizeof(int32_t) * (size_t)d.B * d.M);
  const int group = d.Hkv > 0 ? d.Hq / d.Hkv : 0;
  L.rows = group * d.M;
  L.split_keys = attn_split_keys(d);
  L.max_splits = (int)ceil_div64((int64_t)d.max_blocks * kBlock, L.split_keys);
  L.attn_bytes = sizeof(float) * (size_t)d.B * d.Hkv * L.max_splits * L.rows * (d.D + 1);
  const size_t tc_bytes = d.Hkv > 0 ? sizeof(float) * attn_tc_part_floats(d) : 0;
  if (tc_bytes > L.attn_bytes) L.attn_bytes = tc_bytes;
  L.attn_off = take(L.attn_bytes);
  L.rs_chunk = rs_chunk_elems(d.logits_dtype);
  L.rs_chunks = (int)ceil_div64(d.V, L.rs_chunk);
  L.rs_bytes = sizeof(RowStat) * (size_t)d.B * 2 * d.M * L.rs_chunks;
  L.rs_off = take(L.rs_bytes);
  L.rs_draw_off = take(sizeof(DrawState) * (size_t)d.B);
  L.rs_zsum_off = take(sizeof(double) * (size_t)d.B * L.rs_chunks);
  L.rs_filt_off = take(sizeof(FilterInfo) * (size_t)d.B * 2 * d.M);
  // the chain tail: per request, slices finished, then residual chunks
  // claimed; then the statistics stream's pool counters (claimed, warps done)
  L.rs_tail_off = take(sizeof(uint32_t) * (2 * (size_t)d.B + 2));
  // the LM heads' split statistics (rows B * M, bf16 logits)
  const int64_t lm_units = (int64_t)ceil_div64((int64_t)d.B * d.M, 128) * L.rs_chunks;
  if (d.logits_dtype == SPEC_BF16 && lm_units <= kLmSplitMaxUnits) {
    L.lm_units = lm_units;
    L.lm_part_off = take(sizeof(RowStat) * 2 * (size_t)lm_units * kLmMaxPieces * 128);
    L.lm_cnt_off = take(sizeof(uint32_t) * 2 * (size_t)lm_units * 4);
  }
  off = rsf_layout(d, off, &L);
  L.plain = L.total = off;
  if (view_dims_ok(d)) L.total = view_total(d, L);
  return L;
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

spec_status check_common(const spec_dims* d) {
  if (d == nullptr) return SPEC_ERR_INVALID_ARG;
  if (d->B < 1 || d->M < 1) return SPEC_ERR_INVALID_ARG;
  if (d->M > kMaxNodes) return SPEC_ERR_UNSUPPORTED;
  if (d->block != kBlock) return SPEC_ERR_UNSUPPORTED;
  if ((d->kv_dtype != SPEC_BF16 && d->kv_dtype != SPEC_F32) ||
      (d->logits_dtype != SPEC_BF16 && d->logits_dtype != SPEC_F32))
    return SPEC_ERR_INVALID_ARG;
  if (d->wait_limit_kcycles < 0) return SPEC_ERR_INVALID_ARG;
  if (d->reject_impl < SPEC_REJECT_AUTO || d->reject_impl > SPEC_REJECT_FUSED)
    return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}

static spec_status check_kv(const spec_dims* d) {
  if (d->B > 65535) return SPEC_ERR_UNSUPPORTED;  // grid y/z limit of the attention launch
  if (d->Hq < 1 || d->Hkv < 1 || d->Hq % d->Hkv != 0) return SPEC_ERR_INVALID_ARG;
  if (d->D != 64 && d->D != 128) return SPEC_ERR_UNSUPPORTED;
  if (d->max_blocks < 1 || d->num_blocks < 1) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}

static spec_status check_ws(const spec_dims* d, void* ws, size_t ws_bytes) {
  if (ws == nullptr || !aligned16(ws)) return SPEC_ERR_INVALID_ARG;
  if (ws_bytes < workspace_layout(*d).plain) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}

static spec_status from_cuda(cudaError_t e) { return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA; }

}  // namespace specv

using namespace specv;

extern "C" {

size_t spec_workspace_size(const spec_dims* dims) {
  if (check_common(dims) != SPEC_OK) return 0;
  return workspace_layout(*dims).total;
}

spec_status spec_workspace_init(void* ws, size_t ws_bytes, void* stream) {
  if (ws == nullptr || ws_bytes == 0) return SPEC_ERR_INVALID_ARG;
  return from_cuda(cudaMemsetAsync(ws, 0, ws_bytes, static_cast<cudaStream_t>(stream)));
}

spec_status spec_get_device_status(void* ws, void* stream, int32_t* flags, int32_t clear) {
  if (ws == nullptr || flags == nullptr) return SPEC_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, ws, sizeof(v), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return SPEC_ERR_CUDA;
  *flags = (int32_t)v;
  if (clear) {
    e = cudaMemsetAsync(ws, 0, sizeof(uint32_t), st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return SPEC_ERR_CUDA;
  }
  return SPEC_OK;
}

static spec_status attn_common(const void* q, const void* k_new, const void* v_new, void* k_cache,
                               void* v_cache, const int32_t* block_table, const int32_t* ctx_lens,
                               const int32_t* parent, int32_t window, int32_t sinks,
                               AttnView view, void* out, float* lse, const spec_dims* dims,
                               void* ws, size_t ws_bytes, void* stream) {
  g_launches = 0;
  spec_status s = check_common(dims);
  if (s != SPEC_OK) return s;
  if ((s = check_kv(dims)) != SPEC_OK) return s;
  if ((s = check_ws(dims, ws, ws_bytes)) != SPEC_OK) return s;
  if (!q || !k_new || !v_new || !k_cache || !v_cache || !block_table || !ctx_lens || !out)
    return SPEC_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) ||
      !aligned16(v_cache) || !aligned16(out))
    return SPEC_ERR_INVALID_ARG;
  const int64_t R = (int64_t)(dims->Hq / dims->Hkv) * dims->M;
  // kernel choice: the tensor-core kernel whenever it supports the shape
  // (bf16, D = 128, up to 128 rows per KV head): even a few rows per KV head
  // run faster there than on CUDA cores; CUDA cores otherwise
  const bool tc_ok = attn_tc_ok(*dims);
  const bool simt_ok = R <= 128;
  bool use_tc;
  if (dims->attn_impl == SPEC_ATTN_TENSOR_CORES) {
    if (!tc_ok) return SPEC_ERR_UNSUPPORTED;
    use_tc = true;
  } else if (dims->attn_impl == SPEC_ATTN_CUDA_CORES) {
    if (!simt_ok) return SPEC_ERR_UNSUPPORTED;
    use_tc = false;
  } else if (dims->attn_impl == SPEC_ATTN_AUTO) {
    use_tc = tc_ok;
    if (!use_tc && !simt_ok) return SPEC_ERR_UNSUPPORTED;
  } else {
    return SPEC_ERR_INVALID_ARG;
  }
  const WsLayout lay = workspace_layout(*dims);
  if (view.mode != kViewNone && !view_dims_ok(*dims)) return SPEC_ERR_UNSUPPORTED;
  if (view.mode != kViewNone && ws_bytes < lay.total) return SPEC_ERR_INVALID_ARG;
  // (a pass that the workspace has no room for, were the rule to ask for one where
  // view_total expects none, is not run)
  if (view.mode == kViewPrefix &&
      (prefix_in_requests(*dims, view.prefix_len, use_tc) ||
       view_places(*dims, lay, kViewPrefix, use_tc, lay.plain).end > lay.total))
    view.mode = kViewWhole;
  AttnArgs a;
  a.q = q;
  a.k_new = k_new;
  a.v_new = v_new;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_table = block_table;
  a.ctx_lens = ctx_lens;
  a.parent = parent;
  a.out = out;
  a.lse = lse;
  a.d = *dims;
  a.scale = dims->softmax_scale != 0.f ? dims->softmax_scale : 1.0f / sqrtf((float)dims->D);
  a.window = window;
  a.sinks = sinks;
  a.view = view;
  a.ws = ws;
  if (view.mode != kViewNone) {
    char* w = static_cast<char*>(ws);
    a.at = view_places(*dims, lay, view.mode, use_tc, lay.plain);
    a.view.ctx = reinterpret_cast<int32_t*>(w + a.at.ctx);
    if (view.mode == kViewPrefix) {
      const int pp = view.prefix_len / kBlock;
      a.view.table = block_table + pp;
      a.view.stride_b = dims->max_blocks;
      a.view.stride_h = 0;
      a.view.entries = dims->max_blocks - pp;
    } else if (view.mode == kViewWhole) {
      a.view.table = reinterpret_cast<int32_t*>(w + a.at.table);
      a.view.stride_b = dims->max_blocks;
      a.view.stride_h = 0;
      a.view.entries = dims->max_blocks;
    } else {
      // the selected pages, then those of the context's last partial page and
      // the new rows; together no more than the context and the new rows have
      const int64_t most = (int64_t)view.n_pages + ceil_div(kBlock - 1 + dims->M, kBlock);
      a.view.entries = most < dims->max_blocks ? (int)most : dims->max_blocks;
      a.view.table = reinterpret_cast<int32_t*>(w + a.at.table);
      a.view.stride_h = a.view.entries;
      a.view.stride_b = (int64_t)dims->Hkv * a.view.entries;
    }
  }
  int launches = 0;
  const cudaError_t e = use_tc ? attn_launch_tc(a, lay, static_cast<cudaStream_t>(stream), &launches)
                               : attn_launch_simt(a, lay, static_cast<cudaStream_t>(stream), &launches);
  g_launches = launches;
  return from_cuda(e);
}

spec_status spec_verify_attn(const void* q, const void* k_new, const void* v_new, void* k_cache,
                             void* v_cache, const int32_t* block_table, const int32_t* ctx_lens,
                             const int32_t* parent, void* out, float* lse, const spec_dims* dims,
                             void* ws, size_t ws_bytes, void* stream) {
  return attn_common(q, k_new, v_new, k_cache, v_cache, block_table, ctx_lens, parent, 0, 0,
                     AttnView{}, out, lse, dims, ws, ws_bytes, stream);
}

spec_status spec_verify_attn_window(const void* q, const void* k_new, const void* v_new,
                                    void* k_cache, void* v_cache, const int32_t* block_table,
                                    const int32_t* ctx_lens, const int32_t* parent, int32_t window,
                                    int32_t sinks, void* out, float* lse, const spec_dims* dims,
                                    void* ws, size_t ws_bytes, void* stream) {
  g_launches = 0;
  if (dims == nullptr || window < 1 || sinks < 0) return SPEC_ERR_INVALID_ARG;
  // positions stay below 2^31; a window or sinks past the table's last
  // position mean all of it
  const int64_t cap = (int64_t)dims->max_blocks * kBlock;
  if (cap > INT32_MAX / 2) return SPEC_ERR_UNSUPPORTED;
  const int32_t most = cap > 0 ? (int32_t)cap : 1;
  return attn_common(q, k_new, v_new, k_cache, v_cache, block_table, ctx_lens, parent,
                     window < most ? window : most, sinks < most ? sinks : most, AttnView{}, out,
                     lse, dims, ws, ws_bytes, stream);
}

// What the forms of the attention on views ask of dims beyond attn_common.
static spec_status check_view(const spec_dims* d) {
  if (d == nullptr) return SPEC_ERR_INVALID_ARG;
  if (!(d->softmax_scale >= 0.f) || !(d->softmax_scale < INFINITY)) return SPEC_ERR_INVALID_ARG;
  return view_counts_ok(*d) ? SPEC_OK : SPEC_ERR_UNSUPPORTED;
}

spec_status spec_verify_attn_prefix(const void* q, const void* k_new, const void* v_new,
                                    void* k_cache, void* v_cache, const int32_t* block_table,
                                    const int32_t* ctx_lens, const int32_t* parent,
                                    const int32_t* prefix_table, int32_t prefix_len, void* out,
                                    float* lse, const spec_dims* dims, void* ws, size_t ws_bytes,
                                    void* stream) {
  g_launches = 0;
  const spec_status s = check_view(dims);
  if (s != SPEC_OK) return s;
  if (!prefix_table || prefix_len < kBlock || prefix_len % kBlock != 0 ||
      prefix_len >= (int64_t)dims->max_blocks * kBlock)
    return SPEC_ERR_INVALID_ARG;
  AttnView v = {};
  v.mode = kViewPrefix;
  v.prefix_table = prefix_table;
  v.prefix_len = prefix_len;
  return attn_common(q, k_new, v_new, k_cache, v_cache, block_table, ctx_lens, parent, 0, 0, v, out,
                     lse, dims, ws, ws_bytes, stream);
}

spec_status spec_verify_attn_pages(const void* q, const void* k_new, const void* v_new,
                                   void* k_cache, void* v_cache, const int32_t* block_table,
                                   const int32_t* ctx_lens, const int32_t* parent,
                                   const int32_t* pages, const int32_t* counts, int32_t n_pages,
                                   void* out, float* lse, const spec_dims* dims, void* ws,
                                   size_t ws_bytes, void* stream) {
  g_launches = 0;
  const spec_status s = check_view(dims);
  if (s != SPEC_OK) return s;
  if (!pages || !counts || n_pages < 1) return SPEC_ERR_INVALID_ARG;
  if (n_pages > kSelectMostPages) return SPEC_ERR_UNSUPPORTED;
  AttnView v = {};
  v.mode = kViewPages;
  v.pages = pages;
  v.counts = counts;
  v.n_pages = n_pages;
  return attn_common(q, k_new, v_new, k_cache, v_cache, block_table, ctx_lens, parent, 0, 0, v, out,
                     lse, dims, ws, ws_bytes, stream);
}

// Checks that the calls on pages' bounds and scores share; of the workspace
// they use the status word alone.
static spec_status check_pages(const spec_dims* d, void* ws, size_t ws_bytes) {
  spec_status s = check_common(d);
  if (s != SPEC_OK) return s;
  if ((s = check_kv(d)) != SPEC_OK) return s;
  if ((int64_t)d->max_blocks * kBlock > INT32_MAX / 2 || d->Hkv > 65535) return SPEC_ERR_UNSUPPORTED;
  if (ws == nullptr || ws_bytes < 16 || !aligned16(ws)) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}

spec_status spec_page_bounds(const void* k_cache, const int32_t* block_table,
                             const int32_t* from_lens, const int32_t* ctx_lens, void* bounds,
                             const spec_dims* dims, void* ws, size_t ws_bytes, void* stream) {
  g_launches = 0;
  const spec_status s = check_pages(dims, ws, ws_bytes);
  if (s != SPEC_OK) return s;
  if (!k_cache || !block_table || !ctx_lens || !bounds) return SPEC_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(bounds)) return SPEC_ERR_INVALID_ARG;
  const BoundsArgs a = {k_cache, block_table, from_lens, ctx_lens, bounds, *dims,
                        static_cast<uint32_t*>(ws)};
  int launches = 0;
  const cudaError_t e = page_bounds_launch(a, static_cast<cudaStream_t>(stream), &launches);
  g_launches = launches;
  return from_cuda(e);
}

spec_status spec_page_score(const void* q, const void* bounds, const int32_t* block_table,
                            const int32_t* ctx_lens, float* scores, const spec_dims* dims, void* ws,
                            size_t ws_bytes, void* stream) {
  g_launches = 0;
  const spec_status s = check_pages(dims, ws, ws_bytes);
  if (s != SPEC_OK) return s;
  if (!q || !bounds || !block_table || !ctx_lens || !scores) return SPEC_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(bounds)) return SPEC_ERR_INVALID_ARG;
  const ScoreArgs a = {q, bounds, block_table, ctx_lens, scores, *dims, static_cast<uint32_t*>(ws)};
  int launches = 0;
  const cudaError_t e = page_score_launch(a, static_cast<cudaStream_t>(stream), &launches);
  g_launches = launches;
  return from_cuda(e);
}

spec_status spec_page_select(const float* scores, const int32_t* ctx_lens, int32_t n_pages,
                             int32_t first, int32_t last, int32_t* pages, int32_t* counts,
                             const spec_dims* dims, void* ws, size_t ws_bytes, void* stream) {
  g_launches = 0;
  const spec_status s = check_pages(dims, ws, ws_bytes);
  if (s != SPEC_OK) return s;
  if (!scores || !ctx_lens || !pages || !counts) return SPEC_ERR_INVALID_ARG;
  if (n_pages < 1 || first < 0 || last < 0 || (int64_t)first + last > n_pages)
    return SPEC_ERR_INVALID_ARG;
  if (n_pages > kSelectMostPages) return SPEC_ERR_UNSUPPORTED;
  const SelectArgs a = {scores, ctx_lens, n_pages, first, last, pages, counts, *dims,
                        static_cast<uint32_t*>(ws)};
  int launches = 0;
  const cudaError_t e = page_select_launch(a, static_cast<cudaStream_t>(stream), &launches);
  g_launches = launches;
  return from_cuda(e);
}

static spec_status reject_common(const void* target_logits, const void* draft_logits,
                                 const int32_t* tokens, const int32_t* parent,
                                 const float* temperature, const int32_t* top_k,
                                 const float* top_p, uint64_t seed, uint64_t offset,
                                 uint64_t b_base, int32_t* out_tokens, int32_t* path,
                                 int32_t* accepted_len, float* probe, const spec_dims* dims,
                                 void* ws, size_t ws_bytes, void* stream) {
  g_launches = 0;
  spec_status s = check_common(dims);
  if (s != SPEC_OK) return s;
  if ((s = check_ws(dims, ws, ws_bytes)) != SPEC_OK) return s;
  if (dims->V < 1) return SPEC_ERR_INVALID_ARG;
  if (dims->V > rs_max_vocab(dims->logits_dtype)) return SPEC_ERR_UNSUPPORTED;
  {
    const WsLayout l = workspace_layout(*dims);
    if ((int64_t)l.rs_chunks * 2 * dims->M * dims->B >= (int64_t)1 << 31) return SPEC_ERR_UNSUPPORTED;
  }
  if (!target_logits || !draft_logits || !tokens || !temperature || !out_tokens || !path ||
      !accepted_len)
    return SPEC_ERR_INVALID_ARG;
  if ((top_k != nullptr || top_p != nullptr) && dims->reject_impl == SPEC_REJECT_FUSED)
    return SPEC_ERR_UNSUPPORTED;  // the one-kernel path has no filters
  const WsLayout lay = workspace_layout(*dims);
  RsArgs a;
  a.target = target_logits;
  a.draft = draft_logits;
  a.tokens = tokens;
  a.parent = parent;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.seed = seed;
  a.offset = offset;
  a.b_base = b_base;
  a.out_tokens = out_tokens;
  a.path = path;
  a.accepted_len = accepted_len;
  a.probe = probe;
  a.d = *dims;
  a.ws = ws;
  int launches = 0;
  const cudaError_t e = rs_launch(a, lay, static_cast<cudaStream_t>(stream), &launches);
  g_launches = launches;
  if (e == cudaErrorNotSupported) return SPEC_ERR_UNSUPPORTED;
  return from_cuda(e);
}

spec_status spec_reject_sample(const void* target_logits, const void* draft_logits,
                               const int32_t* tokens, const int32_t* parent,
                               const float* temperature, uint64_t seed, uint64_t offset,
                               uint64_t b_base, int32_t* out_tokens, int32_t* path,
                               int32_t* accepted_len, float* probe, const spec_dims* dims,
                               void* ws, size_t ws_bytes, void* stream) {
  return reject_common(target_logits, draft_logits, tokens, parent, temperature, nullptr,
                       nullptr, seed, offset, b_base, out_tokens, path, accepted_len, probe, dims,
                       ws, ws_bytes, stream);
}

spec_status spec_reject_sample_filtered(const void* target_logits, const void* draft_logits,
                                        const int32_t* tokens, const int32_t* parent,
                                        const float* temperature, const int32_t* top_k,
                                        const float* top_p, uint64_t seed, uint64_t offset,
                                        uint64_t b_base, int32_t* out_tokens, int32_t* path,
                                        int32_t* accepted_len, float* probe,
                                        const spec_dims* dims, void* ws, size_t ws_bytes,
                                        void* stream) {
  return reject_common(target_logits, draft_logits, tokens, parent, temperature, top_k, top_p,
                       seed, offset, b_base, out_tokens, path, accepted_len, probe, dims, ws,
                       ws_bytes, stream);
}

spec_status spec_lm_head(const void* hidden, const void* weight, int32_t rows, int32_t H,
                         int32_t V, void* logits, void* ws, size_t ws_bytes, void* stream) {
  g_launches = 0;
  if (!hidden || !weight || !logits || ws == nullptr || ws_bytes < 16 || !aligned16(ws))
    return SPEC_ERR_INVALID_ARG;
  if (rows < 1 || H < 1 || V < 1) return SPEC_ERR_INVALID_ARG;
  if (!lm_head_supported(rows, H, V)) return SPEC_ERR_UNSUPPORTED;
  if (!aligned16(hidden) || !aligned16(weight) || !aligned16(logits)) return SPEC_ERR_INVALID_ARG;
  spec_dims d;
  memset(&d, 0, sizeof(d));  // the default wait limit
  int launches = 0;
  const cudaError_t e =
      lm_head_launch(hidden, weight, rows, H, V, logits, nullptr, 0, 1, 0, nullptr, d,
                     static_cast<uint32_t*>(ws), nullptr, nullptr,
                     static_cast<cudaStream_t>(stream), &launches);
  g_launches = launches;
  return e == cudaErrorInvalidValue ? SPEC_ERR_UNSUPPORTED : from_cuda(e);
}

spec_status spec_reject_sample_lm_head(const void* hidden_target, const void* weight_target,
                                       int32_t Ht, const void* hidden_draft,
                                       const void* weight_draft, int32_t Hd, void* target_logits,
                                       void* draft_logits, const int32_t* tokens,
                                       const int32_t* parent, const float* temperature,
                                       uint64_t seed, uint64_t offset, uint64_t b_base,
                                       int32_t* out_tokens, int32_t* path, int32_t* accepted_len,
                                       float* probe, const spec_dims* dims, void* ws,
                                       size_t ws_bytes, void* stream) {
  g_launches = 0;
  spec_status s = check_common(dims);
  if (s != SPEC_OK) return s;
  if ((s = check_ws(dims, ws, ws_bytes)) != SPEC_OK) return s;
  if (!hidden_target || !weight_target || !hidden_draft || !weight_draft || !target_logits ||
      !draft_logits || !tokens || !temperature || !out_tokens || !path || !accepted_len)
    return SPEC_ERR_INVALID_ARG;
  if (dims->logits_dtype != SPEC_BF16) return SPEC_ERR_UNSUPPORTED;
  if (dims->reject_impl == SPEC_REJECT_FUSED) return SPEC_ERR_UNSUPPORTED;
  const int R = dims->B * dims->M;
  if ((int64_t)dims->B * dims->M >= ((int64_t)1 << 31) / 2) return SPEC_ERR_UNSUPPORTED;
  if (!lm_head_supported(R, Ht, dims->V) || !lm_head_supported(R, Hd, dims->V))
    return SPEC_ERR_UNSUPPORTED;
  if (!aligned16(hidden_target) || !aligned16(weight_target) || !aligned16(hidden_draft) ||
      !aligned16(weight_draft) || !aligned16(target_logits) || !aligned16(draft_logits))
    return SPEC_ERR_INVALID_ARG;
  const WsLayout lay = workspace_layout(*dims);
  if ((int64_t)lay.rs_chunks * 2 * dims->M * dims->B >= (int64_t)1 << 31) return SPEC_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(ws);
  RowStat* stats = reinterpret_cast<RowStat*>(w + lay.rs_off);
  uint32_t* status = reinterpret_cast<uint32_t*>(w + lay.status_off);
  int launches = 0;
  // the split statistics' workspace, when laid out for these rows
  const bool split = lay.lm_units > 0 && lay.lm_units == lm_head_units(R, dims->V);
  RowStat* part = split ? reinterpret_cast<RowStat*>(w + lay.lm_part_off) : nullptr;
  uint32_t* cnt = split ? reinterpret_cast<uint32_t*>(w + lay.lm_cnt_off) : nullptr;
  cudaError_t e = lm_head_launch(hidden_target, weight_target, R, Ht, dims->V, target_logits,
                                 stats, 0, dims->M, lay.rs_chunks, temperature, *dims, status,
                                 part, cnt, st, &launches);
  if (e == cudaSuccess)
    e = lm_head_launch(hidden_draft, weight_draft, R, Hd, dims->V, draft_logits, stats, 1,
                       dims->M, lay.rs_chunks, temperature, *dims, status, part, cnt, st,
                       &launches);
  if (e != cudaSuccess) {
    g_launches = launches;
    return e == cudaErrorInvalidValue ? SPEC_ERR_UNSUPPORTED : SPEC_ERR_CUDA;
  }
  RsArgs a;
  a.target = target_logits;
  a.draft = draft_logits;
  a.tokens = tokens;
  a.parent = parent;
  a.temperature = temperature;
  a.top_k = nullptr;
  a.top_p = nullptr;
  a.seed = seed;
  a.offset = offset;
  a.b_base = b_base;
  a.out_tokens = out_tokens;
  a.path = path;
  a.accepted_len = accepted_len;
  a.probe = probe;
  a.d = *dims;
  a.d.reject_impl = SPEC_REJECT_STAGED;
  a.ws = ws;
  a.stats_ready = true;
  e = rs_launch(a, lay, st, &launches);
  g_launches = launches;
  return from_cuda(e);
}

spec_status kv_commit(void* k_cache, void* v_cache, const int32_t* block_table,
                      const int32_t* ctx_lens, int32_t* new_ctx_lens, const int32_t* path,
                      const int32_t* accepted_len, const spec_dims* dims, void* ws,
                      size_t ws_bytes, void* stream) {
  g_launches = 0;
  spec_status s = check_common(dims);
  if (s != SPEC_OK) return s;
  if ((s = check_kv(dims)) != SPEC_OK) return s;
  if ((s = check_ws(dims, ws, ws_bytes)) != SPEC_OK) return s;
  if (!k_cache || !v_cache || !block_table || !ctx_lens || !new_ctx_lens || !path || !accepted_len)
    return SPEC_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return SPEC_ERR_INVALID_ARG;
  const WsLayout lay = workspace_layout(*dims);
  CommitArgs a;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_table = block_table;
  a.ctx_lens = ctx_lens;
  a.new_ctx_lens = new_ctx_lens;
  a.path = path;
  a.accepted_len = accepted_len;
  a.d = *dims;
  a.ws = ws;
  int launches = 0;
  const cudaError_t e = commit_launch(a, lay, static_cast<cudaStream_t>(stream), &launches);
  g_launches = launches;
  return from_cuda(e);
}

spec_status spec_block_tables(const int32_t* ctx_lens, const int32_t* row_start,
                              const int32_t* parent, int32_t rows, int32_t window, int32_t sinks,
                              int32_t* block_table, int32_t* span, int32_t* pool,
                              int32_t* pool_state, int64_t* slots, int32_t* positions, int32_t* ok,
                              const spec_dims* dims, void* ws, size_t ws_bytes, void* stream) {
  g_launches = 0;
  spec_status s = check_common(dims);
  if (s != SPEC_OK) return s;
  if (dims->B > 65535) return SPEC_ERR_UNSUPPORTED;
  if (dims->max_blocks < 1 || dims->num_blocks < 1) return SPEC_ERR_INVALID_ARG;
  if ((int64_t)dims->max_blocks * kBlock > INT32_MAX) return SPEC_ERR_UNSUPPORTED;
  // counts of rows and pages, and a grid's stride past them, stay 32-bit
  if (rows > kPagesMaxItems || (int64_t)dims->B * dims->max_blocks > kPagesMaxItems)
    return SPEC_ERR_UNSUPPORTED;
  if ((s = check_ws(dims, ws, ws_bytes)) != SPEC_OK) return s;
  if (!ctx_lens || !block_table || !span || !pool || !pool_state) return SPEC_ERR_INVALID_ARG;
  if (rows > 0 && (!slots || !positions)) return SPEC_ERR_INVALID_ARG;
  if (rows < 0 || window < 0 || sinks < 0) return SPEC_ERR_INVALID_ARG;
  if (row_start != nullptr ? parent != nullptr : (int64_t)dims->B * dims->M > rows)
    return SPEC_ERR_INVALID_ARG;
  const int cap = dims->max_blocks * kBlock;
  PageArgs a;
  a.ctx_lens = ctx_lens;
  a.row_start = row_start;
  a.parent = parent;
  a.rows = rows;
  a.window = window;
  a.sinks = sinks < cap ? sinks : cap;
  a.block_table = block_table;
  a.span = span;
  a.pool = pool;
  a.pool_state = pool_state;
  a.slots = slots;
  a.positions = positions;
  a.ok = ok;
  a.d = *dims;
  a.ws = ws;
  int launches = 0;
  const cudaError_t e = block_tables_launch(a, workspace_layout(*dims),
                                            static_cast<cudaStream_t>(stream), &launches);
  g_launches = launches;
  return from_cuda(e);
}

spec_status spec_qk_norm_rope(const void* q, const void* k, const void* v, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, const void* q_weight,
                              const void* k_weight, float eps, const int32_t* positions,
                              const double* inv_freq, int32_t rot_dim, int32_t interleaved,
                              int32_t rows, void* q_out, void* k_out, const int64_t* slots,
                              void* k_cache, void* v_cache, const spec_dims* dims, void* ws,
                              size_t ws_bytes, void* stream) {
  g_launches = 0;
  spec_status s = check_common(dims);
  if (s != SPEC_OK) return s;
  if ((s = check_kv(dims)) != SPEC_OK) return s;
  if ((s = check_ws(dims, ws, ws_bytes)) != SPEC_OK) return s;
  if (rows < 0 || !(eps >= 0.f) || !(eps < INFINITY)) return SPEC_ERR_INVALID_ARG;
  if (rows == 0) return SPEC_OK;
  if (!q || !k || !positions || !q_out) return SPEC_ERR_INVALID_ARG;
  if (slots != nullptr ? (!v || !k_cache || !v_cache) : !k_out) return SPEC_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim > dims->D || (rot_dim > 0 && !inv_freq)) return SPEC_ERR_INVALID_ARG;
  if (rot_dim % 16 != 0) return SPEC_ERR_UNSUPPORTED;
  const int vec = dims->kv_dtype == SPEC_BF16 ? 8 : 4;
  const int64_t q_row = (int64_t)dims->Hq * dims->D, k_row = (int64_t)dims->Hkv * dims->D;
  if (q_stride < q_row || k_stride < k_row || (slots != nullptr && v_stride < k_row))
    return SPEC_ERR_INVALID_ARG;
  if (q_stride % vec != 0 || k_stride % vec != 0 || (slots != nullptr && v_stride % vec != 0))
    return SPEC_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_out) ||
      !aligned16(k_cache) || !aligned16(v_cache))
    return SPEC_ERR_INVALID_ARG;
  RopeArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.rot_dim = rot_dim;
  a.interleaved = interleaved;
  a.rows = rows;
  a.q_out = q_out;
  a.k_out = k_out;
  a.slots = slots;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.d = *dims;
  a.ws = ws;
  int launches = 0;
  const cudaError_t e = qk_norm_rope_launch(a, workspace_layout(*dims),
                                            static_cast<cudaStream_t>(stream), &launches);
  g_launches = launches;
  return from_cuda(e);
}

spec_status spec_sample(const void* logits, int64_t row_stride, int32_t rows, int32_t V,
                        int32_t logits_dtype, const float* temperature, const int32_t* top_k,
                        const float* top_p, const float* min_p, const float* uniform,
                        int32_t* out_tokens, float* out_prob, void* ws, size_t ws_bytes,
                        void* stream) {
  g_launches = 0;
  if (ws == nullptr || ws_bytes < 16 || !aligned16(ws)) return SPEC_ERR_INVALID_ARG;
  if (logits_dtype != SPEC_BF16 && logits_dtype != SPEC_F32) return SPEC_ERR_INVALID_ARG;
  if (rows < 0 || V < 1 || row_stride < V) return SPEC_ERR_INVALID_ARG;
  if (V > kSampleMaxVocab || rows > (1 << 27)) return SPEC_ERR_UNSUPPORTED;
  if (rows == 0) return SPEC_OK;
  if (!logits || !temperature || !uniform || !out_tokens) return SPEC_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % (logits_dtype == SPEC_BF16 ? 2 : 4) != 0)
    return SPEC_ERR_INVALID_ARG;
  SampleArgs a;
  a.logits = logits;
  a.stride = row_stride;
  a.rows = rows;
  a.V = V;
  a.dtype = logits_dtype;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.uniform = uniform;
  a.out_tokens = out_tokens;
  a.out_prob = out_prob;
  a.status = static_cast<uint32_t*>(ws);
  int launches = 0;
  const cudaError_t e = sample_launch(a, static_cast<cudaStream_t>(stream), &launches);
  g_launches = launches;
  return from_cuda(e);
}

void spec_philox_block(const uint64_t key[2], const uint64_t counter[4], uint64_t out[4]) {
  const Philox4 r = philox4x64_10(counter[0], counter[1], counter[2], counter[3], key[0], key[1]);
  for (int i = 0; i < 4; ++i) out[i] = r.w[i];
}

const char* spec_status_string(int32_t status) {
  switch (status) {
    case SPEC_OK: return "SPEC_OK";
    case SPEC_ERR_INVALID_ARG: return "SPEC_ERR_INVALID_ARG";
    case SPEC_ERR_CAPACITY: return "SPEC_ERR_CAPACITY";
    case SPEC_ERR_UNSUPPORTED: return "SPEC_ERR_UNSUPPORTED";
    case SPEC_ERR_CUDA: return "SPEC_ERR_CUDA";
    case SPEC_ERR_NONFINITE: return "SPEC_ERR_NONFINITE";
    case SPEC_ERR_DEVICE_BOUNDS: return "SPEC_ERR_DEVICE_BOUNDS";
    case SPEC_ERR_TIMEOUT: return "SPEC_ERR_TIMEOUT";
    default: return "SPEC_ERR_UNKNOWN";
  }
}

int32_t spec_last_launch_count(void) { return g_launches; }

}  // extern "C"
