// KV append and verify attention over a paged KV cache.
//
// What is computed (page 1 §2.1, page 2 §3.3, page 3 tree-attention
// section): the M new rows of each request (pending root + drafts, or tree
// nodes) have their K/V appended at positions ctx..ctx+M-1; row i then
// attends to the cached prefix 0..ctx-1 and to the new positions of its
// ancestors and itself, which makes the one-pass result equal to
// token-by-token decoding.
//
// Kernels in this file (CUDA cores; the tensor-core path lives in
// attn_tc.cu):
//   kv_append_kernel   up to eight CTAs per request: each checks the request
//                      (capacity, block ids, topology) and writes its share of
//                      the new K/V and the cleared rest of the last block; the
//                      first records the verdict.
//   attn_split_kernel  split-KV attention: one CTA per (request, KV head,
//                      key range); all group*M query rows that read the KV
//                      head are handled together, so every K/V byte is read
//                      once per range.  Online softmax in base 2.
//   attn_win_split_kernel  the same over a sliding window and sinks.
//   attn_combine_kernel  merges the per-range partials by log-sum-exp, a warp
//                      per row.
#include <math.h>

#include "attn.cuh"
#include "common.cuh"

namespace specv {

// ---------------------------------------------------------------------------
// append + per-request verdict
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256) kv_append_kernel(
    const T* k_new, const T* v_new, T* k_cache, T* v_cache, const int32_t* block_table,
    const int32_t* ctx_lens, const int32_t* parent, spec_dims d, int window, int sinks,
    ulonglong2* anc_ws, int32_t* depth_ws, int32_t* __restrict__ req_ok,
    uint32_t* __restrict__ status) {
  pdl_trigger();
  pdl_wait();  // the inputs and the cache may come from the previous kernel
  const int b = blockIdx.x;
  const int tid = threadIdx.x;
  const int ctx = ctx_lens[b];
  const int64_t L = (int64_t)ctx + d.M;
  const int64_t cap = (int64_t)d.max_blocks * kBlock;
  const int32_t* bt = block_table + (int64_t)b * d.max_blocks;

  // capacity
  const bool cap_ok = ctx >= 0 && L <= cap;
  // block ids of every page the request reads or writes (with a window, not
  // of the pages between the sinks and it)
  int bad_block = 0;
  if (cap_ok) {
    const int pages = (int)ceil_div64(L, kBlock);
    for (int p = tid; p < pages; p += blockDim.x) {
      const int id = bt[p];
      bad_block |= (id < 0 || id >= d.num_blocks) &&
                   (window <= 0 || win_page(p, ctx, window, sinks));
    }
  }
  // topology
  __shared__ int32_t s_par[kMaxNodes];  // for the walks to the root below
  int bad_topo = 0;
  if (parent != nullptr) {
    const int32_t* par = parent + (int64_t)b * d.M;
    for (int n = tid; n < d.M; n += blockDim.x) {
      const int pn = par[n];
      s_par[n] = pn;
      bad_topo |= (n == 0) ? (pn != -1) : (pn < 0 || pn >= n);
    }
  }
  bad_block = __syncthreads_or(bad_block);
  bad_topo = __syncthreads_or(bad_topo);
  const bool ok = cap_ok && !bad_block && !bad_topo;
  if (tid == 0 && blockIdx.y == 0) {
    req_ok[b] = ok ? 1 : 0;
    if (!cap_ok) raise_status(status, SPEC_ERR_CAPACITY);
    if (bad_block) raise_status(status, SPEC_ERR_DEVICE_BOUNDS);
    if (bad_topo) raise_status(status, SPEC_ERR_INVALID_ARG);
  }
  if (!ok) return;
  if (window > 0 && blockIdx.y == 0)
    for (int n = tid; n < d.M; n += blockDim.x)
      win_row_mask(parent != nullptr ? s_par : nullptr, n, ctx, window, sinks,
                   anc_ws + (int64_t)b * d.M + n, depth_ws + (int64_t)b * d.M + n);

  // append: positions ctx .. end-1 where end = ceil(L/16)*16; rows past
  // ctx+M-1 are cleared.
  constexpr int kVec = 16 / sizeof(T);
  const int lanes = d.D / kVec;  // 16-byte vectors per (position, head)
  const int64_t end = ceil_div64(L, kBlock) * kBlock;
  const int npos = (int)(end - ctx);
  const int work = npos * d.Hkv * lanes;
  for (int w = blockIdx.y * blockDim.x + tid; w < work; w += gridDim.y * blockDim.x) {
    const int lane = w % lanes;
    const int h = (w / lanes) % d.Hkv;
    const int i = w / (lanes * d.Hkv);
    const int64_t t = (int64_t)ctx + i;
    const int64_t dst = (((int64_t)bt[t / kBlock] * d.Hkv + h) * kBlock + t % kBlock) * d.D;
    uint4 kv = make_uint4(0, 0, 0, 0), vv = make_uint4(0, 0, 0, 0);
    if (i < d.M) {
      const int64_t src = (((int64_t)b * d.M + i) * d.Hkv + h) * d.D;
      kv = reinterpret_cast<const uint4*>(k_new + src)[lane];
      vv = reinterpret_cast<const uint4*>(v_new + src)[lane];
    }
    reinterpret_cast<uint4*>(k_cache + dst)[lane] = kv;
    reinterpret_cast<uint4*>(v_cache + dst)[lane] = vv;
  }
}

// ---------------------------------------------------------------------------
// split-KV attention on CUDA cores
// ---------------------------------------------------------------------------
// Shared-memory layout (floats):
//   qs [R][D]        queries pre-scaled by softmax_scale*log2(e)
//   ks [32][D+4]     key tile (row padding keeps 16-byte reads conflict-free)
//   vs [32][D]       value tile
//   ps [R][32]       probabilities of the tile
constexpr int kTileKeys = 32;
constexpr int kSimtThreads = 128;
constexpr int kSimtWarps = kSimtThreads / kWarp;
constexpr int kMaxRows = 128;  // new rows per request (tree nodes)
constexpr int kMinWinSplit = 64;  // fewest keys of a range with a window
constexpr int kWinCtas = 3 * 152;

size_t attn_simt_smem_bytes(int R, int D) {
  return sizeof(float) * ((size_t)R * D + kTileKeys * (D + 4) + kTileKeys * D + (size_t)R * kTileKeys) +
         sizeof(unsigned long long) * 2 * kMaxRows;
}

template <typename T, int D, int RPW>
__global__ void __launch_bounds__(kSimtThreads) attn_split_kernel(
    const T* __restrict__ q, const T* __restrict__ k_cache, const T* __restrict__ v_cache,
    const int32_t* __restrict__ block_table, const int32_t* __restrict__ ctx_lens,
    const int32_t* __restrict__ parent, const int32_t* __restrict__ req_ok, spec_dims d,
    float qscale, int split_keys, int max_splits, float* __restrict__ part) {
  constexpr int DPL = D / kWarp;  // d values per lane in the PV step
  static_assert(DPL == 2 || DPL == 4, "D must be 64 or 128");
  const int s = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  if (!req_ok[b]) return;
  const int ctx = ctx_lens[b];
  const int L = ctx + d.M;
  const int k0 = s * split_keys;
  if (k0 >= L) return;
  const int k1 = min(k0 + split_keys, L);
  const int group = d.Hq / d.Hkv;
  const int R = group * d.M;
  const int tid = threadIdx.x, warp = tid / kWarp, lane = tid % kWarp;

  extern __shared__ __align__(16) float smem[];
  float* qs = smem;
  float* ks = qs + R * D;
  float* vs = ks + kTileKeys * (D + 4);
  float* ps = vs + kTileKeys * D;
  // [row][2]: bits 0..63 and 64..127 of each row's mask
  unsigned long long* anc = reinterpret_cast<unsigned long long*>(ps + R * kTileKeys);

  // queries of the rows that read KV head h: row r = i*group + g
  for (int e = tid; e < R * D; e += kSimtThreads) {
    const int r = e / D, dd = e % D;
    const int i = r / group, hq = h * group + r % group;
    qs[e] = to_f32(q[(((int64_t)b * d.M + i) * d.Hq + hq) * D + dd]) * qscale;
  }
  // ancestor-or-self masks of the new rows
  for (int i = tid; i < d.M; i += kSimtThreads) {
    unsigned long long lo = 0, hi = 0;
    if (parent == nullptr) {
      lo = i >= 63 ? ~0ull : ((1ull << (i + 1)) - 1);
      hi = i >= 127 ? ~0ull : (i >= 64 ? ((1ull << (i - 63)) - 1) : 0ull);
    } else {
      // the append kernel has checked the topology (parent[n] < n), so
      // the walk reaches the root
      const int32_t* par = parent + (int64_t)b * d.M;
      for (int n = i, step = 0; step <= kMaxRows && n >= 0; ++step, n = par[n]) {
        if (n < 64) lo |= 1ull << n;
        else hi |= 1ull << (n - 64);
      }
    }
    anc[2 * i] = lo;
    anc[2 * i + 1] = hi;
  }

  float o[RPW][DPL];
  float mrow[RPW], lrow[RPW];
#pragma unroll
  for (int j = 0; j < RPW; ++j) {
    mrow[j] = -INFINITY;
    lrow[j] = 0.f;
#pragma unroll
    for (int c = 0; c < DPL; ++c) o[j][c] = 0.f;
  }

  const int32_t* bt = block_table + (int64_t)b * d.max_blocks;
  constexpr int kVec = 16 / sizeof(T);
  constexpr int kVecPerKey = D / kVec;

  for (int t0 = k0; t0 < k1; t0 += kTileKeys) {
    __syncthreads();  // previous tile fully consumed
    for (int e = tid; e < kTileKeys * kVecPerKey; e += kSimtThreads) {
      const int kk = e / kVecPerKey, vi = e % kVecPerKey;
      const int t = t0 + kk;
      float kf[kVec], vf[kVec];
      if (t < k1) {
        const int64_t base = (((int64_t)bt[t / kBlock] * d.Hkv + h) * kBlock + t % kBlock) * D;
        const uint4 kr = reinterpret_cast<const uint4*>(k_cache + base)[vi];
        const uint4 vr = reinterpret_cast<const uint4*>(v_cache + base)[vi];
        unpack16(kr, kf);
        unpack16(vr, vf);
      } else {
#pragma unroll
        for (int c = 0; c < kVec; ++c) kf[c] = vf[c] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < kVec; ++c) {
        ks[kk * (D + 4) + vi * kVec + c] = kf[c];
        vs[kk * D + vi * kVec + c] = vf[c];
      }
    }
    __syncthreads();

    // scores: lane = key of the tile, rows warp + kSimtWarps*j
    const int t = t0 + lane;
    float sc[RPW];
#pragma unroll
    for (int j = 0; j < RPW; ++j) sc[j] = 0.f;
    const float4* krow = reinterpret_cast<const float4*>(ks + lane * (D + 4));
#pragma unroll 4
    for (int d4 = 0; d4 < D / 4; ++d4) {
      const float4 kv = krow[d4];
#pragma unroll
      for (int j = 0; j < RPW; ++j) {
        const int r = warp + kSimtWarps * j;
        if (r < R) {
          const float4 qv = reinterpret_cast<const float4*>(qs + r * D)[d4];
          sc[j] += qv.x * kv.x + qv.y * kv.y + qv.z * kv.z + qv.w * kv.w;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < RPW; ++j) {
      const int r = warp + kSimtWarps * j;
      if (r >= R) break;  // warp-uniform
      const int i = r / group;
      bool vis = t < k1;
      if (vis && t >= ctx) {
        const int k = t - ctx;  // new position, < M
        vis = (anc[2 * i + (k >> 6)] >> (k & 63)) & 1ull;
      }
      const float sj = vis ? sc[j] : -INFINITY;
      const float mnew = fmaxf(mrow[j], warp_max(sj));
      float p = 0.f, corr = 1.f;
      if (mnew != -INFINITY) {
        p = fast_exp2(sj - mnew);
        corr = exp2f(mrow[j] - mnew);
      }
      lrow[j] = lrow[j] * corr + warp_sum(p);
      mrow[j] = mnew;
      ps[r * kTileKeys + lane] = p;
#pragma unroll
      for (int c = 0; c < DPL; ++c) o[j][c] *= corr;
    }
    __syncwarp();
    // o[r][d] += sum_k p[r][k] * v[k][d], lane owns d = lane*DPL ..
#pragma unroll
    for (int k4 = 0; k4 < kTileKeys / 4; ++k4) {
      float4 p4[RPW];
#pragma unroll
      for (int j = 0; j < RPW; ++j) {
        const int r = warp + kSimtWarps * j;
        p4[j] = (r < R) ? reinterpret_cast<const float4*>(ps + r * kTileKeys)[k4]
                        : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        float vv[DPL];
        if constexpr (DPL == 4) {
          const float4 v4 = reinterpret_cast<const float4*>(vs + (k4 * 4 + kk) * D)[lane];
          vv[0] = v4.x; vv[1] = v4.y; vv[2] = v4.z; vv[3] = v4.w;
        } else {
          const float2 v2 = reinterpret_cast<const float2*>(vs + (k4 * 4 + kk) * D)[lane];
          vv[0] = v2.x; vv[1] = v2.y;
        }
#pragma unroll
        for (int j = 0; j < RPW; ++j) {
          const float pk = kk == 0 ? p4[j].x : kk == 1 ? p4[j].y : kk == 2 ? p4[j].z : p4[j].w;
#pragma unroll
          for (int c = 0; c < DPL; ++c) o[j][c] += pk * vv[c];
        }
      }
    }
  }

  // partial: normalized O and log2-sum-exp per row
  float* pbase = part + (((int64_t)b * d.Hkv + h) * max_splits + s) * (int64_t)R * (D + 1);
#pragma unroll
  for (int j = 0; j < RPW; ++j) {
    const int r = warp + kSimtWarps * j;
    if (r >= R) break;
    const float inv = lrow[j] > 0.f ? 1.f / lrow[j] : 0.f;
    float* prow = pbase + (int64_t)r * (D + 1);
#pragma unroll
    for (int c = 0; c < DPL; ++c)  // zero without a visible key, whatever the others held
      prow[lane * DPL + c] = lrow[j] > 0.f ? o[j][c] * inv : 0.f;
    if (lane == 0) prow[D] = lrow[j] > 0.f ? mrow[j] + log2f(lrow[j]) : -INFINITY;
  }
}

// ---------------------------------------------------------------------------
// the same with a sliding window and sinks
// ---------------------------------------------------------------------------
// The key axis is the sinks' tiles and the window's, without the tiles
// between them.  There are few keys, so the cost is what surrounds the
// products: eight warps share a tile (8 rows a warp at 64 rows), rows are
// padded to whole shares so that nothing in the products is conditional, the
// next tile's keys and values are loaded while a tile is used, masks and
// depths come from the append kernel, tiles that every row sees whole skip
// the mask, and a score's sum runs over two values of D at once (packed fp32
// FMA).  8 trees of 64 rows x 8 heads of 64 fp32 values, window 500: 49 us for
// the call, 35 of them here, where the kernel above with a window took 100 of
// 147; it waits for shared memory (46% of the issue slots used).  Tiles of 64
// keys, two a lane, need a third fewer loads of the queries and leave registers
// for two CTAs an SM instead of three: 52 us.  Three CTAs leave 80 registers, and
// the instances of 8 rows a warp spill (136 bytes of stores a thread for fp32
// heads of 64, 672 for heads of 128).
constexpr int kWinWarps = 8;
constexpr int kWinThreads = kWinWarps * kWarp;

// Rows are padded to whole warps' shares, so that no row of the products is
// conditional.
size_t attn_win_smem_bytes(int rows, int D) {
  return sizeof(float) * ((size_t)rows * D + kTileKeys * (D + 4) + kTileKeys * D +
                          (size_t)rows * kTileKeys) +
         (sizeof(ulonglong2) + sizeof(int)) * (size_t)rows;
}

__device__ __forceinline__ unsigned long long fma_pair(unsigned long long a, unsigned long long b,
                                                       unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

template <typename T, int D, int RPW>
__global__ void __launch_bounds__(kWinThreads, RPW <= 8 ? 3 : (D == 64 ? 2 : 1)) attn_win_split_kernel(
    const T* q, const T* k_cache, const T* v_cache, const int32_t* block_table,
    const int32_t* ctx_lens, const ulonglong2* anc_ws, const int32_t* depth_ws,
    const int32_t* req_ok, spec_dims d, int window, int sinks, float qscale,
    int split_keys, int max_splits, float* __restrict__ part) {
  constexpr int DPL = D / kWarp;  // d values per lane in the PV step
  static_assert(DPL == 2 || DPL == 4, "D must be 64 or 128");
  const int s = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  pdl_trigger();
  pdl_wait();  // the cache, the masks and the verdict come from the append kernel
  if (!req_ok[b]) return;
  const int ctx = ctx_lens[b];
  const int skip = win_skip(ctx, window, sinks, kTileKeys) * kTileKeys;
  const int skip_at = ceil_div(sinks, kTileKeys) * kTileKeys;
  const int L = ctx + d.M - skip;  // keys of the axis
  const int k0 = s * split_keys;
  if (k0 >= L) return;
  const int k1 = min(k0 + split_keys, L);
  const int group = d.Hq / d.Hkv;
  const int R = group * d.M;
  const int tid = threadIdx.x, warp = tid / kWarp, lane = tid % kWarp;

  extern __shared__ __align__(16) float smem[];
  constexpr int kRows = RPW * kWinWarps;
  float* qs = smem;
  float* ks = qs + kRows * D;
  float* vs = ks + kTileKeys * (D + 4);
  float* ps = vs + kTileKeys * D;
  ulonglong2* anc = reinterpret_cast<ulonglong2*>(ps + kRows * kTileKeys);  // mask of each row
  int* first = reinterpret_cast<int*>(anc + kRows);  // first position of its window

  constexpr int kVec = 16 / sizeof(T);
  constexpr int kVecPerKey = D / kVec;
  constexpr int kItems = kTileKeys * kVecPerKey / kWinThreads;  // 16-byte vectors of a thread
  static_assert(kItems >= 1, "a tile has at least one vector per thread");
  const int32_t* bt = block_table + (int64_t)b * d.max_blocks;
  uint4 kr[kItems], vr[kItems];
  // vectors of the tile at t0; keys past the range and keys that no row sees
  // (their pages may not be held, their values may be anything) are zero
  const int wf = win_first(ctx, window);
  auto fetch = [&](int t0) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int e = tid + i * kWinThreads, kk = e / kVecPerKey, vi = e % kVecPerKey;
      const int t = t0 + kk + (t0 >= skip_at ? skip : 0);
      kr[i] = vr[i] = make_uint4(0, 0, 0, 0);
      if (t0 + kk < k1 && (t >= wf || t < sinks)) {
        const int64_t base = (((int64_t)bt[t / kBlock] * d.Hkv + h) * kBlock + t % kBlock) * D;
        kr[i] = reinterpret_cast<const uint4*>(k_cache + base)[vi];
        vr[i] = reinterpret_cast<const uint4*>(v_cache + base)[vi];
      }
    }
  };
  fetch(k0);

  // queries of the rows that read KV head h: row r = i*group + g
  for (int e = tid; e < kRows * kVecPerKey; e += kWinThreads) {
    const int r = e / kVecPerKey, vi = e % kVecPerKey;
    float f[kVec];
    if (r < R) {
      const int i = r / group, hq = h * group + r - i * group;
      unpack16(reinterpret_cast<const uint4*>(q + (((int64_t)b * d.M + i) * d.Hq + hq) * D)[vi], f);
    } else {
#pragma unroll
      for (int c = 0; c < kVec; ++c) f[c] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < kVec; ++c) qs[r * D + vi * kVec + c] = f[c] * qscale;
  }
  for (int r = tid; r < kRows; r += kWinThreads) {
    const int64_t i = (int64_t)b * d.M + min(r, R - 1) / group;
    anc[r] = anc_ws[i];
    first[r] = ctx + depth_ws[i] + 1 - window;
  }

  float o[RPW][DPL];
  float mrow[RPW], lrow[RPW];
#pragma unroll
  for (int j = 0; j < RPW; ++j) {
    mrow[j] = -INFINITY;
    lrow[j] = 0.f;
#pragma unroll
    for (int c = 0; c < DPL; ++c) o[j][c] = 0.f;
  }

  for (int t0 = k0; t0 < k1; t0 += kTileKeys) {
    __syncthreads();  // previous tile fully consumed
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int e = tid + i * kWinThreads, kk = e / kVecPerKey, vi = e % kVecPerKey;
      float kf[kVec], vf[kVec];
      unpack16(kr[i], kf);
      unpack16(vr[i], vf);
#pragma unroll
      for (int c = 0; c < kVec; c += 4) {
        *reinterpret_cast<float4*>(ks + kk * (D + 4) + vi * kVec + c) =
            make_float4(kf[c], kf[c + 1], kf[c + 2], kf[c + 3]);
        *reinterpret_cast<float4*>(vs + kk * D + vi * kVec + c) =
            make_float4(vf[c], vf[c + 1], vf[c + 2], vf[c + 3]);
      }
    }
    __syncthreads();
    if (t0 + kTileKeys < k1) fetch(t0 + kTileKeys);

    // scores: lane = key of the tile, rows warp + kWinWarps*j
    const int t = t0 + lane + (t0 >= skip_at ? skip : 0);
    unsigned long long sc2[RPW];
#pragma unroll
    for (int j = 0; j < RPW; ++j) sc2[j] = 0ull;
    const ulonglong2* krow = reinterpret_cast<const ulonglong2*>(ks + lane * (D + 4));
#pragma unroll 4
    for (int d4 = 0; d4 < D / 4; ++d4) {
      const ulonglong2 kv = krow[d4];
#pragma unroll
      for (int j = 0; j < RPW; ++j) {
        const ulonglong2 qv =
            reinterpret_cast<const ulonglong2*>(qs + (warp + kWinWarps * j) * D)[d4];
        sc2[j] = fma_pair(qv.y, kv.y, fma_pair(qv.x, kv.x, sc2[j]));
      }
    }
    // tiles of cached keys inside every row's window (a depth is at most
    // M - 1), or inside the sinks, need no mask
    const int tt = t - lane;
    const bool plain = t0 + kTileKeys <= k1 && tt + kTileKeys <= ctx &&
                       (tt >= ctx + d.M - window || tt + kTileKeys <= sinks);
#pragma unroll
    for (int j = 0; j < RPW; ++j) {
      const int r = warp + kWinWarps * j;
      float sj = __uint_as_float((uint32_t)sc2[j]) + __uint_as_float((uint32_t)(sc2[j] >> 32));
      if (!plain) {
        bool vis;
        if (t < ctx) {
          vis = t < sinks || t >= first[r];
        } else {
          const int k = t - ctx;  // new position, < M when the key is in the range
          const ulonglong2 m = anc[r];
          vis = ((k < 64 ? m.x : m.y) >> (k & 63)) & 1ull;
        }
        if (!vis || t0 + lane >= k1) sj = -INFINITY;
      }
      const float mnew = fmaxf(mrow[j], warp_max(sj));
      float p = 0.f, corr = 1.f;
      if (mnew != -INFINITY) {
        p = fast_exp2(sj - mnew);
        corr = fast_exp2(mrow[j] - mnew);
      }
      lrow[j] = lrow[j] * corr + p;  // this lane's keys; the lanes are summed at the end
      mrow[j] = mnew;
      ps[r * kTileKeys + lane] = p;
#pragma unroll
      for (int c = 0; c < DPL; ++c) o[j][c] *= corr;
    }
    __syncwarp();
    // o[r][d] += sum_k p[r][k] * v[k][d], lane owns d = lane*DPL ..
#pragma unroll 2
    for (int k4 = 0; k4 < kTileKeys / 4; ++k4) {
      float vv[4][DPL];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const float* vp = vs + (k4 * 4 + kk) * D + lane * DPL;
        if constexpr (DPL == 4) {
          const float4 v4 = *reinterpret_cast<const float4*>(vp);
          vv[kk][0] = v4.x; vv[kk][1] = v4.y; vv[kk][2] = v4.z; vv[kk][3] = v4.w;
        } else {
          const float2 v2 = *reinterpret_cast<const float2*>(vp);
          vv[kk][0] = v2.x; vv[kk][1] = v2.y;
        }
      }
#pragma unroll
      for (int j = 0; j < RPW; ++j) {
        const float4 p4 =
            reinterpret_cast<const float4*>(ps + (warp + kWinWarps * j) * kTileKeys)[k4];
#pragma unroll
        for (int c = 0; c < DPL; ++c)
          o[j][c] = fmaf(p4.w, vv[3][c],
                         fmaf(p4.z, vv[2][c], fmaf(p4.y, vv[1][c], fmaf(p4.x, vv[0][c], o[j][c]))));
      }
    }
  }

  // partial: normalized O and log2-sum-exp per row
  float* pbase = part + (((int64_t)b * d.Hkv + h) * max_splits + s) * (int64_t)R * (D + 1);
#pragma unroll
  for (int j = 0; j < RPW; ++j) {
    const int r = warp + kWinWarps * j;
    if (r >= R) break;
    const float l = warp_sum(lrow[j]);
    const float inv = l > 0.f ? 1.f / l : 0.f;
    float* prow = pbase + (int64_t)r * (D + 1);
#pragma unroll
    for (int c = 0; c < DPL; ++c) prow[lane * DPL + c] = l > 0.f ? o[j][c] * inv : 0.f;
    if (lane == 0) prow[D] = l > 0.f ? mrow[j] + log2f(l) : -INFINITY;
  }
}

// ---------------------------------------------------------------------------
// merge of the split partials
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256) attn_combine_kernel(
    const float* part, const int32_t* ctx_lens, const int32_t* req_ok, spec_dims d, int window,
    int sinks, int split_keys, int max_splits, T* __restrict__ out, float* __restrict__ lse) {
  pdl_trigger();
  pdl_wait();  // the partials come from the previous kernel
  const int h = blockIdx.x, b = blockIdx.z;
  const int group = d.Hq / d.Hkv;
  const int R = group * d.M;
  const int D = d.D;
  const bool ok = req_ok[b] != 0;
  int L = ok ? ctx_lens[b] + d.M : 0;  // keys of the split axis
  if (ok && window > 0) L -= win_skip(ctx_lens[b], window, sinks, kTileKeys) * kTileKeys;
  const int nsp = ok ? ceil_div(L, split_keys) : 0;
  const float* pbase = part + ((int64_t)b * d.Hkv + h) * max_splits * (int64_t)R * (D + 1);
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const int nwarps = gridDim.y * (blockDim.x / kWarp);
  for (int r = blockIdx.y * (blockDim.x / kWarp) + warp; r < R; r += nwarps) {
    const int i = r / group, hq = h * group + r % group;
    // the lanes load the partials' sums side by side, and four partials' rows
    // are on their way at a time (one after another they took 24 us for 10
    // partials of 64 rows)
    float m = -INFINITY;
    for (int s = lane; s < nsp; s += kWarp) m = fmaxf(m, pbase[((int64_t)s * R + r) * (D + 1) + D]);
    m = warp_max(m);
    float wsum = 0.f;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    if (m != -INFINITY) {
#pragma unroll 4
      for (int s = 0; s < nsp; ++s) {
        const float* prow = pbase + ((int64_t)s * R + r) * (D + 1);
        const float w = exp2f(prow[D] - m);  // 0 for a partial without a visible key
        wsum += w;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < D / kWarp) acc[c] += w * prow[lane + c * kWarp];
      }
    }
    T* orow = out + (((int64_t)b * d.M + i) * d.Hq + hq) * D;
    const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
    for (int c = 0; c < D / kWarp; ++c) orow[lane + c * kWarp] = from_f32<T>(acc[c] * inv);
    if (lse != nullptr && lane == 0) {
      lse[((int64_t)b * d.M + i) * d.Hq + hq] =
          wsum > 0.f ? (m + log2f(wsum)) * 0.69314718055994530942f : -INFINITY;
    }
  }
}

// ---------------------------------------------------------------------------
// host launchers
// ---------------------------------------------------------------------------
cudaError_t kv_append_launch(const AttnArgs& a, const WsLayout& lay, cudaStream_t st, int* launches) {
  const spec_dims& d = a.d;
  int32_t* req_ok = reinterpret_cast<int32_t*>(static_cast<char*>(a.ws) + lay.attn_ok_off);
  uint32_t* status = reinterpret_cast<uint32_t*>(static_cast<char*>(a.ws) + lay.status_off);
  ulonglong2* anc = reinterpret_cast<ulonglong2*>(static_cast<char*>(a.ws) + lay.tc_anc_off);
  int32_t* depth = reinterpret_cast<int32_t*>(static_cast<char*>(a.ws) + lay.win_depth_off);
  // one CTA per 1024 vectors of 16 bytes (8 requests of 64 rows x 8 heads x 64
  // fp32 values: 19 us with one CTA each)
  const int64_t work = (int64_t)d.M * d.Hkv * d.D * (d.kv_dtype == SPEC_BF16 ? 2 : 4) / 16;
  const int split = work <= 1024 ? 1 : work >= 8 * 1024 ? 8 : (int)(work / 1024);
  PdlLaunch L(dim3(d.B, split), dim3(256), 0, st);
  cudaError_t e;
  if (d.kv_dtype == SPEC_BF16) {
    using T = __nv_bfloat16;
    e = cudaLaunchKernelEx(&L.cfg, kv_append_kernel<T>, static_cast<const T*>(a.k_new),
                           static_cast<const T*>(a.v_new), static_cast<T*>(a.k_cache),
                           static_cast<T*>(a.v_cache), a.block_table, a.ctx_lens, a.parent, d,
                           a.window, a.sinks, anc, depth, req_ok, status);
  } else {
    e = cudaLaunchKernelEx(&L.cfg, kv_append_kernel<float>, static_cast<const float*>(a.k_new),
                           static_cast<const float*>(a.v_new), static_cast<float*>(a.k_cache),
                           static_cast<float*>(a.v_cache), a.block_table, a.ctx_lens, a.parent,
                           d, a.window, a.sinks, anc, depth, req_ok, status);
  }
  ++*launches;
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
static cudaError_t launch_simt(const AttnArgs& a, const WsLayout& lay, cudaStream_t st, int* launches) {
  const spec_dims& d = a.d;
  const int R = (d.Hq / d.Hkv) * d.M;
  int32_t* req_ok = reinterpret_cast<int32_t*>(static_cast<char*>(a.ws) + lay.attn_ok_off);
  float* part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + lay.attn_off);

  kv_append_launch(a, lay, st, launches);

  const size_t smem = attn_simt_smem_bytes(R, d.D);
  // Key ranges: the layout's, or, with a window, of the fewer keys that a
  // request then has at most, for one wave of three CTAs per SM (the tree case
  // below: 53 us in 448 CTAs of 96 keys, 65 us in 640 of 64, 59 us in 320 of
  // 128), in whole tiles, no more ranges than the partials' workspace holds.
  int split_keys = lay.split_keys, splits = lay.max_splits;
  if (a.window > 0) {
    const int64_t most = min((int64_t)d.max_blocks * kBlock,
                             (int64_t)ceil_div(a.sinks, kTileKeys) * kTileKeys + a.window + d.M +
                                 kTileKeys);
    const int64_t want = max((int64_t)kMinWinSplit, (int64_t)d.B * d.Hkv * most / kWinCtas);
    split_keys = (int)(ceil_div64(max(want, ceil_div64(most, lay.max_splits)), kTileKeys) * kTileKeys);
    splits = (int)ceil_div64(most, split_keys);
  }
  const dim3 grid(splits, d.Hkv, d.B);
  const ulonglong2* anc =
      reinterpret_cast<const ulonglong2*>(static_cast<char*>(a.ws) + lay.tc_anc_off);
  const int32_t* depth =
      reinterpret_cast<const int32_t*>(static_cast<char*>(a.ws) + lay.win_depth_off);
  const float qscale = a.scale * 1.4426950408889634f;
  cudaError_t e = cudaSuccess;
#define SPECV_SIMT(DD, RPW)                                                                   \
  do {                                                                                        \
    auto k = attn_split_kernel<T, DD, RPW>;                                                   \
    /* the most of any call: another thread's may come between this and the launch */       \
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,                  \
                             (int)attn_simt_smem_bytes(RPW * kSimtWarps, DD));                \
    if (e != cudaSuccess) return e;                                                           \
    k<<<grid, kSimtThreads, smem, st>>>(static_cast<const T*>(a.q),                           \
                                        static_cast<const T*>(a.k_cache),                     \
                                        static_cast<const T*>(a.v_cache), a.block_table,      \
                                        a.ctx_lens, a.parent, req_ok, d, qscale,              \
                                        lay.split_keys, lay.max_splits, part);                \
  } while (0)
#define SPECV_WIN(DD, RPW)                                                                    \
  do {                                                                                        \
    auto k = attn_win_split_kernel<T, DD, RPW>;                                               \
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)win_smem);  \
    if (e != cudaSuccess) return e;                                                           \
    PdlLaunch L(grid, dim3(kWinThreads), win_smem, st);                                       \
    e = cudaLaunchKernelEx(&L.cfg, k, static_cast<const T*>(a.q),                             \
                           static_cast<const T*>(a.k_cache), static_cast<const T*>(a.v_cache),\
                           a.block_table, a.ctx_lens, anc, depth, (const int32_t*)req_ok, d,  \
                           a.window, a.sinks, qscale, split_keys, splits, part);              \
    if (e != cudaSuccess) return e;                                                           \
  } while (0)
  const int rpw = ceil_div(R, a.window > 0 ? kWinWarps : kSimtWarps);
  if (a.window > 0) {
    const int pad = rpw <= 1 ? 1 : rpw <= 2 ? 2 : rpw <= 4 ? 4 : rpw <= 8 ? 8 : 16;
    const size_t win_smem = attn_win_smem_bytes(pad * kWinWarps, d.D);
    if (d.D == 128) {
      if (rpw <= 1) SPECV_WIN(128, 1);
      else if (rpw <= 2) SPECV_WIN(128, 2);
      else if (rpw <= 4) SPECV_WIN(128, 4);
      else if (rpw <= 8) SPECV_WIN(128, 8);
      else SPECV_WIN(128, 16);
    } else {
      if (rpw <= 1) SPECV_WIN(64, 1);
      else if (rpw <= 2) SPECV_WIN(64, 2);
      else if (rpw <= 4) SPECV_WIN(64, 4);
      else if (rpw <= 8) SPECV_WIN(64, 8);
      else SPECV_WIN(64, 16);
    }
  } else if (d.D == 128) {
    if (rpw <= 2) SPECV_SIMT(128, 2);
    else if (rpw <= 4) SPECV_SIMT(128, 4);
    else if (rpw <= 8) SPECV_SIMT(128, 8);
    else if (rpw <= 16) SPECV_SIMT(128, 16);
    else SPECV_SIMT(128, 32);
  } else {
    if (rpw <= 2) SPECV_SIMT(64, 2);
    else if (rpw <= 4) SPECV_SIMT(64, 4);
    else if (rpw <= 8) SPECV_SIMT(64, 8);
    else if (rpw <= 16) SPECV_SIMT(64, 16);
    else SPECV_SIMT(64, 32);
  }
#undef SPECV_WIN
#undef SPECV_SIMT
  ++*launches;

  {
    PdlLaunch L(dim3(d.Hkv, ceil_div(R, 8), d.B), dim3(256), 0, st);
    e = cudaLaunchKernelEx(&L.cfg, attn_combine_kernel<T>, (const float*)part, a.ctx_lens,
                           (const int32_t*)req_ok, d, a.window, a.sinks, split_keys, splits,
                           static_cast<T*>(a.out), a.lse);
    if (e != cudaSuccess) return e;
  }
  ++*launches;
  return cudaGetLastError();
}

cudaError_t attn_launch_simt(const AttnArgs& a, const WsLayout& lay, cudaStream_t st, int* launches) {
  if (a.d.kv_dtype == SPEC_BF16) return launch_simt<__nv_bfloat16>(a, lay, st, launches);
  return launch_simt<float>(a, lay, st, launches);
}

}  // namespace specv
