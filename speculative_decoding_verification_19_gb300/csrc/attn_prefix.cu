// Attention of a whole batch over a prefix that its requests share.
//
// softmax(q K^T) V over the keys of the prefix and over a request's own keys
// are two partial sums of one softmax: with their log2-sum-exps l_1, l_2 the
// output is (2^l_1 o_1 + 2^l_2 o_2) / (2^l_1 + 2^l_2).  The prefix' keys are
// the same for every request, so all B * group * M rows that read a KV head are
// one product with them (page 2 §3.3: the cached prefix is reused, here by the
// whole batch): its keys and values are read once, not once a request.  A
// request's own keys go through the verify attention (attn.cu, attn_tc.cu).
//
// Kernels in this file:
//   prefix_simt_kernel   the prefix on CUDA cores (fp32; bf16 goes to the tensor
//                        cores, attn_prefix_tc.cu, unless CUDA cores are asked
//                        for), and views of requests with many rows
//   prefix_merge_kernel  the partials of a row, a warp per row
#include <math.h>

#include "attn.cuh"
#include "common.cuh"
#include "tc_ptx.cuh"

namespace specv {

// ---------------------------------------------------------------------------
// the prefix on CUDA cores
// ---------------------------------------------------------------------------
// A CTA runs 64 rows of a KV head over a range of key tiles.  Both products
// are register tiles of 8 rows per thread: scores 8 x kKeys / 16, summed in two
// halves (even and odd coordinates) so that a packed FMA takes what lies side by
// side in memory, outputs 8 x D / 16, two rows a packed FMA, with the probabilities
// transposed in shared memory.  The next keys are on their way (cp.async) from the
// end of the scores on, the next values from the end of the products with these.
// fp32 throughout.
constexpr int kPfxRows = 64, kPfxThreads = 128;
constexpr int kPfxCtas = 3;  // of an SM (68 KB with heads of 64, 74 KB with heads of 128)
// Ranges of all units together, at least the units: one wave of the CTAs that an
// SM holds, but no more than kPfxSplits lets: a partial in the merge costs 0.2 us, a
// tile in a range some 8.  us with as many ranges as there are tiles / with half of
// them: 8 tiles 29 / 35, 35 tiles 44 / 50, 64 tiles 52 / 44, 256 tiles (228 ranges, 128)
// 95 / 69.
constexpr int kPfxSlots = kPfxCtas * 152;
constexpr int kPfxSplits = 40;  // ranges of a unit: at most the root of this times its tiles

template <int D>
struct PfxTile {
  static constexpr int kKeys = D == 64 ? 64 : 32;
  static constexpr int kLd = kPfxRows + 4;  // padded rows of the transposed probabilities
  static constexpr int kLdK = D + 4;        // 16 keys' vectors: two wavefronts
  // eight rows of queries, then 16 bytes: the two row groups of a warp in other banks
  static constexpr int kQ = kPfxRows * D + 4 * (kPfxRows / 8);
  static constexpr size_t smem =
      sizeof(float) * ((size_t)kQ + kKeys * kLdK + kKeys * D + kKeys * kLd) +
      sizeof(ulonglong2) * kPfxRows;
};

__device__ __forceinline__ unsigned long long pair_of(float a, float b) {
  return (unsigned long long)__float_as_uint(a) | ((unsigned long long)__float_as_uint(b) << 32);
}
__device__ __forceinline__ float lo_of(unsigned long long x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float hi_of(unsigned long long x) {
  return __uint_as_float((uint32_t)(x >> 32));
}

// kOwn: the same tiles over views of the requests (attn_win_split_kernel's work)
// for more than 32 rows per KV head: 64 rows of a request, its view's keys in
// ranges of split_keys, the new rows' masks from the append kernel.  13 requests of
// 36 rows, 4 heads of 128 fp32 values over 45 pages: 61 us for the call, 77 with the
// windowed kernel.  Up to 32 rows a tile would be half empty: 13 requests of 32 rows
// 62 us, 53 with the windowed kernel; 8 of 32, 8 heads of 64 over 33 pages 48, 39.
template <typename T, int D, bool kOwn>
__global__ void __launch_bounds__(kPfxThreads, kPfxCtas) prefix_simt_kernel(
    const T* q, const T* k_cache, const T* v_cache, const int32_t* table, int prefix_len,
    spec_dims d, float qscale, PrefixPlan plan, ViewRanges own, float* __restrict__ part) {
  using Tile = PfxTile<D>;
  constexpr int kKeys = Tile::kKeys, kLd = Tile::kLd, kLdK = Tile::kLdK;
  constexpr int KPT = kKeys / 16;  // keys of a thread
  constexpr int CPT = D / 16;      // output columns of a thread
  constexpr int kVec = 16 / sizeof(T), kVecRow = D / kVec;
  extern __shared__ __align__(16) float smem[];
  float* qs = smem;                // [64][D] queries, scaled, 16 bytes after every eighth
  float* ks = qs + Tile::kQ;       // [kKeys][kLdK]
  float* vs = ks + kKeys * kLdK;   // [kKeys][D]
  float* pt = vs + kKeys * D;      // [kKeys][kLd] probabilities
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int s = blockIdx.x % plan.splits, tile = blockIdx.x / plan.splits, h = blockIdx.y;
  const int group = d.Hq / d.Hkv, R = group * d.M;
  const int rows = kOwn ? R : d.B * R;
  pdl_trigger();
  pdl_wait();  // the queries, the cache and the views may come from the previous kernels
  const int own_b = kOwn ? blockIdx.z : 0;
  int ctx = prefix_len, k0, k1;  // cached keys, and the range of keys
  ulonglong2* anc = reinterpret_cast<ulonglong2*>(pt + kKeys * kLd);  // masks of the rows (kOwn)
  if constexpr (kOwn) {
    if (!__ldcg(own.ok + own_b)) return;
    ctx = __ldcg(own.ctx + own_b);
    k0 = s * own.split_keys;
    k1 = min(k0 + own.split_keys, ctx + d.M);
    if (k0 >= k1) return;
    table += own_b * own.stride_b + h * own.stride_h;
    for (int r = tid; r < kPfxRows; r += kPfxThreads) {
      const int i = min(tile * kPfxRows + r, R - 1) / group;
      anc[r] = own.anc[(int64_t)own_b * d.M + i];
    }
  } else {
    k0 = (int)((int64_t)s * plan.key_tiles / plan.splits) * kKeys;
    k1 = min((int)((int64_t)(s + 1) * plan.key_tiles / plan.splits) * kKeys, prefix_len);
  }

  // keys or values of the tile at t0 by 16-byte vectors, those past the range zero;
  // block ids of its pages in id
  constexpr int kTilePages = kKeys / kBlock;
  auto ids_of = [&](int t0, int(&id)[kTilePages]) {
#pragma unroll
    for (int p = 0; p < kTilePages; ++p) {
      id[p] = t0 + p * kBlock < k1 ? __ldcg(table + t0 / kBlock + p) : 0;
      // no block id: the request check fails every request
      if ((uint32_t)id[p] >= (uint32_t)d.num_blocks) id[p] = 0;
    }
  };
  auto load = [&](const T* cache, int t0, const int(&id)[kTilePages], float* to, int ld) {
    constexpr int kItems = kKeys * kVecRow / kPfxThreads;  // vectors of a thread
    constexpr int kStep = kPfxThreads / kVecRow;           // keys of a round of the threads
    const int vi = tid % kVecRow, kk0 = tid / kVecRow;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int kk = kk0 + i * kStep;
      const bool there = t0 + kk < k1;
      int blk = id[0];  // of page kk / 16
#pragma unroll
      for (int p = 1; p < kTilePages; ++p)
        if (kk / kBlock == p) blk = id[p];
      const T* src = cache + (((int64_t)blk * d.Hkv + h) * kBlock + kk % kBlock) * D + vi * kVec;
      float* dst = to + kk * ld + vi * kVec;
      if constexpr (sizeof(T) == 4) {
        ptx::cp_async16_fill(ptx::smem_u32(dst), src, there ? 16u : 0u);
      } else {
        float f[kVec];
        unpack16(there ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0), f);
#pragma unroll
        for (int c = 0; c < kVec; c += 4)
          *reinterpret_cast<float4*>(dst + c) = make_float4(f[c], f[c + 1], f[c + 2], f[c + 3]);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int id[kTilePages];  // of the tile whose keys are to be loaded next, then its values
  ids_of(k0, id);
  load(k_cache, k0, id, ks, kLdK);
  load(v_cache, k0, id, vs, D);

  for (int e = tid; e < kPfxRows * kVecRow; e += kPfxThreads) {
    const int r = e / kVecRow, vi = e % kVecRow;
    const int gr = tile * kPfxRows + r;
    float f[kVec];
#pragma unroll
    for (int c = 0; c < kVec; ++c) f[c] = 0.f;
    if (gr < rows) {
      const int b = kOwn ? own_b : gr / R, rr = kOwn ? gr : gr - b * R, i = rr / group;
      const int64_t at = (((int64_t)b * d.M + i) * d.Hq + h * group + rr - i * group) * D;
      unpack16(reinterpret_cast<const uint4*>(q + at)[vi], f);
    }
    float* to = qs + r * D + (r >> 3) * 4 + vi * kVec;
#pragma unroll
    for (int c = 0; c < kVec; c += 4)
      *reinterpret_cast<float4*>(to + c) = make_float4(f[c] * qscale, f[c + 1] * qscale,
                                                       f[c + 2] * qscale, f[c + 3] * qscale);
  }

  unsigned long long o[4][CPT];  // row pairs x columns
  float m[8], l[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < CPT; ++c) o[r][c] = 0ull;

  for (int t0 = k0; t0 < k1; t0 += kKeys) {
    const bool more = t0 + kKeys < k1;
    if (more) ids_of(t0 + kKeys, id);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();  // the tile's keys are there

    unsigned long long sc[8][KPT];  // row r, key k * 16 + tx
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int k = 0; k < KPT; ++k) sc[r][k] = 0ull;
    const float* qrow = qs + ty * 8 * D + ty * 4;
    const float* krow = ks + tx * kLdK;
#pragma unroll 2
    for (int dd = 0; dd < D; dd += 4) {
      ulonglong2 kv[KPT];
#pragma unroll
      for (int k = 0; k < KPT; ++k)
        kv[k] = *reinterpret_cast<const ulonglong2*>(krow + k * 16 * kLdK + dd);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const ulonglong2 qv = *reinterpret_cast<const ulonglong2*>(qrow + r * D + dd);
#pragma unroll
        for (int k = 0; k < KPT; ++k) {
          sc[r][k] = fma2(qv.x, kv[k].x, sc[r][k]);
          sc[r][k] = fma2(qv.y, kv[k].y, sc[r][k]);
        }
      }
    }
    __syncthreads();  // the keys are consumed
    if (more) load(k_cache, t0 + kKeys, id, ks, kLdK);
    else asm volatile("cp.async.commit_group;" ::: "memory");
    // softmax: the 16 threads of a row group share its rows
    const int left = k1 - t0 - tx;  // this thread's key k is real if k * 16 is below it
    const bool masked = kOwn && t0 + kKeys > ctx;  // the tile reaches the new rows
    float p[8][KPT];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      float mt = -INFINITY;
#pragma unroll
      for (int k = 0; k < KPT; ++k) {
        const float x = lo_of(sc[r][k]) + hi_of(sc[r][k]);
        bool see = k * 16 < left;
        if (masked && see) {
          const int n = t0 + k * 16 + tx - ctx;  // new row, < M as the key is real
          const ulonglong2 m2 = anc[ty * 8 + r];
          see = n < 0 || ((n < 64 ? m2.x : m2.y) >> (n & 63)) & 1ull;
        }
        p[r][k] = see ? x : -INFINITY;
        mt = fmaxf(mt, p[r][k]);
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, w));
      const float mn = fmaxf(m[r], mt);
      // a tile of a prefix has a key for every row; one of new rows may have none yet
      const float ref = kOwn && mn == -INFINITY ? 0.f : mn;
      const float corr = fast_exp2(m[r] - ref);
      m[r] = mn;
      l[r] *= corr;
#pragma unroll
      for (int k = 0; k < KPT; ++k) {
        p[r][k] = fast_exp2(p[r][k] - ref);
        l[r] += p[r][k];  // this thread's keys; the 16 are summed at the end
      }
      // rescale the row's outputs
#pragma unroll
      for (int c = 0; c < CPT; ++c) {
        const float a = lo_of(o[r / 2][c]), b2 = hi_of(o[r / 2][c]);
        o[r / 2][c] = (r & 1) ? pair_of(a, b2 * corr) : pair_of(a * corr, b2);
      }
    }
#pragma unroll
    for (int k = 0; k < KPT; ++k) {
      float* row = pt + (k * 16 + tx) * kLd + ty * 8;
      *reinterpret_cast<float4*>(row) = make_float4(p[0][k], p[1][k], p[2][k], p[3][k]);
      *reinterpret_cast<float4*>(row + 4) = make_float4(p[4][k], p[5][k], p[6][k], p[7][k]);
    }
    // a row group's probabilities stay inside its warp; the tile's values are there
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
#pragma unroll 4
    for (int k = 0; k < kKeys; ++k) {
      const ulonglong2 pa = *reinterpret_cast<const ulonglong2*>(pt + k * kLd + ty * 8);
      const ulonglong2 pb = *reinterpret_cast<const ulonglong2*>(pt + k * kLd + ty * 8 + 4);
      const unsigned long long pv[4] = {pa.x, pa.y, pb.x, pb.y};
#pragma unroll
      for (int c4 = 0; c4 < CPT / 4; ++c4) {
        const float4 v4 = *reinterpret_cast<const float4*>(vs + k * D + c4 * 64 + tx * 4);
        const float vv[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const unsigned long long v2 = pair_of(vv[c], vv[c]);
#pragma unroll
          for (int r = 0; r < 4; ++r) o[r][c4 * 4 + c] = fma2(pv[r], v2, o[r][c4 * 4 + c]);
        }
      }
    }
    __syncthreads();  // the values are consumed
    if (more) load(v_cache, t0 + kKeys, id, vs, D);
    else asm volatile("cp.async.commit_group;" ::: "memory");
  }

  const int S = kOwn ? D + 1 : tc_part_stride(D);
  float* pbase =
      kOwn ? part + ((((int64_t)own_b * d.Hkv + h) * plan.splits + s) * R + tile * kPfxRows) * (int64_t)S
           : part + (((int64_t)h * plan.tiles + tile) * plan.splits + s) * plan.tile * (int64_t)S;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    float sum = l[r];
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    const int row = ty * 8 + r;
    if (row >= plan.tile || tile * kPfxRows + row >= rows) continue;
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    float* prow = pbase + (int64_t)row * S;
#pragma unroll
    for (int c4 = 0; c4 < CPT / 4; ++c4) {
      float f[4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        f[c] = ((r & 1) ? hi_of(o[r / 2][c4 * 4 + c]) : lo_of(o[r / 2][c4 * 4 + c])) * inv;
      if constexpr (kOwn) {  // rows of the merge's layout start anywhere
#pragma unroll
        for (int c = 0; c < 4; ++c) prow[c4 * 64 + tx * 4 + c] = f[c];
      } else {
        *reinterpret_cast<float4*>(prow + c4 * 64 + tx * 4) = make_float4(f[0], f[1], f[2], f[3]);
      }
    }
    if (tx == 0) prow[D] = sum > 0.f ? m[r] + log2f(sum) : -INFINITY;
  }
}

// ---------------------------------------------------------------------------
// merge
// ---------------------------------------------------------------------------
// A warp per row: a lane has the log2-sum-exp of a partial, then all have columns
// of the outputs and the lanes' weights in turn.
template <typename T>
__global__ void __launch_bounds__(256) prefix_merge_kernel(
    OwnPart own, const float* prefix, PrefixPlan plan, int64_t items, spec_dims d,
    T* __restrict__ out, float* __restrict__ lse) {
  pdl_trigger();
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const int h = blockIdx.y, D = d.D;
  const int group = d.Hq / d.Hkv, R = group * d.M;
  const int64_t gr64 = (int64_t)blockIdx.x * (blockDim.x / kWarp) + warp;
  if (gr64 >= (int64_t)d.B * R) return;
  const int gr = (int)gr64;  // B and R have 16 and 8 bits at most
  const int b = gr / R, r = gr - b * R, i = r / group;
  const int64_t at = ((int64_t)b * d.M + i) * d.Hq + h * group + r - i * group;
  const int tile = gr / plan.tile;
  const int64_t unit = (int64_t)h * plan.tiles + tile;
  const int S = tc_part_stride(D);
  int64_t slot = unit * plan.splits;
  int n_pfx = plan.splits;
  if (plan.ctas > 0) {
    const int c0 = prefix_cta(plan, items, unit * plan.key_tiles);
    slot = unit + c0;
    n_pfx = prefix_cta(plan, items, (unit + 1) * plan.key_tiles - 1) - c0 + 1;
  }
  const int own_step = R * own.stride, pfx_step = plan.tile * S;
  const float* own_row = own.part + (((int64_t)b * d.Hkv + h) * own.splits * R + r) * own.stride;
  const float* pfx_row = prefix + slot * pfx_step + (int64_t)(gr - tile * plan.tile) * S;
  pdl_wait();  // the partials come from the previous kernels
  const int ok = __ldcg(own.ok + b);
  const int n_own = own.splits == 1 ? 1 : ceil_div(__ldcg(own.ctx + b) + d.M, own.split_keys);
  T* orow = out + at * D;
  if (!ok) {  // the request has failed its checks
    for (int c = lane; c < D; c += kWarp) orow[c] = from_f32<T>(0.f);
    if (lse != nullptr && lane == 0) lse[at] = -INFINITY;
    return;
  }
  float mx = -INFINITY, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  auto row_of = [&](int s) {
    return s < n_own ? own_row + (int64_t)s * own_step : pfx_row + (int64_t)(s - n_own) * pfx_step;
  };
  for (int s0 = 0; s0 < n_own + n_pfx; s0 += kWarp) {
    const int n = min(kWarp, n_own + n_pfx - s0);
    const float l = lane < n ? __ldcg(row_of(s0 + lane) + D) : -INFINITY;
    const float mn = fmaxf(mx, warp_max(l));
    const float w = mn == -INFINITY ? 0.f : exp2f(l - mn);
    const float a = mx == -INFINITY ? 0.f : exp2f(mx - mn);
    sum = sum * a + warp_sum(w);
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] *= a;
    mx = mn;
#pragma unroll 8
    for (int s = 0; s < n; ++s) {
      const float* p = row_of(s0 + s) + lane;
      const float ws = __shfl_sync(0xffffffffu, w, s);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c * kWarp < D) acc[c] = fmaf(ws, __ldcg(p + c * kWarp), acc[c]);
    }
  }
  const float inv = 1.f / sum;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (c * kWarp < D) orow[lane + c * kWarp] = from_f32<T>(acc[c] * inv);
  if (lse != nullptr && lane == 0) lse[at] = (mx + log2f(sum)) * 0.69314718055994530942f;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
static PrefixPlan simt_plan(const spec_dims& d, int prefix_len) {
  PrefixPlan p;
  const int64_t rows = (int64_t)d.B * (d.Hq / d.Hkv) * d.M;
  const int keys = d.D == 64 ? PfxTile<64>::kKeys : PfxTile<128>::kKeys;
  p.tile = (int)(rows < kPfxRows ? rows : kPfxRows);
  p.tiles = (int)ceil_div64(rows, kPfxRows);
  p.key_tiles = ceil_div(prefix_len, keys);
  p.ctas = 0;
  const int64_t units = (int64_t)d.Hkv * p.tiles;
  int64_t splits = kPfxSlots / units;
  if (splits > p.key_tiles) splits = p.key_tiles;
  const int most = (int)sqrt((double)kPfxSplits * p.key_tiles);
  if (splits > most) splits = ceil_div(p.key_tiles, ceil_div(p.key_tiles, most));  // even ranges
  p.splits = splits < 1 ? 1 : (int)splits;
  return p;
}

static size_t prefix_simt_part_floats(const spec_dims& d) {
  const int64_t rows = (int64_t)d.B * (d.Hq / d.Hkv) * d.M;
  const int64_t units = (int64_t)d.Hkv * ceil_div64(rows, kPfxRows);
  const int64_t slots = units > kPfxSlots ? units : kPfxSlots;
  return (size_t)slots * (size_t)(rows < kPfxRows ? rows : kPfxRows) * tc_part_stride(d.D);
}

// Of either path; prefix_pass_floats: of the one that a pass with these dims takes.
size_t prefix_part_floats(const spec_dims& d) {
  const size_t simt = prefix_simt_part_floats(d), tc = prefix_tc_part_floats(d);
  return simt > tc ? simt : tc;
}
static bool prefix_on_tensor_cores(const spec_dims& d) {
  return prefix_tc_ok(d) && d.attn_impl != SPEC_ATTN_CUDA_CORES;
}
size_t prefix_pass_floats(const spec_dims& d) {
  return prefix_on_tensor_cores(d) ? prefix_tc_part_floats(d) : prefix_simt_part_floats(d);
}

template <typename T, bool kOwn>
static cudaError_t launch_simt(const AttnArgs& a, const PrefixPlan& p, const ViewRanges& own,
                               float* part, cudaStream_t st) {
  auto kern = a.d.D == 64 ? prefix_simt_kernel<T, 64, kOwn> : prefix_simt_kernel<T, 128, kOwn>;
  const size_t smem = a.d.D == 64 ? PfxTile<64>::smem : PfxTile<128>::smem;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  PdlLaunch L(dim3(p.splits * p.tiles, a.d.Hkv, kOwn ? a.d.B : 1), dim3(kPfxThreads), smem, st);
  return cudaLaunchKernelEx(&L.cfg, kern, static_cast<const T*>(a.q),
                            static_cast<const T*>(a.k_cache), static_cast<const T*>(a.v_cache),
                            kOwn ? a.view.table : a.view.prefix_table, kOwn ? 0 : a.view.prefix_len,
                            a.d, a.scale * 1.4426950408889634f, p, own, part);
}

int view_range_unit(const spec_dims& d) { return d.D == 64 ? PfxTile<64>::kKeys : PfxTile<128>::kKeys; }
int view_ctas() { return kPfxSlots; }

cudaError_t view_split_launch(const AttnArgs& a, const ViewRanges& own, int splits, float* part,
                              cudaStream_t st) {
  PrefixPlan p = {};
  p.tile = kPfxRows;
  p.tiles = ceil_div((a.d.Hq / a.d.Hkv) * a.d.M, kPfxRows);
  p.splits = splits;
  return a.d.kv_dtype == SPEC_BF16 ? launch_simt<__nv_bfloat16, true>(a, p, own, part, st)
                                   : launch_simt<float, true>(a, p, own, part, st);
}

cudaError_t prefix_launch(const AttnArgs& a, const WsLayout& lay, cudaStream_t st, PrefixPlan* plan,
                          int* launches) {
  float* part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + a.at.pfx);
  uint32_t* status = reinterpret_cast<uint32_t*>(static_cast<char*>(a.ws) + lay.status_off);
  cudaError_t e;
  if (prefix_on_tensor_cores(a.d)) {
    e = prefix_tc_launch(a, part, status, st, plan);
    if (e == cudaSuccess) ++*launches;
    return e;
  }
  *plan = simt_plan(a.d, a.view.prefix_len);
  e = a.d.kv_dtype == SPEC_BF16 ? launch_simt<__nv_bfloat16, false>(a, *plan, {}, part, st)
                                : launch_simt<float, false>(a, *plan, {}, part, st);
  if (e == cudaSuccess) ++*launches;
  return e;
}

cudaError_t prefix_merge_launch(const AttnArgs& a, const PrefixPlan& plan, const OwnPart& own,
                                cudaStream_t st, int* launches) {
  const spec_dims& d = a.d;
  const float* part = reinterpret_cast<const float*>(static_cast<char*>(a.ws) + a.at.pfx);
  const int64_t rows = (int64_t)d.B * (d.Hq / d.Hkv) * d.M;
  const int64_t items = (int64_t)d.Hkv * plan.tiles * plan.key_tiles;
  PdlLaunch L(dim3((unsigned)ceil_div64(rows, 8), d.Hkv), dim3(256), 0, st);
  cudaError_t e;
  if (d.kv_dtype == SPEC_BF16)
    e = cudaLaunchKernelEx(&L.cfg, prefix_merge_kernel<__nv_bfloat16>, own, part, plan, items, d,
                           static_cast<__nv_bfloat16*>(a.out), a.lse);
  else
    e = cudaLaunchKernelEx(&L.cfg, prefix_merge_kernel<float>, own, part, plan, items, d,
                           static_cast<float*>(a.out), a.lse);
  if (e == cudaSuccess) ++*launches;
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace specv
