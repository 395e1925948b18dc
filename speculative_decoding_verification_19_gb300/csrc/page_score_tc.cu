// Scores of pages on the 5th-generation tensor cores (bf16 bounds).
//
// q+ . hi + q- . lo is one product of depth 2 D: a page's row of bounds (lo, then
// hi, as they lie in memory) with the row (q-, q+) of every query that reads the
// KV head.  Pages are the M = 128 rows of the MMA (lanes of TMEM), queries its N
// columns, so the maximum over the queries is taken by each thread over its own
// lane.  The products are exact in fp32, their sums round in fp32.  4 D bytes a
// page meet 4 D rows operations: bound by the read of the bounds up to the 128
// rows that the kernel takes.
//
// The tiles of 128 pages of all (request, KV head) pairs, in this order, are
// shared evenly among one CTA per SM.  Per CTA, warp-specialised:
//   warps 4..7   copy a tile's bounds (512 bytes a page for D = 128) by 16-byte
//                cp.async into a ring, in the 128-byte-swizzled operand layout;
//                a tile's block ids are on their way while the last one is copied
//   warps 9, 10  build (q-, q+) of a pair, one pair ahead where shared memory has
//                room for two
//   warp 8       issues the MMAs into two TMEM buffers in turn
//   warps 0..3   maxima and scores
#include <math.h>

#include "page_select.cuh"
#include "tc_ptx.cuh"

namespace specv {
namespace score {

constexpr int kPages = 128;
constexpr int kThreads = 384;
constexpr int kCopyWarp = 4, kCopyThreads = 128, kMmaWarp = 8, kQueryWarp = 9, kQueryThreads = 64;
constexpr int kMaxStages = 4;
constexpr int kHalfBytes = kPages * 128;  // 64 columns of 128 pages
constexpr size_t kSmemMost = 224 * 1024;

struct __align__(8) Bars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t q_full[2], q_empty[2];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int issued[4];        // stages that each copy warp issued
  int64_t first, last;  // the CTA's tiles
  int64_t before;       // tiles of the requests before `b`
  int b;                // the request that holds its first tile
};

// Whole pages of a request; one with a bad length has none.
__device__ __forceinline__ int whole_pages(int ctx, int max_blocks) {
  return ctx > 0 && ctx <= (int64_t)max_blocks * kBlock ? ctx / kBlock : 0;
}

// The CTA's tiles in turn.
struct Walk {
  int64_t x, x1;
  int b, h, tile, nt, full;
  const int32_t* ctx;
  int B, Hkv, mb;
  __device__ Walk(const Bars& s, const int32_t* ctx_lens, const spec_dims& d)
      : x(s.first), x1(s.last), b(s.b), ctx(ctx_lens), B(d.B), Hkv(d.Hkv), mb(d.max_blocks) {
    if (x >= x1) return;
    look();
    const int64_t at = x - s.before;
    h = (int)(at / nt);
    tile = (int)(at - (int64_t)h * nt);
  }
  __device__ void look() {
    full = whole_pages(__ldcg(ctx + b), mb);
    nt = ceil_div(full, kPages);
  }
  __device__ bool more() const { return x < x1; }
  __device__ bool first(int64_t x0) const { return x == x0 || tile == 0; }
  __device__ bool last() const { return x == x1 - 1 || tile == nt - 1; }
  __device__ void next() {
    if (++x >= x1) return;
    if (++tile < nt) return;
    tile = 0;
    if (++h < Hkv) return;
    h = 0;
    do {
      ++b;  // a later request has the tile: x < x1
      look();
    } while (nt == 0);
  }
};

// kShort: the wait limit is short (ptx::mbar_wait_t).
template <int D, bool kShort>
__global__ void __launch_bounds__(kThreads, 1) page_score_tc_kernel(
    const __nv_bfloat16* q, const __nv_bfloat16* bounds, const int32_t* block_table,
    const int32_t* ctx_lens, spec_dims d, int N, int n_stages, int n_q,
    float* __restrict__ scores, uint32_t* __restrict__ status) {
  constexpr int kHalves = 2 * D / 64;
  constexpr int kStageBytes = kHalves * kHalfBytes;
  constexpr int kChunks = kHalves * 8;  // 16-byte chunks of a page's bounds
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* qbuf = smem + (size_t)n_stages * kStageBytes;
  __shared__ Bars bars_s;
  __shared__ int64_t s_sum[kThreads / kWarp];
  Bars* bars = &bars_s;
  const int tid = threadIdx.x, warp = tid / kWarp, lane = tid % kWarp;
  const int group = d.Hq / d.Hkv, R = group * d.M;
  const uint64_t wait = wait_limit_cycles(d);
  volatile int* abort = &bars->abort;
  const uint32_t cols = N <= 16 ? 32 : N <= 32 ? 64 : N <= 64 ? 128 : 256;
  pdl_trigger();

  if (tid == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bars->full[s]), kCopyThreads);
      ptx::mbar_init(ptx::smem_u32(&bars->empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(ptx::smem_u32(&bars->q_full[i]), kQueryThreads);
      ptx::mbar_init(ptx::smem_u32(&bars->q_empty[i]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->acc_full[i]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->acc_empty[i]), 4);
    }
    ptx::mbar_init(ptx::smem_u32(&bars->drain), 1);
    bars->abort = 0;
    ptx::fence_mbar_init();
  }
  pdl_wait();  // the queries, bounds and lengths may come from the previous kernels

  // ---- the CTA's share: tiles of all requests, then the request of its first
  int64_t total = 0;
  int bad = 0;
  for (int base = 0; base < d.B; base += kThreads) {
    const int b = base + tid;
    const int ctx = b < d.B ? __ldcg(ctx_lens + b) : 0;
    bad |= ctx > (int64_t)d.max_blocks * kBlock;
    int64_t n = (int64_t)ceil_div(whole_pages(ctx, d.max_blocks), kPages) * d.Hkv;
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    total += n;  // of this warp's requests
  }
  if (lane == 0) s_sum[warp] = total;
  bad = __syncthreads_or(bad);
  total = 0;
  for (int w = 0; w < kThreads / kWarp; ++w) total += s_sum[w];
  __syncthreads();
  const int64_t x0 = blockIdx.x * total / gridDim.x, x1 = (blockIdx.x + 1) * total / gridDim.x;
  if (tid == 0) {
    bars->first = x0;
    bars->last = x1;
    if (bad && blockIdx.x == 0) raise_status(status, SPEC_ERR_CAPACITY);
  }
  int64_t before = 0;
  for (int base = 0; base < d.B && before <= x0 && x0 < x1; base += kThreads) {
    const int b = base + tid;
    const int ctx = b < d.B ? __ldcg(ctx_lens + b) : 0;
    const int64_t own = (int64_t)ceil_div(whole_pages(ctx, d.max_blocks), kPages) * d.Hkv;
    int64_t upto = own;
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    int64_t all = 0;
    for (int w = 0; w < kThreads / kWarp; ++w) {
      if (w < warp) upto += s_sum[w];
      all += s_sum[w];
    }
    upto += before;
    if (upto - own <= x0 && x0 < upto) {
      bars->b = b;
      bars->before = upto - own;
    }
    before += all;
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    // (behind the wait for the previous kernel: it may need the columns)
    ptx::tmem_alloc(ptx::smem_u32(&bars->tmem_base), cols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp >= kCopyWarp && warp < kCopyWarp + 4) {
    // --------------------------------------------------------------- copies
    const int ct = (warp - kCopyWarp) * kWarp + lane;
    const int c = ct % kChunks;                    // chunk of a page's bounds
    constexpr int kStep = kCopyThreads / kChunks;  // pages of one round of the threads
    const int p0 = ct / kChunks;
    const uint32_t so = (uint32_t)(c >> 3) * kHalfBytes;
    int st = 0, at = 0;
    uint32_t round = 0;
    bool ok = true;
    int ids[kPages / kWarp], nids[kPages / kWarp];  // lane j: blocks of pages j, 32 + j, ...
    auto look_up = [&](const Walk& w, int(&to)[kPages / kWarp]) {
      const int32_t* bt = block_table + (int64_t)w.b * d.max_blocks + w.tile * kPages;
      const int np = w.full - w.tile * kPages;
#pragma unroll
      for (int k = 0; k < kPages / kWarp; ++k)
        to[k] = k * kWarp + lane < np ? __ldcg(bt + k * kWarp + lane) : -1;
    };
    Walk w(*bars, ctx_lens, d);
    if (w.more()) look_up(w, nids);
    while (w.more() && ok) {
      const int h = w.h;
#pragma unroll
      for (int k = 0; k < kPages / kWarp; ++k) ids[k] = nids[k] < d.num_blocks ? nids[k] : -1;
      w.next();
      if (w.more()) look_up(w, nids);
      ok = ptx::mbar_wait_t<kShort>(ptx::smem_u32(&bars->empty[at]), round ^ 1u, abort, wait);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t sb = ptx::smem_u32(smem + (size_t)at * kStageBytes) + so;
#pragma unroll
      for (int k = 0; k < kPages / kWarp; ++k)
#pragma unroll 4
        for (int r = 0; r < kWarp; r += kStep) {
          const int p = k * kWarp + r + p0;
          const int id = __shfl_sync(0xffffffffu, ids[k], r + p0);
          const bool there = id >= 0;  // else zeros
          const __nv_bfloat16* src =
              bounds + ((int64_t)(there ? id : 0) * d.Hkv + h) * 2 * D + c * 8;
          ptx::cp_async16_fill(sb + (uint32_t)p * 128u + ((uint32_t)((c & 7) ^ (p & 7)) << 4), src,
                               there ? 16u : 0u);
        }
      ptx::cp_async_arrive_noinc(ptx::smem_u32(&bars->full[at]));
      ++st;
      if (++at == n_stages) {
        at = 0;
        round ^= 1u;
      }
    }
    // every copy lands before the CTA may exit, also when a wait gave up
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (lane == 0) bars->issued[warp - kCopyWarp] = st;
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (ct == 0) {
      const int all = min(min(bars->issued[0], bars->issued[1]), min(bars->issued[2], bars->issued[3]));
      for (int u = all > n_stages ? all - n_stages : 0; u < all; ++u)
        ptx::mbar_drain(ptx::smem_u32(&bars->full[u % n_stages]), (uint32_t)((u / n_stages) & 1),
                        kDefaultWaitCycles);
    }
  } else if (warp >= kQueryWarp && warp < kQueryWarp + 2) {
    // -------------------------------------------------------------- queries
    const int qt = (warp - kQueryWarp) * kWarp + lane;
    int pairs = 0;
    for (Walk w(*bars, ctx_lens, d); w.more(); w.next()) {
      if (!w.first(x0)) continue;
      const int buf = pairs % n_q;
      if (!__all_sync(0xffffffffu,
                      ptx::mbar_wait_t<kShort>(ptx::smem_u32(&bars->q_empty[buf]),
                                               (uint32_t)((pairs / n_q) & 1) ^ 1u, abort, wait)))
        break;
      ++pairs;
      uint8_t* to = qbuf + (size_t)buf * kHalves * N * 128;
      constexpr int kVec = D / 8, kAtOnce = 6;
      for (int e0 = qt; e0 < N * kVec; e0 += kAtOnce * kQueryThreads) {
        uint4 v[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const int e = e0 + u * kQueryThreads, n = e / kVec, c = e % kVec, i = n / group;
          v[u] = make_uint4(0, 0, 0, 0);
          if (n < R)
            v[u] = __ldcg(reinterpret_cast<const uint4*>(
                              q + (((int64_t)w.b * d.M + i) * d.Hq + w.h * group + n - i * group) * D) + c);
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const int e = e0 + u * kQueryThreads, n = e / kVec, c = e % kVec;
          if (n >= N) break;
          const uint32_t x[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
          uint32_t lo[4], hi[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(lo[k]) : "r"(x[k]), "r"(0u));
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(hi[k]) : "r"(x[k]), "r"(0u));
          }
          const uint32_t o = (uint32_t)(c >> 3) * (uint32_t)N * 128u + (uint32_t)n * 128u +
                             ((uint32_t)((c & 7) ^ (n & 7)) << 4);
          *reinterpret_cast<uint4*>(to + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);  // meets lo
          *reinterpret_cast<uint4*>(to + (kHalves / 2) * N * 128 + o) =
              make_uint4(hi[0], hi[1], hi[2], hi[3]);
        }
      }
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(ptx::smem_u32(&bars->q_full[buf]));
    }
  } else if (warp == kMmaWarp) {
    // ----------------------------------------------------------------- MMAs
    if (lane == 0) {
      const uint64_t da0 = ptx::sdesc_sw128(ptx::smem_u32(smem), 16, 1024);
      const uint64_t db0 = ptx::sdesc_sw128(ptx::smem_u32(qbuf), 16, 1024);
      const uint32_t id = ptx::idesc_bf16_f32(128, N, false, false);
      int at = 0, pairs = 0, qb = 0;
      uint32_t round = 0, t = 0;
      for (Walk w(*bars, ctx_lens, d); w.more(); w.next(), ++t) {
        if (w.first(x0)) {
          qb = pairs % n_q;
          if (!ptx::mbar_wait_t<kShort>(ptx::smem_u32(&bars->q_full[qb]), (uint32_t)((pairs / n_q) & 1),
                                        abort, wait))
            break;
          ++pairs;
        }
        const uint64_t db = db0 + (uint64_t)((qb * kHalves * N * 128) >> 4);
        if (!ptx::mbar_wait_t<kShort>(ptx::smem_u32(&bars->full[at]), round, abort, wait)) break;
        const int buf = t & 1;
        if (!ptx::mbar_wait_t<kShort>(ptx::smem_u32(&bars->acc_empty[buf]), ((t >> 1) & 1) ^ 1u, abort,
                                      wait))
          break;
        ptx::fence_proxy_async_smem();  // the copies' writes, for the tensor cores
        ptx::tc_fence_after();
        const uint64_t da = da0 + (uint64_t)(((size_t)at * kStageBytes) >> 4);
#pragma unroll
        for (int k = 0; k < 2 * D / 16; ++k)
          ptx::mma_ss(tmem + buf * N, da + (uint64_t)(((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4),
                      db + (uint64_t)(((k >> 2) * N * 128 + (k & 3) * 32) >> 4), id, k > 0 ? 1u : 0u);
        ptx::mma_commit(ptx::smem_u32(&bars->acc_full[buf]));
        ptx::mma_commit(ptx::smem_u32(&bars->empty[at]));
        if (w.last()) ptx::mma_commit(ptx::smem_u32(&bars->q_empty[qb]));
        if (++at == n_stages) {
          at = 0;
          round ^= 1u;
        }
      }
      ptx::mma_commit(ptx::smem_u32(&bars->drain));
      ptx::mbar_drain(ptx::smem_u32(&bars->drain), 0, kDefaultWaitCycles);
    }
  } else if (warp < 4) {
    // --------------------------------------------------------------- maxima
    // what no tile covers is -inf: pages that are not whole or not there
    for (int64_t row = blockIdx.x; row < (int64_t)d.B * d.Hkv; row += gridDim.x) {
      const int full = whole_pages(__ldcg(ctx_lens + row / d.Hkv), d.max_blocks);
      for (int p = full + tid; p < d.max_blocks; p += 4 * kWarp)
        scores[row * d.max_blocks + p] = -INFINITY;
    }
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    uint32_t t = 0;
    for (Walk w(*bars, ctx_lens, d); w.more(); w.next(), ++t) {
      const int p = w.tile * kPages + warp * 32 + lane;
      const int id = p < w.full ? __ldcg(block_table + (int64_t)w.b * d.max_blocks + p) : 0;
      const int buf = t & 1;
      if (!__all_sync(0xffffffffu,
                      ptx::mbar_wait_t<kShort>(ptx::smem_u32(&bars->acc_full[buf]),
                                               (t >> 1) & 1, abort, wait)))
        break;
      ptx::tc_fence_after();
      float m[2] = {-INFINITY, -INFINITY};
      for (int n = 0; n < N; n += 16) {
        uint32_t v[16];
        ptx::tmem_ld16(lane_base + buf * N + n, v);
        ptx::tmem_wait_ld(v);
        if (n + 16 > R) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (n + j >= R) v[j] = 0xff800000u;  // -inf: no query
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          m[j & 1] = max_nan(m[j & 1], __uint_as_float(v[j]), __uint_as_float(v[j + 8]));
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars->acc_empty[buf]));
      if (p < w.full) {
        const bool there = id >= 0 && id < d.num_blocks;
        scores[((int64_t)w.b * d.Hkv + w.h) * d.max_blocks + p] = there ? max_nan(m[0], m[1]) : -INFINITY;
        if (!there) raise_status(status, SPEC_ERR_DEVICE_BOUNDS);
      }
    }
  }

  __syncthreads();
  if (tid == 0 && *abort) raise_status(status, SPEC_ERR_TIMEOUT);
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, cols);
  }
}

}  // namespace score

// Rows of a KV head that the kernel takes: the columns of an MMA.
bool page_score_tc_ok(const spec_dims& d) {
  return d.kv_dtype == SPEC_BF16 && (int64_t)(d.Hq / d.Hkv) * d.M <= 128;
}

cudaError_t page_score_tc_launch(const ScoreArgs& a, cudaStream_t st, int* launches) {
  using namespace score;
  const spec_dims& d = a.d;
  const int N = ceil_div((d.Hq / d.Hkv) * d.M, 16) * 16;
  const size_t stage = (size_t)(2 * d.D / 64) * kHalfBytes, qbytes = (size_t)N * 4 * d.D;
  // two buffers of queries where two stages (128 KB of bounds on their way) fit
  // beside them
  const int n_q = 2 * qbytes + 2 * stage <= kSmemMost ? 2 : 1;
  int n_stages = (int)((kSmemMost - n_q * qbytes) / stage);
  if (n_stages > kMaxStages) n_stages = kMaxStages;
  const size_t smem = n_stages * stage + n_q * qbytes + 1024;
  const bool short_wait = wait_limit_cycles(d) < ptx::kShortWait;
  auto kern = d.D == 64 ? (short_wait ? page_score_tc_kernel<64, true> : page_score_tc_kernel<64, false>)
                        : (short_wait ? page_score_tc_kernel<128, true> : page_score_tc_kernel<128, false>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)(kSmemMost + 1024));
  int dev = 0, sms = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // no more CTAs than tiles of the longest requests
  const int64_t most = (int64_t)d.B * d.Hkv * ceil_div(d.max_blocks, kPages);
  PdlLaunch L(dim3((unsigned)(most < sms ? most : sms)), dim3(kThreads), smem, st);
  e = cudaLaunchKernelEx(&L.cfg, kern, static_cast<const __nv_bfloat16*>(a.q),
                         static_cast<const __nv_bfloat16*>(a.bounds), a.block_table, a.ctx_lens, d,
                         N, n_stages, n_q, a.scores, a.status);
  if (e == cudaSuccess) ++*launches;
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace specv
