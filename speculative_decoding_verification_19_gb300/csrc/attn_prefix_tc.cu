// A shared prefix on the 5th-generation tensor cores (tcgen05 + TMEM).
//
// All rows of the batch that read a KV head meet the same keys, so the work is
// two plain products with a softmax between them: 4 rows keys D operations for
// 4 keys D bytes.  From some 290 rows on it is bound by the tensor cores,
// below by the read of the keys and values.
//
// A CTA runs units of 256 rows (two MMA tiles A and B of 128) of a KV head over
// tiles of 128 keys; all (head, unit, key tile) items in that order are shared
// evenly among one CTA per SM, so a unit may be split over CTAs: each leaves a
// partial (normalised output and log2-sum-exp of its keys) for the merge.
//
// A and B are two pipelines that share the K/V ring and nothing else:
//   warps 0..3, 4..7  softmax of A, of B: a thread per row (TMEM lane), 64 scores
//                     in registers at a time, P written back as bf16 over the
//                     scores in TMEM
//   warps 8, 9        issue A's, B's MMAs: S = Q K^T, then O += P V when P is there,
//                     the first 64 keys of P while the softmax does the others.
//                     The next S is issued when P V is done, as it overwrites P;
//                     the other pipeline's MMAs fill the wait
//   warps 10, 11      copy: Q rows, and the pages' keys and values by 16-byte
//                     cp.async into a ring of five 32 KB stages, K and V in turn,
//                     in the 128-byte-swizzled layout of the operands
//
// O is rescaled in TMEM by the softmax threads only when a row's running
// maximum grows by more than 2^8 (O's last P V is done by then: the scores they
// hold were issued after it).  Scores, maxima, sums and O are fp32, the
// probabilities bf16 for P V (attn_tc.cu says what that costs).
//
// TMEM: S_A [0, 128) with P_A in its first half, S_B [128, 256), O_A [256, 384),
// O_B [384, 512).
#include <math.h>

#include "attn.cuh"
#include "common.cuh"
#include "tc_ptx.cuh"

namespace specv {
namespace pfx {

constexpr int kKeys = 128;
constexpr int kPages = kKeys / kBlock;  // 8
constexpr int kTileRows = 128;          // rows of an MMA tile; two make a unit
constexpr int kUnitRows = 2 * kTileRows;
constexpr int kStages = 5;
constexpr int kThreads = 384;
constexpr int kIssueWarp = 8;  // and 9
constexpr int kCopyWarp = 10;  // and 11
constexpr int kCopyThreads = 64;
constexpr int kHalfBytes = kKeys * 128;  // 64 columns of 128 rows
constexpr int kTmemCols = 512;
constexpr int kOCol = 256;

struct __align__(8) Bars {
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t q_full, q_empty;
  uint64_t s_full[2];
  uint64_t p_half[2][2];
  uint64_t o_done[2];
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort;
  int issued[2];  // stages that each copy warp issued
  int units[2];   // units whose queries it issued
};

// The CTA's items x0 .. x1 - 1 in turn.
struct Walk {
  int64_t x, x0, x1, unit;
  int kt, tile, h, nt, tiles;
  __device__ Walk(int64_t from, int64_t to, const PrefixPlan& p)
      : x(from), x0(from), x1(to), unit(from / p.key_tiles), nt(p.key_tiles), tiles(p.tiles) {
    kt = (int)(from - unit * nt);
    h = (int)(unit / tiles);
    tile = (int)(unit - (int64_t)h * tiles);
  }
  __device__ bool more() const { return x < x1; }
  __device__ bool first() const { return x == x0 || kt == 0; }
  __device__ bool last() const { return x == x1 - 1 || kt == nt - 1; }
  __device__ void next() {
    ++x;
    if (++kt < nt) return;
    kt = 0;
    ++unit;
    if (++tile < tiles) return;
    tile = 0;
    ++h;
  }
};

template <int D>
struct Shape {
  static constexpr int kHalves = D / 64;
  static constexpr int kStageBytes = kHalves * kHalfBytes;
  static constexpr int kQBytes = 2 * kHalves * kHalfBytes;
  static constexpr size_t kSmem = (size_t)kStages * kStageBytes + kQBytes + sizeof(Bars) + 1024;
};

__device__ __forceinline__ unsigned long long pack2(uint32_t a, uint32_t b) {
  return (unsigned long long)a | ((unsigned long long)b << 32);
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b,
                                                   unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float lo_of(unsigned long long x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float hi_of(unsigned long long x) {
  return __uint_as_float((uint32_t)(x >> 32));
}

// kShort: the wait limit is short (ptx::mbar_wait_t).
template <int D, bool kShort>
__global__ void __launch_bounds__(kThreads, 1) prefix_tc_kernel(
    const __nv_bfloat16* q, const __nv_bfloat16* k_cache, const __nv_bfloat16* v_cache,
    const int32_t* table, int prefix_len, spec_dims d, float qscale2, PrefixPlan plan,
    float* __restrict__ part, uint32_t* __restrict__ status) {
  using S = Shape<D>;
  constexpr int kHalves = S::kHalves;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* stages = smem;
  uint8_t* qbuf = smem + kStages * S::kStageBytes;
  Bars* bars = reinterpret_cast<Bars*>(qbuf + S::kQBytes);

  const int tid = threadIdx.x, warp = tid / kWarp, lane = tid % kWarp;
  const int Hkv = d.Hkv, group = d.Hq / d.Hkv, R = group * d.M;
  const int64_t rows = (int64_t)d.B * R;
  const int64_t items = (int64_t)Hkv * plan.tiles * plan.key_tiles;
  const int c = blockIdx.x;
  const int64_t x0 = c * items / plan.ctas, x1 = (c + 1) * items / plan.ctas;
  const uint64_t wait = wait_limit_cycles(d);
  // rows of a head all in tile A: B has no part in the call
  const int pipes = rows > kTileRows ? 2 : 1;
  pdl_trigger();

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bars->full[s]), kCopyThreads);
      ptx::mbar_init(ptx::smem_u32(&bars->empty[s]), pipes);
    }
    ptx::mbar_init(ptx::smem_u32(&bars->q_full), kCopyThreads);
    ptx::mbar_init(ptx::smem_u32(&bars->q_empty), pipes);
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(ptx::smem_u32(&bars->s_full[a]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->p_half[a][0]), 4);
      ptx::mbar_init(ptx::smem_u32(&bars->p_half[a][1]), 4);
      ptx::mbar_init(ptx::smem_u32(&bars->o_done[a]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->drain[a]), 1);
    }
    bars->abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kCopyWarp) {
    ptx::tmem_alloc(ptx::smem_u32(&bars->tmem_base), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  volatile int* abort = &bars->abort;
  pdl_wait();  // the queries and the cache may come from the previous kernels

  if (warp >= kIssueWarp) {
    if (warp >= kCopyWarp) {
      // ------------------------------------------------------------- copies
      const int ct = (warp - kCopyWarp) * kWarp + lane;  // copy thread 0..63
      const int c16 = ct % (8 * kHalves);                // 16-byte chunk of a row
      const int r0 = ct / (8 * kHalves);
      constexpr int kRowStep = kCopyThreads / (8 * kHalves);
      const uint32_t swz_half = (uint32_t)(c16 >> 3) * kHalfBytes;
      int64_t st = 0;  // stage number: K and V of a tile in turn
      int seg = 0;
      int ids = 0;
      int have = -1;  // window of 32 pages that ids holds
      bool ok = true;
      for (Walk w(x0, x1, plan); w.more() && ok; w.next()) {
        const int kt = w.kt, h = w.h;
        if (w.first()) {
          // the unit's queries, when the last unit's products are done: 128 rows
          // a warp, a lane finds the place of a row for all
          ok = ptx::mbar_wait_t<kShort>(ptx::smem_u32(&bars->q_empty), (uint32_t)((seg & 1) ^ 1),
                                        abort, wait);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const int64_t row0 = (int64_t)w.tile * kUnitRows + (warp - kCopyWarp) * kTileRows;
          const uint32_t qb = ptx::smem_u32(qbuf) + (warp - kCopyWarp) * kHalves * kHalfBytes + swz_half;
          for (int r32 = 0; r32 < kTileRows && row0 < rows; r32 += kWarp) {
            const int64_t gr = row0 + r32 + lane;
            int at = -1;
            if (gr < rows) {
              const int b = (int)(gr / R), rr = (int)(gr - (int64_t)b * R), i = rr / group;
              at = (int)(((int64_t)b * d.M + i) * d.Hq + h * group + rr - i * group);
            }
            constexpr int kPer = kWarp / (8 * kHalves);  // rows of a copy
#pragma unroll 4
            for (int k = 0; k < kWarp; k += kPer) {
              const int rl = k + lane / (8 * kHalves), rr = r32 + rl;
              const int from = __shfl_sync(0xffffffffu, at, rl);
              ptx::cp_async16_fill(qb + (uint32_t)rr * 128u + ((uint32_t)((c16 & 7) ^ (rr & 7)) << 4),
                                   q + (from < 0 ? 0 : (int64_t)from * D + c16 * 8),
                                   from < 0 ? 0u : 16u);
            }
          }
          ptx::cp_async_arrive_noinc(ptx::smem_u32(&bars->q_full));
          ++seg;
        }
        // lane j holds the block of page j of a window of 32 (four tiles)
        if ((kt >> 2) != have) {
          have = kt >> 2;
          const int p = have * 32 + lane;
          ids = p * kBlock < prefix_len ? __ldcg(table + p) : 0;
          // no block id: the request check fails every request
          if ((uint32_t)ids >= (uint32_t)d.num_blocks) ids = 0;
        }
        const int np = min(kPages, prefix_len / kBlock - kt * kPages);
        int64_t blk[kPages];
#pragma unroll
        for (int p = 0; p < kPages; ++p)
          blk[p] = ((int64_t)__shfl_sync(0xffffffffu, ids, (kt & 3) * kPages + p) * Hkv + h) * kBlock;
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++st) {
          const int sl = (int)(st % kStages);
          ok = ptx::mbar_wait_t<kShort>(ptx::smem_u32(&bars->empty[sl]),
                                        (uint32_t)((st / kStages) & 1) ^ 1u, abort, wait);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t sb = ptx::smem_u32(stages + sl * S::kStageBytes) + swz_half;
          const __nv_bfloat16* src = (kv == 0 ? k_cache : v_cache) + c16 * 8;
#pragma unroll
          for (int p = 0; p < kPages; ++p) {
            if (p < np) {
#pragma unroll
              for (int k = 0; k < kBlock / kRowStep; ++k) {
                const int r = r0 + k * kRowStep;
                ptx::cp_async16(sb + (uint32_t)(p * kBlock + r) * 128u +
                                    ((uint32_t)((c16 & 7) ^ (r & 7)) << 4),
                                src + (blk[p] + r) * D);
              }
            }
          }
          ptx::cp_async_arrive_noinc(ptx::smem_u32(&bars->full[sl]));
        }
      }
      // every copy lands before the CTA may exit, also when a wait gave up and
      // the two warps stopped at different stages: their own copies, then the
      // barriers that both arrived on
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (lane == 0) {
        bars->issued[warp - kCopyWarp] = (int)st;
        bars->units[warp - kCopyWarp] = seg;
      }
      asm volatile("bar.sync 2, 64;" ::: "memory");
      if (ct == 0) {
        const int64_t both = min(bars->issued[0], bars->issued[1]);
        for (int64_t u = both > kStages ? both - kStages : 0; u < both; ++u)
          ptx::mbar_drain(ptx::smem_u32(&bars->full[u % kStages]), (uint32_t)((u / kStages) & 1),
                          kDefaultWaitCycles);
        const int units = min(bars->units[0], bars->units[1]);
        if (units > 0)
          ptx::mbar_drain(ptx::smem_u32(&bars->q_full), (uint32_t)((units - 1) & 1), kDefaultWaitCycles);
      }
    } else if (lane == 0 && warp - kIssueWarp < pipes) {
      // ---------------------------------------------------------------- MMAs
      const int a = warp - kIssueWarp;
      const uint64_t dq = ptx::sdesc_sw128(ptx::smem_u32(qbuf) + a * kHalves * kHalfBytes, 16, 1024);
      const uint64_t dk0 = ptx::sdesc_sw128(ptx::smem_u32(stages), 16, 1024);
      const uint64_t dv0 = ptx::sdesc_sw128(ptx::smem_u32(stages), kHalfBytes, 1024);
      const uint32_t id_qk = ptx::idesc_bf16_f32(128, kKeys, false, false);
      const uint32_t id_pv = ptx::idesc_bf16_f32(128, D, false, true);
      const uint32_t scol = tmem + a * kKeys, ocol = tmem + kOCol + a * 128;
      int64_t st = 0;
      int seg = 0;
      int64_t t = 0;  // tiles that this pipeline has run
      for (Walk w(x0, x1, plan); w.more(); w.next()) {
        const int kt = w.kt;
        const bool first = w.first(), last = w.last();
        const bool mine = a == 0 || (int64_t)w.tile * kUnitRows + kTileRows < rows;
        if (first) {
          if (!ptx::mbar_wait_t<kShort>(ptx::smem_u32(&bars->q_full), (uint32_t)(seg & 1), abort, wait))
            break;
          ++seg;
        }
        const int ks = (int)(st % kStages), vs = (int)((st + 1) % kStages);
        const uint32_t kph = (uint32_t)((st / kStages) & 1), vph = (uint32_t)(((st + 1) / kStages) & 1);
        st += 2;
        if (!ptx::mbar_wait_t<kShort>(ptx::smem_u32(&bars->full[ks]), kph, abort, wait)) break;
        if (!mine) {  // no rows of this unit in the tile
          ptx::mbar_arrive(ptx::smem_u32(&bars->empty[ks]));
          if (last) ptx::mbar_arrive(ptx::smem_u32(&bars->q_empty));
          if (!ptx::mbar_wait_t<kShort>(ptx::smem_u32(&bars->full[vs]), vph, abort, wait)) break;
          ptx::mbar_arrive(ptx::smem_u32(&bars->empty[vs]));
          continue;
        }
        const int np = min(kPages, prefix_len / kBlock - kt * kPages);
        const uint32_t idqk = np == kPages ? id_qk : ptx::idesc_bf16_f32(128, np * kBlock, false, false);
        ptx::fence_proxy_async_smem();  // the copies' writes, for the tensor cores
        ptx::tc_fence_after();
        const uint64_t dk = dk0 + (uint64_t)((ks * S::kStageBytes) >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t o = (uint64_t)(((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4);
          ptx::mma_ss(scol, dq + o, dk + o, idqk, k > 0 ? 1u : 0u);
        }
        ptx::mma_commit(ptx::smem_u32(&bars->s_full[a]));
        ptx::mma_commit(ptx::smem_u32(&bars->empty[ks]));
        if (last) ptx::mma_commit(ptx::smem_u32(&bars->q_empty));
        if (!ptx::mbar_wait_t<kShort>(ptx::smem_u32(&bars->full[vs]), vph, abort, wait)) break;
        ptx::fence_proxy_async_smem();
        const uint64_t dv = dv0 + (uint64_t)((vs * S::kStageBytes) >> 4);
        bool ok = true;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          ok = ptx::mbar_wait_t<kShort>(ptx::smem_u32(&bars->p_half[a][hf]), (uint32_t)(t & 1), abort,
                                        wait);
          if (!ok) break;
          ptx::tc_fence_after();
#pragma unroll
          for (int j = hf * 4; j < hf * 4 + 4; ++j)
            if (j < np)
              ptx::mma_ts(ocol, scol + j * 8, dv + (uint64_t)((j * 2 * 1024) >> 4), id_pv,
                          (first && j == 0) ? 0u : 1u);
        }
        if (!ok) break;
        ptx::mma_commit(ptx::smem_u32(&bars->o_done[a]));
        ptx::mma_commit(ptx::smem_u32(&bars->empty[vs]));
        if (!ptx::mbar_wait_t<kShort>(ptx::smem_u32(&bars->o_done[a]), (uint32_t)(t & 1), abort, wait))
          break;
        ++t;
      }
      // all MMAs of this thread complete before TMEM is released
      ptx::mma_commit(ptx::smem_u32(&bars->drain[a]));
      ptx::mbar_drain(ptx::smem_u32(&bars->drain[a]), 0, kDefaultWaitCycles);
    }
  } else {
    // --------------------------------------------------------------- softmax
    const int a = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t scol = lane_base + a * kKeys, ocol = lane_base + kOCol + a * 128;
    const unsigned long long qs2 = pack2(__float_as_uint(qscale2), __float_as_uint(qscale2));
    float m = -INFINITY, l = 0.f;
    int64_t t = 0;
    for (Walk w(x0, x1, plan); w.more() && a < pipes; w.next()) {
      const int kt = w.kt;
      const bool first = w.first(), last = w.last();
      const int64_t gr = (int64_t)w.tile * kUnitRows + a * kTileRows + row;
      if (gr - row >= rows) continue;  // no rows of this unit in the tile
      if (!__all_sync(0xffffffffu, ptx::mbar_wait_t<kShort>(ptx::smem_u32(&bars->s_full[a]),
                                                            (uint32_t)(t & 1), abort, wait)))
        break;
      ptx::tc_fence_after();
      const int nk = min(kKeys, prefix_len - kt * kKeys);
      uint32_t s[2][32];  // 64 scores of the row
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      auto load = [&](int hf) {
        ptx::tmem_ld32(scol + hf * 64, s[0]);
        ptx::tmem_ld32(scol + hf * 64 + 32, s[1]);
        ptx::tmem_wait_ld();
        if (nk < kKeys) {  // columns that the product did not write
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (hf * 64 + k * 32 + j >= nk) s[k][j] = 0xff800000u;
        }
      };
#pragma unroll
      for (int hf = 1; hf >= 0; --hf) {
        load(hf);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < 32; j += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mx[e] = fmaxf(fmaxf(mx[e], __uint_as_float(s[k][j + e])), __uint_as_float(s[k][j + e + 4]));
      }
      const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * qscale2;
      if (first) {
        m = mt;
        l = 0.f;
      } else {
        const bool need = mt > m + 8.0f;
        if (__any_sync(0xffffffffu, need)) {
          const float f = need ? exp2f(m - mt) : 1.f;
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            ptx::tmem_ld32(ocol + cc * 32, o);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            ptx::tmem_st32(ocol + cc * 32, o);
          }
          ptx::tmem_wait_st();
          if (need) {
            l *= f;
            m = mt;
          }
        }
      }
      const unsigned long long nm2 = pack2(__float_as_uint(-m), __float_as_uint(-m));
      unsigned long long sum[2] = {0ull, 0ull};
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if (hf == 1) load(1);  // again: 128 scores do not fit the registers
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const unsigned long long e =
                fma2(pack2(s[k][2 * j], s[k][2 * j + 1]), qs2, nm2);
            const float pa = fast_exp2(lo_of(e)), pb = fast_exp2(hi_of(e));
            sum[j & 1] = add2(sum[j & 1], pack2(__float_as_uint(pa), __float_as_uint(pb)));
            pk[j] = ptx::pack_bf16x2(pa, pb);
          }
          ptx::tmem_st16(scol + hf * 32 + k * 16, pk);
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars->p_half[a][hf]));
      }
      const unsigned long long both = add2(sum[0], sum[1]);
      l += lo_of(both) + hi_of(both);
      if (last) {
        if (!__all_sync(0xffffffffu, ptx::mbar_wait_t<kShort>(ptx::smem_u32(&bars->o_done[a]),
                                                              (uint32_t)(t & 1), abort, wait)))
          break;
        ptx::tc_fence_after();
        constexpr int stride = tc_part_stride(D);
        float* prow = part + ((w.unit + c) * plan.tile + a * kTileRows + row) * (int64_t)stride;
        const float inv = 1.f / l;
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          ptx::tmem_ld32(ocol + cc * 32, o);
          ptx::tmem_wait_ld();
          if (gr < rows) {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<float4*>(prow + cc * 32 + j) = make_float4(
                  __uint_as_float(o[j]) * inv, __uint_as_float(o[j + 1]) * inv,
                  __uint_as_float(o[j + 2]) * inv, __uint_as_float(o[j + 3]) * inv);
          }
        }
        if (gr < rows) prow[D] = m + log2f(l);
        ptx::tc_fence_before();
      }
      ++t;
    }
  }

  __syncthreads();
  if (tid == 0 && *abort) raise_status(status, SPEC_ERR_TIMEOUT);
  if (warp == kCopyWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace pfx

bool prefix_tc_ok(const spec_dims& d) {
  return d.kv_dtype == SPEC_BF16 && (d.D == 64 || d.D == 128) &&
         (int64_t)d.B * d.M * d.Hq < INT32_MAX;
}

size_t prefix_tc_part_floats(const spec_dims& d) {
  const int64_t rows = (int64_t)d.B * (d.Hq / d.Hkv) * d.M;
  const int64_t units = (int64_t)d.Hkv * ceil_div64(rows, pfx::kUnitRows);
  return (size_t)(units + kMaxPrefixCtas) * (size_t)(rows < pfx::kUnitRows ? rows : pfx::kUnitRows) *
         tc_part_stride(d.D);
}

cudaError_t prefix_tc_launch(const AttnArgs& a, float* part, uint32_t* status, cudaStream_t st,
                             PrefixPlan* plan) {
  using namespace pfx;
  const spec_dims& d = a.d;
  const int64_t rows = (int64_t)d.B * (d.Hq / d.Hkv) * d.M;
  PrefixPlan p;
  p.tile = (int)(rows < kUnitRows ? rows : kUnitRows);
  p.tiles = (int)ceil_div64(rows, kUnitRows);
  p.key_tiles = ceil_div(a.view.prefix_len, kKeys);
  p.splits = 0;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)d.Hkv * p.tiles * p.key_tiles;
  int64_t G = sms < kMaxPrefixCtas ? sms : kMaxPrefixCtas;
  if (G > items) G = items;
  p.ctas = (int)G;
  *plan = p;
  const bool short_wait = wait_limit_cycles(d) < ptx::kShortWait;
  auto kern = d.D == 64 ? (short_wait ? prefix_tc_kernel<64, true> : prefix_tc_kernel<64, false>)
                        : (short_wait ? prefix_tc_kernel<128, true> : prefix_tc_kernel<128, false>);
  const size_t smem = d.D == 64 ? Shape<64>::kSmem : Shape<128>::kSmem;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  PdlLaunch L(dim3(p.ctas), dim3(kThreads), smem, st);
  return cudaLaunchKernelEx(&L.cfg, kern, static_cast<const __nv_bfloat16*>(a.q),
                            static_cast<const __nv_bfloat16*>(a.k_cache),
                            static_cast<const __nv_bfloat16*>(a.v_cache), a.view.prefix_table,
                            a.view.prefix_len, d, a.scale * 1.4426950408889634f, p, part, status);
}

}  // namespace specv
