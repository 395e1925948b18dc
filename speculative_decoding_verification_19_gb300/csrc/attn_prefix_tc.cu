// A shared prefix on the 5th-generation tensor cores (tcgen05 + TMEM).
//
// All rows of the batch that read a KV head meet the same keys, so the work is
// two plain products with a softmax between them: 4 rows keys D operations for
// 4 keys D bytes.  From some 290 rows on it is bound by the tensor cores,
// below by the read of the keys and values.
//
// A CTA runs units of 256 rows (two MMA tiles A and B of 128) of a KV head over
// tiles of 80 keys; all (head, unit, key tile) items in that order are shared
// evenly among one CTA per SM, so a unit may be split over CTAs: each leaves a
// partial (normalised output and log2-sum-exp of its keys) for the merge.
//
//   warps 0..3, 4..7  softmax of A, of B: a thread per row (TMEM lane), its 80
//                     scores in registers, P written to TMEM as bf16
//   warps 8, 9        issue S = Q K^T of A, of B as soon as the softmax has read the
//                     last S
//   warps 10, 11      issue O += P V of A, of B when P is there (a warp each: a
//                     wait and a batch of MMAs with its commits take an issuer
//                     some 900 cycles, and one warp for all S took 2300 a tile)
//   warps 12, 13      copy: Q rows, and the pages' keys and values by 16-byte
//                     cp.async into a ring of eight 20 KB stages, K and V in
//                     turn, in the 128-byte-swizzled layout of the operands
//
// Why 80 keys.  TMEM has 512 columns; the two O take 256, and with S and P in
// places of their own (80 + 40 columns each) the next tile's S is computed while
// the softmax works on this one.  With tiles of 128 keys P has to go over S: S,
// softmax, P V and the next S follow one another, and a tile took 3700 to 4700
// cycles (A and B half a tile apart, or in step), where the tensor cores need
// 2048.  80 keys cost the products of S 51 cycles instead of 40 each (both
// operands come from shared memory, 128 bytes a cycle).
//
// 64 requests of 5 rows, 64/8 heads, behind 32768 positions: 268 us, 1.28
// PFLOP/s, 0.66 of the measured bf16 rate; a tile of 80 keys takes some 2150 cycles
// of which the tensor cores work 1456.  Bound by the softmax' chain (loads of S 240
// cycles, exponentials 1000, P's store 400, the next S 400) at two softmax warps a
// scheduler.
//
// O is rescaled in TMEM by the softmax threads only when a row's maximum grows by
// more than 2^8.
//
// Rounding.  Scores, maxima, sums and O are fp32.  The probabilities are rounded to
// bf16 for P V, as in attn_tc.cu, and the sums take them unrounded: an output is off
// by 0.0023 of its size (2-norm) against fp64, where probabilities of twice the bits
// leave 0.0017, the output's own rounding.  Those take a second product with what
// the rounding leaves, and as many columns again, so tiles of 64 keys.  us for the
// call with two products / with one in tiles of 64 keys / as it is: 64 chains of 5,
// 64/8 heads, behind 32768 positions 409 / 357 / 344; 16 of them behind 8192 67 / 62 /
// 62; 64 of them with heads of 64 behind 8192 128 / 112 / 108.
//
// TMEM: O_A [0, 128), O_B [128, 256), S_A [256, 336), S_B [336, 416), P_A [416,
// 456), P_B [464, 504).
#include <math.h>

#include "attn.cuh"
#include "common.cuh"
#include "tc_ptx.cuh"

namespace specv {
namespace pfx {

constexpr int kKeys = 80;
constexpr int kPages = kKeys / kBlock;  // 5
constexpr int kTileRows = 128;          // rows of an MMA tile; two make a unit
constexpr int kUnitRows = 2 * kTileRows;
constexpr int kStages = 8;
constexpr int kThreads = 512;  // warps 14 and 15 only make up a group of four
constexpr int kScoreWarp = 8;   // and 9: issue S of A, of B
constexpr int kValueWarp = 10;  // and 11: issue P V
constexpr int kCopyWarp = 12;   // and 13
constexpr int kCopyThreads = 64;
constexpr int kQHalfBytes = kTileRows * 128;  // 64 columns of 128 rows
constexpr int kHalfBytes = kKeys * 128;       // of 80 keys
constexpr int kTmemCols = 512;
constexpr int kSCol = 256, kPCol = 416, kPStep = 48;
// Registers: 512 threads start with 128 each; the softmax warps take 168, the
// others keep 88 (256 * 168 + 256 * 88 = 65536, all of them).

struct __align__(8) Bars {
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t q_full, q_empty;
  uint64_t s_full[2];
  uint64_t s_read[2];
  uint64_t p_full[2];
  uint64_t o_done[2];
  uint64_t drain[4];
  uint32_t tmem_base;
  int abort;
  int issued[2];  // stages that each copy warp issued
  int units[2];   // units whose queries it issued
};

// A place in the ring and the parity of its round.
struct Place {
  int at = 0;
  uint32_t round = 0;
  __device__ void next() {
    if (++at == kStages) {
      at = 0;
      round ^= 1u;
    }
  }
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
  static constexpr int kQBytes = 2 * kHalves * kQHalfBytes;
  static constexpr size_t kSmem = (size_t)kStages * kStageBytes + kQBytes + sizeof(Bars) + 1024;
};

__device__ __forceinline__ unsigned long long pack2(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(unsigned long long x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// fast_exp2 where it stands (volatile): the order of the softmax is the source's.
__device__ __forceinline__ float exp2_now(float x) {
  float y;
  asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Scores from the n-th on to -inf.
template <int N>
__device__ __forceinline__ void hide(uint32_t (&x)[N], int n) {
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (j >= n) x[j] = 0xff800000u;
}

__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(1000u)
      : "memory");
  return ok != 0;
}
// Waits for the phase of `parity`, with ptx::mbar_wait's rules for giving up; a poll
// suspends the warp for up to a microsecond.  (No function call: that and
// setmaxnreg do not go together.)
template <bool kShort>
__device__ __forceinline__ bool await(const uint64_t* bar, uint32_t parity, volatile int* abort,
                                      uint64_t timeout_cycles) {
  const uint32_t at = ptx::smem_u32(bar);
  if (!kShort && try_wait(at, parity)) return true;
  const long long t0 = clock64();
  for (uint32_t it = 1;; ++it) {
    if (kShort ? ptx::mbar_test_wait(at, parity) : try_wait(at, parity)) return true;
    if ((it & 15u) != 0) continue;
    if (*abort) return false;
    if ((uint64_t)(clock64() - t0) > timeout_cycles) {
      *abort = 1;
      return false;
    }
  }
}
// The same by a whole warp, which goes on converged.
template <bool kShort>
__device__ __forceinline__ bool await_all(const uint64_t* bar, uint32_t parity, volatile int* abort,
                                          uint64_t timeout_cycles) {
  return __all_sync(0xffffffffu, await<kShort>(bar, parity, abort, timeout_cycles));
}
__device__ __forceinline__ void drain(const uint64_t* bar, uint32_t parity) {
  int never = 0;  // the work lands whatever the caller's limit is
  await<false>(bar, parity, &never, kDefaultWaitCycles);
}

// One thread of a converged warp, the same every time.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}

// kShort: the wait limit is short.
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
  pdl_trigger();

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bars->full[s]), kCopyThreads);
      ptx::mbar_init(ptx::smem_u32(&bars->empty[s]), 2);
    }
    ptx::mbar_init(ptx::smem_u32(&bars->q_full), kCopyThreads);
    ptx::mbar_init(ptx::smem_u32(&bars->q_empty), 2);
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(ptx::smem_u32(&bars->s_full[a]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->s_read[a]), 4);
      ptx::mbar_init(ptx::smem_u32(&bars->p_full[a]), 4);
      ptx::mbar_init(ptx::smem_u32(&bars->o_done[a]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->drain[a]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->drain[2 + a]), 1);
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

  if (warp >= kScoreWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp >= kCopyWarp + 2) {
      // no part
    } else if (warp >= kCopyWarp) {
      // ------------------------------------------------------------- copies
      const int ct = (warp - kCopyWarp) * kWarp + lane;  // copy thread 0..63
      const int c16 = ct % (8 * kHalves);                // 16-byte chunk of a row
      const int r0 = ct / (8 * kHalves);
      constexpr int kRowStep = kCopyThreads / (8 * kHalves);
      const uint32_t swz_half = (uint32_t)(c16 >> 3) * kHalfBytes;
      Place pl;     // K and V of a tile in turn
      int st = 0;   // stages issued
      int seg = 0;
      // lane j has the block of page j of the tile, and of the next one
      auto block_of = [&](int kt) {
        const int p = kt * kPages + lane;
        const int id = lane < kPages && p * kBlock < prefix_len ? __ldcg(table + p) : 0;
        // no block id: the request check fails every request
        return (uint32_t)id < (uint32_t)d.num_blocks ? id : 0;
      };
      int next_id = 0;
      bool ok = true;
      for (Walk w(x0, x1, plan); w.more() && ok; w.next()) {
        const int kt = w.kt, h = w.h;
        if (w.first()) {
          // the unit's queries, when the last unit's products are done: 128 rows
          // a warp, a lane finds the place of a row for all
          ok = await<kShort>(&bars->q_empty, (uint32_t)((seg & 1) ^ 1),
                                        abort, wait);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const int64_t row0 = (int64_t)w.tile * kUnitRows + (warp - kCopyWarp) * kTileRows;
          const uint32_t qb = ptx::smem_u32(qbuf) + (warp - kCopyWarp) * kHalves * kQHalfBytes +
                              (uint32_t)(c16 >> 3) * kQHalfBytes;
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
        const int id = w.x == x0 ? block_of(kt) : next_id;
        next_id = block_of(kt + 1 < w.nt ? kt + 1 : 0);
        const int np = min(kPages, prefix_len / kBlock - kt * kPages);
        int64_t blk[kPages];
#pragma unroll
        for (int p = 0; p < kPages; ++p)
          blk[p] = ((int64_t)__shfl_sync(0xffffffffu, id, p) * Hkv + h) * kBlock;
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++st, pl.next()) {
          const int sl = pl.at;
          ok = await<kShort>(&bars->empty[sl], pl.round ^ 1u, abort, wait);
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
        bars->issued[warp - kCopyWarp] = st;
        bars->units[warp - kCopyWarp] = seg;
      }
      asm volatile("bar.sync 2, 64;" ::: "memory");
      if (ct == 0) {
        const int both = min(bars->issued[0], bars->issued[1]);
        for (int u = both > kStages ? both - kStages : 0; u < both; ++u)
          drain(&bars->full[u % kStages], (uint32_t)((u / kStages) & 1));
        const int units = min(bars->units[0], bars->units[1]);
        if (units > 0)
          drain(&bars->q_full, (uint32_t)((units - 1) & 1));
      }
    } else {
      // ---------------------------------------------------------------- MMAs
      // Whole warps walk, one thread issues.
      const bool scores = warp < kValueWarp;
      const int a = warp & 1;
      const uint64_t dq =
          ptx::sdesc_sw128(ptx::smem_u32(qbuf) + a * kHalves * kQHalfBytes, 16, 1024);
      const uint64_t dk0 = ptx::sdesc_sw128(ptx::smem_u32(stages), 16, 1024);
      const uint64_t dv0 = ptx::sdesc_sw128(ptx::smem_u32(stages), kHalfBytes, 1024);
      const uint32_t id_qk = ptx::idesc_bf16_f32(128, kKeys, false, false);
      const uint32_t id_pv = ptx::idesc_bf16_f32(128, D, false, true);
      const uint32_t scol = tmem + kSCol + a * kKeys, pcol = tmem + kPCol + a * kPStep;
      Place pl;
      int seg = 0;
      uint32_t t = 0;  // tiles run
      bool ok = true;
      for (Walk w(x0, x1, plan); ok && w.more(); w.next()) {
        const int np = min(kPages, prefix_len / kBlock - w.kt * kPages);
        const bool first = w.first(), last = w.last();
        const bool mine = a == 0 || (int64_t)w.tile * kUnitRows + kTileRows < rows;
        if (!scores) pl.next();
        const int sl = pl.at;
        if (scores && first) ok = await_all<kShort>(&bars->q_full, (uint32_t)(seg++ & 1), abort, wait);
        if (ok) ok = await_all<kShort>(&bars->full[sl], pl.round, abort, wait);
        if (!ok) break;
        pl.next();
        if (scores) pl.next();
        if (!mine) {  // B has no rows of the unit
          if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars->empty[sl]));
          if (lane == 0 && scores && last) ptx::mbar_arrive(ptx::smem_u32(&bars->q_empty));
          continue;
        }
        ptx::fence_proxy_async_smem();  // the copies' writes, for the tensor cores
        if (scores) {
          const uint32_t idqk = np == kPages ? id_qk : ptx::idesc_bf16_f32(128, np * kBlock, false, false);
          const uint64_t dk = dk0 + (uint64_t)((sl * S::kStageBytes) >> 4);
          if (t > 0) ok = await_all<kShort>(&bars->s_read[a], (t - 1) & 1u, abort, wait);
          if (!ok) break;
          ptx::tc_fence_after();
          if (elected()) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              ptx::mma_ss(scol, dq + (uint64_t)(((k >> 2) * kQHalfBytes + (k & 3) * 32) >> 4),
                          dk + (uint64_t)(((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4), idqk,
                          k > 0 ? 1u : 0u);
            ptx::mma_commit(ptx::smem_u32(&bars->s_full[a]));
            ptx::mma_commit(ptx::smem_u32(&bars->empty[sl]));
            if (last) ptx::mma_commit(ptx::smem_u32(&bars->q_empty));
          }
        } else {
          const uint64_t dv = dv0 + (uint64_t)((sl * S::kStageBytes) >> 4);
          ok = await_all<kShort>(&bars->p_full[a], t & 1u, abort, wait);
          if (!ok) break;
          ptx::tc_fence_after();
          if (elected()) {
#pragma unroll
            for (int j = 0; j < kPages; ++j)
              if (j < np)
                ptx::mma_ts(tmem + a * 128, pcol + j * 8, dv + (uint64_t)((j * 2 * 1024) >> 4), id_pv,
                            (first && j == 0) ? 0u : 1u);
            ptx::mma_commit(ptx::smem_u32(&bars->o_done[a]));
            ptx::mma_commit(ptx::smem_u32(&bars->empty[sl]));
          }
        }
        __syncwarp();
        ++t;
      }
      // all MMAs of this warp complete before TMEM is released
      __syncwarp();
      if (elected()) ptx::mma_commit(ptx::smem_u32(&bars->drain[warp - kScoreWarp]));
      drain(&bars->drain[warp - kScoreWarp], 0);
    }
  } else {
    // --------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    const int a = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t scol = lane_base + kSCol + a * kKeys, pcol = lane_base + kPCol + a * kPStep;
    const uint32_t ocol = lane_base + a * 128;
    const unsigned long long qs2 = pack2(qscale2, qscale2);
    float m = -INFINITY, l = 0.f;
    uint32_t t = 0;
    for (Walk w(x0, x1, plan); w.more(); w.next()) {
      const bool first = w.first(), last = w.last();
      const int64_t gr = (int64_t)w.tile * kUnitRows + a * kTileRows + row;
      if (gr - row >= rows) continue;  // no rows of this unit in the tile
      if (!await_all<kShort>(&bars->s_full[a], t & 1u, abort, wait)) break;
      ptx::tc_fence_after();
      uint32_t s[2][32], s2[16];
      ptx::tmem_ld32(scol, s[0]);
      ptx::tmem_ld32(scol + 32, s[1]);
      ptx::tmem_ld16(scol + 64, s2);
      ptx::tmem_wait_ld(s[0]);
      ptx::tmem_wait_ld(s[1]);
      ptx::tmem_wait_ld(s2);
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars->s_read[a]));
      const int nk = min(kKeys, prefix_len - w.kt * kKeys);
      if (nk < kKeys) {  // columns that the product did not write
        hide(s[0], nk);
        hide(s[1], nk - 32);
        hide(s2, nk - 64);
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < 32; ++j)
        mx[j & 3] = fmaxf(fmaxf(mx[j & 3], __uint_as_float(s[0][j])), __uint_as_float(s[1][j]));
#pragma unroll
      for (int j = 0; j < 8; ++j)
        mx[j & 3] = fmaxf(fmaxf(mx[j & 3], __uint_as_float(s2[j])), __uint_as_float(s2[j + 8]));
      const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * qscale2;
      // P and O are free when the last tile's P V is done
      bool done = first;
      if (first) {
        m = mt;
        l = 0.f;
      } else {
        const bool need = mt > m + 8.0f;
        if (__any_sync(0xffffffffu, need)) {
          if (!await_all<kShort>(&bars->o_done[a], (t - 1) & 1u, abort, wait)) break;
          done = true;
          ptx::tc_fence_after();
          const float f = need ? exp2f(m - mt) : 1.f;
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            ptx::tmem_ld32(ocol + cc * 32, o);
            ptx::tmem_wait_ld(o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            ptx::tmem_st32(ocol + cc * 32, o);
          }
          if (need) {
            l *= f;
            m = mt;
          }
        }
      }
      const unsigned long long nm2 = pack2(-m, -m);
      unsigned long long sum[2] = {0ull, 0ull};
      // eight pairs at a time, each instruction for all of them before the next
      auto exps = [&](const uint32_t* x, uint32_t* out) {
        unsigned long long e[8];
        float f[16];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          e[j] = fma2(pack2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), qs2, nm2);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          unpack2(e[j], f[2 * j], f[2 * j + 1]);
          f[2 * j] = exp2_now(f[2 * j]);
          f[2 * j + 1] = exp2_now(f[2 * j + 1]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          sum[j & 1] = add2(sum[j & 1], pack2(f[2 * j], f[2 * j + 1]));
          out[j] = ptx::pack_bf16x2(f[2 * j], f[2 * j + 1]);
        }
      };
      uint32_t pk[32], pk2[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) exps(&s[j >> 1][16 * (j & 1)], &pk[8 * j]);
      exps(s2, pk2);
      if (!done) {
        if (!await_all<kShort>(&bars->o_done[a], (t - 1) & 1u, abort, wait)) break;
        ptx::tc_fence_after();
      }
      ptx::tmem_st32(pcol, pk);
      ptx::tmem_st8(pcol + 32, pk2);
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars->p_full[a]));
      float la, lb;
      unpack2(add2(sum[0], sum[1]), la, lb);
      l += la + lb;
      if (last) {
        if (!await_all<kShort>(&bars->o_done[a], t & 1u, abort, wait))
          break;
        ptx::tc_fence_after();
        constexpr int stride = tc_part_stride(D);
        float* prow = part + ((w.unit + c) * plan.tile + a * kTileRows + row) * (int64_t)stride;
        const float inv = 1.f / l;
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          ptx::tmem_ld32(ocol + cc * 32, o);
          ptx::tmem_wait_ld(o);
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
