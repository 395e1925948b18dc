// Block tables, slot map and positions of a step's new rows, from the
// requests' lengths (page 2 §4.3 and page 3: the cache is paged, a block table
// maps a request's positions to blocks; page 2 §3.3: a rollback frees what lies
// past the accepted prefix).
//
// What is computed, for request b with c cached tokens and n new rows, pages
// of 16 positions, a window of W tokens and S sink tokens (sp = ceil(S/16)
// pages):
//   hi' = ceil((c + n) / 16),  lo' = max(0, c - W + 1) / 16  (0 without a window)
//   wanted(p) = p < hi' and (p < sp or p >= lo')
//   held(p)   = p < hi  and (p < sp or p >= lo)      (lo, hi: the span kept)
// Pages held and not wanted go to the tail of the ring of free pages, pages
// wanted and not held come from its head, both in (request, page) order.  As
// lo <= lo', what is taken is at most two runs of pages and what is given
// back at most three, so a request's counts are interval arithmetic and a
// page's rank inside its request is too; ranks across requests are prefix
// sums.
//
// The ring makes one pass enough: a call takes ids from [head, head + count)
// and writes ids to [head + count, ..), which never overlap, so no CTA waits
// for another's writes (a stack would pop entries that the same call pushes).
// Pages given back are free from the next call on.
//
// The work is a few bytes per row and page; what bounds it is latency: one
// dependent chain of lengths -> prefix sums -> table or ring entry -> slot.
// So it is one launch.  Every CTA repeats the prefix sums over all requests
// (512 at a time, one per thread: 20 bytes a request, from L2 after the
// first CTA) and then does its share of the items: pages given back, pages
// taken, rows.  Spans, ring state and verdicts are written by the CTA that
// arrives last, when every CTA has read the old ones.
//
// An entry of a table or of the ring that is no block id (a corrupt state) must
// not reach another request.  A CTA that meets one says so with its arrival, and
// only then does the last CTA look through the pages that the requests take or
// write, refuse the requests with such a page, and close the gaps among the ids
// given back; a sound state pays for nothing but the flag.
#include "block_tables.cuh"

namespace specv {
namespace pages {

constexpr int kThreads = 512;  // also the requests of one round
constexpr int kWarps = kThreads / kWarp;
constexpr int kMaxCtas = 152;
// Items of one CTA when the call has more than that (host rule): below it the
// launch is one CTA, which needs no arrival count.  One item a thread: 65541
// rows of 512 requests take 7.6 us so, 11.2 us with four (2048 items a CTA).
constexpr int kItemsPerCta = kThreads;

struct Shared {
  // exclusive prefixes over the round's requests, relative to its first
  int take_pre[kThreads + 1];
  int give_pre[kThreads + 1];
  int row0[kThreads + 1];  // first row of each request
  int ctx[kThreads];
  int lo[kThreads], hi[kThreads], lo2[kThreads], hi2[kThreads];
  // 2: rows get slots, 1: a request without rows to serve, 0: unchanged; 3: of
  // the first kind, but one of its pages is no block
  int good[kThreads];
  int64_t warp_need[kWarps];
  int warp_give[kWarps], warp_take[kWarps];
  int last;
  int corrupt;  // an entry that is no block id was met
};

// What the rounds carry from request to request.
struct Carry {
  int64_t need;  // pages asked for, by requests that failed too
  int take, give;
};

__device__ __forceinline__ int pos_part(int x) { return x > 0 ? x : 0; }

// Pages of [hi, hi2) a request takes: [hi, min(sp, hi2)) and
// [max(hi, lo2, sp), hi2).
__device__ __forceinline__ int take_low(int hi, int hi2, int sp) { return pos_part(min(sp, hi2) - hi); }
__device__ __forceinline__ int take_from(int hi, int lo2, int sp) { return max(hi, max(lo2, sp)); }

// Rows [r0, r1) that cannot be a request's.
__device__ __forceinline__ bool bad_rows(int r0, int r1, int rows) {
  return r0 < 0 || r1 < r0 || r1 > rows;
}

// One round: the records and prefixes of requests base .. base + 511.  rows_ok:
// row_start ascends within the rows (found here when the round is the only one).
__device__ void plan_round(Shared& sh, const PageArgs& a, int base, int sp, bool pool_ok, int count,
                           bool& rows_ok, Carry& carry, uint32_t* status, bool report) {
  const int tid = threadIdx.x, lane = tid % kWarp, warp = tid / kWarp;
  const int B = a.d.B, M = a.d.M, mb = a.d.max_blocks;
  const int b = base + tid;
  int ctx = -1, r0 = 0, r1 = 0, lo = 0, hi = 0, lo2 = 0, hi2 = 0, good = 0, take = 0, give = 0;
  int64_t need = 0;
  if (b < B) {
    ctx = a.ctx_lens[b];
    lo = a.span[2 * (int64_t)b];
    hi = a.span[2 * (int64_t)b + 1];
    if (a.row_start != nullptr) {
      r0 = a.row_start[b];
      r1 = a.row_start[b + 1];
    } else {
      r0 = b * M;
      r1 = r0 + M;
    }
  }
  if (a.row_start != nullptr && B <= kThreads)
    rows_ok = !__syncthreads_or(b < B && bad_rows(r0, r1, a.rows));
  if (b < B) {
    int code = 0;
    if (!pool_ok || lo < 0 || lo > hi || hi > mb) code = SPEC_ERR_DEVICE_BOUNDS;
    else if (ctx < -1 || !rows_ok) code = SPEC_ERR_INVALID_ARG;
    if (a.parent != nullptr && ctx >= 0) {
      const int32_t* par = a.parent + (int64_t)b * M;
      bool bad = par[0] != -1;
      for (int n = 1; n < M; ++n) {
        const int p = par[n];
        bad |= p < 0 || p >= n;
      }
      if (bad) code = SPEC_ERR_INVALID_ARG;
    }
    if (code == 0 && ctx >= 0) {
      const int64_t end = (int64_t)ctx + (r1 - r0);
      const int low = a.window > 0 ? max(0, ctx - a.window + 1) / kBlock : 0;
      if (end > (int64_t)mb * kBlock) code = SPEC_ERR_CAPACITY;
      else if (low < lo && hi > 0) code = SPEC_ERR_INVALID_ARG;  // pages given back are needed again
      else {
        lo2 = low;
        hi2 = (int)ceil_div64(end, kBlock);
        good = 2;
        const int t = take_low(hi, hi2, sp) + pos_part(hi2 - take_from(hi, lo2, sp));
        need = t;
      }
    } else if (code == 0) {
      good = 1;  // ended: everything goes back
    }
    if (code != 0) {
      if (report) raise_status(status, code);
      lo2 = lo;  // unchanged
      hi2 = hi;
    }
  }
  // inclusive prefix of the pages asked for
  int64_t incl = need;
#pragma unroll
  for (int o = 1; o < kWarp; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == kWarp - 1) sh.warp_need[warp] = incl;
  __syncthreads();
  // lane w holds warp w's sum: those of the warps before, and all of them
  const int64_t wn = lane < kWarps ? sh.warp_need[lane] : 0;
  int64_t before_need = lane < warp ? wn : 0, total_need = wn;
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) {
    before_need += __shfl_xor_sync(0xffffffffu, before_need, o);
    total_need += __shfl_xor_sync(0xffffffffu, total_need, o);
  }
  incl += __shfl_sync(0xffffffffu, before_need, 0);
  total_need = __shfl_sync(0xffffffffu, total_need, 0);
  if (good == 2 && need > 0 && carry.need + incl > count) {
    if (report) raise_status(status, SPEC_ERR_CAPACITY);
    good = 1;            // gives back what it no longer needs, takes nothing
    hi2 = min(hi, hi2);
    lo2 = min(lo2, hi2);  // a span stays ordered (no page past hi2 is held)
  } else {
    take = (int)need;    // carry.need + incl <= count, an int
  }
  if (b < B) {
    // [hi2, min(sp, hi)), [max(lo, sp), min(hi, lo2)), [max(lo, sp, hi2), hi)
    const int w0 = max(lo, sp);
    give = pos_part(min(sp, hi) - hi2) + pos_part(min(hi, lo2) - w0) + pos_part(hi - max(w0, hi2));
  }
  // exclusive prefixes of what is taken and given
  int it = take, ig = give;
#pragma unroll
  for (int o = 1; o < kWarp; o <<= 1) {
    const int yt = __shfl_up_sync(0xffffffffu, it, o), yg = __shfl_up_sync(0xffffffffu, ig, o);
    if (lane >= o) {
      it += yt;
      ig += yg;
    }
  }
  if (lane == kWarp - 1) {
    sh.warp_take[warp] = it;
    sh.warp_give[warp] = ig;
  }
  __syncthreads();
  const int wt = lane < kWarps ? sh.warp_take[lane] : 0, wg = lane < kWarps ? sh.warp_give[lane] : 0;
  it += __reduce_add_sync(0xffffffffu, lane < warp ? wt : 0);
  ig += __reduce_add_sync(0xffffffffu, lane < warp ? wg : 0);
  const int tt = __reduce_add_sync(0xffffffffu, wt), tg = __reduce_add_sync(0xffffffffu, wg);
  sh.take_pre[tid] = it - take;
  sh.give_pre[tid] = ig - give;
  const int n = min(kThreads, B - base);
  if (tid < n) sh.row0[tid] = r0;
  if (tid == n - 1) sh.row0[n] = r1;
  sh.ctx[tid] = ctx;
  sh.lo[tid] = lo;
  sh.hi[tid] = hi;
  sh.lo2[tid] = lo2;
  sh.hi2[tid] = hi2;
  sh.good[tid] = good;
  if (tid == 0) {
    sh.take_pre[kThreads] = tt;
    sh.give_pre[kThreads] = tg;
  }
  __syncthreads();
  carry.need += total_need;
}

// The last request r of the round with pre[r] <= x (pre ascending).
__device__ __forceinline__ int find(const int* pre, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Whether every page that request r of the round takes, or that its rows are
// written to, is a block (the table after the call; read past L1, as other CTAs
// wrote it).
__device__ __noinline__ bool pages_sound(const Shared& sh, const PageArgs& a, int base, int r,
                                         int sp) {
  const int32_t* table = a.block_table + (int64_t)(base + r) * a.d.max_blocks;
  auto sound = [&](int p0, int p1) {
    bool good = true;
    for (int p = p0; p < p1; ++p) {
      const int id = __ldcg(table + p);
      good &= id >= 0 && id < a.d.num_blocks;
    }
    return good;
  };
  const int hi = sh.hi[r], hi2 = sh.hi2[r];
  return sound(hi, min(sp, hi2)) && sound(take_from(hi, sh.lo2[r], sp), hi2) &&
         (sh.row0[r + 1] == sh.row0[r] || sound(sh.ctx[r] / kBlock, hi2));
}

// Moves the block ids among the `given` entries behind the ring's first `count`
// together, in their order, and clears the places left over (one warp).
// Returns how many ids there are.
__device__ __noinline__ int close_gaps(int32_t* pool, int head, int count, int given, int nb) {
  const int lane = threadIdx.x % kWarp;
  const int64_t first = (int64_t)head + count;
  int kept = 0;
  for (int j0 = 0; j0 < given; j0 += kWarp) {
    const int id = j0 + lane < given ? __ldcg(pool + (first + j0 + lane) % nb) : -1;
    const bool good = id >= 0 && id < nb;
    const unsigned mask = __ballot_sync(0xffffffffu, good);  // every lane has read
    if (good) pool[(first + kept + __popc(mask & ((1u << lane) - 1))) % nb] = id;
    kept += __popc(mask);
    __syncwarp();
  }
  for (int j = kept + lane; j < given; j += kWarp) pool[(first + j) % nb] = -1;
  return kept;
}

__global__ void __launch_bounds__(kThreads) block_tables_kernel(PageArgs a, uint32_t* arrivals,
                                                                uint32_t* status) {
  __shared__ Shared sh;
  pdl_trigger();
  pdl_wait();  // lengths and page state may come from the previous kernel
  const int tid = threadIdx.x;
  const int B = a.d.B, M = a.d.M, mb = a.d.max_blocks, nb = a.d.num_blocks;
  const int sp = a.window > 0 ? ceil_div(a.sinks, kBlock) : 0;
  const int head = a.pool_state[0], count = a.pool_state[1];
  const bool pool_ok = head >= 0 && head < nb && count >= 0 && count <= nb;
  if (!pool_ok && blockIdx.x == 0 && tid == 0) raise_status(status, SPEC_ERR_DEVICE_BOUNDS);
  if (tid == 0) sh.corrupt = 0;  // plan_round's barriers stand before its uses
  auto is_block = [&](int id) {
    if (id >= 0 && id < nb) return true;
    raise_status(status, SPEC_ERR_DEVICE_BOUNDS);
    sh.corrupt = 1;
    return false;
  };
  const int gt = blockIdx.x * kThreads + tid, gn = gridDim.x * kThreads;
  bool rows_ok = true;  // one entry out of order leaves no row certain
  if (a.row_start != nullptr && B > kThreads) {
    int bad = 0;
    for (int b = tid; b < B; b += kThreads) bad |= bad_rows(a.row_start[b], a.row_start[b + 1], a.rows);
    rows_ok = !__syncthreads_or(bad);
  }
  Carry carry{0, 0, 0};
  for (int base = 0; base < B; base += kThreads) {
    plan_round(sh, a, base, sp, pool_ok, count, rows_ok, carry, status, blockIdx.x == 0);
    const int n = min(kThreads, B - base);
    const int n_take = sh.take_pre[kThreads], n_give = sh.give_pre[kThreads];
    // pages given back: to the ring's tail, their table entries cleared
    for (int j = gt; j < n_give; j += gn) {
      const int r = find(sh.give_pre, n, j);
      const int hi2 = sh.hi2[r], hi = sh.hi[r], w0 = max(sh.lo[r], sp);
      int k = j - sh.give_pre[r], p;
      const int n1 = pos_part(min(sp, hi) - hi2), n2 = pos_part(min(hi, sh.lo2[r]) - w0);
      if (k < n1) p = hi2 + k;
      else if (k < n1 + n2) p = w0 + k - n1;
      else p = max(w0, hi2) + k - n1 - n2;
      int32_t* entry = a.block_table + (int64_t)(base + r) * mb + p;
      const int id = *entry;
      const int64_t g = (int64_t)count + carry.give + j;
      if (is_block(id) && g >= nb) raise_status(status, SPEC_ERR_DEVICE_BOUNDS);
      if (g < nb) a.pool[(head + g) % nb] = id;
      *entry = -1;
    }
    // pages taken: from the ring's head, in order
    for (int j = gt; j < n_take; j += gn) {
      const int r = find(sh.take_pre, n, j);
      const int hi = sh.hi[r], low = take_low(hi, sh.hi2[r], sp);
      const int k = j - sh.take_pre[r];
      const int p = k < low ? hi + k : take_from(hi, sh.lo2[r], sp) + k - low;
      const int id = a.pool[((int64_t)head + carry.take + j) % nb];
      a.block_table[(int64_t)(base + r) * mb + p] = is_block(id) ? id : -1;
    }
    // rows: slot and position; an entry of a page taken by this call is read
    // from the ring, not from the table that another CTA may be writing
    // (row_start out of order: every row is none's)
    const int row_lo = rows_ok ? sh.row0[0] : 0;
    const int row_hi = rows_ok ? sh.row0[n] : (base == 0 ? a.rows : 0);
    for (int row = row_lo + gt; row < row_hi; row += gn) {
      const int r = !rows_ok ? 0 : a.row_start != nullptr ? find(sh.row0, n, row) : row / M - base;
      int64_t slot = -1;
      int pos = -1;
      if (sh.good[r] == 2) {
        const int i = row - sh.row0[r], t = sh.ctx[r] + i, p = t / kBlock;
        const int hi = sh.hi[r];
        int id;
        if (p < hi) {
          id = a.block_table[(int64_t)(base + r) * mb + p];
        } else {
          const int rank = p < sp ? p - hi
                                  : take_low(hi, sh.hi2[r], sp) + p - take_from(hi, sh.lo2[r], sp);
          id = a.pool[((int64_t)head + carry.take + sh.take_pre[r] + rank) % nb];
        }
        if (is_block(id)) slot = (int64_t)id * kBlock + t % kBlock;
        pos = t;
        if (a.parent != nullptr) {
          // depth: steps to the root (checked above: every step goes down)
          const int32_t* par = a.parent + (int64_t)(base + r) * M;
          int depth = 0;
          for (int k = i; k > 0; k = par[k]) ++depth;
          pos = sh.ctx[r] + depth;
        }
      }
      a.slots[row] = slot;
      a.positions[row] = pos;
    }
    carry.take += n_take;
    carry.give += n_give;
    __syncthreads();  // the round's records are read
  }
  // ---- the new page state, by the last CTA to arrive (arrivals in the lower
  // half of the word, those with a corrupt entry in the upper)
  if (gridDim.x > 1) {
    if (tid == 0) {
      __threadfence();
      const uint32_t before = atomicAdd(arrivals, sh.corrupt ? 0x10001u : 1u);
      sh.last = (before & 0xffffu) == gridDim.x - 1;
      if (before >> 16) sh.corrupt = 1;
    }
    __syncthreads();
    if (!sh.last) return;
    __threadfence();
  }
  const bool corrupt = sh.corrupt;
  Carry again{0, 0, 0};
  for (int base = 0; base < B; base += kThreads) {
    if (B > kThreads) plan_round(sh, a, base, sp, pool_ok, count, rows_ok, again, status, false);
    const int b = base + tid;
    if (corrupt) {
      const int n = min(kThreads, B - base);
      if (b < B && sh.good[tid] == 2 && !pages_sound(sh, a, base, tid, sp)) sh.good[tid] = 3;
      __syncthreads();
      for (int r = 0; r < n; ++r) {
        if (sh.good[r] != 3) continue;
        for (int row = sh.row0[r] + tid; row < sh.row0[r + 1]; row += kThreads) {
          a.slots[row] = -1;
          a.positions[row] = -1;
        }
      }
    }
    if (b < B) {
      if (a.ok != nullptr) a.ok[b] = sh.good[tid] == 2;
      a.span[2 * (int64_t)b] = sh.lo2[tid];
      a.span[2 * (int64_t)b + 1] = sh.hi2[tid];
    }
    __syncthreads();
  }
  int given = (int)min((int64_t)carry.give, (int64_t)nb - count);
  if (corrupt && pool_ok && tid < kWarp) given = close_gaps(a.pool, head, count, given, nb);
  if (tid == 0) {
    if (pool_ok) {
      a.pool_state[0] = (int)(((int64_t)head + carry.take) % nb);
      a.pool_state[1] = count + given - carry.take;
    }
    if (gridDim.x > 1) *arrivals = 0;
  }
}

}  // namespace pages

cudaError_t block_tables_launch(const PageArgs& a, const WsLayout& lay, cudaStream_t st,
                                int* launches) {
  using namespace pages;
  char* ws = static_cast<char*>(a.ws);
  // rows are counted on the host; pages are at most a table's size, and one in
  // 64 of its entries moves in an ordinary step
  const int64_t items = max((int64_t)a.rows, (int64_t)a.d.B * a.d.max_blocks / 64);
  const int G = (int)min((int64_t)kMaxCtas, max((int64_t)1, items / kItemsPerCta));
  PdlLaunch L(dim3(G), dim3(kThreads), 0, st);
  const cudaError_t e = cudaLaunchKernelEx(
      &L.cfg, block_tables_kernel, a, reinterpret_cast<uint32_t*>(ws + lay.pg_sync_off),
      reinterpret_cast<uint32_t*>(ws + lay.status_off));
  ++*launches;
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace specv
