// Which pages of a long cache a verify step reads.
//
// Page 1 §2.1 has every query see the whole context; at long contexts most of
// a softmax' mass lies in a few pages.  For a page whose keys have least and
// largest coordinates lo, hi, no query q has a score above
//   sum_d max(q_d lo_d, q_d hi_d) = q+ . hi + q- . lo,   q+ = max(q, 0), q- = min(q, 0)
// with any of its keys.  Bounds of 2 D numbers a page and KV head stand for 16
// D of keys, and the pages with the largest bounds are read.
//
//   page_bounds_kernel   lo and hi of the pages that a step has filled
//   page_score_kernel    the bound of every page, the largest over the rows
//                        that read the KV head (fp32, and more than 128 rows;
//                        bf16 goes to the tensor cores, page_score_tc.cu)
//   page_select_kernel   the first and last pages and those of largest score
#include <math.h>

#include "page_select.cuh"

namespace specv {

// ---------------------------------------------------------------------------
// bounds
// ---------------------------------------------------------------------------
__device__ __forceinline__ void widen(uint4& lo, uint4& hi, const uint4& v, float) {
  float a[4], b[4], c[4];
  unpack16(lo, a);
  unpack16(hi, b);
  unpack16(v, c);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = fminf(a[i], c[i]);
    b[i] = fmaxf(b[i], c[i]);
  }
  lo = make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(a[2]), __float_as_uint(a[3]));
  hi = make_uint4(__float_as_uint(b[0]), __float_as_uint(b[1]), __float_as_uint(b[2]), __float_as_uint(b[3]));
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void widen(uint4& lo, uint4& hi, const uint4& v, __nv_bfloat16) {
  lo = make_uint4(min2(lo.x, v.x), min2(lo.y, v.y), min2(lo.z, v.z), min2(lo.w, v.w));
  hi = make_uint4(max2(hi.x, v.x), max2(hi.y, v.y), max2(hi.z, v.z), max2(hi.w, v.w));
}
__device__ __forceinline__ uint4 shfl_xor16(const uint4& v, int m) {
  return make_uint4(__shfl_xor_sync(0xffffffffu, v.x, m), __shfl_xor_sync(0xffffffffu, v.y, m),
                    __shfl_xor_sync(0xffffffffu, v.z, m), __shfl_xor_sync(0xffffffffu, v.w, m));
}

// A warp per page and KV head: 16 rows of D keys in 16-byte vectors, minima and
// maxima in registers, then across the lanes that hold the same columns.
template <typename T, int D>
__global__ void __launch_bounds__(256) page_bounds_kernel(const T* k_cache,
                                                          const int32_t* block_table,
                                                          const int32_t* from_lens,
                                                          const int32_t* ctx_lens, spec_dims d,
                                                          T* bounds, uint32_t* status) {
  constexpr int kVecRow = D * (int)sizeof(T) / 16;  // vectors of a row: 8, 16 or 32
  constexpr int kLoads = kVecRow / 2;               // of a lane
  constexpr int kRowsPer = kWarp / kVecRow;         // rows of one load of the warp
  pdl_trigger();
  pdl_wait();  // the cache and the lengths may come from the previous kernels
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const int b = blockIdx.y;
  const int ctx = __ldcg(ctx_lens + b);
  if (ctx <= 0) return;
  const int from = from_lens != nullptr ? __ldcg(from_lens + b) : 0;
  if (from < 0 || ctx > (int64_t)d.max_blocks * kBlock) {
    if (blockIdx.x == 0 && threadIdx.x == 0)
      raise_status(status, from < 0 ? SPEC_ERR_INVALID_ARG : SPEC_ERR_CAPACITY);
    return;
  }
  const int p0 = from / kBlock, p1 = ceil_div(ctx, kBlock);
  const int64_t n = (int64_t)(p1 - p0) * d.Hkv;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x / kWarp);
  for (int64_t w = (int64_t)blockIdx.x * (blockDim.x / kWarp) + warp; w < n; w += step) {
    const int p = p0 + (int)(w / d.Hkv), h = (int)(w % d.Hkv);
    const int id = __ldcg(block_table + (int64_t)b * d.max_blocks + p);
    if (id < 0 || id >= d.num_blocks) {
      if (lane == 0) raise_status(status, SPEC_ERR_DEVICE_BOUNDS);
      continue;
    }
    const int last = min(kBlock, ctx - p * kBlock) - 1;  // rows past it repeat it
    const int64_t blk = (int64_t)id * d.Hkv + h;
    const uint4* keys = reinterpret_cast<const uint4*>(k_cache + blk * kBlock * D);
    const int r0 = lane / kVecRow, c = lane % kVecRow;
    uint4 v[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) v[i] = __ldcg(keys + min(r0 + i * kRowsPer, last) * kVecRow + c);
    uint4 lo = v[0], hi = v[0];
#pragma unroll
    for (int i = 1; i < kLoads; ++i) widen(lo, hi, v[i], T());
#pragma unroll
    for (int m = kVecRow; m < kWarp; m <<= 1) {
      const uint4 a = shfl_xor16(lo, m), e = shfl_xor16(hi, m);
      uint4 t = a;
      widen(lo, t, a, T());
      t = e;
      widen(t, hi, e, T());
    }
    uint4* dst = reinterpret_cast<uint4*>(bounds + blk * 2 * D);
    if (lane < kVecRow) dst[lane] = lo;
    if (kVecRow == kWarp) dst[kVecRow + lane] = hi;
    else if (lane >= kVecRow && lane < 2 * kVecRow) dst[lane] = hi;
  }
}

// ---------------------------------------------------------------------------
// scores
// ---------------------------------------------------------------------------
// A CTA per kTile pages of a KV head; the product q+ . hi + q- . lo in register
// tiles of RPT rows x kTile / 16 pages, the rows' maximum in registers, then across
// the eight row groups.  64 pages a CTA, or 16 where those would not fill the GPU
// twice: 11 requests of 17 rows, 4 heads of 128 fp32 values, up to 310 pages 16 us
// (25 with 64), 3 of 116 rows, one head of 64, up to 390 pages 12 us (20).
constexpr int kScoreThreads = 128;

template <int D, int RPT, int kTile>
constexpr size_t score_smem() {
  return sizeof(float) * ((size_t)2 * D * (kTile + 4) + (size_t)D * (8 * RPT + 4) + 8 * kTile);
}

template <typename T, int D, int RPT, int kTile>
__global__ void __launch_bounds__(kScoreThreads) page_score_kernel(
    const T* q, const T* bounds, const int32_t* block_table, const int32_t* ctx_lens, spec_dims d,
    float* __restrict__ scores, uint32_t* __restrict__ status) {
  constexpr int kLd = kTile + 4, kRows = 8 * RPT, kLdQ = kRows + 4, PPT = kTile / 16;
  static_assert(PPT == 4 || PPT == 1, "a thread has four pages or one");
  constexpr int kVec = 16 / sizeof(T), kVecRow = D / kVec;
  extern __shared__ __align__(16) float smem[];
  float* lo = smem;               // [D][kLd]
  float* hi = lo + D * kLd;       // [D][kLd]
  float* qs = hi + D * kLd;       // [D][kLdQ]
  float* red = qs + D * kLdQ;     // [8][kTile]
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int h = blockIdx.y, b = blockIdx.z, page0 = blockIdx.x * kTile;
  const int group = d.Hq / d.Hkv, R = group * d.M;
  pdl_trigger();
  pdl_wait();  // the queries, bounds and lengths may come from the previous kernels
  const int ctx = __ldcg(ctx_lens + b);
  const bool fits = ctx <= (int64_t)d.max_blocks * kBlock;
  const int full = fits && ctx > 0 ? ctx / kBlock : 0;
  if (!fits && page0 == 0 && h == 0 && tid == 0) raise_status(status, SPEC_ERR_CAPACITY);
  float* out = scores + ((int64_t)b * d.Hkv + h) * d.max_blocks;
  if (page0 >= full) {
    for (int p = page0 + tid; p < min(page0 + kTile, d.max_blocks); p += kScoreThreads)
      out[p] = -INFINITY;
    return;
  }
  for (int e = tid; e < kTile * 2 * kVecRow; e += kScoreThreads) {
    const int p = e % kTile, vi = e / kTile;  // vectors of lo, then of hi
    float f[kVec];
#pragma unroll
    for (int c = 0; c < kVec; ++c) f[c] = 0.f;
    if (page0 + p < full) {
      const int id = __ldcg(block_table + (int64_t)b * d.max_blocks + page0 + p);
      if (id >= 0 && id < d.num_blocks)
        unpack16(__ldcg(reinterpret_cast<const uint4*>(bounds + ((int64_t)id * d.Hkv + h) * 2 * D) + vi), f);
    }
#pragma unroll
    for (int c = 0; c < kVec; ++c) lo[(vi * kVec + c) * kLd + p] = f[c];
  }
  float best[PPT];
#pragma unroll
  for (int k = 0; k < PPT; ++k) best[k] = -INFINITY;
  for (int r0 = 0; r0 < R; r0 += kRows) {
    __syncthreads();
    for (int e = tid; e < kRows * kVecRow; e += kScoreThreads) {
      const int r = e % kRows, vi = e / kRows;
      const int rr = min(r0 + r, R - 1), i = rr / group;  // rows past the last repeat it
      float f[kVec];
      unpack16(__ldcg(reinterpret_cast<const uint4*>(
                          q + (((int64_t)b * d.M + i) * d.Hq + h * group + rr - i * group) * D) + vi), f);
#pragma unroll
      for (int c = 0; c < kVec; ++c) qs[(vi * kVec + c) * kLdQ + r] = f[c];
    }
    __syncthreads();
    float acc[RPT][PPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r)
#pragma unroll
      for (int k = 0; k < PPT; ++k) acc[r][k] = 0.f;
#pragma unroll 2
    for (int dd = 0; dd < D; ++dd) {
      float a[PPT], c[PPT];
      if constexpr (PPT == 4) {
        const float4 a4 = *reinterpret_cast<const float4*>(lo + dd * kLd + tx * 4);
        const float4 c4 = *reinterpret_cast<const float4*>(hi + dd * kLd + tx * 4);
        a[0] = a4.x; a[1] = a4.y; a[2] = a4.z; a[3] = a4.w;
        c[0] = c4.x; c[1] = c4.y; c[2] = c4.z; c[3] = c4.w;
      } else {
        a[0] = lo[dd * kLd + tx];
        c[0] = hi[dd * kLd + tx];
      }
#pragma unroll
      for (int r = 0; r < RPT; ++r) {
        const float qv = qs[dd * kLdQ + ty * RPT + r];
        const float qp = max_nan(qv, 0.f), qn = min_nan(qv, 0.f);
#pragma unroll
        for (int k = 0; k < PPT; ++k) acc[r][k] = fmaf(qp, c[k], fmaf(qn, a[k], acc[r][k]));
      }
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r)
#pragma unroll
      for (int k = 0; k < PPT; ++k) best[k] = max_nan(best[k], acc[r][k]);
  }
#pragma unroll
  for (int k = 0; k < PPT; ++k) red[ty * kTile + tx * PPT + k] = best[k];
  __syncthreads();
  if (tid < kTile && page0 + tid < d.max_blocks) {
    float m = red[tid];
#pragma unroll
    for (int k = 1; k < 8; ++k) m = max_nan(m, red[k * kTile + tid]);
    bool there = page0 + tid < full;
    if (there) {
      const int id = __ldcg(block_table + (int64_t)b * d.max_blocks + page0 + tid);
      if (id < 0 || id >= d.num_blocks) {
        there = false;
        raise_status(status, SPEC_ERR_DEVICE_BOUNDS);
      }
    }
    out[page0 + tid] = there ? m : -INFINITY;
  }
}

// ---------------------------------------------------------------------------
// selection
// ---------------------------------------------------------------------------
// A CTA per (request, KV head).  Scores become keys whose order is the scores';
// the key of the last page taken is found digit by digit from the top of the
// competing keys' range (histograms of 256 counts; the range, because scores of
// one row share their exponents), then those above it and the first of those
// equal to it are written in the pages' order.
//
// Keys stay in shared memory, so a row is read once, and all passes go over it
// with many warps an SM (keys in registers, 32 a thread: half the warps, unrolled
// code past the instruction cache, 26 to 42 us where this takes 25).
// What is left is a chain of some fifteen barriers and about 40 instructions a key, and
// with 8192 pages 42 KB a CTA, so five CTAs an SM: 128 requests x 8 heads, 18 MB, are
// 1.35 waves of rows and take 25 us, one request 4.8 us, where four passes over memory
// with the leading digits in few bins took 61 and 11.
constexpr int kSelThreads = 256;

__device__ __forceinline__ uint32_t order_key(float x) {
  // -0 counts as 0; NaN as the lowest value of all (no number has a key of 0 or 1)
  if (x != x) return 1u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Bits 0 .. n - 1 of a word.
__device__ __forceinline__ uint32_t first_bits(int n) {
  return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
}

// Exclusive prefix of one count per thread over the CTA (s: a place per warp and
// one for the sum, which is returned too).
template <int kWarps>
__device__ __forceinline__ int cta_prefix(int own, int* s, int* sum) {
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  int x = own;
#pragma unroll
  for (int o = 1; o < kWarp; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == kWarp - 1) s[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int y = s[w];
    before += w < warp ? y : 0;
    all += y;
  }
  *sum = all;
  return before + x - own;
}

// kHeld: the keys fit shared memory (else they are read again for every pass).
template <int kThreads, bool kHeld>
__global__ void __launch_bounds__(kThreads) page_select_kernel(
    const float* scores, const int32_t* ctx_lens, int n_pages, int first, int last, spec_dims d,
    int32_t* __restrict__ pages, int32_t* __restrict__ counts, uint32_t* __restrict__ status) {
  constexpr int kWarps = kThreads / kWarp;
  constexpr int kRun = 32;    // rounds of pages between two scans: a word of 32 pages a thread
  constexpr int kAtOnce = 8;  // loads of a thread on their way
  constexpr int kList = 1024;
  extern __shared__ uint32_t s_keys[];  // 0 for pages that do not compete
  __shared__ int s_hist[256];
  __shared__ int s_digit, s_want, s_count, s_n;
  __shared__ uint32_t s_lo[kWarps], s_hi[kWarps];
  __shared__ int s_sum[2][kWarps];
  __shared__ uint32_t s_above[kRun * kWarps], s_equal[kRun * kWarps];
  __shared__ uint32_t s_list[kList];
  const int tid = threadIdx.x, warp = tid / kWarp, lane = tid % kWarp;
  const int h = blockIdx.x, b = blockIdx.y;
  pdl_trigger();
  pdl_wait();  // the scores and lengths may come from the previous kernels
  const float* x = scores + ((int64_t)b * d.Hkv + h) * d.max_blocks;
  // all of the row's places are there: the first loads need not wait for the length
  float v[kAtOnce];
#pragma unroll
  for (int i = 0; i < kAtOnce; ++i) {
    const int p = i * kThreads + tid;
    v[i] = kHeld && p < d.max_blocks ? __ldcg(x + p) : 0.f;
  }
  const int ctx = __ldcg(ctx_lens + b);
  const bool fits = ctx <= (int64_t)d.max_blocks * kBlock;
  const int full = fits && ctx > 0 ? ctx / kBlock : 0;
  const int count = min(full, n_pages);
  int32_t* list = pages + ((int64_t)b * d.Hkv + h) * n_pages;
  if (tid == 0 && h == 0) {
    counts[b] = count;
    if (!fits) raise_status(status, SPEC_ERR_CAPACITY);
  }
  for (int j = count + tid; j < n_pages; j += kThreads) list[j] = -1;
  if (full <= n_pages) {  // every page
    for (int j = tid; j < count; j += kThreads) list[j] = j;
    return;
  }
  // pages c0 .. c1 - 1 compete for `want` places
  const int c0 = first, c1 = full - last;
  int want = n_pages - first - last;
  const int rounds = ceil_div(full, kThreads);
  auto make_key = [&](int i, float score) {
    const int p = i * kThreads + tid;
    return p >= c0 && p < c1 ? order_key(score) : 0u;
  };
  // the key of this thread's i-th page
  auto key_of = [&](int i) {
    const int p = i * kThreads + tid;
    if constexpr (kHeld) return s_keys[p];
    else return make_key(i, p < full ? __ldcg(x + p) : 0.f);
  };
  uint32_t lo = 0xffffffffu, hi = 0;
  auto see = [&](uint32_t k) {
    lo = min(lo, k - 1u);  // 0 becomes the largest value
    hi = max(hi, k);
  };
  if constexpr (kHeld) {
    for (int i0 = 0; i0 < rounds; i0 += kAtOnce) {
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int p = (i0 + i) * kThreads + tid;
        if (i0 > 0) v[i] = p < full ? __ldcg(x + p) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (i0 + i < rounds) {
          const uint32_t k = make_key(i0 + i, v[i]);
          s_keys[(i0 + i) * kThreads + tid] = k;
          see(k);
        }
    }
  } else {
#pragma unroll 4
    for (int i = 0; i < rounds; ++i) see(key_of(i));
  }
  const int bad = lo == 0u;
  lo += 1u;
  // (no competing page in this thread: lo wraps to 0)
  lo = __reduce_min_sync(0xffffffffu, lo - 1u) + 1u;
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    s_lo[warp] = lo;
    s_hi[warp] = hi;
  }
  if (__syncthreads_or(bad) && tid == 0) raise_status(status, SPEC_ERR_NONFINITE);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    lo = min(lo - 1u, s_lo[w] - 1u) + 1u;
    hi = max(hi, s_hi[w]);
  }
  // Taken are the keys above `edge` and the first `want` of those equal to it.
  // `edge` is known down to bit `shift` (relative to lo).
  uint32_t edge = lo;
  int shift = 32 - __clz(hi - lo);  // 0 if all are equal
  if (want == 0) {
    edge = hi;  // nothing is above it
    shift = 0;
  }
  int listed = -1;  // keys in s_list: all that are still open (-1: no list yet)
  while (shift > 0) {
    const int bits = min(8, shift), top = shift;
    const uint32_t above = top < 32 ? (edge - lo) >> top : 0u;
    shift -= bits;
    if (tid < 256) s_hist[tid] = 0;
    __syncthreads();
    auto digit = [&](uint32_t k) { atomicAdd(&s_hist[(k >> shift) & ((1u << bits) - 1u)], 1); };
    if (listed >= 0) {
      for (int e = tid; e < listed; e += kThreads)
        if ((s_list[e] >> top) == above) digit(s_list[e]);
    } else {
#pragma unroll 4
      for (int i = 0; i < rounds; ++i) {
        const uint32_t k = key_of(i);
        if (k != 0u && (top >= 32 || ((k - lo) >> top) == above)) digit(k - lo);
      }
    }
    __syncthreads();
    if (warp == 0) {
      // lane j has the digits 255 - 8 j and the seven below
      int c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = s_hist[255 - 8 * lane - i];
        sum += c[i];
      }
      int before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
      }
      before -= sum;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (before < want && want <= before + c[i]) {
          s_digit = 255 - 8 * lane - i;
          s_want = want - before;
          s_count = c[i];
        }
        before += c[i];
      }
      if (lane == 0) s_n = 0;
    }
    __syncthreads();
    edge += (uint32_t)s_digit << shift;
    want = s_want;
    const int open = s_count;  // keys with the digits of `edge` so far
    if (want == open) {  // all of them are taken: the keys from `edge` on (keys are above 0)
      --edge;
      want = 0;
      break;
    }
    if (listed < 0 && shift > 0 && open <= kList) {  // the later digits of these alone
      const uint32_t now = (edge - lo) >> shift;
#pragma unroll 4
      for (int i = 0; i < rounds; ++i) {
        const uint32_t k = key_of(i);
        if (k != 0u && ((k - lo) >> shift) == now) s_list[atomicAdd(&s_n, 1)] = k - lo;
      }
      listed = open;
      __syncthreads();
    }
  }
  // words of 32 pages in order: those above the edge (and the first and last
  // pages), those equal to it
  int done = 0, equal = 0;
  for (int r0 = 0; r0 < rounds; r0 += kRun) {
    auto word = [&](int i) {
      const uint32_t k = key_of(i);
      const uint32_t m = __ballot_sync(0xffffffffu, k > edge);
      const uint32_t e = __ballot_sync(0xffffffffu, k == edge);
      if (lane == 0) {
        s_above[(i - r0) * kWarps + warp] = m;
        s_equal[(i - r0) * kWarps + warp] = e;
      }
    };
#pragma unroll 4
    for (int i = r0; i < min(rounds, r0 + kRun); ++i) word(i);
    __syncthreads();
    const bool mine = tid < kRun * kWarps && r0 * kWarps + tid < rounds * kWarps;
    const int page0 = r0 * kThreads + tid * kWarp;
    uint32_t m = 0, e = 0;
    if (mine) {
      m = s_above[tid] | first_bits(c0 - page0) | (first_bits(full - page0) & ~first_bits(c1 - page0));
      e = want > 0 ? s_equal[tid] : 0u;
    }
    int sum;
    if (want > 0) {
      const int before = equal + cta_prefix<kWarps>(__popc(e), s_sum[0], &sum);
      equal += sum;
      for (int left = want - before; e != 0 && left > 0; --left) {  // the lowest of them
        m |= e & (0u - e);
        e &= e - 1u;
      }
    }
    int at = done + cta_prefix<kWarps>(__popc(m), s_sum[1], &sum);
    done += sum;
    for (; m != 0; m &= m - 1u, ++at)
      if (at < n_pages) list[at] = page0 + __ffs(m) - 1;
    if (r0 + kRun < rounds) __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <typename T>
static cudaError_t launch_bounds(const BoundsArgs& a, cudaStream_t st) {
  const spec_dims& d = a.d;
  // one warp a (page, head); no more CTAs a request than its table has work for,
  // eight CTAs an SM over the batch
  const int64_t most = ceil_div64((int64_t)d.max_blocks * d.Hkv, 8);
  int64_t x = ceil_div64(8 * 152, d.B);
  if (x > most) x = most;
  PdlLaunch L(dim3((unsigned)x, d.B), dim3(256), 0, st);
  return cudaLaunchKernelEx(&L.cfg, d.D == 64 ? page_bounds_kernel<T, 64> : page_bounds_kernel<T, 128>,
                            static_cast<const T*>(a.k_cache), a.block_table, a.from_lens,
                            a.ctx_lens, d, static_cast<T*>(a.bounds), a.status);
}

cudaError_t page_bounds_launch(const BoundsArgs& a, cudaStream_t st, int* launches) {
  const cudaError_t e = a.d.kv_dtype == SPEC_BF16 ? launch_bounds<__nv_bfloat16>(a, st)
                                                  : launch_bounds<float>(a, st);
  if (e == cudaSuccess) ++*launches;
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int D, int RPT, int kTile>
static cudaError_t launch_score(const ScoreArgs& a, cudaStream_t st) {
  const spec_dims& d = a.d;
  auto k = page_score_kernel<T, D, RPT, kTile>;
  constexpr size_t smem = score_smem<D, RPT, kTile>();
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  PdlLaunch L(dim3(ceil_div(d.max_blocks, kTile), d.Hkv, d.B), dim3(kScoreThreads), smem, st);
  return cudaLaunchKernelEx(&L.cfg, k, static_cast<const T*>(a.q), static_cast<const T*>(a.bounds),
                            a.block_table, a.ctx_lens, d, a.scores, a.status);
}

template <typename T, int D, int kTile>
static cudaError_t launch_score(const ScoreArgs& a, cudaStream_t st) {
  const int R = (a.d.Hq / a.d.Hkv) * a.d.M;
  if (R <= 8) return launch_score<T, D, 1, kTile>(a, st);
  if (R <= 16) return launch_score<T, D, 2, kTile>(a, st);
  if (R <= 32) return launch_score<T, D, 4, kTile>(a, st);
  return launch_score<T, D, 8, kTile>(a, st);
}

template <typename T, int D>
static cudaError_t launch_score(const ScoreArgs& a, cudaStream_t st) {
  const int64_t ctas = (int64_t)ceil_div(a.d.max_blocks, 64) * a.d.Hkv * a.d.B;
  return ctas < 2 * 152 ? launch_score<T, D, 16>(a, st) : launch_score<T, D, 64>(a, st);
}

cudaError_t page_score_launch(const ScoreArgs& a, cudaStream_t st, int* launches) {
  if (page_score_tc_ok(a.d)) return page_score_tc_launch(a, st, launches);
  cudaError_t e;
  if (a.d.kv_dtype == SPEC_BF16)
    e = a.d.D == 64 ? launch_score<__nv_bfloat16, 64>(a, st) : launch_score<__nv_bfloat16, 128>(a, st);
  else
    e = a.d.D == 64 ? launch_score<float, 64>(a, st) : launch_score<float, 128>(a, st);
  if (e == cudaSuccess) ++*launches;
  return e != cudaSuccess ? e : cudaGetLastError();
}

constexpr int kSelMost = 48 * 1024;  // keys that fit shared memory

template <int kThreads, bool kHeld>
static cudaError_t launch_select(const SelectArgs& a, cudaStream_t st) {
  auto k = page_select_kernel<kThreads, kHeld>;
  // whole rounds of the threads
  const size_t smem = kHeld ? sizeof(uint32_t) * ceil_div(a.d.max_blocks, kThreads) * kThreads : 0;
  if (kHeld) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)(sizeof(uint32_t) * kSelMost));
    if (e != cudaSuccess) return e;
  }
  PdlLaunch L(dim3(a.d.Hkv, a.d.B), dim3(kThreads), smem, st);
  return cudaLaunchKernelEx(&L.cfg, k, a.scores, a.ctx_lens, a.n_pages, a.first, a.last, a.d,
                            a.pages, a.counts, a.status);
}

cudaError_t page_select_launch(const SelectArgs& a, cudaStream_t st, int* launches) {
  // few threads a row where there are many rows' worth of warps anyway
  const int n = a.d.max_blocks;
  const cudaError_t e = n <= 16 * 1024    ? launch_select<kSelThreads, true>(a, st)
                        : n <= kSelMost   ? launch_select<1024, true>(a, st)
                                          : launch_select<1024, false>(a, st);
  if (e == cudaSuccess) ++*launches;
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace specv
