// Sampling of one token per logits row from given uniforms: temperature,
// top-k, top-p and min-p (page 1 §3.3 temperature; page 2 §5.1 the filters).
// A draft model draws its tokens with it, and so does plain decoding, which a
// request falls back to when speculation does not pay.
//
// What is computed for a row x with temperature T and filters k, t, r:
//   w_i = exp((x_i - max x) / T)
//   order the tokens by x, largest first, the smaller index first among equal
//   ones; keep the first k; of those the shortest prefix whose mass reaches t
//   times their mass; of those the tokens with w_i >= r
//   C_i = sum of the kept weights of tokens 0..i, Z their total
//   token = the smallest i with C_i > u Z,  prob = w_i / Z
// A kept set is {x > tau} and the first c tokens equal to tau, so the filters
// come down to a threshold and a count.
//
// Rounding.  The token is a whole number that hangs on a comparison of sums;
// with 150k tokens every second row has a step of C within fp32's error of
// u Z.  Sums add 2^-40 of their value at most.  Weights come as double-floats
// (fp32 pairs): the exponential by table and polynomial (P. T. P. Tang,
// "Table-driven implementation of the exponential function", ACM TOMS 1989),
// 2^(j/32) from the table and four terms of the series for the rest r.  They
// are off by 2^-28.9 of their value at worst, 2^-31.5 on average: r (up to 2^-6)
// is one fp32 number, 2^-31 off, or 2^-30 just above 2^-6; so is the series, whose
// last product and sum round 2^-31 each; and the table's low word is not
// multiplied by it, 2^-31.5.  With a few tokens a step of C is off by as much; with
// many the errors average out.  (T above 2^100 loses more: log2(e) / T has no low
// word left there.)  GB300's fp64 rate is a hundredth of its fp32 rate, so
// nothing here is a per-element fp64 operation.  Masses that the filters
// compare are 42-bit fixed-point integers: their sums do not depend on the
// order of the atomics that form them.
//
// Two kernels read the logits.  Without filters sample_plain_kernel streams a
// row through registers once (its comment has the arithmetic).  With any
// filter sample_kernel takes a row with one cluster of up to 8 CTAs, each with
// a slice of the row in shared memory: the row is read from HBM once, whatever
// the filters ask for, and what the CTAs tell one another (maxima, candidates,
// histograms, masses) goes through distributed shared memory.  Slices that do
// not fit are read again through L2.  Its steps:
//   1   slice to shared memory, maximum, rows without a distribution
//   2a  with top-k or top-p: the tokens at or above a bound go to the first
//       CTA, which finishes the row alone.  The bound comes from the threads'
//       maxima: if n of them reach v, at least n tokens do; for top-k that
//       makes it safe, for top-p the candidates' mass is checked
//   2   else (a large k, a top-p that reaches far down) a select over the
//       slices' order keys, on counts or on masses, gives the threshold: for
//       bf16 over the values themselves, else level by level
//   3   the kept mass of every warp's run of tokens, exchanged; the warp that
//       holds u Z walks its run in order
// Measured (queued calls, us): 640 rows of 152064 bf16 logits, temperature
// alone, 72 (195 MB: 29 at the copy rate; the stream 50, the marked rows 21);
// 33 rows of 32001 fp32 logits with mixed filters 26 to 31 (44 by the selects over
// the cluster alone); one row of 32000: 9 without filters, 13 with top-k 50,
// 18 with top-p 0.9; 33 rows of 128256 bf16 logits with a top-p that keeps
// 30000 tokens 80.  A filtered row is bound by its chain of barriers, not by
// bytes; the slowest are rows whose top-p reaches past the candidates.
#include <cooperative_groups.h>
#include <math.h>

#include "rs_device.cuh"
#include "sample.cuh"

namespace specv {
namespace smp {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / kWarp;
constexpr int kMaxCluster = 8;
constexpr int kBinBits = 9;
constexpr int kBins = 1 << kBinBits;  // one per thread
constexpr uint32_t kKeyNegInf = 0x007fffffu;  // order key of -inf
constexpr int kUnroll = 4;
constexpr int kLongRun = 5 * kWarp;  // vectors; above it the walk is shared
constexpr size_t kMaxSharedBytes = 224 * 1024;  // static and dynamic, of an SM's CTAs

// Lets launches of `kern` ask for up to `most` bytes of dynamic shared memory.
// The limit is the same in every call: it belongs to the kernel, and another
// thread's call may stand between this one's setting and its launch.
template <typename K>
cudaError_t allow_shared(K kern, size_t most) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
}

// 2^(j/32) as hi + lo
__device__ const float2 kPow2[32] = {
    {0x1p+0f, 0.f}, {0x1.059b0ep+0f, -0x1.9d4f52p-25f},
    {0x1.0b5586p+0f, 0x1.9f3122p-25f}, {0x1.11301ep+0f, -0x1.fdb496p-25f},
    {0x1.172b84p+0f, -0x1.c15742p-27f}, {0x1.1d4874p+0f, -0x1.d2e8cap-25f},
    {0x1.2387a6p+0f, 0x1.ceac48p-25f}, {0x1.29e9ep+0f, -0x1.5c0424p-25f},
    {0x1.306fep+0f, 0x1.4636e2p-25f}, {0x1.371a74p+0f, -0x1.18aac6p-25f},
    {0x1.3dea64p+0f, 0x1.824684p-25f}, {0x1.44e086p+0f, 0x1.8624b4p-30f},
    {0x1.4bfdaep+0f, -0x1.593abcp-25f}, {0x1.5342b6p+0f, -0x1.2c561p-25f},
    {0x1.5ab07ep+0f, -0x1.5bd5ecp-27f}, {0x1.6247ecp+0f, -0x1.f8b55p-25f},
    {0x1.6a09e6p+0f, 0x1.9fcef4p-26f}, {0x1.71f75ep+0f, 0x1.1d8beep-25f},
    {0x1.7a1148p+0f, -0x1.829fdp-25f}, {0x1.82589ap+0f, -0x1.accc7cp-26f},
    {0x1.8ace54p+0f, 0x1.15506ep-27f}, {0x1.93737cp+0f, -0x1.e64744p-25f},
    {0x1.9c4918p+0f, 0x1.51f848p-27f}, {0x1.a5503cp+0f, -0x1.b83b54p-25f},
    {0x1.ae89fap+0f, -0x1.a94b14p-26f}, {0x1.b7f77p+0f, -0x1.a09438p-25f},
    {0x1.c199bep+0f, -0x1.3d56b2p-27f}, {0x1.cb720ep+0f, -0x1.8837ccp-27f},
    {0x1.d5818ep+0f, -0x1.822dbcp-27f}, {0x1.dfc974p+0f, -0x1.908c94p-25f},
    {0x1.ea4afap+0f, 0x1.52486cp-27f}, {0x1.f50766p+0f, -0x1.246ebp-26f}};

// What the exact draw exchanges.
struct DrawShared {
  float2 pow2[32];
  float2 mass[kMaxCluster * kWarps];
  int ties[kMaxCluster * kWarps];
  int pick, pick_ties;
  float2 pick_base, pick_z;
  float2 part[kWarps];  // of the chosen run, by warp
  int part_ties[kWarps];
};

struct Shared {
  DrawShared draw;
  alignas(16) uint32_t hist[2][4][kBins];  // counts, then the masses' three 14-bit limbs
  float ex_max[kMaxCluster];
  uint32_t ex_bad[kMaxCluster], ex_theta[kMaxCluster], ex_low[kMaxCluster];
  float2 ex_z[kMaxCluster];
  long long ex_mass[kMaxCluster];
  int ex_n[kMaxCluster];
  int ex_first[kMaxCluster];
  int n_list;
  float red[kWarps];
  uint32_t red_low[kWarps];
  uint32_t scan_cnt[kWarps];
  long long scan_mass[kWarps];
  int sel_bin;
  uint32_t sel_above, sel_count;
  long long sel_mass;
  uint32_t mid[3];  // value_select: mass of the values about zero, in limbs
};

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}

// Order key: unsigned, ascending with the value; -0 and +0 are equal.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

struct Law {
  float m, c_hi, c_lo;  // maximum; log2(e) / T as a double-float
  const float2* pow2;
  // log2(e) / T: log2(e) as a double-float, the quotient's remainder exact
  __device__ __forceinline__ Law(float max, float T, const float2* table)
      : m(max), c_hi(1.44269502f / T), pow2(table) {
    c_lo = (fmaf(-c_hi, T, 1.44269502f) + 1.92596303e-8f) / T;
  }
  // exp((x - m) / T) as a double-float, off by 2^-28.9 of it at most; 0 below 2^-120
  __device__ __forceinline__ dfloat weight(float x) const {
    const dfloat d = df_two_sum(x, -m);
    const float y = __fmul_rn(d.hi, c_hi);
    if (!(y > -120.f)) return dfloat{0.f, 0.f};  // -inf (and its NaN error term) too
    float yl = fmaf(d.hi, c_hi, -y);
    yl = fmaf(d.hi, c_lo, yl);
    yl = fmaf(d.lo, c_hi, yl);
    const float t = __fadd_rn(__fmul_rn(y, 32.f), 12582912.f);  // rounds to a whole number
    const int ki = __float_as_int(t) - 0x4b400000;
    const float r = fmaf(__fsub_rn(t, 12582912.f), -0.03125f, y) + yl;
    // 2^r - 1, |r| <= 1/64: the terms (r ln 2)^n / n!, n <= 4
    float p = fmaf(r, 9.61812911e-3f, 5.55041087e-2f);
    p = fmaf(r, p, 2.40226507e-1f);
    p = fmaf(r, p, 6.93147181e-1f);
    p = __fmul_rn(r, p);
    const float2 e = pow2[ki & 31];
    const float s = __int_as_float((127 + (ki >> 5)) << 23);
    const float hi = fmaf(e.x, p, e.x);
    const float lo = fmaf(e.x, p, __fsub_rn(e.x, hi)) + e.y;
    return dfloat{hi * s, lo * s};
  }
};

// w / z, rounded once (the quotient of the high words, and its remainder).
__device__ __forceinline__ float df_quotient(dfloat w, dfloat z) {
  const float q = w.hi / z.hi;
  const float rest = fmaf(-q, z.hi, w.hi) + fmaf(-q, z.lo, w.lo);
  return q + rest / z.hi;
}

// A weight as a 42-bit fixed-point fraction, in three limbs of 14 bits, none
// negative (the limbs of 2^17 weights add up in 32 bits).
__device__ __forceinline__ void fixed_limbs(dfloat w, uint32_t (&l)[3]) {
  float a = floorf(w.hi * 0x1p14f);
  if (fmaf(a, -0x1p-14f, w.hi) + w.lo < 0.f) a -= 1.f;
  const float r1 = fmaf(a, -0x1p-14f, w.hi);
  const float b = floorf((r1 + w.lo) * 0x1p28f);
  const float r2 = fmaf(b, -0x1p-28f, r1) + w.lo;
  l[0] = (uint32_t)a;
  l[1] = (uint32_t)b;
  l[2] = (uint32_t)__float2int_rn(fmaxf(0.f, r2 * 0x1p42f));
}
__device__ __forceinline__ long long limbs_value(long long a, long long b, long long c) {
  return (a << 28) + (b << 14) + c;
}
__device__ __forceinline__ long long fixed_value(dfloat w) {
  uint32_t l[3];
  fixed_limbs(w, l);
  return limbs_value(l[0], l[1], l[2]);
}
// t times a fixed-point mass, rounded up.
__device__ __forceinline__ long long mass_target(float t, long long z) {
  return max(1ll, __double2ll_ru((double)t * (double)z));
}
__device__ __forceinline__ int ties_for(long long missing, long long each, int most) {
  if (each <= 0) return most;
  const long long c = (missing + each - 1) / each;
  return c < most ? (int)c : most;
}

// A CTA's slice of a row, as 16-byte vectors counted from the 16-byte
// boundary at or below its first element (elements outside it read as -inf).
template <typename T, bool kSmem>
struct Slice {
  static constexpr int kVec = 16 / sizeof(T);
  const T* src;  // first element
  int off;       // elements between the boundary and it
  int n;         // elements
  const uint4* sm;

  __device__ __forceinline__ uint4 load(int v) const {
    const int p = v * kVec - off;
    if (p >= 0 && p + kVec <= n) return *reinterpret_cast<const uint4*>(src + p);
    uint4 r;
    T* e = reinterpret_cast<T*>(&r);
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      e[i] = p + i >= 0 && p + i < n ? src[p + i] : from_f32<T>(-INFINITY);
    return r;
  }
  __device__ __forceinline__ uint4 get(int v) const { return kSmem ? sm[v] : load(v); }
};

// Inclusive running sums of a count and a mass over the CTA's threads.
__device__ __forceinline__ void block_running(Shared& sh, uint32_t& c, long long& m, bool with_mass) {
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
#pragma unroll
  for (int o = 1; o < kWarp; o <<= 1) {
    const uint32_t yc = __shfl_up_sync(0xffffffffu, c, o);
    if (lane >= o) c += yc;
    if (with_mass) {
      const long long ym = __shfl_up_sync(0xffffffffu, m, o);
      if (lane >= o) m += ym;
    }
  }
  if (lane == kWarp - 1) {
    sh.scan_cnt[warp] = c;
    sh.scan_mass[warp] = m;
  }
  __syncthreads();
  // the sums of the warps before, lane w holding warp w's
  uint32_t wc = lane < warp ? sh.scan_cnt[lane] : 0;
  wc = __reduce_add_sync(0xffffffffu, wc);
  c += wc;
  if (with_mass) {
    long long wm = lane < warp ? sh.scan_mass[lane] : 0;
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) wm += __shfl_xor_sync(0xffffffffu, wm, o);
    m += __shfl_sync(0xffffffffu, wm, 0);
  }
}

struct Selected {
  bool found;
  uint32_t tau;   // order key of the threshold
  uint32_t above, ties;
  long long mass;  // of the tokens above tau (when masses were summed)
};

// Select for bf16 logits, arguments as in radix_select below: a 16-bit value
// has few neighbours, so a bin holds one value, tokens are only counted and a
// bin's mass is its count times one weight -- one level, one atomic a token,
// no weight a token.  The bins run down from the largest value: kDirectBins
// values, those within 2^-10 of zero (36000 of the 65536) together in one bin
// whose mass is summed.  Not resolved (false) if the place lies in that bin or
// past the last one.  Each CTA sums its share of the bins over the cluster and
// the place is found by running sums over the shares.  (33 rows of 128256
// logits, top-p 0.9 of a normal law of deviation 2: 81 us, against 157 with
// the levels below; top-k 5000 and that: 56 against 122; 32001 logits: 37
// against 43 and 34 against 46.)  `buf` is -1 before any select, 2 after this
// one.
constexpr int kDirectBins = 8 * kBins;
// The order key of a bf16 value from its upper half: the bits below are zeros,
// or ones for a negative value.
__device__ __forceinline__ uint32_t full_key(uint32_t key) {
  return key & 0x8000u ? key << 16 : (key << 16) | 0xffffu;
}
constexpr uint32_t kMidHigh = 0xba80u, kMidLow = 0x457fu;  // keys of 2^-10 and -2^-10

template <typename T, bool kSmem>
__device__ bool value_select(Shared& sh, const Slice<T, kSmem>& sl, int nv, const Law& law,
                             uint32_t low, uint32_t high, bool by_mass, bool with_mass,
                             long long rank, long long mass, int C, int& buf, Selected& r) {
  constexpr int kVec = Slice<T, kSmem>::kVec, kPer = kDirectBins / kThreads;
  static_assert(kPer == 8 && sizeof(sh.hist) == kDirectBins * 4, "both buffers, 8 bins a thread");
  const int tid = threadIdx.x, rank_of = blockIdx.x % C;
  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t top = high >> 16;
  const int mid = top >= kMidHigh ? (int)(top - kMidHigh) + 1 : top > kMidLow ? 0 : -1;
  if (buf == 2) __syncthreads();  // the last select's sel_* are read
  else if (buf >= 0) cluster_sync();  // and its bins, by the other CTAs
  buf = 2;
  uint32_t* hist = &sh.hist[0][0][0];
  for (int i = tid; i < kDirectBins; i += kThreads) hist[i] = 0;
  if (tid < 3) sh.mid[tid] = 0;
  if (tid == 0) sh.sel_bin = -1;
  __syncthreads();
  for (int v = tid; v < nv; v += kThreads) {
    const uint4 raw = sl.get(v);
    float x[kVec];
    unpack16(raw, x);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const uint32_t full = order_key(x[i]), key = full >> 16;
      if (full < low || full <= kKeyNegInf) continue;
      const uint32_t at = mid < 0 || key >= kMidHigh ? top - key
                          : key > kMidLow            ? (uint32_t)mid
                                                     : mid + 1 + (kMidLow - key);
      if (at >= (uint32_t)kDirectBins) continue;
      atomicAdd(hist + at, 1u);
      if (with_mass && (int)at == mid) {
        uint32_t l[3];
        fixed_limbs(law.weight(x[i]), l);
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (l[j] != 0) atomicAdd(&sh.mid[j], l[j]);
      }
    }
  }
  cluster_sync();
  // each CTA sums its share of the bins over the cluster, 8 / C of them a thread
  const int per = kPer / C, b0 = (rank_of * kThreads + tid) * per;
  uint32_t cnt[kPer], c = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) cnt[i] = 0;
#pragma unroll
  for (int q = 0; q < kMaxCluster; ++q) {
    if (q >= C) break;
    const uint32_t* h = cluster.map_shared_rank(hist, q) + b0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < per) cnt[i] += h[i];
  }
  long long mid_mass = 0;
  if (with_mass && mid >= b0 && mid < b0 + per)
    for (int q = 0; q < C; ++q) {
      const uint32_t* l = cluster.map_shared_rank(&sh.mid[0], q);
      mid_mass += limbs_value(l[0], l[1], l[2]);
    }
  // mass of a bin's tokens
  auto bin_mass = [&](int i) -> long long {
    const int at = b0 + i;
    if (at == mid) return mid_mass;
    const uint32_t key = mid < 0 || at < mid ? top - at : kMidLow - (at - mid - 1);
    return cnt[i] == 0 ? 0 : cnt[i] * fixed_value(law.weight(key_value(full_key(key))));
  };
  long long m = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    c += cnt[i];
    if (with_mass) m += bin_mass(i);
  }
  uint32_t ci = c;
  long long mi = m;
  block_running(sh, ci, mi, with_mass);
  if (tid == kThreads - 1)
    for (int q = 0; q < C; ++q) {
      *cluster.map_shared_rank(&sh.ex_n[rank_of], q) = (int)ci;
      *cluster.map_shared_rank(&sh.ex_mass[rank_of], q) = mi;
    }
  cluster_sync();
  for (int q = 0; q < rank_of; ++q) {
    ci += sh.ex_n[q];
    mi += sh.ex_mass[q];
  }
  const long long want = by_mass ? mass : rank;
  if ((by_mass ? mi - m : (long long)(ci - c)) < want && want <= (by_mass ? mi : (long long)ci)) {
    uint32_t above = ci - c, count = 0;
    long long over = mi - m;
    int bin = -1;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i >= per || bin >= 0) continue;
      const long long bm = with_mass ? bin_mass(i) : 0;
      if (want <= (by_mass ? over + bm : (long long)(above + cnt[i]))) {
        bin = b0 + i;
        count = cnt[i];
      } else {
        above += cnt[i];
        over += bm;
      }
    }
    for (int q = 0; q < C; ++q) {
      *cluster.map_shared_rank(&sh.sel_bin, q) = bin;
      *cluster.map_shared_rank(&sh.sel_above, q) = above;
      *cluster.map_shared_rank(&sh.sel_mass, q) = over;
      *cluster.map_shared_rank(&sh.sel_count, q) = count;
    }
  }
  cluster_sync();
  const int at = sh.sel_bin;
  if (at < 0 || at == mid) return false;
  const uint32_t key = mid < 0 || at < mid ? top - at : kMidLow - (at - mid - 1);
  r.found = true;
  r.tau = full_key(key);
  r.above = sh.sel_above;
  r.ties = sh.sel_count;
  r.mass = sh.sel_mass;
  return true;
}

// Radix select over the tokens with order key >= low (the largest key being
// `high`): the value of rank `rank` (1 = largest), or, with by_mass, the first
// at which the running mass reaches `mass`.  Not found when all of them
// together fall short.  A level cuts the range of keys that is left into 512
// bins; keys are counted from `low`, so that the bins fill evenly and a range
// of a few octaves takes one level for bf16 and three for fp32 (digits of the
// key itself put every candidate into two or three bins: their atomics then
// run one after another).
template <typename T, bool kSmem>
__device__ Selected radix_select(Shared& sh, const Slice<T, kSmem>& sl, int nv, const Law& law,
                                 uint32_t low, uint32_t high, bool by_mass, bool with_mass,
                                 long long rank, long long mass, int C, int& buf) {
  constexpr int kVec = Slice<T, kSmem>::kVec;
  constexpr int kShift = sizeof(T) == 2 ? 16 : 0;  // bits that a key of this type does not use
  const int tid = threadIdx.x;
  cg::cluster_group cluster = cg::this_cluster();
  Selected r{true, 0, 0, 0, 0};
  // counts alone are as quick in the levels below while a slice is short (one
  // row, top-k 5000: 32001 logits 14 us, 18 by value_select, 128256 24 and 27;
  // 33 of those rows, slices of 32064: 52 and 42)
  constexpr int kShortSlice = 20000;
  if constexpr (sizeof(T) == 2) {
    if ((with_mass || nv * kVec > kShortSlice) &&
        value_select<T, kSmem>(sh, sl, nv, law, low, high, by_mass, with_mass, rank, mass, C, buf, r))
      return r;
  }
  if (buf == 2) __syncthreads();  // value_select's sel_* are read
  if (buf != 1) buf = 0;
  if (low <= kKeyNegInf) low = kKeyNegInf + 1;
  uint32_t base = low >> kShift;
  int bits = 32 - __clz((high >> kShift) - base);  // keys base .. base + 2^bits - 1
  do {
    const int sh_bits = max(0, bits - kBinBits);
    const uint32_t span = bits < 32 ? (1u << bits) - 1 : ~0u;
    // the other CTAs read this buffer two levels ago, before they arrived at
    // the last level's barrier
    for (int i = tid; i < 4 * kBins; i += kThreads) (&sh.hist[buf][0][0])[i] = 0;
    if (tid == 0) sh.sel_bin = -1;
    __syncthreads();
    for (int v = tid; v < nv; v += kThreads) {
      const uint4 raw = sl.get(v);
      float x[kVec];
      unpack16(raw, x);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const uint32_t key = order_key(x[i]);
        const uint32_t at = (key >> kShift) - base;
        if (key >= low && at <= span) {
          const uint32_t bin = at >> sh_bits;
          atomicAdd(&sh.hist[buf][0][bin], 1u);
          if (with_mass) {
            uint32_t l[3];
            fixed_limbs(law.weight(x[i]), l);
#pragma unroll
            for (int j = 0; j < 3; ++j)
              if (l[j] != 0) atomicAdd(&sh.hist[buf][1 + j][bin], l[j]);
          }
        }
      }
    }
    cluster_sync();
    // thread i: bin 511 - i, summed over the cluster, then the running sums
    const int bin = kBins - 1 - tid;
    uint32_t cnt = 0;
    long long ms = 0;
    for (int q = 0; q < C; ++q) {
      const uint32_t* h = cluster.map_shared_rank(&sh.hist[buf][0][0], q);
      cnt += h[bin];
      if (with_mass) ms += limbs_value(h[kBins + bin], h[2 * kBins + bin], h[3 * kBins + bin]);
    }
    uint32_t ci = cnt;
    long long mi = ms;
    block_running(sh, ci, mi, with_mass);
    const long long before = by_mass ? r.mass + mi - ms : (long long)r.above + ci - cnt;
    const long long upto = by_mass ? r.mass + mi : (long long)r.above + ci;
    const long long want = by_mass ? mass : rank;
    if (before < want && want <= upto) {
      sh.sel_bin = bin;
      sh.sel_above = ci - cnt;
      sh.sel_mass = mi - ms;
      sh.sel_count = cnt;
    }
    __syncthreads();
    buf ^= 1;
    if (sh.sel_bin < 0) {
      r.found = false;
      return r;
    }
    r.above += sh.sel_above;
    r.mass += sh.sel_mass;
    r.ties = sh.sel_count;
    base += (uint32_t)sh.sel_bin << sh_bits;
    bits = sh_bits;
    __syncthreads();  // sel_* are read
  } while (bits > 0);
  r.tau = sizeof(T) == 2 ? full_key(base) : base;
  return r;
}

// The draw, exactly: the kept mass of every warp's run of tokens (warp_vecs
// vectors of the CTA's slice, which begins at token `first`), exchanged over
// the cluster; the warp whose run holds u Z walks it in vocabulary order.  A
// long run is first shared out among its CTA's warps in the same way, and the
// warp whose share holds u Z walks that (300 rows of 128256 bf16 logits, runs
// of 502 vectors: 51 us instead of 60; runs of 32: 2 us slower, of 149: equal).
// Kept are the tokens above tau, the first keep_ties of those equal to it
// (everything for tau = kKeyNegInf), and of these the ones of weight >= mp.
template <int kW, typename T, bool kSmem>
__device__ void exact_draw(DrawShared& sh, const Slice<T, kSmem>& sl, const Law& law, uint32_t tau,
                           int keep_ties, float mp, float u, int warp_vecs, int C, int rank,
                           int first, const SampleArgs& a, int64_t row) {
  constexpr int kVec = Slice<T, kSmem>::kVec;
  const int tid = threadIdx.x, lane = tid % kWarp, warp = tid / kWarp;
  cg::cluster_group cluster = cg::this_cluster();
  const bool filtered = tau != kKeyNegInf || mp > 0.f;
  dfloat w_tau = df_make(0.f);
  if (tau != kKeyNegInf) {
    w_tau = law.weight(key_value(tau));
    if ((w_tau.hi - mp) + w_tau.lo < 0.f) w_tau = df_make(0.f);
  }
  // mass (without the tokens at tau) and tokens at tau of vectors lo .. hi - 1
  auto run_mass = [&](int lo, int hi, int& ties) {
    // four sums, so that one's chain of additions does not wait for another's
    dfloat acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = df_make(0.f);
    ties = 0;
    for (int v = lo + lane; v < hi; v += kWarp) {
      const uint4 raw = sl.get(v);
      float x[kVec];
      unpack16(raw, x);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        if (filtered) {
          const uint32_t key = order_key(x[i]);
          ties += key == tau && tau != kKeyNegInf;
          if (key <= tau) continue;
        }
        dfloat w = law.weight(x[i]);
        if ((w.hi - mp) + w.lo < 0.f) w = df_make(0.f);
        const dfloat s = df_two_sum(acc[i & 3].hi, w.hi);
        acc[i & 3].hi = s.hi;
        acc[i & 3].lo += s.lo + w.lo;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = df_norm(acc[i].hi, acc[i].lo);
    ties = (int)__reduce_add_sync(0xffffffffu, (unsigned)ties);
    return df_warp_sum(df_add(df_add(acc[0], acc[1]), df_add(acc[2], acc[3])));
  };
  {
    int ties;
    const dfloat z = run_mass(warp * warp_vecs, (warp + 1) * warp_vecs, ties);
    if (lane < C) {
      *cluster.map_shared_rank(&sh.mass[rank * kW + warp], lane) = make_float2(z.hi, z.lo);
      *cluster.map_shared_rank(&sh.ties[rank * kW + warp], lane) = ties;
    }
  }
  cluster_sync();  // from here on each CTA touches only its own shared memory
  if (warp == 0) {
    const int per = kMaxCluster * kW / kWarp;  // runs of a lane
    const int runs = C * kW;
    int t[per], ts = 0;
#pragma unroll
    for (int i = 0; i < per; ++i) {
      t[i] = lane * per + i < runs ? sh.ties[lane * per + i] : 0;
      ts += t[i];
    }
    int before = ts;
#pragma unroll
    for (int o = 1; o < kWarp; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
    }
    before -= ts;
    dfloat own[per], sum = df_make(0.f);
    int tb = before;
#pragma unroll
    for (int i = 0; i < per; ++i) {
      own[i] = df_make(0.f);
      if (lane * per + i < runs) {
        const float2 ms = sh.mass[lane * per + i];
        const int kept = max(0, min(keep_ties - tb, t[i]));
        own[i] = df_add(dfloat{ms.x, ms.y}, df_mul_f(w_tau, (float)kept));
      }
      tb += t[i];
      sum = df_add(sum, own[i]);
    }
    const dfloat incl = df_warp_scan(sum);
    const dfloat Z = df_shfl(incl, kWarp - 1);
    const dfloat thr = df_mul_f(Z, u);
    const unsigned past = __ballot_sync(0xffffffffu, sum.hi > 0.f && df_gt(incl, thr));
    const unsigned any = __ballot_sync(0xffffffffu, sum.hi > 0.f);
    const int owner = past != 0 ? __ffs(past) - 1 : 31 - __clz(any);
    if (lane == owner) {
      dfloat cum = df_sub(incl, sum), base = cum;
      int pick = -1, pick_ties = 0;
      tb = before;
#pragma unroll
      for (int i = 0; i < per; ++i) {
        if ((pick < 0 || !df_gt(cum, thr)) && own[i].hi > 0.f) {
          pick = lane * per + i;  // the first run past u Z, or the lane's last
          pick_ties = tb;
          base = cum;
          cum = df_add(cum, own[i]);
        }
        tb += t[i];
      }
      sh.pick = pick;
      sh.pick_ties = pick_ties;
      sh.pick_base = make_float2(base.hi, base.lo);
      sh.pick_z = make_float2(Z.hi, Z.lo);
    }
  }
  __syncthreads();
  const int pick = sh.pick;
  if (pick / kW != rank) return;
  const dfloat Z{sh.pick_z.x, sh.pick_z.y};
  const dfloat thr = df_mul_f(Z, u);
  dfloat cum{sh.pick_base.x, sh.pick_base.y};
  int tie_base = sh.pick_ties;
  int v_lo = pick % kW * warp_vecs, v_hi = v_lo + warp_vecs;
  if (warp_vecs <= kLongRun) {
    if (pick % kW != warp) return;
  } else {
    const int share = ceil_div(warp_vecs, kW);
    v_lo += warp * share;
    v_hi = min(v_lo + share, v_hi);
    int t;
    const dfloat z = run_mass(v_lo, v_hi, t);
    if (lane == 0) {
      sh.part[warp] = make_float2(z.hi, z.lo);
      sh.part_ties[warp] = t;
    }
    __syncthreads();
    // lane w: warp w's share
    dfloat own = df_make(0.f);
    t = 0;
    if (lane < kW) {
      own = dfloat{sh.part[lane].x, sh.part[lane].y};
      t = sh.part_ties[lane];
    }
    int before = t;
#pragma unroll
    for (int o = 1; o < kWarp; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
    }
    before += tie_base - t;
    own = df_add(own, df_mul_f(w_tau, (float)max(0, min(keep_ties - before, t))));
    const dfloat incl = df_add(cum, df_warp_scan(own));
    const unsigned past = __ballot_sync(0xffffffffu, own.hi > 0.f && df_gt(incl, thr));
    const unsigned any = __ballot_sync(0xffffffffu, own.hi > 0.f);
    const int owner = past != 0 ? __ffs(past) - 1 : 31 - __clz(any);
    if (owner != warp) return;
    cum = df_shfl(df_sub(incl, own), warp);
    tie_base = __shfl_sync(0xffffffffu, before, warp);
  }
  int last = -1;        // this lane's last kept token so far
  dfloat last_w = df_make(0.f);
  for (int v0 = v_lo; v0 < v_hi; v0 += kWarp) {
    const int v = v0 + lane;
    float x[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) x[i] = -INFINITY;
    if (v < v_hi) {
      const uint4 raw = sl.get(v);
      unpack16(raw, x);
    }
    int nt = 0;
    if (tau != kKeyNegInf) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) nt += order_key(x[i]) == tau;
    }
    int it = nt;
    if (tau != kKeyNegInf) {
#pragma unroll
      for (int o = 1; o < kWarp; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, it, o);
        if (lane >= o) it += y;
      }
    }
    int tr = tie_base + it - nt;
    dfloat w[kVec], sum = df_make(0.f);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      w[i] = df_make(0.f);
      const uint32_t key = order_key(x[i]);
      if (filtered && key == tau && tau != kKeyNegInf) {
        if (tr++ < keep_ties) w[i] = w_tau;
      } else if (!filtered || key > tau) {
        w[i] = law.weight(x[i]);
        if ((w[i].hi - mp) + w[i].lo < 0.f) w[i] = df_make(0.f);
      }
      if (w[i].hi > 0.f) {
        last = v * kVec + i;
        last_w = w[i];
      }
      sum = df_add(sum, w[i]);
    }
    tie_base += __shfl_sync(0xffffffffu, it, kWarp - 1);
    const dfloat incl = df_add(cum, df_warp_scan(sum));
    const unsigned past = __ballot_sync(0xffffffffu, sum.hi > 0.f && df_gt(incl, thr));
    if (past != 0) {
      if (lane == __ffs(past) - 1) {
        dfloat c = df_sub(incl, sum);
        int at = -1;
        dfloat wt = df_make(0.f);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          if ((at < 0 || !df_gt(c, thr)) && w[i].hi > 0.f) {
            c = df_add(c, w[i]);
            at = v * kVec + i;
            wt = w[i];
          }
        }
        a.out_tokens[row] = first + at - sl.off;
        if (a.out_prob != nullptr) a.out_prob[row] = df_quotient(wt, Z);
      }
      return;
    }
    cum = df_shfl(incl, kWarp - 1);
  }
  // u Z at the very end of what is walked, within the sums' rounding: its last
  // kept token
  const int top = __reduce_max_sync(0xffffffffu, last);
  if (last == top && top >= 0) {
    a.out_tokens[row] = first + top - sl.off;
    if (a.out_prob != nullptr) a.out_prob[row] = df_quotient(last_w, Z);
  }
}

// Sum and maximum of one number a thread over the CTA.
__device__ __forceinline__ long long block_sum(Shared& sh, long long v) {
#pragma unroll
  for (int o = kWarp / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (threadIdx.x % kWarp == 0) sh.scan_mass[threadIdx.x / kWarp] = v;
  __syncthreads();
  v = 0;
  for (int w = 0; w < kWarps; ++w) v += sh.scan_mass[w];
  __syncthreads();
  return v;
}
__device__ __forceinline__ long long block_max(Shared& sh, long long v) {
#pragma unroll
  for (int o = kWarp / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if (threadIdx.x % kWarp == 0) sh.scan_mass[threadIdx.x / kWarp] = v;
  __syncthreads();
  v = sh.scan_mass[0];
  for (int w = 1; w < kWarps; ++w) v = max(v, sh.scan_mass[w]);
  __syncthreads();
  return v;
}

// ---------------------------------------------------------------------------
// the candidates of a filtered row in one CTA
// ---------------------------------------------------------------------------
// When few tokens can matter they are sent to the cluster's first CTA (at
// most kListCap / C from each), and the filters and the draw run there on
// registers: a level of the select is then a few block barriers, where one
// over the cluster's slices costs a cluster barrier and 32 remote loads a
// thread.  Masses are 40-bit fractions in two limbs of 20 bits (the limbs of
// up to 4096 weights add up in 32 bits).
// candidates of a row; a CTA has its share of the places (28 KB: two CTAs with
// a quarter of 128k bf16 logits each fit an SM)
constexpr int kListCap = 7 * kThreads;
constexpr int kListEach = kListCap / kThreads;  // of a thread of the first CTA
// Of a CTA's 512 threads' maxima, how many have to reach the candidates' lower
// bound: n of them leave about 512 ln(512 / (512 - n)) candidates, the more
// tokens a thread has.  For top-p as many as fill seven eighths of the CTA's
// places; for top-k the count asked for, up to the one that fills two thirds.
__device__ __forceinline__ int list_need_p(int C) {
  return C == 8 ? 274 : C == 4 ? 401 : C == 2 ? 488 : 511;
}
__device__ __forceinline__ int list_most_k(int C) {
  return C == 8 ? 226 : C == 4 ? 352 : C == 2 ? 462 : 507;
}

struct Picked {
  bool found;
  uint32_t key;  // the key at the place asked for
  uint32_t above, ties;
  long long mass;  // of the keys above it
};

__device__ __forceinline__ void fixed_pair(dfloat w, uint32_t& hi, uint32_t& lo) {
  float a = floorf(w.hi * 0x1p20f);
  if (fmaf(a, -0x1p-20f, w.hi) + w.lo < 0.f) a -= 1.f;
  const float r = fmaf(a, -0x1p-20f, w.hi) + w.lo;
  hi = (uint32_t)a;
  lo = (uint32_t)__float2int_rn(r * 0x1p40f);
}

// Sum of such fractions as a double-float.
__device__ __forceinline__ dfloat pair_sum(long long z) {
  const float hi = (float)z;
  return dfloat{hi * 0x1p-40f, (float)(z - (long long)hi) * 0x1p-40f};
}

__device__ __forceinline__ long long pair_value(uint32_t hi, uint32_t lo) {
  return ((long long)hi << 20) + lo;
}

// Among the CTA's keys (those of bit i in `active`, all in [base, base +
// 2^bits)), in descending order: the key of rank `want`, or at which the
// running mass reaches `want`.  sh.hist[buf] is zero on entry, and on return.
__device__ Picked list_select(Shared& sh, const uint32_t (&key)[kListEach],
                              const uint32_t (&mh)[kListEach], const uint32_t (&ml)[kListEach],
                              uint32_t active, uint32_t base, int bits, bool by_mass,
                              long long want, int& buf) {
  const int tid = threadIdx.x;
  Picked r{true, 0, 0, 0, 0};
  do {
    uint32_t(&hist)[4][kBins] = sh.hist[buf];
    const int sh_bits = max(0, bits - kBinBits);
    const uint32_t span = bits < 32 ? (1u << bits) - 1 : ~0u;
#pragma unroll
    for (int i = 0; i < kListEach; ++i) {
      const uint32_t at = key[i] - base;
      if (((active >> i) & 1u) && at <= span) {
        const uint32_t bin = at >> sh_bits;
        atomicAdd(&hist[0][bin], 1u);
        if (mh[i] != 0) atomicAdd(&hist[1][bin], mh[i]);
        if (ml[i] != 0) atomicAdd(&hist[2][bin], ml[i]);
      }
    }
    if (tid == 0) sh.sel_bin = -1;  // the last level's sel_* are read: its last barrier but one
    __syncthreads();
    const int bin = kBins - 1 - tid;
    const uint32_t cnt = hist[0][bin];
    const long long ms = pair_value(hist[1][bin], hist[2][bin]);
    hist[0][bin] = 0;
    hist[1][bin] = 0;
    hist[2][bin] = 0;
    uint32_t ci = cnt;
    long long mi = ms;
    block_running(sh, ci, mi, true);
    const long long before = by_mass ? r.mass + mi - ms : (long long)r.above + ci - cnt;
    const long long upto = by_mass ? r.mass + mi : (long long)r.above + ci;
    if (before < want && want <= upto) {
      sh.sel_bin = bin;
      sh.sel_above = ci - cnt;
      sh.sel_mass = mi - ms;
      sh.sel_count = cnt;
    }
    __syncthreads();
    const int got = sh.sel_bin;
    const uint32_t above = sh.sel_above, count = sh.sel_count;
    const long long mass = sh.sel_mass;
    buf ^= 1;
    __syncthreads();  // sel_* are read
    if (got < 0) {
      r.found = false;
      return r;
    }
    r.above += above;
    r.mass += mass;
    r.ties = count;
    base += (uint32_t)got << sh_bits;
    bits = sh_bits;
  } while (bits > 0);
  r.key = base;
  return r;
}

// The filters and the draw over a short list, n <= kShortList tokens: every
// token is compared with every other, two threads a token, so that its rank
// and the mass of the tokens before it (by value, then by index) come without
// a select.  Two passes and a few barriers: n = 80 takes 3 us where the
// selects below take 16.
constexpr int kShortList = 256;

__device__ void short_draw(Shared& sh, const uint2* list, const Law& law, int C, int n, int k,
                           long long want_p, float tp, float mp, float u, const SampleArgs& a,
                           int64_t row) {
  static_assert(kThreads == 2 * kShortList, "two threads a token");
  // token j: order key, index, mass; the list's places are dealt out in turn
  uint4* tok = reinterpret_cast<uint4*>(&sh.hist[0][0][0]);
  const int tid = threadIdx.x, e = tid >> 1, part = tid & 1;
  uint32_t key = 0, idx = 0;
  float x = 0.f;
  dfloat w = df_make(0.f);
  long long mass = 0;
  if (e < n) {
    int q = 0, at = e;
    while (at >= sh.ex_n[q]) at -= sh.ex_n[q++];  // e < n: q stays below C
    const uint2 t = list[q * (kListCap / C) + at];
    x = __uint_as_float(t.x);
    key = order_key(x);
    idx = t.y;
    w = law.weight(x);
    uint32_t hi, lo;
    fixed_pair(w, hi, lo);
    mass = pair_value(hi, lo);
    if (part == 0) tok[e] = make_uint4(key, idx, (uint32_t)mass, (uint32_t)(mass >> 32));
  }
  __syncthreads();
  const int j0 = part * (kShortList / 2), j1 = min(n, j0 + kShortList / 2);
  int rank = 0;
  long long before = 0, all = 0;
  for (int j = j0; j < j1; ++j) {
    const uint4 o = tok[j];
    const long long m = (long long)o.z | ((long long)o.w << 32);
    const bool first = o.x > key || (o.x == key && o.y < idx);
    rank += first;
    if (first) before += m;
    all += m;
  }
  rank += __shfl_xor_sync(0xffffffffu, rank, 1);
  before += __shfl_xor_sync(0xffffffffu, before, 1);
  all += __shfl_xor_sync(0xffffffffu, all, 1);
  if (tp < 1.f && want_p == 0) {  // the mass of the first k, from the token of rank k - 1
    if (e < n && part == 0 && rank == k - 1) sh.sel_mass = before + mass;
    __syncthreads();
    want_p = mass_target(tp, n >= k ? sh.sel_mass : all);
  }
  const bool keep = e < n && (k == 0 || rank < k) && (tp >= 1.f || before < want_p) &&
                    (w.hi - mp) + w.lo >= 0.f;
  const long long kept = keep ? mass : 0;
  __syncthreads();  // tok is read
  if (e < n && part == 0) tok[e] = make_uint4(0, idx, (uint32_t)kept, (uint32_t)(kept >> 32));
  __syncthreads();
  long long z = 0;
  before = 0;
  for (int j = j0; j < j1; ++j) {
    const uint4 o = tok[j];
    const long long m = (long long)o.z | ((long long)o.w << 32);
    if (o.y < idx) before += m;
    z += m;
  }
  before += __shfl_xor_sync(0xffffffffu, before, 1);
  z += __shfl_xor_sync(0xffffffffu, z, 1);
  const long long past = __double2ll_rd((double)u * (double)z);
  if (part == 0 && kept > 0 && before <= past && past < before + kept) {
    a.out_tokens[row] = (int)idx;
    if (a.out_prob != nullptr) a.out_prob[row] = df_quotient(w, pair_sum(z));
  }
}

// The filters and the draw over the list (the first CTA; n[q] tokens (value,
// index) of CTA q at list[q * (kListCap / C)]).
template <typename T>
__device__ void list_draw(Shared& sh, const uint2* list, const Law& law, int C, int k, bool has_k,
                          long long want_p, float tp, float mp, float u, uint32_t low,
                          const SampleArgs& a, int64_t row) {
  constexpr int kShift = sizeof(T) == 2 ? 16 : 0;
  const int tid = threadIdx.x;
  int n = 0, buf = 0;
  for (int q = 0; q < C; ++q) n += sh.ex_n[q];
  if (n <= kShortList) {
    short_draw(sh, list, law, C, n, has_k ? k : 0, want_p, tp, mp, u, a, row);
    return;
  }
  for (int i = tid; i < 2 * 4 * kBins; i += kThreads) (&sh.hist[0][0][0])[i] = 0;
  __syncthreads();
  uint32_t key[kListEach], idx[kListEach], mh[kListEach], ml[kListEach];
  float x[kListEach];
  uint32_t active = 0;
#pragma unroll
  for (int q = 0; q < kListEach; ++q) {
    key[q] = idx[q] = mh[q] = ml[q] = 0;
    x[q] = 0.f;
    const int at = q * kThreads + tid, cta = at / (kListCap / C);
    if (at % (kListCap / C) < sh.ex_n[cta]) {
      const uint2 e = list[at];
      x[q] = __uint_as_float(e.x);
      idx[q] = e.y;
      key[q] = order_key(x[q]) >> kShift;
      fixed_pair(law.weight(x[q]), mh[q], ml[q]);
      active |= 1u << q;
    }
  }
  const uint32_t base = max(low, kKeyNegInf + 1) >> kShift;
  const int bits = 32 - __clz((order_key(law.m) >> kShift) - base);
  uint32_t tau = 0;
  int keep_ties = 0, ties = 0;  // kept of the tokens at tau, all of them (tau 0: every token)
  long long each = 0;
  if (has_k) {
    const Picked s = list_select(sh, key, mh, ml, active, base, bits, false, k, buf);
    if (s.found) {
      tau = s.key;
      ties = (int)s.ties;
      keep_ties = k - (int)s.above;
      if (tp < 1.f) {
#pragma unroll
        for (int q = 0; q < kListEach; ++q)
          if (((active >> q) & 1u) && key[q] == tau) each = pair_value(mh[q], ml[q]);
        each = block_max(sh, each);
        want_p = mass_target(tp, s.mass + each * keep_ties);
        if (s.mass < want_p) {
          keep_ties = ties_for(want_p - s.mass, each, keep_ties);
          want_p = 0;
        }
      }
    } else if (tp < 1.f) {  // fewer tokens than k: all of them
      long long z = 0;
#pragma unroll
      for (int q = 0; q < kListEach; ++q) z += pair_value(mh[q], ml[q]);
      want_p = mass_target(tp, block_sum(sh, z));
    }
  }
  if (want_p > 0) {
    const Picked s = list_select(sh, key, mh, ml, active, base, bits, true, want_p, buf);
    if (s.found) {
      tau = s.key;
      ties = (int)s.ties;
      each = 0;
#pragma unroll
      for (int q = 0; q < kListEach; ++q)
        if (((active >> q) & 1u) && key[q] == tau) each = pair_value(mh[q], ml[q]);
      each = block_max(sh, each);
      keep_ties = ties_for(want_p - s.mass, each, ties);
    }
  }
  // kept: above tau, and at tau the first keep_ties by index
  uint32_t cut = ~0u;
  const uint32_t kTop = a.V - 1;  // descending keys of ascending indices
  const int idx_bits = 32 - __clz(kTop);
  uint32_t back[kListEach];
#pragma unroll
  for (int q = 0; q < kListEach; ++q) back[q] = kTop - idx[q];
  if (keep_ties < ties) {
    uint32_t at_tau = 0;
#pragma unroll
    for (int q = 0; q < kListEach; ++q)
      if (((active >> q) & 1u) && key[q] == tau) at_tau |= 1u << q;
    cut = kTop - list_select(sh, back, mh, ml, at_tau, 0, idx_bits, false, keep_ties, buf).key;
  }
  long long z = 0;
#pragma unroll
  for (int q = 0; q < kListEach; ++q) {
    const dfloat w = law.weight(x[q]);
    const bool keep = ((active >> q) & 1u) && (key[q] > tau || (key[q] == tau && idx[q] <= cut)) &&
                      (w.hi - mp) + w.lo >= 0.f;
    if (!keep) active &= ~(1u << q);
    else z += pair_value(mh[q], ml[q]);
  }
  z = block_sum(sh, z);
  const long long past = __double2ll_rd((double)u * (double)z) + 1;  // C_i > u Z
  const Picked s = list_select(sh, back, mh, ml, active, 0, idx_bits, true, past, buf);
#pragma unroll
  for (int q = 0; q < kListEach; ++q) {
    if (((active >> q) & 1u) && back[q] == s.key) {
      a.out_tokens[row] = (int)idx[q];
      if (a.out_prob != nullptr)
        a.out_prob[row] = df_quotient(law.weight(x[q]), pair_sum(z));
    }
  }
}

template <typename T, bool kSmem>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(SampleArgs a, int C, int slice,
                                                          int warp_vecs) {
  constexpr int kVec = 16 / sizeof(T);
  __shared__ Shared sh;
  extern __shared__ uint4 data[];
  const int tid = threadIdx.x, lane = tid % kWarp, warp = tid / kWarp;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = blockIdx.x % C;
  const int64_t row = blockIdx.x / C;
  pdl_trigger();
  cluster_arrive();  // every CTA of the cluster runs before its shared memory is written
  if (tid < 32) sh.draw.pow2[tid] = kPow2[tid];
  pdl_wait();  // the logits may come from the previous kernel

  const float T_ = a.temperature[row], u = a.uniform[row];
  const int k = a.top_k != nullptr ? a.top_k[row] : 0;
  const float tp = a.top_p != nullptr ? a.top_p[row] : 1.f;
  const float mp = a.min_p != nullptr ? a.min_p[row] : 0.f;
  const bool valid = temperature_valid(T_) && u >= 0.f && u < 1.f && k >= 0 && tp > 0.f &&
                     tp <= 1.f && mp >= 0.f && mp <= 1.f;
  const bool greedy = T_ == 0.f;
  const bool has_k = !greedy && k > 0 && k < a.V, has_p = !greedy && tp < 1.f;

  Slice<T, kSmem> sl;
  sl.src = static_cast<const T*>(a.logits) + row * a.stride + (int64_t)rank * slice;
  sl.off = (int)((reinterpret_cast<uintptr_t>(sl.src) & 15u) / sizeof(T));
  sl.n = max(0, min(slice, a.V - rank * slice));
  sl.sm = data;
  const int nv = kWarps * warp_vecs;

  // ---- 1: the slice, its maximum, elements that make the row fail
  float tmax = -INFINITY;
  int bad = 0;
  for (int v0 = tid; v0 < nv; v0 += kUnroll * kThreads) {
    uint4 raw[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
      if (v0 + j * kThreads < nv) raw[j] = sl.load(v0 + j * kThreads);
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      if (v0 + j * kThreads >= nv) break;
      if (kSmem) data[v0 + j * kThreads] = raw[j];
      float x[kVec];
      unpack16(raw[j], x);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        bad |= !(x[i] < INFINITY);  // NaN or +inf
        tmax = fmaxf(tmax, x[i]);
      }
    }
  }
  const float wm = warp_max(tmax);
  const uint32_t wl = __reduce_min_sync(0xffffffffu, order_key(tmax));
  if (lane == 0) {
    sh.red[warp] = wm;
    sh.red_low[warp] = wl;
  }
  bad = __syncthreads_or(bad);
  float m = sh.red[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) m = fmaxf(m, sh.red[w]);
  // lower bound of the tokens that can matter: the largest 16-bit key that at
  // least `need` of the threads' maxima reach
  uint32_t theta = 0;
  const int need = has_k ? ceil_div(k, C) : list_need_p(C);
  if (valid && (has_k || has_p)) {
    if (need <= kThreads) {
      const uint32_t key = order_key(tmax) >> 16;
      for (uint32_t bit = 0x8000u; bit != 0; bit >>= 1)
        if (__syncthreads_count(key >= (theta | bit)) >= need) theta |= bit;
    }
  }
  cluster_wait();
  if (tid < C) {
    *cluster.map_shared_rank(&sh.ex_max[rank], tid) = m;
    *cluster.map_shared_rank(&sh.ex_bad[rank], tid) = (uint32_t)bad;
    *cluster.map_shared_rank(&sh.ex_theta[rank], tid) = theta << 16;
    uint32_t low = sh.red_low[0];
    for (int w = 1; w < kWarps; ++w) low = min(low, sh.red_low[w]);
    *cluster.map_shared_rank(&sh.ex_low[rank], tid) = low;
  }
  cluster_sync();
  for (int q = 0; q < C; ++q) {
    m = fmaxf(m, sh.ex_max[q]);
    bad |= (int)sh.ex_bad[q];
    // for top-k every CTA's share has to lie above it; for top-p no CTA may
    // send more than its place
    theta = q == 0 ? sh.ex_theta[0]
            : has_k ? min(theta, sh.ex_theta[q]) : max(theta, sh.ex_theta[q]);
  }
  if (!valid || bad || m == -INFINITY) {
    if (rank == 0 && tid == 0) {
      raise_status(a.status, valid ? SPEC_ERR_NONFINITE : SPEC_ERR_INVALID_ARG);
      a.out_tokens[row] = -1;
      if (a.out_prob != nullptr) a.out_prob[row] = 0.f;
    }
    return;
  }
  if (greedy) {
    int first = 0x7fffffff;
    for (int v = tid; v < nv; v += kThreads) {
      const uint4 raw = sl.get(v);
      float x[kVec];
      unpack16(raw, x);
#pragma unroll
      for (int i = kVec - 1; i >= 0; --i)
        if (x[i] == m) first = min(first, rank * slice + v * kVec - sl.off + i);
    }
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) sh.draw.ties[warp] = first;
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < kWarps; ++w) first = min(first, sh.draw.ties[w]);
      *cluster.map_shared_rank(&sh.ex_first[rank], 0) = first;
    }
    cluster_sync();
    if (rank == 0 && tid == 0) {
      for (int q = 0; q < C; ++q) first = min(first, sh.ex_first[q]);
      a.out_tokens[row] = first;
      if (a.out_prob != nullptr) a.out_prob[row] = 1.f;
    }
    return;
  }

  const Law law(m, T_, sh.draw.pow2);
  // below it tokens weigh nothing (2^-120 of the largest: those masked by a low
  // value, for instance) and need no place, whatever the filters keep of them
  const uint32_t weightless = max(kKeyNegInf + 1, order_key(m - 120.5f / law.c_hi));

  // ---- 2a: few candidates go to the first CTA, which finishes the row
  dfloat total = df_make(0.f);  // mass of every token (top-p without top-k)
  const bool want_list = has_k ? need <= list_most_k(C) : has_p;
  const int places = kListCap / C;
  if (want_list) {
    if (tid == 0) sh.n_list = 0;
    __syncthreads();
    uint2* list = reinterpret_cast<uint2*>(data + (kSmem ? nv : 0));
    uint2* to = cluster.map_shared_rank(list, 0) + rank * places;
    const uint32_t low = max(theta, weightless);
    dfloat z = df_make(0.f);
    long long mass = 0;
    for (int v0 = 0; v0 < nv; v0 += kThreads) {
      const int v = v0 + tid;
      float x[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) x[i] = -INFINITY;
      if (v < nv) unpack16(sl.get(v), x);
      int n = 0;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const bool in = order_key(x[i]) >= low;
        n += in;
        if (!has_k) {
          const dfloat w = law.weight(x[i]);
          const dfloat s = df_two_sum(z.hi, w.hi);
          z.hi = s.hi;
          z.lo += s.lo + w.lo;
          if (in) {
            uint32_t hi, lo;
            fixed_pair(w, hi, lo);
            mass += pair_value(hi, lo);
          }
        }
      }
      if (__any_sync(0xffffffffu, n > 0)) {
        int at = n;
#pragma unroll
        for (int o = 1; o < kWarp; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, at, o);
          if (lane >= o) at += y;
        }
        int first = 0;
        if (lane == kWarp - 1) first = atomicAdd(&sh.n_list, at);
        at += __shfl_sync(0xffffffffu, first, kWarp - 1) - n;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          if (order_key(x[i]) >= low) {
            if (at < places)
              to[at] = make_uint2(__float_as_uint(x[i]), rank * slice + v * kVec - sl.off + i);
            ++at;
          }
      }
    }
    if (!has_k) {
      z = df_warp_sum(df_norm(z.hi, z.lo));
      if (lane == 0) sh.draw.mass[warp] = make_float2(z.hi, z.lo);
      mass = block_sum(sh, mass);
      z = df_make(0.f);
      for (int w = 0; w < kWarps; ++w) z = df_add(z, dfloat{sh.draw.mass[w].x, sh.draw.mass[w].y});
    } else {
      __syncthreads();
    }
    if (tid < C) {
      *cluster.map_shared_rank(&sh.ex_z[rank], tid) = make_float2(z.hi, z.lo);
      *cluster.map_shared_rank(&sh.ex_mass[rank], tid) = mass;
      *cluster.map_shared_rank(&sh.ex_n[rank], tid) = sh.n_list;
    }
    cluster_sync();
    bool fits = true;
    z = df_make(0.f);
    mass = 0;
    for (int q = 0; q < C; ++q) {
      fits &= sh.ex_n[q] <= places;
      z = df_add(z, dfloat{sh.ex_z[q].x, sh.ex_z[q].y});
      mass += sh.ex_mass[q];
    }
    total = z;
    const long long want =
        has_k ? 0 : mass_target(tp, __float2ll_rn(z.hi * 0x1p40f) + __float2ll_rn(z.lo * 0x1p40f));
    if (fits && mass >= want) {  // the same in every CTA
      if (rank == 0)
        list_draw<T>(sh, list, law, C, k, has_k, want, tp, mp, u, low, a, row);
      return;
    }
  }

  // ---- 2: the filters' threshold tau and how many tokens equal to it are kept
  uint32_t tau = kKeyNegInf;
  int keep_ties = 0;
  int buf = -1;
  const uint32_t high = order_key(m);
  if (has_k) {
    Selected s = radix_select<T, kSmem>(sh, sl, nv, law, theta, high, false, has_p, k, 0, C, buf);
    if (s.found) {
      tau = s.tau;
      keep_ties = k - (int)s.above;
      if (has_p) {
        const long long each = fixed_value(law.weight(key_value(tau)));
        const long long want = mass_target(tp, s.mass + each * keep_ties);
        if (s.mass >= want) {
          const Selected p =
              radix_select<T, kSmem>(sh, sl, nv, law, tau + 1, high, true, true, 0, want, C,
                                            buf);
          tau = p.tau;
          keep_ties = ties_for(want - p.mass, fixed_value(law.weight(key_value(tau))), (int)p.ties);
        } else {
          keep_ties = ties_for(want - s.mass, each, keep_ties);
        }
      }
    }
  }
  if (has_p && tau == kKeyNegInf) {  // no top-k, or fewer tokens than k
    // the mass of every token: known from 2a, or formed here
    dfloat z = total;
    if (has_k) {
      z = df_make(0.f);
      for (int v = tid; v < nv; v += kThreads) {
        const uint4 raw = sl.get(v);
        float x[kVec];
        unpack16(raw, x);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const dfloat w = law.weight(x[i]);
          const dfloat s = df_two_sum(z.hi, w.hi);
          z.hi = s.hi;
          z.lo += s.lo + w.lo;
        }
      }
      z = df_warp_sum(df_norm(z.hi, z.lo));
      if (lane == 0) sh.draw.mass[warp] = make_float2(z.hi, z.lo);
      __syncthreads();
      if (tid < C) {
        z = df_make(0.f);
        for (int w = 0; w < kWarps; ++w) z = df_add(z, dfloat{sh.draw.mass[w].x, sh.draw.mass[w].y});
        *cluster.map_shared_rank(&sh.ex_z[rank], tid) = make_float2(z.hi, z.lo);
      }
      cluster_sync();
      z = df_make(0.f);
      for (int q = 0; q < C; ++q) z = df_add(z, dfloat{sh.ex_z[q].x, sh.ex_z[q].y});
    }
    const long long zi = __float2ll_rn(z.hi * 0x1p42f) + __float2ll_rn(z.lo * 0x1p42f);
    const long long want = mass_target(tp, zi);
    // fp32: first the tokens that no thread's maximum is below, if they hold
    // enough
    uint32_t low = has_k || sizeof(T) == 2 ? weightless : sh.ex_low[0];
    if (!has_k && sizeof(T) == 4) {
      for (int q = 1; q < C; ++q) low = min(low, sh.ex_low[q]);
      low = max(low, weightless);
    }
    Selected p = radix_select<T, kSmem>(sh, sl, nv, law, low, high, true, true, 0, want, C, buf);
    if (!p.found && low > weightless)
      p = radix_select<T, kSmem>(sh, sl, nv, law, weightless, high, true, true, 0, want, C, buf);
    if (p.found) {
      tau = p.tau;
      keep_ties = ties_for(want - p.mass, fixed_value(law.weight(key_value(tau))), (int)p.ties);
    }
  }

  // ---- 3
  exact_draw<kWarps>(sh.draw, sl, law, tau, keep_ties, mp, u, warp_vecs, C, rank, rank * slice, a, row);
}

// ---------------------------------------------------------------------------
// rows without filters
// ---------------------------------------------------------------------------
// The row streams through registers once: a warp takes a chunk of 256
// vectors, its maximum, and its mass relative to that maximum with the
// hardware's exp2 -- five instructions an element against 45 for an exact
// weight.  The chunk that holds u Z is then walked with exact weights, and
// the token stands if u Z is further from both its steps than the masses can
// be off: per weight 1.47e-7 (ex2.approx: 2^-22.73 is the largest error over
// all arguments in [-126, 0], measured) and 2 * 2^-24 ln2 |y| for the two
// roundings of its exponent y, 3 * 2^-24 for the sum of two vectors' eight
// pairs (these sums and the lanes' add up as double-floats); sum w |y| is
// formed with the mass.  The
// rounding of log2(e)/T itself is taken out to first order by the same sum.
// Else (a few rows in a hundred at 150k tokens) the row is drawn exactly.
// (Copying a warp's next chunk to shared memory while it works made no
// difference: 640 rows of 152064 logits take about 41 us of streaming, at 58%
// of the issue slots, and 9 of start, choice and walk.)
constexpr uint32_t kMarkMask = 0xfffff;
constexpr int kPlainThreads = 256;
constexpr int kPlainWarps = kPlainThreads / kWarp;
constexpr int kChunkVecs = 256;  // 8 vectors a lane
constexpr int kMarkedClusters = 38;  // clusters of 8 CTAs that share the marked rows

struct PlainShared {
  DrawShared draw;
  // maximum, mass (hi, lo) and error of each chunk, relative to its maximum;
  // then mass (hi, lo) and error relative to the row's, and the maximum
  float4 stat[(kSampleMaxVocab / 4 + 8) / kChunkVecs + 1];
  float2 warp_mass[kPlainWarps];
  float pick_err;
  int sure;
};

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Two fp32 numbers in one register pair and the packed operations on them.
struct pair2 {
  unsigned long long v;
};
__device__ __forceinline__ pair2 pk(float a, float b) {
  pair2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpk(pair2 p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v));
}
__device__ __forceinline__ pair2 add2(pair2 a, pair2 b) {
  pair2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ pair2 sub2(pair2 a, pair2 b) {
  pair2 r;
  asm("{.reg .b64 m; mov.b64 m, 0xbf800000bf800000; fma.rn.f32x2 %0, %2, m, %1;}"
      : "=l"(r.v)
      : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ pair2 mul2(pair2 a, pair2 b) {
  pair2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ pair2 fma2(pair2 a, pair2 b, pair2 c) {
  pair2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// Maximum of a lane's vectors, NaN if any element is.
template <int N>
__device__ __forceinline__ float lane_max(const uint4 (&r)[N], __nv_bfloat16) {
  __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&r[0].x);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const uint32_t w[4] = {r[j].x, r[j].y, r[j].z, r[j].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __hmax2_nan(m, *reinterpret_cast<const __nv_bfloat162*>(&w[i]));
  }
  return max_nan(__low2float(m), __high2float(m));
}
template <int N>
__device__ __forceinline__ float lane_max(const uint4 (&r)[N], float) {
  float m = __uint_as_float(r[0].x);
#pragma unroll
  for (int j = 0; j < N; ++j)
    m = max_nan(max_nan(max_nan(m, __uint_as_float(r[j].x)), __uint_as_float(r[j].y)),
                max_nan(__uint_as_float(r[j].z), __uint_as_float(r[j].w)));
  return m;
}

// Elements of a vector, none below `low` (whose weight is 0), in pairs.
__device__ __forceinline__ void vec_pairs(const uint4& r, __nv_bfloat16 low, pair2 (&p)[4]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  const __nv_bfloat162 l2 = __halves2bfloat162(low, low);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), l2);
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&m);
    p[i] = pk(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
}
__device__ __forceinline__ void vec_pairs(const uint4& r, float low, pair2 (&p)[2]) {
  p[0] = pk(fmaxf(__uint_as_float(r.x), low), fmaxf(__uint_as_float(r.y), low));
  p[1] = pk(fmaxf(__uint_as_float(r.z), low), fmaxf(__uint_as_float(r.w), low));
}
// The type's lowest finite value.
__device__ __forceinline__ float lowest(__nv_bfloat16) { return __uint_as_float(0xff7f0000u); }
__device__ __forceinline__ float lowest(float) { return __uint_as_float(0xff7fffffu); }
// A value of the type at or below m - gap, and below m (a finite one if m is
// not the lowest).
__device__ __forceinline__ __nv_bfloat16 below(float m, float gap, __nv_bfloat16) {
  const uint32_t b = __float_as_uint(m) >> 16;  // m is a bf16
  const uint32_t next = m > 0.f ? b - 1 : (m < 0.f ? b + 1 : 0x8001u);
  return __float2bfloat16_rd(fminf(m - gap, __uint_as_float(next << 16)));
}
__device__ __forceinline__ float below(float m, float gap, float) {
  return fminf(m - gap, nextafterf(m, -INFINITY));
}

// This lane's vectors of a chunk of the row.
template <typename T>
__device__ __forceinline__ void load_chunk(const Slice<T, false>& row, int ch,
                                           uint4 (&raw)[kChunkVecs / kWarp]) {
  constexpr int kVec = 16 / sizeof(T);
  const int lane = threadIdx.x % kWarp;
  const int p = ch * kChunkVecs * kVec - row.off;
  if (p >= 0 && p + kChunkVecs * kVec <= row.n) {  // wholly inside
    const uint4* q = reinterpret_cast<const uint4*>(row.src + p) + lane;
#pragma unroll
    for (int j = 0; j < kChunkVecs / kWarp; ++j) raw[j] = __ldcs(q + j * kWarp);
  } else {
#pragma unroll
    for (int j = 0; j < kChunkVecs / kWarp; ++j)
      raw[j] = row.load(ch * kChunkVecs + j * kWarp + lane);
  }
}

// kDefer: rows that need the exact draw are marked for sample_marked_kernel.
template <typename T, bool kDefer>
__global__ void __launch_bounds__(kPlainThreads, 5)
    sample_plain_kernel(SampleArgs a, int C, int chunks, int slice, int warp_vecs) {
  constexpr int kVec = 16 / sizeof(T), kPairs = kVec / 2;
  constexpr int kLaneVecs = kChunkVecs / kWarp;
  constexpr int kSets = kLaneVecs / kPlainWarps;
  __shared__ PlainShared sh;
  const int tid = threadIdx.x, lane = tid % kWarp, warp = tid / kWarp;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = blockIdx.x % C;
  const int64_t row = blockIdx.x / C;
  pdl_trigger();
  cluster_arrive();  // every CTA of the cluster runs before its shared memory is written
  if (tid < 32) sh.draw.pow2[tid] = kPow2[tid];
  if (tid == 0) sh.sure = 0;
  pdl_wait();  // the logits may come from the previous kernel

  const float T_ = a.temperature[row], u = a.uniform[row];
  const bool valid = temperature_valid(T_) && u >= 0.f && u < 1.f;
  const bool greedy = T_ == 0.f;
  Slice<T, false> whole;  // the row
  whole.src = static_cast<const T*>(a.logits) + row * a.stride;
  whole.off = (int)((reinterpret_cast<uintptr_t>(whole.src) & 15u) / sizeof(T));
  whole.n = a.V;
  whole.sm = nullptr;
  const Law scale(0.f, valid && !greedy ? T_ : 1.f, sh.draw.pow2);
  const float c = scale.c_hi;
  cluster_wait();

  for (int ch = rank * kPlainWarps + warp; ch < chunks; ch += C * kPlainWarps) {
    uint4 raw[kLaneVecs];
    load_chunk(whole, ch, raw);
    float m = lane_max(raw, T());
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    float4 st = make_float4(m, 0.f, 0.f, 0.f);
    if (m == lowest(T())) {
      // a wholly masked chunk: its tokens at the lowest value weigh 1 each (no
      // value is below it but -inf, whose exponent would spoil the moment)
      int n = 0;
#pragma unroll
      for (int j = 0; j < kLaneVecs; ++j) {
        float x[kVec];
        unpack16(raw[j], x);
#pragma unroll
        for (int i = 0; i < kVec; ++i) n += x[i] == m;
      }
      st.y = (float)__reduce_add_sync(0xffffffffu, n);
    } else if (m < INFINITY && m > -INFINITY && !greedy) {
      const pair2 neg = pk(-m, -m), c2 = pk(c, c);
      const T low = below(m, 300.f / c, T());  // weights below 2^-300 are 0
      pair2 sum = pk(0.f, 0.f), lost = sum, moment = sum;
#pragma unroll
      for (int j = 0; j < kLaneVecs; j += 2) {
        pair2 p[2 * kPairs];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          pair2 x[kPairs];
          vec_pairs(raw[j + v], low, x);
#pragma unroll
          for (int i = 0; i < kPairs; ++i) {
            const pair2 d = add2(x[i], neg);
            float y0, y1;
            unpk(mul2(d, c2), y0, y1);
            const pair2 e = pk(fast_exp2(y0), fast_exp2(y1));
            moment = fma2(e, d, moment);
            p[v * kPairs + i] = e;
          }
        }
#pragma unroll
        for (int w = 1; w < 2 * kPairs; w *= 2)
#pragma unroll
          for (int i = 0; i + w < 2 * kPairs; i += 2 * w) p[i] = add2(p[i], p[i + w]);
        // the two vectors' sum joins the lane's, with what the addition
        // rounds off
        const pair2 s = add2(sum, p[0]), b = sub2(s, sum);
        lost = add2(lost, add2(sub2(sum, sub2(s, b)), sub2(p[0], b)));
        sum = s;
      }
      float s0, s1, l0, l1, a0, a1;
      unpk(sum, s0, s1);
      unpk(lost, l0, l1);
      unpk(moment, a0, a1);
      const dfloat s = df_warp_sum(df_add(df_two_sum(s0, s1), df_make(l0 + l1)));
      const float mom = warp_sum(a0 + a1);  // sum w (x - m), negative
      const dfloat fixed = df_add(s, df_make(mom * 0.693147181f * scale.c_lo));
      st.y = fixed.hi;
      st.z = fixed.lo;
      st.w = s.hi * (1.47e-7f + 3 * 0x1p-24f) - mom * c * (2 * 0.6931472f * 0x1p-24f);
    }
    if (lane < C) *cluster.map_shared_rank(&sh.stat[ch], lane) = st;
  }
  cluster_sync();  // every CTA has every chunk's statistics
  float m = -INFINITY;
  for (int ch = lane; ch < chunks; ch += kWarp) m = max_nan(m, sh.stat[ch].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (!valid || !(m < INFINITY) || m == -INFINITY) {
    if (rank == 0 && tid == 0) {
      raise_status(a.status, valid ? SPEC_ERR_NONFINITE : SPEC_ERR_INVALID_ARG);
      a.out_tokens[row] = -1;
      if (a.out_prob != nullptr) a.out_prob[row] = 0.f;
    }
    return;
  }
  if (greedy) {
    if (rank != 0 || warp != 0) return;
    int ch = 0x7fffffff;  // the first chunk that holds the maximum
    for (int i = chunks - 1 - lane; i >= 0; i -= kWarp)
      if (sh.stat[i].x == m) ch = i;
    ch = __reduce_min_sync(0xffffffffu, ch);
    int first = 0x7fffffff;
    for (int j = 0; j < kLaneVecs; ++j) {
      const int v = ch * kChunkVecs + j * kWarp + lane;
      const uint4 raw = whole.load(v);
      float x[kVec];
      unpack16(raw, x);
#pragma unroll
      for (int i = kVec - 1; i >= 0; --i)
        if (x[i] == m) first = min(first, v * kVec + i - whole.off);
    }
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) {
      a.out_tokens[row] = first;
      if (a.out_prob != nullptr) a.out_prob[row] = 1.f;
    }
    return;
  }
  const Law law(m, T_, sh.draw.pow2);
  __syncthreads();  // the maxima are read
  for (int ch = tid; ch < chunks; ch += kPlainThreads) {
    const float4 st = sh.stat[ch];
    const dfloat f = law.weight(st.x);
    const dfloat mass = df_add(df_mul_f(f, st.y), df_make(f.hi * st.z));
    sh.stat[ch] = make_float4(mass.hi, mass.lo, f.hi * st.w, st.x);
  }
  __syncthreads();
  if (warp == 0) {
    const int per = ceil_div(chunks, kWarp), c0 = lane * per, c1 = min(chunks, c0 + per);
    dfloat sum = df_make(0.f);
    float err = 0.f;
    for (int ch = c0; ch < c1; ++ch) {
      const float4 st = sh.stat[ch];
      sum = df_add(sum, dfloat{st.x, st.y});
      err += st.z;
    }
    const dfloat incl = df_warp_scan(sum);
    float err_to = err;  // errors of the chunks up to this lane's last
#pragma unroll
    for (int o = 1; o < kWarp; o <<= 1) {
      const float y = __shfl_up_sync(0xffffffffu, err_to, o);
      if (lane >= o) err_to += y;
    }
    const float err_all = __shfl_sync(0xffffffffu, err_to, kWarp - 1);
    const dfloat Z = df_shfl(incl, kWarp - 1), thr = df_mul_f(Z, u);
    const unsigned past = __ballot_sync(0xffffffffu, sum.hi > 0.f && df_gt(incl, thr));
    const int owner = past != 0 ? __ffs(past) - 1 : -1;
    if (lane == owner) {
      dfloat cum = df_sub(incl, sum);
      int ch = c0;
      float before = fmaxf(0.f, err_to - err);
      for (; ch + 1 < c1; ++ch) {
        const float4 st = sh.stat[ch];
        const dfloat next = df_add(cum, dfloat{st.x, st.y});
        if (df_gt(next, thr)) break;
        cum = next;
        before += st.z;
      }
      sh.draw.pick = ch;
      sh.draw.pick_base = make_float2(cum.hi, cum.lo);
      sh.draw.pick_z = make_float2(Z.hi, Z.lo);
      // C_i - u Z is off by at most (1 - u) times the error of the masses up to
      // i and u times that of the others (the chunk's own counted in both;
      // 1.0001 for the roundings of these sums)
      sh.pick_err = 1.0001f * ((1.f - u) * (before + sh.stat[ch].z) + u * (err_all - before));
    }
    if (owner < 0 && lane == 0) sh.draw.pick = -1;
  }
  __syncthreads();
  // one CTA walks the chunk and tells the others whether the token stands
  const int pick = sh.draw.pick;
  if (pick >= 0 && pick % C == rank) {
    // warp w holds the vectors [w, w + 1) * 256 / warps of the chunk, 32 at a time
    dfloat w[kSets][kVec], incl[kSets], sum[kSets], total = df_make(0.f);
    const int v0 = pick * kChunkVecs + warp * kSets * kWarp + lane;
#pragma unroll
    for (int j = 0; j < kSets; ++j) {
      const uint4 raw = whole.load(v0 + j * kWarp);
      float x[kVec];
      unpack16(raw, x);
      sum[j] = df_make(0.f);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        w[j][i] = law.weight(x[i]);
        sum[j] = df_add(sum[j], w[j][i]);
      }
      incl[j] = df_add(total, df_warp_scan(sum[j]));
      total = df_shfl(incl[j], kWarp - 1);
    }
    if (lane == 0) sh.warp_mass[warp] = make_float2(total.hi, total.lo);
    __syncthreads();
    dfloat base{sh.draw.pick_base.x, sh.draw.pick_base.y};
    for (int i = 0; i < warp; ++i)
      base = df_add(base, dfloat{sh.warp_mass[i].x, sh.warp_mass[i].y});
    const dfloat Z{sh.draw.pick_z.x, sh.draw.pick_z.y}, thr = df_mul_f(Z, u);
#pragma unroll
    for (int j = 0; j < kSets; ++j) {
      const dfloat upto = df_add(base, incl[j]);
      dfloat cum = df_sub(upto, sum[j]);
      if (sum[j].hi > 0.f && df_gt(upto, thr) && !df_gt(cum, thr)) {  // one thread at most
        int at = -1;
        dfloat wt = df_make(0.f), before = cum;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          if ((at < 0 || !df_gt(cum, thr)) && w[j][i].hi > 0.f) {
            before = cum;
            cum = df_add(cum, w[j][i]);
            at = i;
            wt = w[j][i];
          }
        }
        const float gap = fminf(df_to_f(df_sub(thr, before)), df_to_f(df_sub(cum, thr)));
        if (gap > sh.pick_err) {
          for (int q = 0; q < C; ++q) *cluster.map_shared_rank(&sh.sure, q) = 1;
          a.out_tokens[row] = (v0 + j * kWarp) * kVec + at - whole.off;
          if (a.out_prob != nullptr) a.out_prob[row] = df_quotient(wt, Z);
        }
      }
    }
  }
  cluster_sync();
  if (sh.sure) return;
  if (kDefer) {
    if (rank == 0 && tid == 0)
      a.out_tokens[row] = -2 - (int)(atomicAdd(a.status + 1, 1u) & kMarkMask);
    return;
  }
  Slice<T, false> sl;
  sl.src = whole.src + (int64_t)rank * slice;
  sl.off = (int)((reinterpret_cast<uintptr_t>(sl.src) & 15u) / sizeof(T));
  sl.n = max(0, min(slice, a.V - rank * slice));
  sl.sm = nullptr;
  exact_draw<kPlainWarps>(sh.draw, sl, law, kKeyNegInf, 0, 0.f, u, warp_vecs, C, rank, rank * slice,
                          a, row);
}

// The exact draw of the rows that sample_plain_kernel<T, true> marked with a
// token of -2 - i (i counts the marks): cluster i % G of the G takes them.  A
// few rows in a hundred come here, so the whole GPU shares them, where a CTA
// that drew its own row exactly kept the others waiting at the end (640 rows
// of 152064 bf16 logits: 105 us, against 75 us with this kernel at the time).
constexpr int kMarkedRows = 4;  // rows a thread looks at in one round

struct MarkedShared {
  DrawShared draw;
  float ex_max[kMaxCluster];
  float red[kWarps];
  int warp_n[kWarps];
  int list[kMarkedRows * kThreads];
};

template <typename T, bool kSmem>
__global__ void __launch_bounds__(kThreads) sample_marked_kernel(SampleArgs a, int C, int slice,
                                                                 int warp_vecs) {
  constexpr int kVec = 16 / sizeof(T);
  __shared__ MarkedShared sh;
  extern __shared__ uint4 data[];
  const int tid = threadIdx.x, lane = tid % kWarp, warp = tid / kWarp;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = blockIdx.x % C, G = gridDim.x / C, mine = blockIdx.x / C;
  pdl_trigger();
  cluster_arrive();
  if (tid < 32) sh.draw.pow2[tid] = kPow2[tid];
  pdl_wait();
  cluster_wait();
  for (int base = 0; base < a.rows; base += kMarkedRows * kThreads) {
    // marked rows of this block of rows that are this cluster's, in order
    // (other clusters may be writing tokens over their own marks)
    int mark[kMarkedRows], n = 0;
#pragma unroll
    for (int j = 0; j < kMarkedRows; ++j) {
      const int r = base + tid * kMarkedRows + j;
      mark[j] = r < a.rows ? -2 - a.out_tokens[r] : -1;
    }
#pragma unroll
    for (int j = 0; j < kMarkedRows; ++j) n += mark[j] >= 0 && mark[j] % G == mine;
    int at = n;
#pragma unroll
    for (int o = 1; o < kWarp; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += y;
    }
    if (lane == kWarp - 1) sh.warp_n[warp] = at;
    __syncthreads();
    at -= n;
    n = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += sh.warp_n[w];
      n += sh.warp_n[w];
    }
#pragma unroll
    for (int j = 0; j < kMarkedRows; ++j)
      if (mark[j] >= 0 && mark[j] % G == mine) sh.list[at++] = base + tid * kMarkedRows + j;
    __syncthreads();
    for (int i = 0; i < n; ++i) {
      const int64_t row = sh.list[i];
      Slice<T, kSmem> sl;
      sl.src = static_cast<const T*>(a.logits) + row * a.stride + (int64_t)rank * slice;
      sl.off = (int)((reinterpret_cast<uintptr_t>(sl.src) & 15u) / sizeof(T));
      sl.n = max(0, min(slice, a.V - rank * slice));
      sl.sm = data;
      float m = -INFINITY;
      for (int v = tid; v < kWarps * warp_vecs; v += kThreads) {
        const uint4 raw = sl.load(v);
        if (kSmem) data[v] = raw;
        float x[kVec];
        unpack16(raw, x);
#pragma unroll
        for (int j = 0; j < kVec; ++j) m = fmaxf(m, x[j]);
      }
      m = warp_max(m);
      if (lane == 0) sh.red[warp] = m;
      __syncthreads();
      if (tid < C) {
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sh.red[w]);
        *cluster.map_shared_rank(&sh.ex_max[rank], tid) = m;
      }
      cluster_sync();
      for (int q = 0; q < C; ++q) m = fmaxf(m, sh.ex_max[q]);
      const Law law(m, a.temperature[row], sh.draw.pow2);
      exact_draw<kWarps>(sh.draw, sl, law, kKeyNegInf, 0, 0.f, a.uniform[row], warp_vecs, C, rank,
                         rank * slice, a, row);
      cluster_sync();  // the exchange is read
    }
    __syncthreads();  // the list is read
  }
}

struct ClusterLaunch {  // use in place: cfg points at attr
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg;
  ClusterLaunch(int64_t rows, int C, int threads, size_t smem, cudaStream_t st) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg = cudaLaunchConfig_t{};
    cfg.gridDim = dim3((unsigned)(rows * C));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
  ClusterLaunch(const ClusterLaunch&) = delete;
  ClusterLaunch& operator=(const ClusterLaunch&) = delete;
};

template <typename T>
static cudaError_t launch_t(const SampleArgs& a, cudaStream_t st, int* launches) {
  constexpr int kVec = 16 / sizeof(T);
  const bool plain = a.top_k == nullptr && a.top_p == nullptr && a.min_p == nullptr;
  int C = 1;
  if (plain) {
    const int chunks = ceil_div(ceil_div(a.V, kVec) + 1, kChunkVecs);
    auto slice_of = [&](int c) { return ceil_div(ceil_div(a.V, c), kVec) * kVec; };
    auto vecs_of = [&](int c, int warps) { return ceil_div(slice_of(c) / kVec + 1, warps); };
    // enough CTAs to fill the GPU twice over, as long as each has a chunk a warp
    while (C < kMaxCluster && C * kPlainWarps < chunks && (int64_t)a.rows * C < 608) C *= 2;
    const bool defer = C <= 2 && chunks > 8;
    {
      ClusterLaunch L(a.rows, C, kPlainThreads, 0, st);
      const cudaError_t e = cudaLaunchKernelEx(
          &L.cfg, defer ? sample_plain_kernel<T, true> : sample_plain_kernel<T, false>, a, C, chunks,
          slice_of(C), vecs_of(C, kPlainWarps));
      ++*launches;
      if (e != cudaSuccess || !defer) return e;
    }
    C = kMaxCluster;
    const int vecs = vecs_of(C, kWarps);
    const size_t bytes = (size_t)kWarps * vecs * 16;
    const bool fits = bytes + sizeof(MarkedShared) <= kMaxSharedBytes;
    auto kern = fits ? sample_marked_kernel<T, true> : sample_marked_kernel<T, false>;
    const size_t smem = fits ? bytes : 0;
    const cudaError_t e = allow_shared(kern, fits ? kMaxSharedBytes - sizeof(MarkedShared) : 0);
    if (e != cudaSuccess) return e;
    ClusterLaunch L(min(kMarkedClusters, a.rows), C, kThreads, smem, st);
    ++*launches;
    return cudaLaunchKernelEx(&L.cfg, kern, a, C, slice_of(C), vecs);
  }
  // CTAs per row: those of the least estimated time.  A row takes about 12 us
  // for its chain of barriers, and for each KB of a slice 0.05 us with top-k
  // alone and about 0.2 where every token is weighted (top-p, min-p).  An SM
  // holds two CTAs, or one when their shared memory is over half of it, and a
  // cluster stays inside one of eight parts of 19 SMs.  (33 rows of 32001 fp32
  // logits, top-k 50: 24 us with 8 CTAs a row, which makes two waves, 18 with
  // 4; 33 rows of 128256 bf16, top-p 0.9: 45 us with 8, 61 with 2; 256 of them,
  // top-k 50: 122 us with 8, 78 with 2.)
  auto slice_of = [&](int c) { return ceil_div(ceil_div(a.V, c), kVec) * kVec; };
  // a row may start anywhere in a 16-byte vector: up to one more vector
  auto vecs_of = [&](int c) { return ceil_div(slice_of(c) / kVec + 1, kWarps); };
  const size_t list = sizeof(uint2) * kListCap;
  const int64_t per_kb = a.top_p == nullptr && a.min_p == nullptr ? 50 : 200;
  C = kMaxCluster;
  int64_t best = INT64_MAX;
  for (int c = kMaxCluster; c >= 1; c /= 2) {
    const size_t bytes = (size_t)kWarps * vecs_of(c) * 16, all = bytes + list + sizeof(Shared);
    if (all > kMaxSharedBytes) break;
    const int per_sm = 2 * (all + 1024) <= 228 * 1024 ? 2 : 1;
    const int64_t waves = ceil_div64(a.rows, 8 * (19 * per_sm / c));
    const int64_t ns = waves * (12000 + per_kb * (int64_t)(bytes / 1024));
    if (ns < best) {
      best = ns;
      C = c;
    }
  }
  const bool fits = best != INT64_MAX;
  const int warp_vecs = vecs_of(C);
  auto kern = fits ? sample_kernel<T, true> : sample_kernel<T, false>;
  const size_t smem = (fits ? (size_t)kWarps * warp_vecs * 16 : 0) + list;
  const cudaError_t e = allow_shared(kern, fits ? kMaxSharedBytes - sizeof(Shared) : list);
  if (e != cudaSuccess) return e;
  ClusterLaunch L(a.rows, C, kThreads, smem, st);
  ++*launches;
  return cudaLaunchKernelEx(&L.cfg, kern, a, C, slice_of(C), warp_vecs);
}

}  // namespace smp

cudaError_t sample_launch(const SampleArgs& a, cudaStream_t st, int* launches) {
  const cudaError_t e = a.dtype == SPEC_BF16 ? smp::launch_t<__nv_bfloat16>(a, st, launches)
                                             : smp::launch_t<float>(a, st, launches);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace specv
