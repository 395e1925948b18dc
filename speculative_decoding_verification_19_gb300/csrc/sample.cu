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
// Rounding.  The token is a whole number that hangs on a comparison of sums,
// so the sums are held to about 2^-40 of their value, not to fp32's 2^-24
// (with 150k tokens every second row has a step of C within fp32's error of
// u Z).  Weights come as double-floats (fp32 pairs; exact to about 2^-32 of
// each weight): the exponential by table and polynomial (P. T. P. Tang,
// "Table-driven implementation of the exponential function", ACM TOMS 1989),
// 2^(j/32) from the table and four terms of the series for the rest, sums as
// double-floats.  GB300's fp64 rate is a hundredth of its fp32 rate, so
// nothing here is a per-element fp64 operation.  Masses that the filters
// compare are 42-bit fixed-point integers: their sums do not depend on the
// order of the atomics that form them.
//
// One cluster of up to 16 CTAs per row, each with a slice of the row in shared
// memory: the row is read from HBM once, whatever the filters ask for, and
// what the CTAs tell one another (maxima, histograms, masses) goes through
// distributed shared memory.  Rows whose slices do not fit are read again
// through L2 instead.  Steps:
//   1  slice to shared memory, maximum, rows without a distribution
//   2  with top-k or top-p: a radix select over the order keys, 8 bits a
//      level, on counts or on masses.  Only tokens that can matter take part:
//      for top-k those at or above a lower bound of the k-th value taken from
//      the threads' maxima (n threads' maxima >= v make n tokens >= v), for
//      top-p those above every thread's maximum's minimum, if they hold the
//      mass that is asked for (checked; else all)
//   3  the kept mass of every warp's run of tokens, exchanged; the warp that
//      holds u Z walks its run in order
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
constexpr int kBins = 256;
constexpr uint32_t kKeyNegInf = 0x007fffffu;  // order key of -inf
constexpr int kUnroll = 4;
constexpr size_t kMaxSliceBytes = 200 * 1024;

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

struct Shared {
  float2 pow2[32];
  uint32_t hist[2][4][kBins];  // counts, then the masses' three 14-bit limbs
  float2 mass[kMaxCluster * kWarps];
  int ties[kMaxCluster * kWarps];
  float ex_max[kMaxCluster];
  uint32_t ex_bad[kMaxCluster], ex_theta[kMaxCluster];
  float2 ex_z[kMaxCluster];
  int ex_first[kMaxCluster];
  float red[kWarps];
  uint32_t scan_cnt[kBins / kWarp];
  long long scan_mass[kBins / kWarp];
  int sel_bin;
  uint32_t sel_above, sel_count;
  long long sel_mass;
  int pick, pick_ties;
  float2 pick_base, pick_z;
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
  // exp((x - m) / T) as a double-float; 0 below 2^-120
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

struct Selected {
  bool found;
  uint32_t tau;   // order key of the threshold
  uint32_t above, ties;
  long long mass;  // of the tokens above tau (when masses were summed)
};

// Radix select over the tokens with order key >= low: the value of rank
// `rank` (1 = largest), or, with by_mass, the first at which the running mass
// reaches `mass`.  Not found when all of them together fall short.
template <typename T, bool kSmem>
__device__ Selected radix_select(Shared& sh, const Slice<T, kSmem>& sl, int nv, const Law& law,
                                 uint32_t low, bool by_mass, bool with_mass, long long rank,
                                 long long mass, int C, int& buf) {
  constexpr int kVec = Slice<T, kSmem>::kVec;
  const int tid = threadIdx.x, lane = tid % kWarp;
  cg::cluster_group cluster = cg::this_cluster();
  Selected r{true, 0, 0, 0, 0};
  uint32_t prefix = 0, mask = 0;
  constexpr int kLast = sizeof(T) == 2 ? 16 : 0;
  if (low <= kKeyNegInf) low = kKeyNegInf + 1;
  for (int shift = 24; shift >= kLast; shift -= 8) {
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
        if (key >= low && (key & mask) == prefix) {
          const int bin = (key >> shift) & (kBins - 1);
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
    // thread i: bin 255 - i, summed over the cluster, then the running sums
    uint32_t cnt = 0, ci = 0;
    long long ms = 0, mi = 0;
    if (tid < kBins) {
      const int bin = kBins - 1 - tid;
      for (int q = 0; q < C; ++q) {
        const uint32_t* h = cluster.map_shared_rank(&sh.hist[buf][0][0], q);
        cnt += h[bin];
        if (with_mass)
          ms += limbs_value(h[kBins + bin], h[2 * kBins + bin], h[3 * kBins + bin]);
      }
      ci = cnt;
      mi = ms;
#pragma unroll
      for (int o = 1; o < kWarp; o <<= 1) {
        const uint32_t yc = __shfl_up_sync(0xffffffffu, ci, o);
        const long long ym = __shfl_up_sync(0xffffffffu, mi, o);
        if (lane >= o) {
          ci += yc;
          mi += ym;
        }
      }
      if (lane == kWarp - 1) {
        sh.scan_cnt[tid / kWarp] = ci;
        sh.scan_mass[tid / kWarp] = mi;
      }
    }
    __syncthreads();
    if (tid < kBins) {
      for (int w = 0; w < tid / kWarp; ++w) {
        ci += sh.scan_cnt[w];
        mi += sh.scan_mass[w];
      }
      const long long before = by_mass ? r.mass + mi - ms : (long long)r.above + ci - cnt;
      const long long upto = by_mass ? r.mass + mi : (long long)r.above + ci;
      const long long want = by_mass ? mass : rank;
      if (before < want && want <= upto) {
        sh.sel_bin = kBins - 1 - tid;
        sh.sel_above = ci - cnt;
        sh.sel_mass = mi - ms;
        sh.sel_count = cnt;
      }
    }
    __syncthreads();
    buf ^= 1;
    const int bin = sh.sel_bin;
    if (bin < 0) {
      r.found = false;
      return r;
    }
    r.above += sh.sel_above;
    r.mass += sh.sel_mass;
    r.ties = sh.sel_count;
    prefix |= (uint32_t)bin << shift;
    mask |= (uint32_t)(kBins - 1) << shift;
    __syncthreads();  // sel_* are read
  }
  // the bits below a bf16 key: zeros, or ones for a negative value
  r.tau = sizeof(T) == 2 && !(prefix & 0x80000000u) ? prefix | 0xffffu : prefix;
  return r;
}

template <typename T, bool kSmem>
__global__ void __launch_bounds__(kThreads) sample_kernel(SampleArgs a, int C, int slice,
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
  if (tid < 32) sh.pow2[tid] = kPow2[tid];
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
  if (lane == 0) sh.red[warp] = wm;
  bad = __syncthreads_or(bad);
  float m = sh.red[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) m = fmaxf(m, sh.red[w]);
  // lower bound of the tokens that can matter: the largest 16-bit key that at
  // least `need` of the threads' maxima reach
  uint32_t theta = 0;
  if (valid && (has_k || has_p)) {
    const int need = has_k ? ceil_div(k, C) : kThreads;
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
  }
  cluster_sync();
  for (int q = 0; q < C; ++q) {
    m = fmaxf(m, sh.ex_max[q]);
    bad |= (int)sh.ex_bad[q];
    theta = q == 0 ? sh.ex_theta[0] : min(theta, sh.ex_theta[q]);
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
    if (lane == 0) sh.ties[warp] = first;
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < kWarps; ++w) first = min(first, sh.ties[w]);
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

  Law law;
  law.m = m;
  law.pow2 = sh.pow2;
  // log2(e) / T: log2(e) as a double-float, the quotient's remainder exact
  law.c_hi = 1.44269502f / T_;
  law.c_lo = (fmaf(-law.c_hi, T_, 1.44269502f) + 1.92596303e-8f) / T_;

  // ---- 2: the filters' threshold tau and how many tokens equal to it are kept
  uint32_t tau = kKeyNegInf;
  int keep_ties = 0;
  int buf = 0;
  if (has_k) {
    Selected s = radix_select<T, kSmem>(sh, sl, nv, law, theta, false, has_p, k, 0, C, buf);
    if (s.found) {
      tau = s.tau;
      keep_ties = k - (int)s.above;
      if (has_p) {
        const long long each = fixed_value(law.weight(key_value(tau)));
        const long long want = mass_target(tp, s.mass + each * keep_ties);
        if (s.mass >= want) {
          const Selected p =
              radix_select<T, kSmem>(sh, sl, nv, law, tau + 1, true, true, 0, want, C, buf);
          tau = p.tau;
          keep_ties = ties_for(want - p.mass, fixed_value(law.weight(key_value(tau))), (int)p.ties);
        } else {
          keep_ties = ties_for(want - s.mass, each, keep_ties);
        }
      }
    }
  }
  if (has_p && tau == kKeyNegInf) {  // no top-k, or fewer tokens than k
    dfloat z = df_make(0.f);
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
    if (lane == 0) sh.mass[warp] = make_float2(z.hi, z.lo);
    __syncthreads();
    if (tid < C) {
      z = df_make(0.f);
      for (int w = 0; w < kWarps; ++w) z = df_add(z, dfloat{sh.mass[w].x, sh.mass[w].y});
      *cluster.map_shared_rank(&sh.ex_z[rank], tid) = make_float2(z.hi, z.lo);
    }
    cluster_sync();
    z = df_make(0.f);
    for (int q = 0; q < C; ++q) z = df_add(z, dfloat{sh.ex_z[q].x, sh.ex_z[q].y});
    const long long zi = __float2ll_rn(z.hi * 0x1p42f) + __float2ll_rn(z.lo * 0x1p42f);
    const long long want = mass_target(tp, zi);
    Selected p = radix_select<T, kSmem>(sh, sl, nv, law, has_k ? 0u : theta, true, true, 0, want,
                                        C, buf);
    if (!p.found && !has_k)
      p = radix_select<T, kSmem>(sh, sl, nv, law, 0u, true, true, 0, want, C, buf);
    if (p.found) {
      tau = p.tau;
      keep_ties = ties_for(want - p.mass, fixed_value(law.weight(key_value(tau))), (int)p.ties);
    }
  }

  // ---- 3: kept masses of the warps' runs, in vocabulary order
  const bool filtered = tau != kKeyNegInf || mp > 0.f;
  dfloat w_tau = df_make(0.f);
  if (tau != kKeyNegInf) {
    w_tau = law.weight(key_value(tau));
    if ((w_tau.hi - mp) + w_tau.lo < 0.f) w_tau = df_make(0.f);
  }
  const int v_lo = warp * warp_vecs, v_hi = v_lo + warp_vecs;
  {
    dfloat z = df_make(0.f);
    int ties = 0;
    for (int v = v_lo + lane; v < v_hi; v += kWarp) {
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
        const dfloat s = df_two_sum(z.hi, w.hi);
        z.hi = s.hi;
        z.lo += s.lo + w.lo;
      }
    }
    z = df_warp_sum(df_norm(z.hi, z.lo));
    ties = (int)__reduce_add_sync(0xffffffffu, (unsigned)ties);
    if (lane < C) {
      *cluster.map_shared_rank(&sh.mass[rank * kWarps + warp], lane) = make_float2(z.hi, z.lo);
      *cluster.map_shared_rank(&sh.ties[rank * kWarps + warp], lane) = ties;
    }
  }
  cluster_sync();  // from here on each CTA touches only its own shared memory
  if (warp == 0) {
    const int per = kMaxCluster * kWarps / kWarp;  // runs of a lane
    const int runs = C * kWarps;
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
  if (pick / kWarps != rank || pick % kWarps != warp) return;
  const dfloat Z{sh.pick_z.x, sh.pick_z.y};
  const dfloat thr = df_mul_f(Z, u);
  dfloat cum{sh.pick_base.x, sh.pick_base.y};
  int tie_base = sh.pick_ties;
  int last = -1;        // this lane's last kept token so far
  float last_w = 0.f;
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
#pragma unroll
    for (int o = 1; o < kWarp; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, it, o);
      if (lane >= o) it += y;
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
        last_w = w[i].hi;
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
        float wt = 0.f;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          if ((at < 0 || !df_gt(c, thr)) && w[i].hi > 0.f) {
            c = df_add(c, w[i]);
            at = v * kVec + i;
            wt = w[i].hi;
          }
        }
        a.out_tokens[row] = rank * slice + at - sl.off;
        if (a.out_prob != nullptr) a.out_prob[row] = wt / df_to_f(Z);
      }
      return;
    }
    cum = df_shfl(incl, kWarp - 1);
  }
  // u Z at the run's very end, within the sums' rounding: its last kept token
  const int top = __reduce_max_sync(0xffffffffu, last);
  if (last == top && top >= 0) {
    a.out_tokens[row] = rank * slice + top - sl.off;
    if (a.out_prob != nullptr) a.out_prob[row] = last_w / df_to_f(Z);
  }
}

template <typename T>
static cudaError_t launch_t(const SampleArgs& a, cudaStream_t st) {
  constexpr int kVec = 16 / sizeof(T);
  // CTAs per row: slices of at most 24 KB, so that several clusters share an SM
  int C = 1;
  while (C < kMaxCluster && ceil_div64(a.V, C) * (int)sizeof(T) > 8192) C *= 2;
  const int slice = ceil_div(ceil_div(a.V, C), kVec) * kVec;
  // a row may start anywhere in a 16-byte vector: up to one more vector
  const int warp_vecs = ceil_div(slice / kVec + 1, kWarps);
  const size_t bytes = (size_t)kWarps * warp_vecs * 16;
  const bool fits = bytes <= kMaxSliceBytes;
  auto kern = fits ? sample_kernel<T, true> : sample_kernel<T, false>;
  const size_t smem = fits ? bytes : 0;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((int64_t)a.rows * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a, C, slice, warp_vecs);
}

}  // namespace smp

cudaError_t sample_launch(const SampleArgs& a, cudaStream_t st, int* launches) {
  const cudaError_t e =
      a.dtype == SPEC_BF16 ? smp::launch_t<__nv_bfloat16>(a, st) : smp::launch_t<float>(a, st);
  ++*launches;
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace specv
