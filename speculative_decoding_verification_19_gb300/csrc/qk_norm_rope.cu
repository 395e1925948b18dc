// RMS norm of every query and key head and the position rotation in one pass,
// with an optional write of the keys and values to the paged cache.
//
// What is computed for a head x of D values at position t, with weight w and
// inverse frequencies f_j (j < rot/2):
//   y = x * rsqrt(mean(x^2) + eps) * w          (y = x without a weight)
//   (y_a, y_b) -> (y_a cos(t f_j) - y_b sin(t f_j), y_b cos(t f_j) + y_a sin(t f_j))
// for the pairs (a, b) = (j, j + rot/2), or (2j, 2j + 1) interleaved.  All in
// fp32, rounded once when stored.
//
// The angle.  t f_j in fp32 loses t * 2^-24 of a radian, which is everything
// at far positions.  A turn is a fraction of 2^64 here: f_j / 2 pi is turned
// into a 64-bit fixed-point fraction once per CTA (in fp64), and t times it,
// modulo 2^64, is the angle in turns by one integer product -- the reduction
// modulo 2 pi is the overflow.  Its error is t * 2^-54 turns (the fp64
// product's rounding).  The top 32 bits, less the nearest quarter turn, go to
// sincospif.
//
// Every byte is read once and written once, so the bound is HBM.  One warp
// takes a run of query heads, or of key and value heads, of one token: a head
// is 8..32 lanes of 16 bytes, so the sum of squares and the partner of a pair
// are shuffles (of the packed values), and no shared memory or barrier sits
// between a load and its store.  A warp forms its token's cosines and sines
// once, two a lane, hands them round by shuffles and multiplies the head's
// weight into them: w_a cos and w_b sin stay in registers, which leaves few
// enough of them for 32 warps an SM with four loads each in flight.
// 16384 rows of 64 + 8 bf16 heads of 128 with the cache written (705 MB):
// 118 us (104 at the copy rate); 178 us with the weights and both kinds of
// heads in one loop at 16 warps an SM.
// (Packed fp32 pairs for the products took 135 us: pairing the unpacked halves
// costs more than the packed instructions save.)
#include "qk_norm_rope.cuh"

namespace specv {
namespace rope {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / kWarp;
constexpr int kUnroll = 4;  // 16-byte loads in flight per lane
constexpr int kMaxHalf = 64;

// cos and sin of turns / 2^64 of a full turn.
__device__ __forceinline__ void turn_cos_sin(uint64_t turns, float* c, float* s) {
  const uint32_t t = (uint32_t)(turns >> 32);
  const uint32_t quarter = (t + 0x20000000u) >> 30;        // nearest quarter turn, modulo 4
  const int32_t rest = (int32_t)(t - (quarter << 30));     // [-2^29, 2^29)
  float sn, cs;
  sincospif((float)rest * 0x1p-31f, &sn, &cs);
  const float a = (quarter & 1u) ? sn : cs, b = (quarter & 1u) ? cs : sn;
  // quarters 0..3: (cs, sn), (-sn, cs), (-cs, -sn), (sn, -cs)
  *c = (quarter == 1u || quarter == 2u) ? -a : a;
  *s = (quarter >= 2u) ? -b : b;
}

template <int N>
__device__ __forceinline__ uint4 pack16(const float (&f)[N]);
template <>
__device__ __forceinline__ uint4 pack16<4>(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}
template <>
__device__ __forceinline__ uint4 pack16<8>(const float (&f)[8]) {
  uint4 r;
  uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return r;
}

// Work of a warp: `units` runs of heads per row, the first uq of them query
// heads (q_run each), the others key and value heads (kv_run each).
struct Split {
  int uq, units, q_run, kv_run;
};

template <typename T, int D, bool kInter>
__global__ void __launch_bounds__(kThreads, 4) qk_norm_rope_kernel(RopeArgs a, Split sp,
                                                                   uint32_t* status) {
  constexpr int kVec = 16 / sizeof(T);      // elements of a lane
  constexpr int kLanes = D / kVec;          // lanes of a head: 8, 16 or 32
  constexpr int kHeads = kWarp / kLanes;    // heads of a warp's load
  __shared__ uint64_t freq[kMaxHalf];
  const int tid = threadIdx.x, lane = tid % kWarp;
  const int sub = lane % kLanes, hsub = lane / kLanes, e0 = sub * kVec;
  const int half = a.rot_dim / 2;
  const int Hq = a.d.Hq, Hkv = a.d.Hkv;
  pdl_trigger();
  pdl_wait();  // the projections and positions may come from the previous kernel
  for (int j = tid; j < kMaxHalf; j += kThreads) {
    const double f = j < half ? a.inv_freq[j] * 0.15915494309189533577 : 0.0;  // turns per position
    freq[j] = (uint64_t)((f - floor(f)) * 18446744073709551616.0);
  }
  __syncthreads();

  const bool cached = a.slots != nullptr;
  const int kv_heads = cached ? 2 * Hkv : Hkv;
  const int64_t n_units = (int64_t)a.rows * sp.units;
  const int64_t warps = (int64_t)gridDim.x * kWarps;
  const bool turned = e0 < a.rot_dim;
  // the lane that holds the other element of this lane's pairs (half-split)
  const int partner = (!turned || kInter) ? lane
                      : e0 < half         ? lane + half / kVec
                                          : lane - half / kVec;
  for (int64_t u = (int64_t)blockIdx.x * kWarps + tid / kWarp; u < n_units; u += warps) {
    const int64_t row = u / sp.units;
    const int part = (int)(u - row * sp.units);
    const bool is_q = part < sp.uq;
    const int h0 = is_q ? part * sp.q_run : (part - sp.uq) * sp.kv_run;
    const int h1 = min(is_q ? Hq : kv_heads, h0 + (is_q ? sp.q_run : sp.kv_run));
    // heads below hk are turned, the others are values
    const int hk = is_q ? h1 : min(h1, Hkv);
    const T* src = (is_q ? static_cast<const T*>(a.q) + row * a.q_stride
                         : static_cast<const T*>(a.k) + row * a.k_stride) + e0;
    const T* vsrc = static_cast<const T*>(a.v) + row * a.v_stride - (int64_t)Hkv * D + e0;
    const int pos = a.positions[row];
    int64_t slot = -1;
    if (cached && !is_q) {
      slot = a.slots[row];
      if (slot >= (int64_t)a.d.num_blocks * kBlock) {
        if (lane == 0) raise_status(status, SPEC_ERR_DEVICE_BOUNDS);
        slot = -1;
      }
      if (pos < 0 || slot < 0) slot = -1;
    }
    const int64_t page = slot < 0 ? 0 : slot / kBlock * Hkv * kBlock + slot % kBlock;
    T* out = is_q ? static_cast<T*>(a.q_out) + row * Hq * D + e0
                  : static_cast<T*>(a.k_out) + row * Hkv * D + e0;
    const bool write = is_q || a.k_out != nullptr;
    const bool norm = (is_q ? a.q_weight : a.k_weight) != nullptr;
    float wc[kVec], ws[kVec];  // weight times cosine; partner's weight times +-sine
    bool ready = false;
    for (int h = h0; h < h1; h += kUnroll * kHeads) {
      uint4 raw[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int hh = h + k * kHeads + hsub;
        raw[k] = make_uint4(0, 0, 0, 0);
        if (hh < h1)
          raw[k] = *reinterpret_cast<const uint4*>((hh < hk ? src : vsrc) + (int64_t)hh * D);
      }
      if (!ready) {  // after the first loads are on their way
        ready = true;
        // lane l forms the angles of frequencies 2l and 2l + 1
        float c2[2], s2[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          turn_cos_sin((uint64_t)(uint32_t)pos * freq[2 * lane + i], &c2[i], &s2[i]);
        const T* w = static_cast<const T*>(is_q ? a.q_weight : a.k_weight);
        const int j0 = kInter ? e0 / 2 : (e0 < half || !turned ? e0 : e0 - half);
        const int mate = kInter ? e0 : (!turned ? e0 : e0 < half ? e0 + half : e0 - half);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const int j = kInter ? i / 2 : i;  // j0 is even: frequency j0 + j is held at [j & 1]
          const float c = __shfl_sync(0xffffffffu, c2[j & 1], ((j0 + j) >> 1) & 31);
          const float s = __shfl_sync(0xffffffffu, s2[j & 1], ((j0 + j) >> 1) & 31);
          const bool first = kInter ? (i & 1) == 0 : e0 < half;
          wc[i] = turned ? c : 1.f;
          ws[i] = turned ? (first ? -s : s) : -0.f;
          if (norm) {
            wc[i] *= to_f32(w[e0 + i]);
            ws[i] *= to_f32(w[kInter ? mate + (i ^ 1) : mate + i]);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int hh = h + k * kHeads + hsub;
        if (h + k * kHeads >= h1) break;  // the same for the whole warp
        float x[kVec], xp[kVec], y[kVec];
        unpack16(raw[k], x);
        if (kInter) {
#pragma unroll
          for (int i = 0; i < kVec; ++i) xp[i] = turned ? x[i ^ 1] : 0.f;
        } else {
          uint4 o;
          o.x = __shfl_sync(0xffffffffu, raw[k].x, partner);
          o.y = __shfl_sync(0xffffffffu, raw[k].y, partner);
          o.z = __shfl_sync(0xffffffffu, raw[k].z, partner);
          o.w = __shfl_sync(0xffffffffu, raw[k].w, partner);
          if (!turned) o = make_uint4(0, 0, 0, 0);
          unpack16(o, xp);
        }
        float r = 1.f;
        if (norm) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < kVec; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          r = rsqrtf(ss * (1.f / D) + a.eps);
        }
        // what does not turn: 0 * -0 + x, which is x also for infinities and zeros
#pragma unroll
        for (int i = 0; i < kVec; ++i) y[i] = fmaf(xp[i], ws[i], x[i] * wc[i]) * r;
        if (hh >= h1) continue;
        if (hh < hk) {
          const uint4 w = pos < 0 ? make_uint4(0, 0, 0, 0) : pack16<kVec>(y);
          if (write) *reinterpret_cast<uint4*>(out + (int64_t)hh * D) = w;
          if (slot >= 0)
            *reinterpret_cast<uint4*>(static_cast<T*>(a.k_cache) +
                                      (page + (int64_t)hh * kBlock) * D + e0) = w;
        } else if (slot >= 0) {
          *reinterpret_cast<uint4*>(static_cast<T*>(a.v_cache) +
                                    (page + (int64_t)(hh - Hkv) * kBlock) * D + e0) = raw[k];
        }
      }
    }
  }
}

template <typename T, int D, bool kInter>
static cudaError_t launch_t(const RopeArgs& a, uint32_t* status, cudaStream_t st) {
  constexpr int kHeads = kWarp / (D * (int)sizeof(T) / 16);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int step = kUnroll * kHeads;  // heads of one round of loads
  const int q_rounds = ceil_div(a.d.Hq, step);
  const int kv_rounds = ceil_div(a.slots != nullptr ? 2 * a.d.Hkv : a.d.Hkv, step);
  // A warp takes half of a token's query heads, or all its key and value
  // heads, when the tokens alone fill the GPU (the angles are then formed
  // three times per token), else one round of loads.  With all query heads in
  // one run every second unit was four times the other, and as the number of
  // warps is even each warp kept to one kind: 136 us against 117 (124 in three
  // to six runs, 149 in eight).
  const bool whole = a.rows >= (int64_t)sms * 16;
  Split sp;
  sp.q_run = whole ? ceil_div(q_rounds, 2) * step : step;
  sp.uq = ceil_div(q_rounds * step, sp.q_run);
  sp.kv_run = whole ? kv_rounds * step : step;
  sp.units = sp.uq + (whole ? 1 : kv_rounds);
  const int64_t ctas = ceil_div64((int64_t)a.rows * sp.units, kWarps);
  const int64_t wave = (int64_t)sms * 4;  // CTAs that the launch bounds keep resident
  PdlLaunch L(dim3((unsigned)(ctas < wave ? ctas : wave)), dim3(kThreads), 0, st);
  return cudaLaunchKernelEx(&L.cfg, qk_norm_rope_kernel<T, D, kInter>, a, sp, status);
}

template <typename T>
static cudaError_t launch_type(const RopeArgs& a, uint32_t* status, cudaStream_t st) {
  if (a.interleaved)
    return a.d.D == 128 ? launch_t<T, 128, true>(a, status, st) : launch_t<T, 64, true>(a, status, st);
  return a.d.D == 128 ? launch_t<T, 128, false>(a, status, st) : launch_t<T, 64, false>(a, status, st);
}

}  // namespace rope

cudaError_t qk_norm_rope_launch(const RopeArgs& a, const WsLayout& lay, cudaStream_t st,
                                int* launches) {
  uint32_t* status = reinterpret_cast<uint32_t*>(static_cast<char*>(a.ws) + lay.status_off);
  const cudaError_t e = a.d.kv_dtype == SPEC_BF16 ? rope::launch_type<__nv_bfloat16>(a, status, st)
                                                  : rope::launch_type<float>(a, status, st);
  ++*launches;
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace specv
