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
// takes a run of heads of one token: a head is 8..32 lanes of 16 bytes, so the
// sum of squares and the partner of a pair are shuffles, and no shared memory
// or barrier sits between a load and its store.  The token's cosines and sines
// are formed once per warp and unit and stay in registers.
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

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(RopeArgs a, int unit_heads,
                                                                int units_per_row,
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
  for (int j = tid; j < half; j += kThreads) {
    const double f = a.inv_freq[j] * 0.15915494309189533577;  // turns per position
    freq[j] = (uint64_t)((f - floor(f)) * 18446744073709551616.0);
  }
  // the lane's weights, the same for every head
  float wq[kVec], wk[kVec];
  const bool norm_q = a.q_weight != nullptr, norm_k = a.k_weight != nullptr;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    wq[i] = norm_q ? to_f32(static_cast<const T*>(a.q_weight)[e0 + i]) : 1.f;
    wk[i] = norm_k ? to_f32(static_cast<const T*>(a.k_weight)[e0 + i]) : 1.f;
  }
  __syncthreads();

  const bool cached = a.slots != nullptr;
  const int heads = Hq + (cached ? 2 * Hkv : Hkv);
  const int64_t n_units = (int64_t)a.rows * units_per_row;
  const int64_t warps = (int64_t)gridDim.x * kWarps;
  const bool turned = e0 < a.rot_dim;
  // the lane that holds the other element of this lane's pairs (half-split)
  const int partner = (!turned || a.interleaved) ? lane
                      : e0 < half                ? lane + half / kVec
                                                 : lane - half / kVec;
  const T* qp = static_cast<const T*>(a.q) + e0;
  const T* kp = static_cast<const T*>(a.k) + e0;
  const T* vp = static_cast<const T*>(a.v) + e0;
  for (int64_t u = (int64_t)blockIdx.x * kWarps + tid / kWarp; u < n_units; u += warps) {
    const int64_t row = u / units_per_row;
    const int h0 = (int)(u - row * units_per_row) * unit_heads;
    const int h1 = min(heads, h0 + unit_heads);
    const int pos = a.positions[row];
    int64_t slot = -1;
    if (cached) {
      slot = a.slots[row];
      if (slot >= (int64_t)a.d.num_blocks * kBlock) {
        if (lane == 0) raise_status(status, SPEC_ERR_DEVICE_BOUNDS);
        slot = -1;
      }
      if (pos < 0 || slot < 0) slot = -1;
    }
    const int64_t page = slot < 0 ? 0 : slot / kBlock * Hkv * kBlock + slot % kBlock;
    float c[kVec], s[kVec];
    bool ready = false;
    for (int h = h0; h < h1; h += kUnroll * kHeads) {
      uint4 raw[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int hh = h + k * kHeads + hsub;
        raw[k] = make_uint4(0, 0, 0, 0);
        if (hh < h1) {
          const T* src = hh < Hq          ? qp + row * a.q_stride + (int64_t)hh * D
                         : hh < Hq + Hkv  ? kp + row * a.k_stride + (int64_t)(hh - Hq) * D
                                          : vp + row * a.v_stride + (int64_t)(hh - Hq - Hkv) * D;
          raw[k] = *reinterpret_cast<const uint4*>(src);
        }
      }
      if (!ready) {  // after the first loads are on their way
        ready = true;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          c[i] = 1.f;
          s[i] = 0.f;
        }
        if (turned) {
          if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < kVec; i += 2) {
              turn_cos_sin((uint64_t)(uint32_t)pos * freq[(e0 + i) / 2], &c[i], &s[i + 1]);
              c[i + 1] = c[i];
              s[i] = -s[i + 1];
            }
          } else {
            const int j0 = e0 < half ? e0 : e0 - half;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
              turn_cos_sin((uint64_t)(uint32_t)pos * freq[j0 + i], &c[i], &s[i]);
              if (e0 < half) s[i] = -s[i];
            }
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int hh = h + k * kHeads + hsub;
        if (h + k * kHeads >= h1) break;  // the same for the whole warp
        float x[kVec], y[kVec];
        unpack16(raw[k], x);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < kVec; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const bool is_q = hh < Hq;
        const float r = (is_q ? norm_q : norm_k) ? rsqrtf(ss * (1.f / D) + a.eps) : 1.f;
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[i] *= r * (is_q ? wq[i] : wk[i]);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const float other = a.interleaved ? x[i ^ 1] : __shfl_sync(0xffffffffu, x[i], partner);
          y[i] = fmaf(other, s[i], x[i] * c[i]);
        }
        if (hh >= h1) continue;
        if (hh < Hq + Hkv) {
          const uint4 w = pos < 0 ? make_uint4(0, 0, 0, 0) : pack16<kVec>(y);
          T* dst = is_q ? static_cast<T*>(a.q_out) + (row * Hq + hh) * D + e0
                        : static_cast<T*>(a.k_out) + (row * Hkv + hh - Hq) * D + e0;
          if (is_q || a.k_out != nullptr) *reinterpret_cast<uint4*>(dst) = w;
          if (!is_q && slot >= 0)
            *reinterpret_cast<uint4*>(static_cast<T*>(a.k_cache) +
                                      (page + (int64_t)(hh - Hq) * kBlock) * D + e0) = w;
        } else if (slot >= 0) {
          *reinterpret_cast<uint4*>(static_cast<T*>(a.v_cache) +
                                    (page + (int64_t)(hh - Hq - Hkv) * kBlock) * D + e0) = raw[k];
        }
      }
    }
  }
}

template <typename T, int D>
static cudaError_t launch_t(const RopeArgs& a, uint32_t* status, cudaStream_t st) {
  constexpr int kHeads = kWarp / (D * (int)sizeof(T) / 16);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int heads = a.d.Hq + (a.slots != nullptr ? 2 : 1) * a.d.Hkv;
  const int step = kUnroll * kHeads;  // heads of one round of loads
  const int rounds = ceil_div(heads, step);
  // A warp takes all heads of a token when the tokens alone fill the GPU (the
  // angles are then formed once per token), else one round of loads.
  const int64_t full = (int64_t)sms * 16;
  const int per_unit = a.rows >= full ? rounds : 1;
  const int units = ceil_div(rounds, per_unit);
  const int64_t ctas = ceil_div64((int64_t)a.rows * units, kWarps);
  // CTAs an SM holds: a property of the kernel, asked for once
  static const int per_sm = [] {
    int n = 0;
    const cudaError_t q =
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, qk_norm_rope_kernel<T, D>, kThreads, 0);
    return q == cudaSuccess && n > 0 ? n : 1;
  }();
  const int64_t wave = (int64_t)sms * per_sm;
  PdlLaunch L(dim3((unsigned)(ctas < wave ? ctas : wave)), dim3(kThreads), 0, st);
  return cudaLaunchKernelEx(&L.cfg, qk_norm_rope_kernel<T, D>, a, per_unit * step, units, status);
}

}  // namespace rope

cudaError_t qk_norm_rope_launch(const RopeArgs& a, const WsLayout& lay, cudaStream_t st,
                                int* launches) {
  uint32_t* status = reinterpret_cast<uint32_t*>(static_cast<char*>(a.ws) + lay.status_off);
  cudaError_t e;
  if (a.d.kv_dtype == SPEC_BF16)
    e = a.d.D == 128 ? rope::launch_t<__nv_bfloat16, 128>(a, status, st)
                     : rope::launch_t<__nv_bfloat16, 64>(a, status, st);
  else
    e = a.d.D == 128 ? rope::launch_t<float, 128>(a, status, st)
                     : rope::launch_t<float, 64>(a, status, st);
  ++*launches;
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace specv
