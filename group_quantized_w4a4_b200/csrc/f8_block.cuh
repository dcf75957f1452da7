// f8_block.cuh -- block-scaled FP8 (E4M3) quantization: activations in groups of 1 x 128,
// weights in blocks of 128 x 128, one fp32 scale each.
//
// Rule, for a group (or block) with largest magnitude a:
//   s = fp32_rne(a / 448)                      (IEEE fp32 division; 448 is E4M3's maximum)
//   q = E4M3(x / s), the exact quotient rounded once, half to even (q = 0 when s == 0)
// A NaN in the group makes s and every q NaN; an infinity makes s infinite (a NaN once
// multiplied).  The exact quotient, not its fp32 rounding, decides: t = fl(x * r), r within an
// ulp of 1/s, is within 3 ulp of it, so unless t lies within 4 ulp of a middle m between two
// E4M3 values both round alike; there the sign of x - m * s (one fma) decides.  Exact ties are
// common: 16-bit values and the scale of one of them make about one in a thousand.
// Whether a value needs that is seen from its codes: bounds of the quotient, x * r * (1 +- 2^-21),
// that round to one code leave nothing to decide (rounding is monotonic), which costs a packed
// multiply and a conversion more instead of five integer operations a value.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "ptx.cuh"

namespace apex {

enum DType : int { DT_F16 = 0, DT_BF16 = 1, DT_F32 = 2 };

template <int DT> struct DTraits;
template <> struct DTraits<DT_F16> {
  using T = __half;
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ __half one(float a) { return __float2half_rn(a); }
  static __device__ __forceinline__ float up(__half a) { return __half2float(a); }
};
template <> struct DTraits<DT_BF16> {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ __nv_bfloat16 one(float a) { return __float2bfloat16_rn(a); }
  static __device__ __forceinline__ float up(__nv_bfloat16 a) { return __bfloat162float(a); }
};
template <> struct DTraits<DT_F32> {
  using T = float;
  static __device__ __forceinline__ float up(float a) { return a; }
};

// 8 consecutive elements as fp32.
template <int DT>
__device__ __forceinline__ void load8(const void* base, size_t at, float (&v)[8]) {
  if constexpr (DT == DT_F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(
        static_cast<const typename DTraits<DT>::T*>(base) + at));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = DTraits<DT>::unpack(u[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

// Magnitudes compare as their bit patterns, with infinity above every number and NaN above
// infinity, so an integer maximum keeps a NaN.
__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint32_t absmax8_bits(const float (&v)[8]) {
  uint32_t m = abs_bits(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max(m, abs_bits(v[i]));
  return m;
}

// A group's scale and its reciprocal.  `exact`: the scale is out of the safe range (subnormal,
// huge or non-finite), every quotient is formed in 64 bits.
struct F8Scale {
  float s, r;
  bool exact;
};
__device__ __forceinline__ float rcp_approx(float x) {   // within 1 ulp
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ F8Scale f8_scale(uint32_t amax_bits) {
  const float a = __uint_as_float(amax_bits);
  F8Scale q;
  // a / 448 by Markstein's correction: the product with the rounded 1/448 is within an ulp, and one
  // residual step (exact in an fma) makes it the correctly rounded quotient
  const float k = 1.0f / 448.0f;
  const float q0 = __fmul_rn(a, k);
  q.s = __fmaf_rn(__fmaf_rn(-q0, 448.0f, a), k, q0);
  q.exact = !(amax_bits - 0x10000000u < 0x60000000u);   // a outside [2^-95, 2^97): 0 and NaN too
  if (q.exact) {
    q.s = __fdiv_rn(a, 448.0f);
    q.exact = q.s != 0.0f;
  }
  q.r = q.s == 0.0f ? 0.0f : rcp_approx(q.s);
  return q;
}

// fp32 value that rounds to E4M3 as the exact x / s does (round to odd of the 64-bit quotient).
__device__ __noinline__ float f8_quotient_exact(float x, float s) {
  if (s == 0.0f) return 0.0f;
  const double q = (double)x / (double)s;
  const float f = __double2float_rz(q);
  if ((double)f == q || !(fabs(q) <= 3.0e38)) return f;   // exact, or infinite / NaN
  return __uint_as_float(__float_as_uint(f) | 1u);
}

// t = fl(x * r) lies within 4 ulp of the middle between two neighbouring E4M3 values.  From
// 2^-6 on E4M3 keeps 3 mantissa bits: middles have the next 20 bits at 0x80000.  Below, the
// values are multiples of 2^-9 and the middles (odd multiples of 2^-10) have at most four
// significant bits: the low 20 bits of the mantissa are 0.  Under 2^-11 there is no middle.
__device__ __forceinline__ bool f8_near_middle(float t) {
  const uint32_t b = abs_bits(t);
  const uint32_t shift = b >= 0x3C800000u ? 0x80004u : 4u;      // 2^-6
  return ((b + shift) & 0xFFFFFu) <= 8u && b >= 0x3A000000u;    // 2^-11
}

__device__ __forceinline__ uint32_t f8_pair(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// A value beside the quotient x / s that rounds to E4M3 as the quotient does, from a t that is
// near a middle: the middle itself for a tie, else its fp32 neighbour on the quotient's side.
__device__ __forceinline__ float f8_settle(float x, float s, float t) {
  const uint32_t b = abs_bits(t);
  uint32_t m = b >= 0x3C800000u ? (b & 0xFFF00000u) | 0x80000u : (b + 4u) & 0xFFF00000u;
  const float e = __fmaf_rn(-__uint_as_float(m), s, fabsf(x));
  m += e > 0.0f ? 1u : e < 0.0f ? 0xFFFFFFFFu : 0u;
  return copysignf(__uint_as_float(m), t);
}

// One value's rounding input.
__device__ __forceinline__ float f8_quotient(float x, const F8Scale& q) {
  if (q.exact) return f8_quotient_exact(x, q.s);
  const float t = __fmul_rn(x, q.r);
  return f8_near_middle(t) ? f8_settle(x, q.s, t) : t;
}

// The E4M3 codes of 8 values of one group, where some value is near a middle or the scale is out
// of its safe range.
__device__ __forceinline__ uint2 f8_codes8_near(const float (&v)[8], const F8Scale& q) {
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t[i] = __fmul_rn(v[i], q.r);
    if (f8_near_middle(t[i])) t[i] = f8_settle(v[i], q.s, t[i]);
  }
  return make_uint2(f8_pair(t[0], t[1]) | (f8_pair(t[2], t[3]) << 16),
                    f8_pair(t[4], t[5]) | (f8_pair(t[6], t[7]) << 16));
}
__device__ __noinline__ uint2 f8_codes8_rare(float v0, float v1, float v2, float v3, float v4,
                                             float v5, float v6, float v7, float s, float r,
                                             bool exact) {
  const float v[8] = {v0, v1, v2, v3, v4, v5, v6, v7};
  F8Scale q;
  q.s = s;
  q.r = r;
  q.exact = exact;
  if (!exact) return f8_codes8_near(v, q);
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = f8_quotient_exact(v[i], s);
  return make_uint2(f8_pair(t[0], t[1]) | (f8_pair(t[2], t[3]) << 16),
                    f8_pair(t[4], t[5]) | (f8_pair(t[6], t[7]) << 16));
}

// The E4M3 codes of 8 values of one group.  RARE: the values are fp32 results, which are near a
// middle once in 10^5, so that case is a call; 16-bit values are so in one warp of five.
template <bool RARE>
__device__ __forceinline__ uint2 f8_codes8(const float (&v)[8], const F8Scale& q) {
  const float rl = q.r * (1.0f - 0x1p-21f), rh = q.r * (1.0f + 0x1p-21f);
  const float2 rl2 = make_float2(rl, rl), rh2 = make_float2(rh, rh);
  uint32_t lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = make_float2(v[2 * i], v[2 * i + 1]);
    const float2 l = __fmul2_rn(x, rl2), h = __fmul2_rn(x, rh2);
    lo[i] = f8_pair(l.x, l.y);
    hi[i] = f8_pair(h.x, h.y);
  }
  uint2 c = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
  const uint2 d = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
  if constexpr (RARE) {
    if (q.exact || c.x != d.x || c.y != d.y)
      c = f8_codes8_rare(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], q.s, q.r, q.exact);
  } else {
    if (c.x != d.x || c.y != d.y) c = f8_codes8_near(v, q);
    if (q.exact)
      c = f8_codes8_rare(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], q.s, q.r, true);
  }
  return c;
}

// Maximum over the 16 lanes of this half-warp.
__device__ __forceinline__ uint32_t half_warp_max(uint32_t v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Activations [M][K] (K % 16 == 0) -> E4M3 codes [M][K] and scales [M][G], G = ceil(K / 128).
// Bound: the issue slots for a large batch (the exact rounding; HBM's 2 bytes in and 1 + 4/128 out
// an element take half as long), latency for a small one.  A half-warp owns one (row, group): one
// 16-byte load a lane, a shuffle maximum, one 8-byte store a lane.  Measured: 4096 x 8192 29.5 us
// (bf16 34.7; 15 at the copy rate), a decode step's 16 x 8192 1.7 us.  Two groups in flight a
// half-warp were slower at every size but one (32.8 us, 2.2; 512 x 8192: 4.9 against 5.1).
template <int DT>
__global__ void __launch_bounds__(128) f8_quantize_act_kernel(const void* __restrict__ x, int M,
                                                              int K, int G, int g_shift,
                                                              uint8_t* __restrict__ codes,
                                                              float* __restrict__ scales) {
  grid_dep_wait();
  grid_dep_launch();
  const int hl = threadIdx.x & 15;
  const long long units = (long long)M * G;
  const long long step = (long long)gridDim.x * 8;
  // every lane of a warp runs the same number of rounds (the shuffles are warp-wide)
  for (long long u0 = (long long)blockIdx.x * 8 + (threadIdx.x >> 5) * 2; u0 < units; u0 += step) {
    const long long u = u0 + ((threadIdx.x >> 4) & 1);
    const uint32_t w = (uint32_t)(u < units ? u : 0);
    const int row = g_shift >= 0 ? (int)(w >> g_shift) : (int)(w / (uint32_t)G);
    const int g = (int)w - row * G;
    const bool in = u < units && g * 128 + hl * 8 < K;
    const size_t at = (size_t)row * K + g * 128 + hl * 8;
    float v[8] = {};
    if (in) load8<DT>(x, at, v);
    const F8Scale q = f8_scale(half_warp_max(absmax8_bits(v)));
    if (in) *reinterpret_cast<uint2*>(codes + at) = f8_codes8<DT == DT_F32>(v, q);
    if (hl == 0 && u < units) scales[(size_t)row * G + g] = q.s;
  }
}

// Weights [E][N][K] (K % 16 == 0, any N) -> codes [E][N][K], scales [E][ceil(N/128)][G].
// Offline.  One CTA per 128 x 128 block; a thread keeps its 8 chunks of 8 values, so the
// block is read once.
template <int DT>
__global__ void __launch_bounds__(256) f8_pack_weights_kernel(const void* __restrict__ w, int N,
                                                              int K, int G, int NB,
                                                              uint8_t* __restrict__ codes,
                                                              float* __restrict__ scales) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ uint32_t s_max[8];
  const int g = blockIdx.x % G;
  const int nb = (blockIdx.x / G) % NB;
  const long long e = blockIdx.x / G / NB;
  const int c = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  const int k = g * 128 + c * 8;
  float v[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = nb * 128 + r0 + 16 * i;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    if (n < N && k < K) load8<DT>(w, ((size_t)e * N + n) * K + k, v[i]);
    m = max(m, absmax8_bits(v[i]));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, s_max[i]);
  const F8Scale q = f8_scale(m);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = nb * 128 + r0 + 16 * i;
    if (n < N && k < K)
      *reinterpret_cast<uint2*>(codes + ((size_t)e * N + n) * K + k) = f8_codes8<DT == DT_F32>(v[i], q);
  }
  if (threadIdx.x == 0) scales[((size_t)e * NB + nb) * G + g] = q.s;
}

}  // namespace apex
