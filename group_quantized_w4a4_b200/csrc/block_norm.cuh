// block_norm.cuh -- what stands between two blocks of a model, in one pass over a token:
//
//   z = x                                                     (the block's output)
//   z = z * rsqrt(mean(z^2) + eps) * (off + post_weight)      (optional: norm behind the block)
//   z = z * gate                                              (optional)
//   h = residual + alpha * z                                  (the new residual stream)
//   y = h * rsqrt(mean(h^2) + eps) * (off + pre_weight)       (optional: norm before the next)
//
// with h and y stored in x's type, and y also as the next product's block-scaled E4M3 operand
// (f8_block.cuh).  Everything between is fp32: h is rounded where it is stored, y and its codes
// are formed from the unrounded values.  The combine of the experts' products is here too: a
// weighted sum over a token's choices.
// Measured in a graph, 4096 x 8192 fp16: everything on 61 us (302 MB, 46 at the copy rate; the issue
// slots are 70 % busy), without the gate 53, pre-norm and residual alone with codes 43, with values
// 42, the residual alone 29 (201 MB: 31).  One token: 4.0 us with everything, 1.7 the residual alone;
// two reductions over a CTA and a launch.
#pragma once
#include <stdint.h>

#include "f8_block.cuh"
#include "ptx.cuh"

namespace apex {

struct NormArgs {
  const void *x, *residual, *post, *gate, *pre;   // all but x may be null
  int T, H, G;             // G = ceil(H / 128)
  int rows_per_gate;       // row t takes gate row t / rows_per_gate
  float alpha, eps, off;
  void *h, *y;             // may be null
  uint8_t* codes;          // may be null
  float* scales;
};

// Sum over the CTA; every thread gets it.  One slot array per call site.
__device__ __forceinline__ float block_sum(float v, float* s_part, int warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = (threadIdx.x & 31) < warps ? s_part[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}

// 8 consecutive 16-bit elements as they are stored, and as fp32.
__device__ __forceinline__ uint4 raw8(const void* base, size_t at) {
  return __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
}
template <int DT>
__device__ __forceinline__ void widen8(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = DTraits<DT>::unpack(u[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
template <int DT>
__device__ __forceinline__ uint4 narrow8(const float (&v)[8]) {
  return make_uint4(DTraits<DT>::pack(v[0], v[1]), DTraits<DT>::pack(v[2], v[3]),
                    DTraits<DT>::pack(v[4], v[5]), DTraits<DT>::pack(v[6], v[7]));
}

// One CTA per token; thread i holds chunks i, i + blockDim, ... of 8 elements in registers, so
// every tensor is read and written once.  Bound: HBM for many tokens (x and residual in; h, y
// and codes out), latency for a few.  A few tokens take one chunk a thread, the shortest chain;
// many take two or four, in CTAs of up to 256 threads, several of which share an SM, so that
// one's loads cover the others' reductions.  (A CTA that keeps the weights in registers and
// walks through tokens, the next one's loads ahead, took half as long again.)
template <int DT, int NC, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) block_norm_kernel(const NormArgs a) {
  using D = DTraits<DT>;
  __shared__ float s_part[2][32];
  grid_dep_wait();
  grid_dep_launch();
  const int warps = blockDim.x >> 5;
  const size_t base = (size_t)blockIdx.x * a.H;
  uint4 xr[NC], rr[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8;
    xr[i] = rr[i] = make_uint4(0u, 0u, 0u, 0u);
    if (c < a.H) {
      xr[i] = raw8(a.x, base + c);
      if (a.residual) rr[i] = raw8(a.residual, base + c);
    }
  }
  float z[NC][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    widen8<DT>(xr[i], z[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(z[i][j], z[i][j], ss);
  }
  float rs = 1.0f;
  if (a.post) rs = __frsqrt_rn(block_sum(ss, s_part[0], warps) / (float)a.H + a.eps);
  const size_t gbase = a.gate ? (size_t)(blockIdx.x / a.rows_per_gate) * a.H : 0;
  ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8;
    if (c >= a.H) continue;
    float w[8];
    if (a.post) {
      widen8<DT>(raw8(a.post, c), w);
#pragma unroll
      for (int j = 0; j < 8; ++j) z[i][j] = z[i][j] * rs * (a.off + w[j]);
    }
    if (a.gate) {
      widen8<DT>(raw8(a.gate, gbase + c), w);
#pragma unroll
      for (int j = 0; j < 8; ++j) z[i][j] *= w[j];
    }
    widen8<DT>(rr[i], w);   // 0 without a residual
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      z[i][j] = fmaf(a.alpha, z[i][j], w[j]);
      ss = fmaf(z[i][j], z[i][j], ss);
    }
    if (a.h) *reinterpret_cast<uint4*>(static_cast<typename D::T*>(a.h) + base + c) = narrow8<DT>(z[i]);
  }
  if (!a.pre) return;
  rs = __frsqrt_rn(block_sum(ss, s_part[1], warps) / (float)a.H + a.eps);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * 8;
    const bool in = c < a.H;
    if (in) {
      float w[8];
      widen8<DT>(raw8(a.pre, c), w);
#pragma unroll
      for (int j = 0; j < 8; ++j) z[i][j] = z[i][j] * rs * (a.off + w[j]);
      if (a.y) *reinterpret_cast<uint4*>(static_cast<typename D::T*>(a.y) + base + c) = narrow8<DT>(z[i]);
    }
    if (a.codes) {   // 16 lanes hold one group (the shuffles are warp-wide)
      const F8Scale q = f8_scale(half_warp_max(absmax8_bits(z[i])));
      if (in) {
        *reinterpret_cast<uint2*>(a.codes + base + c) = f8_codes8<true>(z[i], q);
        if ((threadIdx.x & 15) == 0) a.scales[(size_t)blockIdx.x * a.G + c / 128] = q.s;
      }
    }
  }
}

// out[t] = sum_j weights[t,j] * y[row of t * k + j] over the choices with an id in [0, E), in the
// order of j, in fp32 and rounded once; the row is the flat index itself, or slot_of[it].  Bound:
// the fp32 rows (4096 tokens x 8 x 2048: 46 us, 285 MB, 0.95 of the copy rate).
template <int DT>
__global__ void __launch_bounds__(256) combine_kernel(const float* __restrict__ y,
                                                      const float* __restrict__ weights,
                                                      const int32_t* __restrict__ ids,
                                                      const int32_t* __restrict__ slot_of, int T,
                                                      int H, int k, int E, void* __restrict__ out) {
  using D = DTraits<DT>;
  grid_dep_wait();
  grid_dep_launch();
  const int chunks = H / 8;
  const long long n = (long long)T * chunks;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n;
       i += (long long)gridDim.x * 256) {
    const long long t = i / chunks;
    const int c = (int)(i - t * chunks) * 8;
    float acc[8] = {};
    for (int j0 = 0; j0 < k; j0 += 4) {   // four rows in flight
      float r[4][8];
      float w[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int id = j0 + u < k ? __ldg(ids + t * k + j0 + u) : -1;
        w[u] = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) r[u][e] = 0.0f;
        if (id >= 0 && id < E) {
          int row = (int)(t * k) + j0 + u;
          if (slot_of) row = __ldg(slot_of + row);
          if (row >= 0 && row < T * k) {   // (no order's slots lead out of y)
            w[u] = __ldg(weights + t * k + j0 + u);
            load8<DT_F32>(y, (size_t)row * H + c, r[u]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = fmaf(w[u], r[u][e], acc[e]);
      }
    }
    *reinterpret_cast<uint4*>(static_cast<typename D::T*>(out) + (size_t)t * H + c) =
        make_uint4(D::pack(acc[0], acc[1]), D::pack(acc[2], acc[3]), D::pack(acc[4], acc[5]),
                   D::pack(acc[6], acc[7]));
  }
}

}  // namespace apex
