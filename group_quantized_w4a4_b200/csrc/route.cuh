// route.cuh -- routing of tokens to experts, and the grouping of the routed tokens by expert.
//
// For every token with logits z[E]:
//   p = softmax(z) or 1 / (1 + exp(-z))                       (scores)
//   v = p + bias                                              (values that are compared)
//   groups > 1: a group of E / groups neighbouring experts is worth the sum of its two largest
//   v; experts of the topk_groups best groups stay in the choice
//   ids = the k largest v, ties to the lowest index;  weights = scale * p[ids], divided by
//   their sum first when renormalized.
// Without a bias and groups the order of v is the order of z, which is compared itself.
// Otherwise v is formed in 64 bits, so that the choice does not hang on an exponential's last
// bits.  A NaN is chosen last; a softmax row of -inf alone has scores 0; weights whose sum is
// 0 stay 0.
#pragma once
#include <stdint.h>

#include "f8_block.cuh"
#include "ptx.cuh"

namespace apex {

struct RouteArgs {
  const void* logits;      // [T][E]
  const float* bias;       // [E] or null
  const uint8_t* mask;     // [T] or null: 0 = the token takes no part
  int T, E, k, G, TG;
  int sigmoid, renorm;
  float scale;
  int32_t* ids;            // [T][k]
  float* weights;          // [T][k]
};

constexpr int kRouteWarps = 4;

// One warp per token; lane l holds experts l, l + 32, ...
template <int DT, int EPL>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  extern __shared__ double s_v[];   // [kRouteWarps][E] when groups are used
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int E = a.E;
  const double ninf = -__longlong_as_double(0x7FF0000000000000ll);
  for (long long t = (long long)blockIdx.x * kRouteWarps + warp; t < a.T;
       t += (long long)gridDim.x * kRouteWarps) {
    if (a.mask && !a.mask[t]) {
      if (lane < a.k) {
        a.ids[t * a.k + lane] = -1;
        a.weights[t * a.k + lane] = 0.0f;
      }
      continue;
    }
    const typename DTraits<DT>::T* z = static_cast<const typename DTraits<DT>::T*>(a.logits) + t * E;
    double v[EPL], p[EPL];
    float zf[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      zf[i] = lane + 32 * i < E ? DTraits<DT>::up(z[lane + 32 * i]) : __int_as_float(0xFF800000);
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) p[i] = 1.0 / (1.0 + exp(-(double)zf[i]));
    } else {
      float m = zf[0];
#pragma unroll
      for (int i = 1; i < EPL; ++i) m = fmaxf(m, zf[i]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      double sum = 0.0;
      const bool none = m == __int_as_float(0xFF800000);
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const bool in = lane + 32 * i < E;
        // the row's NaNs reach every score through the sum; a row of -inf alone scores 0
        p[i] = !in || (none && zf[i] == m) ? 0.0 : exp((double)zf[i] - (double)m);
        sum += p[i];
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
      for (int i = 0; i < EPL; ++i) p[i] = sum == 0.0 ? 0.0 : p[i] / sum;
    }
    const bool plain = a.bias == nullptr && a.G == 1;
    uint32_t left = 0;   // this lane's experts that can still be chosen
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      v[i] = ninf;
      if (e < E) {
        left |= 1u << i;
        v[i] = plain ? (double)zf[i] : p[i] + (a.bias ? (double)a.bias[e] : 0.0);
        if (!(v[i] == v[i])) v[i] = ninf;
      }
    }
    if (a.G > 1) {
      double* sv = s_v + (size_t)warp * E;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (lane + 32 * i < E) sv[lane + 32 * i] = v[i];
      __syncwarp();
      const int epg = E / a.G;
      double best = ninf, second = ninf;
      if (lane < a.G) {
        for (int i = 0; i < epg; ++i) {
          const double w = sv[lane * epg + i];
          if (w > best) { second = best; best = w; }
          else if (w > second) second = w;
        }
      }
      __syncwarp();
      const double worth = epg > 1 ? best + second : best;
      int rank = 0;
      for (int g = 0; g < a.G; ++g) {
        const double other = __shfl_sync(0xffffffffu, worth, g);
        rank += other > worth || (other == worth && g < lane);
      }
      const uint32_t open = __ballot_sync(0xffffffffu, lane < a.G && rank < a.TG);
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (lane + 32 * i < E && !((open >> ((lane + 32 * i) / epg)) & 1u)) left &= ~(1u << i);
    }
    int my_id = -1;
    float my_w = 0.0f;
    double total = 0.0;
    for (int j = 0; j < a.k; ++j) {
      double bv = ninf;
      int be = 0x7FFFFFFF;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (((left >> i) & 1u) && (v[i] > bv || be == 0x7FFFFFFF)) { bv = v[i]; be = lane + 32 * i; }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const double ov = __shfl_xor_sync(0xffffffffu, bv, o);
        const int oe = __shfl_xor_sync(0xffffffffu, be, o);
        const bool take = oe != 0x7FFFFFFF && (be == 0x7FFFFFFF || ov > bv || (ov == bv && oe < be));
        if (take) { bv = ov; be = oe; }
      }
      double pw = 0.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (be == lane + 32 * i) { pw = p[i]; left &= ~(1u << i); }
      pw = __shfl_sync(0xffffffffu, pw, be & 31);
      total += pw;
      if (lane == j) { my_id = be; my_w = 0.0f; }
      if (lane == j) my_w = __double2float_rn(pw);
    }
    if (lane < a.k) {
      float w = my_w;
      if (a.renorm) w = total == 0.0 ? 0.0f : __double2float_rn((double)w / total);
      a.ids[t * a.k + lane] = my_id;
      a.weights[t * a.k + lane] = w * a.scale;
    }
  }
}

// Groups flat indices f = t * k + j by ids[f]: order = the f of expert 0 in ascending order,
// of expert 1, ...; entries behind offsets[E] are -1.  An id outside [0, E) belongs to none.
// One CTA per expert: a first pass counts the ids below its own and its own, a second writes.
__global__ void __launch_bounds__(256) plan_kernel(const int32_t* __restrict__ ids, int S, int E,
                                                   int32_t* __restrict__ offsets,
                                                   int32_t* __restrict__ order) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ int s_below[8], s_mine[8];
  const int e = blockIdx.x;   // E: the CTA that writes offsets[E] and the entries behind it
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int below = 0;
  for (int i = threadIdx.x; i < S; i += 256) {
    const int id = __ldg(ids + i);
    below += id >= 0 && id < e;
  }
  below = __reduce_add_sync(0xffffffffu, below);
  if (lane == 0) s_below[warp] = below;
  __syncthreads();
  int at = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) at += s_below[w];
  if (threadIdx.x == 0) offsets[e] = at;
  if (e == E) {
    for (int i = at + threadIdx.x; i < S; i += 256) order[i] = -1;
    return;
  }
  for (int i0 = 0; i0 < S; i0 += 256) {
    const int i = i0 + threadIdx.x;
    const bool mine = i < S && __ldg(ids + i) == e;
    const uint32_t b = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) s_mine[warp] = __popc(b);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      if (w < warp) before += s_mine[w];
      all += s_mine[w];
    }
    if (mine) order[at + before + __popc(b & ((1u << lane) - 1u))] = i;
    at += all;
    __syncthreads();
  }
}

}  // namespace apex
