// route.cuh -- routing of tokens to experts, and the grouping of the routed tokens by expert.
//
// For every token with logits z[E]:
//   p = softmax(z) or 1 / (1 + exp(-z))                       (scores)
//   v = p + bias                                              (values that are compared)
//   groups > 1: a group of E / groups neighbouring experts is worth the sum of its two largest
//   v; experts of the topk_groups best groups stay in the choice
//   ids = the k largest v, ties to the lowest index;  weights = scale * p[ids], divided by
//   their sum first when renormalized.
// The choice is that of v in 64 bits; without a bias and groups the order of v is the order of
// z, which is compared itself.  A NaN is chosen last; a softmax row of -inf alone has scores 0;
// weights whose sum is 0 stay 0.
//
// 64-bit exponentials of every logit cost 230 us for 16384 tokens x 256 experts, sixty times
// the time of reading them.  So v is formed in fp32 with a bound f on its error, and the choice
// is made on these; where two values that an order was decided between lie within their bounds
// of each other (and do not come from the same logit and bias), the token is decided again in
// 64 bits, which well under 1 % of random rows need.  Scores of the chosen experts are always
// 64-bit.
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

__device__ __forceinline__ float ninf_f() { return __int_as_float(0xFF800000); }
__device__ __forceinline__ double ninf_d() { return -__longlong_as_double(0x7FF0000000000000ll); }

// Order-preserving key of a value that is not NaN; every key is above 0, which marks an expert
// that cannot be chosen.
__device__ __forceinline__ uint32_t route_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);   // -0 and 0 are one value
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// Top two of `best >= second` and another such pair.
template <typename F>
__device__ __forceinline__ void merge2(F& best, F& second, F b2, F s2) {
  second = best >= b2 ? (second >= b2 ? second : b2) : (best >= s2 ? best : s2);
  best = best >= b2 ? best : b2;
}

// Worth of the group of lanes 32/P.. (P = groups rounded up to a power of two) from the values
// sv[E] in shared memory: every lane returns its group's (lanes of groups past G: -inf), and
// the largest error bound sf[] of its members.
template <typename F>
__device__ __forceinline__ F group_worth(const F* sv, const float* sf, int E, int G, int lane,
                                         int lanes_per, F ninf, float* fmax_out) {
  const int epg = E / G, g = lane / lanes_per, s = lane % lanes_per;
  F best = ninf, second = ninf;
  float f = 0.0f;
  if (g < G) {
    const int n = (epg + lanes_per - 1) / lanes_per;
    // groups start at different places of their round, so that they meet different banks
    int i = g % n;
    for (int c = 0; c < n; ++c) {
      const int at = s + lanes_per * i;
      if (at < epg) {
        const F w = sv[g * epg + at];
        if (w > best) { second = best; best = w; }
        else if (w > second) second = w;
        if (sf) f = fmaxf(f, sf[g * epg + at]);
      }
      i = i + 1 == n ? 0 : i + 1;
    }
  }
  for (int o = 1; o < lanes_per; o <<= 1) {
    const F b2 = __shfl_xor_sync(0xffffffffu, best, o);
    const F s2 = __shfl_xor_sync(0xffffffffu, second, o);
    f = fmaxf(f, __shfl_xor_sync(0xffffffffu, f, o));
    merge2(best, second, b2, s2);
  }
  if (fmax_out) *fmax_out = f;
  return epg > 1 ? best + second : best;
}

// The bit set of the TG groups of largest worth, ties to the lowest.
template <typename F>
__device__ __forceinline__ uint32_t open_groups(F worth, int G, int TG, int lane, int lanes_per) {
  const int mine = lane / lanes_per;
  int rank = 0;
  for (int g = 0; g < G; ++g) {
    const F other = __shfl_sync(0xffffffffu, worth, g * lanes_per);
    rank += other > worth || (other == worth && g < mine);
  }
  uint32_t set = mine < G && rank < TG && lane % lanes_per == 0 ? 1u << mine : 0u;
  return __reduce_or_sync(0xffffffffu, set);
}

__device__ __forceinline__ int lanes_per_group(int G) {
  int p = 32;
  while (G > 32 / p) p >>= 1;   // 32 / p >= G groups of p lanes
  return p;
}

// The whole choice in 64 bits; returns lane j's j-th expert.
template <int DT, int EPL>
__device__ __noinline__ int route_exact(const typename DTraits<DT>::T* z, const RouteArgs& a,
                                        float m, double* sv, int lane) {
  const int E = a.E;
  double v[EPL];
  double sum = 0.0;
#pragma unroll 1
  for (int i = 0; i < EPL; ++i) {
    double w = ninf_d();
    if (lane + 32 * i < E) {
      const float zi = DTraits<DT>::up(z[lane + 32 * i]);
      if (a.sigmoid) w = 1.0 / (1.0 + exp(-(double)zi));
      else w = m == ninf_f() && zi == m ? 0.0 : exp((double)zi - (double)m);
      sum += w;
    }
#pragma unroll
    for (int c = 0; c < EPL; ++c) v[c] = c == i ? w : v[c];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  uint32_t left = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    if (e < E) {
      left |= 1u << i;
      if (!a.sigmoid) v[i] = sum == 0.0 ? 0.0 : v[i] / sum;
      if (a.bias) v[i] += (double)a.bias[e];
      if (!(v[i] == v[i])) v[i] = ninf_d();
    }
  }
  if (a.G > 1) {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + 32 * i < E) sv[lane + 32 * i] = v[i];
    __syncwarp();
    const int lp = lanes_per_group(a.G);
    const double worth = group_worth<double>(sv, nullptr, E, a.G, lane, lp, ninf_d(), nullptr);
    __syncwarp();
    const uint32_t open = open_groups(worth, a.G, a.TG, lane, lp);
    const int epg = E / a.G;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + 32 * i < E && !((open >> ((lane + 32 * i) / epg)) & 1u)) left &= ~(1u << i);
  }
  int mine = -1;
  for (int j = 0; j < a.k; ++j) {
    double bv = ninf_d();
    int be = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (((left >> i) & 1u) && (v[i] > bv || be == 0x7FFFFFFF)) { bv = v[i]; be = lane + 32 * i; }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double ov = __shfl_xor_sync(0xffffffffu, bv, o);
      const int oe = __shfl_xor_sync(0xffffffffu, be, o);
      if (oe != 0x7FFFFFFF && (be == 0x7FFFFFFF || ov > bv || (ov == bv && oe < be))) {
        bv = ov;
        be = oe;
      }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (be == lane + 32 * i) left &= ~(1u << i);
    if (lane == j) mine = be;
  }
  return mine;
}

// One token by one warp; lane l holds experts l, l + 32, ...  sv: E doubles of this warp's
// shared memory (used with groups only).
template <int DT, int EPL>
__device__ __forceinline__ void route_token(const RouteArgs& a, long long t, double* sv, int lane) {
  if (a.mask && !a.mask[t]) {
    if (lane < a.k) {
      a.ids[t * a.k + lane] = -1;
      a.weights[t * a.k + lane] = 0.0f;
    }
    return;
  }
  const int E = a.E;
  const typename DTraits<DT>::T* z = static_cast<const typename DTraits<DT>::T*>(a.logits) + t * E;
  const bool plain = a.bias == nullptr && a.G == 1;
  float zf[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    zf[i] = lane + 32 * i < E ? DTraits<DT>::up(z[lane + 32 * i]) : ninf_f();
  float m = ninf_f();
  bool poison = false;    // softmax: a NaN or +inf logit makes every score NaN
  double sum = 0.0;       // softmax: of exp(z - m) over the row
  float v[EPL], f[EPL];   // fp32 values that are compared, and bounds on their errors
  if (!a.sigmoid) {
    bool nan = false;
    uint32_t mk = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      nan |= !(zf[i] == zf[i]);
      mk = max(mk, zf[i] == zf[i] ? route_key(zf[i]) : 0u);
    }
    mk = __reduce_max_sync(0xffffffffu, mk);
    m = mk == 0u ? ninf_f() : __uint_as_float((mk & 0x80000000u) ? mk & 0x7FFFFFFFu : ~mk);
    poison = __any_sync(0xffffffffu, nan) || m == -ninf_f();
    if (!(plain && a.renorm)) {
      // exp(z - m) with the rounding of z - m made good: within 1.5 ulp of the exact value
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const float d = zf[i] - m;
        const float lost = fabsf(zf[i]) > fabsf(m) ? -m - (d - zf[i]) : zf[i] - (d + m);
        const float e = zf[i] == ninf_f() ? 0.0f : expf(d);
        v[i] = fabsf(lost) < 1.0f ? fmaf(e, lost, e) : e;
        if (lane + 32 * i >= E) v[i] = 0.0f;
        sum += (double)v[i];
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
  }
  if (plain) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = zf[i];
  } else {
    const float inv = sum == 0.0 ? 0.0f : __double2float_rn(1.0 / sum);
    // relative error bounds: softmax 1.5 ulp of the exponential, as much of the sum, 1/sum and
    // the product (one rounding each): under 2^-20; sigmoid: 1 ulp of the exponential and the
    // roundings of the sum and the quotient: under 2^-21
    const float rel = a.sigmoid ? 0x1p-21f : 0x1p-20f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float p = a.sigmoid ? __fdiv_rn(1.0f, 1.0f + expf(-zf[i])) : v[i] * inv;
      v[i] = p;
      if (a.bias && lane + 32 * i < E) v[i] = p + __ldg(a.bias + lane + 32 * i);
      f[i] = p * rel + fabsf(v[i]) * 0x1p-23f + 0x1p-126f;
      if (!(f[i] < 1e30f)) f[i] = 1e30f;   // NaN or huge: decide in 64 bits
    }
  }
  uint32_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    key[i] = lane + 32 * i >= E ? 0u : v[i] == v[i] ? route_key(v[i]) : route_key(ninf_f());
  bool unsure = false;
  if (a.G > 1) {
    float* s32 = reinterpret_cast<float*>(sv);   // v, then f
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + 32 * i < E) {
        s32[lane + 32 * i] = v[i] == v[i] ? v[i] : ninf_f();
        s32[E + lane + 32 * i] = f[i];
      }
    __syncwarp();
    const int lp = lanes_per_group(a.G);
    float ferr;
    const float worth = group_worth<float>(s32, s32 + E, E, a.G, lane, lp, ninf_f(), &ferr);
    __syncwarp();
    const uint32_t open = open_groups(worth, a.G, a.TG, lane, lp);
    if (a.TG < a.G) {
      // two values, each within ferr, and the rounding of their sum
      const float err = 2.0f * ferr + fabsf(worth) * 0x1p-23f;
      const int g = lane / lp;
      const bool kept = g < a.G && ((open >> g) & 1u);
      float low = kept ? worth - err : -ninf_f();
      float high = g < a.G && !kept ? worth + err : ninf_f();
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
        high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
      }
      unsure = !(low > high);
    }
    const int epg = E / a.G;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + 32 * i < E && !((open >> ((lane + 32 * i) / epg)) & 1u)) key[i] = 0u;
  }
  int mine = -1;             // lane j: the j-th choice
  float mine_v = 0.0f, mine_f = 0.0f, mine_z = 0.0f, mine_b = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    uint32_t bk = key[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < EPL; ++i)
      if (key[i] > bk) { bk = key[i]; bi = i; }
    const uint32_t top = __reduce_max_sync(0xffffffffu, bk);
    const uint32_t be =
        __reduce_min_sync(0xffffffffu, bk == top ? (uint32_t)(lane + 32 * bi) : 0xFFFFFFFFu);
    if (lane == j) mine = (int)be;
    if ((be & 31u) == (uint32_t)lane) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if ((int)(be >> 5) == i) key[i] = 0u;
    }
  }
  if (!plain) {
    // every chosen value against the next, and the last against all that were left (the ones
    // still with a key)
    const int src = mine < 0 ? 0 : mine;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      // lane j's expert lives in lane (mine & 31), register mine >> 5
      const float vv = __shfl_sync(0xffffffffu, v[i], src & 31);
      const float ff = __shfl_sync(0xffffffffu, f[i], src & 31);
      const float zz = __shfl_sync(0xffffffffu, zf[i], src & 31);
      if ((src >> 5) == i) { mine_v = vv; mine_f = ff; mine_z = zz; }
    }
    mine_b = a.bias ? __ldg(a.bias + src) : 0.0f;
    const float nv = __shfl_down_sync(0xffffffffu, mine_v, 1);
    const float nf = __shfl_down_sync(0xffffffffu, mine_f, 1);
    const float nz = __shfl_down_sync(0xffffffffu, mine_z, 1);
    const float nb = __shfl_down_sync(0xffffffffu, mine_b, 1);
    if (lane + 1 < a.k)
      unsure |= !(mine_v - nv > mine_f + nf) && !(mine_z == nz && mine_b == nb);
    const float lv = __shfl_sync(0xffffffffu, mine_v, a.k - 1);
    const float lf = __shfl_sync(0xffffffffu, mine_f, a.k - 1);
    const float lz = __shfl_sync(0xffffffffu, mine_z, a.k - 1);
    const float lb = __shfl_sync(0xffffffffu, mine_b, a.k - 1);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (key[i] != 0u && !(lv - v[i] > lf + f[i]) &&
          !(zf[i] == lz && (!a.bias || __ldg(a.bias + lane + 32 * i) == lb)))
        unsure = true;
    if (__any_sync(0xffffffffu, unsure)) mine = route_exact<DT, EPL>(z, a, m, sv, lane);
  }
  // the chosen scores in 64 bits
  double p = 0.0;
  if (lane < a.k) {
    const float zm = DTraits<DT>::up(z[mine]);
    if (a.sigmoid) p = 1.0 / (1.0 + exp(-(double)zm));
    else p = m == ninf_f() && zm == m ? 0.0 : exp((double)zm - (double)m);
    if (poison) p = __longlong_as_double(0x7FF8000000000000ll);
    if (!a.sigmoid && !a.renorm && sum != 0.0) p /= sum;
  }
  if (a.renorm) {
    double total = p;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    p = total == 0.0 ? 0.0 : p / total;
  }
  if (lane < a.k) {
    a.ids[t * a.k + lane] = mine;
    a.weights[t * a.k + lane] = __double2float_rn(p * (double)a.scale);
  }
}

template <int DT, int EPL>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  extern __shared__ double s_v[];   // [kRouteWarps][E] with groups
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (long long t = (long long)blockIdx.x * kRouteWarps + warp; t < a.T;
       t += (long long)gridDim.x * kRouteWarps)
    route_token<DT, EPL>(a, t, s_v + (a.G > 1 ? (size_t)warp * a.E : 0), lane);
}

// Groups the flat indices i = t * k + j of ids by expert, in ascending order within each:
// order, offsets; entries behind offsets[E] are -1.  An id outside [0, E) belongs to none.
// A stable counting sort by one CTA, or by the CTAs of one cluster, which pass each other their
// counts through shared memory.  Every warp owns a run of consecutive entries: it counts them
// by expert (equal ids of 32 entries at once), the counts become the places of its first
// entry of each expert, and a second walk writes.  No atomics: the result does not depend on
// the order in which the warps run.
struct PlanShared {
  int* cnt;     // [warps][E]
  int* tot;     // [E] of this CTA (read by the cluster's other CTAs)
  int* base;    // [E]
  int* part;    // [32]
};

__device__ __forceinline__ void plan_experts_cta(const int32_t* ids, int S, int E,
                                                 int32_t* offsets, int32_t* order,
                                                 const PlanShared& s, int rank, int ctas) {
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int run = (S + ctas * warps - 1) / (ctas * warps);
  run = (run + 31) & ~31;
  const int begin = min(S, (rank * warps + warp) * run);
  const int end = min(S, begin + run);
  int* mine = s.cnt + warp * E;
  for (int e = lane; e < E; e += 32) mine[e] = 0;
  __syncwarp();
  for (int i = begin + lane; i - lane < end; i += 32) {
    const int id = i < end ? ids[i] : -1;
    const bool in = id >= 0 && id < E;
    const uint32_t same = __match_any_sync(0xffffffffu, in ? id : -1);
    if (in && lane == __ffs(same) - 1) mine[id] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // counts -> exclusive sums over this CTA's warps, and the CTA's totals
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int sum = 0;
    for (int w = 0; w < warps; ++w) {
      const int c = s.cnt[w * E + e];
      s.cnt[w * E + e] = sum;
      sum += c;
    }
    s.tot[e] = sum;
  }
  __syncthreads();
  if (ctas > 1) {
    cluster_arrive();
    cluster_wait();
  }
  // all CTAs' totals of expert e, and those of the CTAs before this one
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    int all = 0, before = 0;
    if (e < E) {
      for (int c = 0; c < ctas; ++c) {
        int n = s.tot[e];
        if (ctas > 1) {
          const uint32_t remote = cluster_map(smem_u32(s.tot + e), (uint32_t)c);
          asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(n) : "r"(remote) : "memory");
        }
        all += n;
        if (c < rank) before += n;
      }
    }
    int v = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) s.part[warp] = v;
    __syncthreads();
    int below = carry, whole = 0;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) below += s.part[w];
      whole += s.part[w];
    }
    if (e < E) {
      s.base[e] = below + v - all + before;
      if (rank == 0) offsets[e] = below + v - all;
    }
    carry += whole;
    __syncthreads();
  }
  if (rank == 0 && threadIdx.x == 0) offsets[E] = carry;
  for (int e = lane; e < E; e += 32) mine[e] += s.base[e];
  __syncwarp();
  for (int i = begin + lane; i - lane < end; i += 32) {
    const int id = i < end ? ids[i] : -1;
    const bool in = id >= 0 && id < E;
    const uint32_t same = __match_any_sync(0xffffffffu, in ? id : -1);
    const int at = in ? mine[id] : 0;
    __syncwarp();
    if (in) {
      order[at + __popc(same & ((1u << lane) - 1u))] = i;
      if (lane == __ffs(same) - 1) mine[id] = at + __popc(same);
    }
    __syncwarp();
  }
  for (int i = carry + rank * (int)blockDim.x + (int)threadIdx.x; i < S; i += ctas * blockDim.x)
    order[i] = -1;
  if (ctas > 1) {   // no CTA leaves while another may still read its totals
    cluster_arrive();
    cluster_wait();
  }
}

__device__ __forceinline__ PlanShared plan_shared(int* smem, int E, int warps) {
  PlanShared s;
  s.cnt = smem;
  s.tot = smem + warps * E;
  s.base = s.tot + E;
  s.part = s.base + E;
  return s;
}
constexpr int plan_smem(int E, int warps) { return (warps * E + 2 * E + 32) * 4; }

__global__ void __launch_bounds__(1024) plan_kernel(const int32_t* __restrict__ ids, int S, int E,
                                                    int32_t* __restrict__ offsets,
                                                    int32_t* __restrict__ order) {
  grid_dep_wait();
  grid_dep_launch();
  extern __shared__ int s_plan[];
  plan_experts_cta(ids, S, E, offsets, order, plan_shared(s_plan, E, blockDim.x >> 5),
                   (int)blockIdx.x, (int)gridDim.x);
}

// Routing and grouping of a few tokens in one CTA: a decode step is bound by its launches.
template <int DT, int EPL>
__global__ void __launch_bounds__(512) route_plan_kernel(const RouteArgs a, int32_t* offsets,
                                                         int32_t* order) {
  grid_dep_wait();
  grid_dep_launch();
  extern __shared__ double s_v[];   // [warps][E] with groups; the counting sort's arrays after
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  for (int t = warp; t < a.T; t += warps)
    route_token<DT, EPL>(a, t, s_v + (a.G > 1 ? (size_t)warp * a.E : 0), lane);
  __syncthreads();   // the ids in global memory are this CTA's own writes
  plan_experts_cta(a.ids, a.T * a.k, a.E, offsets, order,
                   plan_shared(reinterpret_cast<int*>(s_v), a.E, warps), 0, 1);
}

}  // namespace apex
