// route.cuh -- routing of tokens to experts, and the grouping of the routed tokens by expert.
//
// For every token with logits z[E]:
//   p = softmax(z) or 1 / (1 + exp(-z))                       (scores)
//   v = p + bias                                              (values that are compared)
//   groups > 1: a group of E / groups neighbouring experts is worth the sum of its two largest
//   v, or its largest alone; experts of the topk_groups best groups stay in the choice
//   ids = the k largest v, ties to the lowest index;  weights = scale * p[ids], divided by
//   their sum first when renormalized.
// The choice is that of v in 64 bits; without a bias the order of v is the order of z, which is
// compared itself (by groups' largest too, so that nothing is left to decide there).  A NaN is chosen last; a softmax row of -inf alone has scores 0; weights
// whose sum is 0 stay 0.
//
// 64-bit exponentials of every logit cost 230 us for 16384 tokens x 256 experts, sixty times
// the time of reading them.  So the choice is made on fp32 values with a bound on their errors
// for the row.  Where two neighbours in the chosen order (or the last chosen and the best left)
// are closer than their bounds, the chosen and the next few are compared again in 64 bits, a lane
// each; where groups on either side of the border are, the groups are; with NaNs, or more near
// ties than that, the whole token is.  The chosen experts' scores are 64-bit.  What divides them in a
// softmax without renormalization is a 64-bit sum of fp32 exponentials, each within 1.5 ulp: such
// weights are within 2^-22 of the exact ones with their rounding, others within 2^-24.
//
// The largest values are taken in turn.  Every lane first sorts its values as 32-bit keys whose
// low bits are replaced by the register's number, so that a comparator is a maximum and a
// minimum; a round is then one warp-wide maximum and a shift in the lane that had it.  (Values
// that come from 16-bit logits as they are have those bits free: their keys hold the expert's
// number and decide exactly, ties to the lowest index.)
// Measured: 16384 tokens x 256 experts, fp32: softmax 18 us, sigmoid with a bias and 8 groups 32
// us.  Instructions bound it (59 % of the issue slots); the logits take 2.6 us to read.
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
  int group_max;           // a group is worth its largest value alone
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

// A lane's part in the groups' worths: 1 << shift neighbouring lanes share a group.  Made once a
// warp: the divisions would be a third of a token's instructions.
struct RouteGroups {
  int shift;     // lane >> shift: this lane's group (G and above: none)
  int mine;
  int n;         // values of a group a lane reads, at most
  int start;     // the first of them: groups start at different places, for different banks
  int at;        // this lane's value 0
  int left;      // values of the group from there on
  bool pairs;    // a group is worth the sum of two experts' values
};

__device__ __forceinline__ RouteGroups route_groups(const RouteArgs& a, int lane) {
  RouteGroups q;
  const int G = a.G;
  q.shift = 5;
  while (G > 32 >> q.shift) --q.shift;
  const int epg = a.E / G, s = lane & ((1 << q.shift) - 1);
  q.mine = lane >> q.shift;
  q.n = (epg + (1 << q.shift) - 1) >> q.shift;
  q.start = q.mine % q.n;
  q.at = q.mine * epg + s;
  q.left = q.mine < G ? epg - s : 0;
  q.pairs = epg > 1 && !a.group_max;
  return q;
}

// Worth of this lane's group from the values sv[E] in shared memory (lanes of no group: -inf).
// size: the two values' magnitudes together.
template <typename F>
__device__ __forceinline__ F group_worth(const F* sv, const RouteGroups& q, F ninf, F& size) {
  F best = ninf, second = ninf;
  const F* v = sv + q.at;
  int i = q.start;
#pragma unroll 4
  for (int c = 0; c < q.n; ++c) {
    const int off = i << q.shift;
    const F w = off < q.left ? v[off] : ninf;
    second = w > best ? best : w > second ? w : second;
    best = w > best ? w : best;
    i = i + 1 == q.n ? 0 : i + 1;
  }
  for (int o = 1; o < 1 << q.shift; o <<= 1) {
    const F b2 = __shfl_xor_sync(0xffffffffu, best, o);
    const F s2 = __shfl_xor_sync(0xffffffffu, second, o);
    merge2(best, second, b2, s2);
  }
  size = q.pairs ? fabs(best) + fabs(second) : fabs(best);
  return q.pairs ? best + second : best;
}

// The bit set of the TG groups of largest worth, ties to the lowest.
template <typename F>
__device__ __forceinline__ uint32_t open_groups(F worth, int G, int TG, const RouteGroups& q,
                                                int lane) {
  int rank = 0;
#pragma unroll 4
  for (int g = 0; g < G; ++g) {
    const F other = __shfl_sync(0xffffffffu, worth, g << q.shift);
    rank += other > worth || (other == worth && g < q.mine);
  }
  const bool first = (lane & ((1 << q.shift) - 1)) == 0;
  const uint32_t set = q.mine < G && rank < TG && first ? 1u << q.mine : 0u;
  return __reduce_or_sync(0xffffffffu, set);
}

// A logit's score before normalization, in 64 bits.
__device__ __forceinline__ double route_score64(float z, bool sigmoid, float m) {
  if (sigmoid) return 1.0 / (1.0 + exp(-(double)z));
  return m == ninf_f() && z == m ? 0.0 : exp((double)z - (double)m);
}

// The sum of a softmax row's scores in 64 bits.
template <int DT>
__device__ __forceinline__ double route_sum64(const typename DTraits<DT>::T* z, int E, float m,
                                              int lane) {
  double sum = 0.0;
#pragma unroll 2
  for (int e = lane; e < E; e += 32) sum += route_score64(DTraits<DT>::up(z[e]), false, m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// Whether values are compared as logits: their order is that of the scores, and no sum of two
// scores is asked for.
__device__ __forceinline__ bool route_by_logits(const RouteArgs& a) {
  return a.bias == nullptr && (a.G == 1 || a.group_max);
}

// The groups that stay open, by 64-bit values.
template <int DT>
__device__ __noinline__ uint32_t route_open64(const typename DTraits<DT>::T* z, const RouteArgs& a,
                                              float m, bool poison, double* sv, int lane) {
  // (without a bias a softmax row's sum divides every group's worth)
  const double sum = a.bias && !a.sigmoid ? route_sum64<DT>(z, a.E, m, lane) : 1.0;
#pragma unroll 4
  for (int e = lane; e < a.E; e += 32) {
    const float ze = DTraits<DT>::up(z[e]);
    double w = route_by_logits(a) ? (double)ze : route_score64(ze, a.sigmoid, m);
    if (a.bias) w = (a.sigmoid ? w : sum == 0.0 ? 0.0 : w / sum) + (double)__ldg(a.bias + e);
    sv[e] = w == w && !poison ? w : ninf_d();   // poison: every score is NaN
  }
  __syncwarp();
  const RouteGroups q = route_groups(a, lane);
  double size;
  const double worth = group_worth<double>(sv, q, ninf_d(), size);
  __syncwarp();
  return open_groups(worth, a.G, a.TG, q, lane);
}

// The whole choice in 64 bits; returns lane j's j-th expert.
template <int DT, int EPL>
__device__ __noinline__ int route_exact(const typename DTraits<DT>::T* z, const RouteArgs& a,
                                        float m, bool poison, double* sv, int lane) {
  const int E = a.E;
  const uint32_t open = a.G > 1 ? route_open64<DT>(z, a, m, poison, sv, lane) : 0xffffffffu;
  const double sum = a.bias && !a.sigmoid ? route_sum64<DT>(z, E, m, lane) : 1.0;
  const int epg = E / a.G;
  double v[EPL];
  uint32_t left = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    v[i] = ninf_d();
    if (e < E && (a.G == 1 || ((open >> (e / epg)) & 1u))) {
      left |= 1u << i;
      const float zi = DTraits<DT>::up(z[e]);
      double w = (double)zi;   // without a bias: the order of the logits
      if (a.bias) {
        w = route_score64(zi, a.sigmoid, m);
        w = (a.sigmoid ? w : sum == 0.0 ? 0.0 : w / sum) + (double)__ldg(a.bias + e);
      }
      if (w == w) v[i] = w;
    }
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

// Lane c < n holds candidate expert `id`, all of a token's choice among them: their order by the
// exact values; returns lane j's j-th.
template <int DT>
__device__ __noinline__ int route_candidates(const typename DTraits<DT>::T* z, const RouteArgs& a,
                                             float m, int id, int n, int lane) {
  const double sum = a.bias && !a.sigmoid ? route_sum64<DT>(z, a.E, m, lane) : 1.0;
  double v = ninf_d();
  if (lane < n) {
    const float zi = DTraits<DT>::up(z[id]);
    v = !a.bias ? (double)zi : route_score64(zi, a.sigmoid, m);
    if (a.bias) v = (a.sigmoid ? v : sum == 0.0 ? 0.0 : v / sum) + (double)a.bias[id];
    if (!(v == v)) v = ninf_d();
  }
  int rank = 0;
  for (int c = 0; c < n; ++c) {
    const double o = __shfl_sync(0xffffffffu, v, c);
    const int oid = __shfl_sync(0xffffffffu, id, c);
    rank += o > v || (o == v && oid < id);
  }
  int mine = -1;
  for (int c = 0; c < n; ++c) {
    const int r = __shfl_sync(0xffffffffu, rank, c);
    const int oid = __shfl_sync(0xffffffffu, id, c);
    if (r == lane) mine = oid;
  }
  return mine;
}

// What the last step needs of a token whose experts are chosen.
struct RouteChoice {
  int id;         // lane j: the j-th expert (-1: the token is masked)
  float m;        // softmax: the row's largest logit
  double sum;     // softmax without renormalization: the sum of exp(z - m)
  bool poison;    // softmax: a NaN or +inf logit makes every score NaN
};

// Sorts EPL keys in descending order (Batcher's odd-even merge sort network; EPL a power of two).
template <int EPL>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[EPL]) {
#pragma unroll
  for (int p = 1; p < EPL; p <<= 1)
#pragma unroll
    for (int q = p; q >= 1; q >>= 1)
#pragma unroll
      for (int j = q % p; j + q < EPL; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < EPL && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const uint32_t x = k[i + j], y = k[i + j + q];
            k[i + j] = max(x, y);
            k[i + j + q] = min(x, y);
          }
}

// One token by one warp; lane l holds experts l, l + 32, ...  sv: E doubles of this warp's
// shared memory (used with groups only).
template <int DT, int EPL>
__device__ __forceinline__ void route_load(const RouteArgs& a, long long t, int lane,
                                           float (&zv)[EPL]) {
  const typename DTraits<DT>::T* z =
      static_cast<const typename DTraits<DT>::T*>(a.logits) + t * a.E;
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    zv[i] = lane + 32 * i < a.E ? DTraits<DT>::up(z[lane + 32 * i]) : ninf_f();
}

template <int DT, int EPL, bool GROUPS>
__device__ __forceinline__ RouteChoice route_choose(const RouteArgs& a, long long t,
                                                    const float (&zv)[EPL],
                                                    const RouteGroups& q,
                                                    const uint32_t (&of)[EPL / 4 + 1], double* sv,
                                                    int lane) {
  RouteChoice r;
  r.id = -1;
  r.m = ninf_f();
  r.sum = 0.0;
  r.poison = false;
  if (a.mask && !a.mask[t]) return r;
  const int E = a.E;
  const typename DTraits<DT>::T* z = static_cast<const typename DTraits<DT>::T*>(a.logits) + t * E;
  const bool plain = a.bias == nullptr && (!GROUPS || a.group_max);   // (route_by_logits)
  float v[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) v[i] = zv[i];
  float F = 0.0f;   // bound on the error of every v before the bias
  if (!a.sigmoid) {
    bool nan = false;
    float m = ninf_f();
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      nan |= !(v[i] == v[i]);
      m = fmaxf(m, v[i]);
    }
    const uint32_t mk = __reduce_max_sync(0xffffffffu, route_key(m));
    m = __uint_as_float((mk & 0x80000000u) ? mk & 0x7FFFFFFFu : ~mk);
    r.m = m;
    r.poison = __any_sync(0xffffffffu, nan) || m == -ninf_f();
    if (!plain || !a.renorm) {
      float sum = 0.0f;
      float e[EPL];
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        // exp(z - m) with the rounding of z - m made good: within 1.5 ulp of the exact value
        const float d = v[i] - m;
        const float lost = fabsf(v[i]) > fabsf(m) ? -m - (d - v[i]) : v[i] - (d + m);
        e[i] = v[i] == ninf_f() ? 0.0f : a.renorm ? __expf(d) : expf(d);
        e[i] = fabsf(lost) < 1.0f ? fmaf(e[i], lost, e[i]) : e[i];
        sum += e[i];
        r.sum += (double)e[i];
      }
      if (!a.renorm) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) r.sum += __shfl_xor_sync(0xffffffffu, r.sum, o);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (!plain) {
        const float inv = sum == 0.0f ? 0.0f : __frcp_rn(sum);
        // The sum: EPL + 5 roundings (under 2^-19.5 together) and its terms' errors, the fast
        // exponential's (2 + 1.2 |d|) 2^-23 with |d| = 7 at most on average.  A score's own:
        // 2^-22 of it, and 1.2 |d| p 2^-23 <= 0.5 top 2^-23.
        F = inv * 0x1p-18f + 0x1p-23f;   // inv: the largest score
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[i] = e[i] * inv;
      }
    }
  } else if (!plain) {
    // 1 / (1 + exp(-z)): the fast exponential's relative error (2 + 1.2 |z|) 2^-23 counts
    // p (1 - p) times, p (1 - p) |z| < 0.23; with the sum's rounding and the reciprocal's ulp
    // under 2^-22 in all
    F = 0x1p-21f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = rcp_approx(1.0f + __expf(-v[i]));
  }
  if (!plain) {
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (lane + 32 * i < E) v[i] += __ldg(a.bias + lane + 32 * i);
    }
  }
  uint32_t open = 0xffffffffu;
  bool unsure = false;
  if (GROUPS) {
    float* s32 = reinterpret_cast<float*>(sv);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + 32 * i < E)
        s32[lane + 32 * i] = v[i] == v[i] && !(plain && r.poison) ? v[i] : ninf_f();
    __syncwarp();
    float size;
    const float worth = group_worth<float>(s32, q, ninf_f(), size);
    __syncwarp();
    open = open_groups(worth, a.G, a.TG, q, lane);
    if (a.TG < a.G && !plain) {
      // two values, each within F and the rounding of its sum with the bias, and the rounding of
      // their sum, on either side of the border; an infinite worth lies beyond every finite one
      const float err = size < -ninf_f() ? 2.0f * F + size * 0x1p-23f : 0.0f;
      const int g = q.mine;
      const bool kept = g < a.G && ((open >> g) & 1u);
      // (as keys, for one warp-wide minimum and maximum; a NaN decides nothing: 64 bits)
      const uint32_t low = kept ? route_key(worth - err) : 0xffffffffu;
      const uint32_t high = g < a.G && !kept ? route_key(worth + err) : 0u;
      if (__reduce_min_sync(0xffffffffu, low) <= __reduce_max_sync(0xffffffffu, high))
        open = route_open64<DT>(z, a, r.m, r.poison, sv, lane);
    }
  }
  // keys: the value (without a bias: the logit) in the upper bits, NaN as -inf and a closed or
  // absent expert as 0; below it the register's number, or the whole expert's where 16-bit
  // logits leave those bits free
  constexpr bool HALF = DT != DT_F32;
  const bool whole = HALF && a.bias == nullptr;
  const uint32_t low_bits = whole ? 511u : (uint32_t)(EPL - 1);
  uint32_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    const bool in =
        e < E && (!GROUPS || (__funnelshift_r(open, 0u, of[i / 4] >> (8 * (i % 4))) & 1u));
    const float w = a.bias ? v[i] : zv[i];
    const uint32_t k32 = route_key(w == w ? w : ninf_f());
    const uint32_t low = low_bits - (whole ? (uint32_t)e : (uint32_t)i);
    key[i] = in ? (k32 & ~low_bits) | low : 0u;
    unsure |= !(w == w);   // NaNs tie with -inf (whole keys tell them apart as 64 bits would)
  }
  sort_keys<EPL>(key);
  uint32_t mine = 0;   // lane j: the j-th largest key
  auto rounds = [&](int from, int to) {
    for (int j = from; j < to; ++j) {
      const uint32_t top = __reduce_max_sync(0xffffffffu, key[0]);
      const int winner = __ffs(__ballot_sync(0xffffffffu, key[0] == top)) - 1;
      if (lane == j) {
        mine = top;
        r.id = whole ? (int)(511u - (top & 511u)) : winner + 32 * (int)(low_bits - (top & low_bits));
      }
      if (lane == winner) {
#pragma unroll
        for (int i = 0; i + 1 < EPL; ++i) key[i] = key[i + 1];
        key[EPL - 1] = 0u;
      }
    }
  };
  if (whole) {
    rounds(0, a.k);
  } else {
    rounds(0, min(32, a.k + 1));
    if (a.bias == nullptr) F = 0.0f;   // logits are compared as they are
    // neighbours in the order that are not clearly apart (key 0: nothing was left)
    auto decode = [](uint32_t k) {
      return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
    };
    // what the keys' low bits hide, EPL - 1 units, and the rounding of the sum with the bias
    const float cut = (float)EPL * 0x1p-23f;
    auto apart = [&](uint32_t hi, uint32_t lo) {
      const float x = decode(hi), y = decode(lo);
      return lo == 0u || x - y > 2.0f * F + cut * (fabsf(x) + fabsf(y)) + 0x1p-120f;
    };
    const uint32_t next = __shfl_down_sync(0xffffffffu, mine, 1);
    const bool close = lane < a.k && !(lane < 31 && apart(mine, next));
    if (__any_sync(0xffffffffu, close || unsure)) {
      const int n = min(32, a.k + 8);   // candidates: the choice is among them if the last is out
      rounds(min(32, a.k + 1), n);
      const uint32_t kth = __shfl_sync(0xffffffffu, mine, a.k - 1);
      const uint32_t last = __shfl_sync(0xffffffffu, mine, n - 1);
      if (!__any_sync(0xffffffffu, unsure) && n > a.k && apart(kth, last))
        r.id = route_candidates<DT>(z, a, r.m, r.id,
                                    __popc(__ballot_sync(0xffffffffu, lane < n && mine != 0u)), lane);
      else
        r.id = route_exact<DT, EPL>(z, a, r.m, r.poison, sv, lane);
    }
  }
  return r;
}

// The weights of up to 32 / kp tokens at once, kp lanes each: lane b * kp + j has the j-th choice
// of token t0 + b.  Scores in 64 bits (but for a softmax's whole sum), one rounding.
template <int DT>
__device__ __forceinline__ void route_write(const RouteArgs& a, long long t0, int batch, int kp,
                                            const RouteChoice& r, int lane) {
  const int b = lane / kp, j = lane - b * kp;
  const long long t = t0 + b;
  const bool mine = b < batch && j < a.k && t < a.T;
  double p = 0.0;
  if (mine && r.id >= 0) {
    const float zm = DTraits<DT>::up(
        static_cast<const typename DTraits<DT>::T*>(a.logits)[t * a.E + r.id]);
    if (a.sigmoid) p = 1.0 / (1.0 + exp(-(double)zm));
    else p = r.m == ninf_f() && zm == r.m ? 0.0 : exp((double)zm - (double)r.m);
    if (r.poison) p = __longlong_as_double(0x7FF8000000000000ll);
    if (!a.sigmoid && !a.renorm && r.sum != 0.0) p /= r.sum;
  }
  if (a.renorm) {
    double total = p;
    for (int o = kp >> 1; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    p = total == 0.0 ? 0.0 : p / total;
  }
  if (mine) {
    a.ids[t * a.k + j] = r.id;
    a.weights[t * a.k + j] = __double2float_rn(p * (double)a.scale);
  }
}

// Tokens first, first + step, ..., `batch` (32 / kp at most) neighbours at a time.
template <int DT, int EPL, bool GROUPS>
__device__ __forceinline__ void route_tokens(const RouteArgs& a, long long first, long long step,
                                             int batch, double* sv, int lane) {
  int kp = 1;
  while (kp < a.k) kp <<= 1;
  RouteGroups q = {};
  if (GROUPS) q = route_groups(a, lane);
  uint32_t of[EPL / 4 + 1];   // the groups of this lane's experts, a byte each
#pragma unroll
  for (int i = 0; i < EPL / 4 + 1; ++i) of[i] = 0u;
  if (GROUPS) {
    const int epg = a.E / a.G;
#pragma unroll
    for (int i = 0; i < EPL; ++i) of[i / 4] |= (uint32_t)((lane + 32 * i) / epg) % 32u << (8 * (i % 4));
  }
  for (long long t0 = first * batch; t0 < a.T; t0 += step * batch) {
    RouteChoice all;
    all.id = -1;
    all.m = 0.0f;
    all.sum = 0.0;
    all.poison = false;
    float zv[EPL];
    route_load<DT, EPL>(a, t0, lane, zv);
    for (int b = 0; b < batch && t0 + b < a.T; ++b) {
      float zn[EPL];   // the next token's logits are on their way meanwhile
      if (b + 1 < batch && t0 + b + 1 < a.T) route_load<DT, EPL>(a, t0 + b + 1, lane, zn);
      const RouteChoice r = route_choose<DT, EPL, GROUPS>(a, t0 + b, zv, q, of, sv, lane);
#pragma unroll
      for (int i = 0; i < EPL; ++i) zv[i] = zn[i];
      const int id = __shfl_sync(0xffffffffu, r.id, lane & (kp - 1));
      if (lane / kp == b) {
        all = r;
        all.id = id;
      }
    }
    route_write<DT>(a, t0, batch, kp, all, lane);
  }
}

template <int DT, int EPL, bool GROUPS>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteArgs a, int batch) {
  grid_dep_wait();
  grid_dep_launch();
  extern __shared__ double s_v[];   // [kRouteWarps][E] with groups
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  route_tokens<DT, EPL, GROUPS>(a, (long long)blockIdx.x * kRouteWarps + warp,
                        (long long)gridDim.x * kRouteWarps, batch,
                        s_v + (GROUPS ? (size_t)warp * a.E : 0), lane);
}

// Groups the flat indices i = t * k + j of ids by expert, in ascending order within each:
// order, offsets; entries behind offsets[E] are -1.  An id outside [0, E) belongs to none.
// A stable counting sort by one CTA, or by the CTAs of one cluster, which pass each other their
// counts through shared memory.  Every warp owns a run of consecutive entries: it counts them
// by expert, the counts become the places of its first entry of each expert, and a second walk
// writes, with the places of equal ids among 32 from one ballot for each bit of an id (a
// hardware match takes 60 cycles of a unit that the whole SM shares).  The atomics only count:
// the result does not depend on the order in which the warps run.  Bound: a few dependent steps
// for few choices (4662: 4.6 us), the ballots for many (131072: 11.2 us).
constexpr int kPlanBatch = 16;    // loads in flight
constexpr int kPlanClusterMax = 16;
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
  int bits = 0;
  while ((1 << bits) < E + 1) ++bits;
  int id[kPlanBatch];   // a run of one batch stays here for the second walk
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kPlanBatch; ++u) {
      const int i = i0 + 32 * u + lane;
      id[u] = i < end ? ids[i] : E;
      if (id[u] < 0 || id[u] >= E) id[u] = E;   // none
    }
  };
  for (int i0 = begin; i0 < end; i0 += 32 * kPlanBatch) {
    load(i0);
#pragma unroll
    for (int u = 0; u < kPlanBatch; ++u)
      if (id[u] < E) atomicAdd(mine + id[u], 1);   // counts alone: any order
  }
  __syncthreads();
  // counts -> exclusive sums over this CTA's warps, and the CTA's totals
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int sum = 0;
    for (int w0 = 0; w0 < warps; w0 += 8) {   // (warps is a multiple of 8)
      int c[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) c[u] = s.cnt[(w0 + u) * E + e];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        s.cnt[(w0 + u) * E + e] = sum;
        sum += c[u];
      }
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
      if (ctas > 1) {
        int n[kPlanClusterMax];
#pragma unroll
        for (int c = 0; c < kPlanClusterMax; ++c) {
          n[c] = 0;
          if (c >= ctas) continue;
          const uint32_t remote = cluster_map(smem_u32(s.tot + e), (uint32_t)c);
          asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(n[c]) : "r"(remote) : "memory");
        }
#pragma unroll
        for (int c = 0; c < kPlanClusterMax; ++c) {
          all += n[c];
          before += c < rank ? n[c] : 0;
        }
      } else {
        all = s.tot[e];
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
    int p = lane < warps ? s.part[lane] : 0;   // every warp: the sums of the warps before it
    const int mine_w = p;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, p, o);
      if (lane >= o) p += u;
    }
    const int whole = __shfl_sync(0xffffffffu, p, 31);
    const int below = carry + __shfl_sync(0xffffffffu, p - mine_w, warp);
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
  const bool again = run > 32 * kPlanBatch;
  for (int i0 = begin; i0 < end; i0 += 32 * kPlanBatch) {
    if (again) load(i0);
#pragma unroll
    for (int u = 0; u < kPlanBatch; ++u) {
      if (i0 + 32 * u >= end) break;
      uint32_t same = 0xffffffffu;   // the lanes with this lane's id
      for (int b = 0; b < bits; ++b) {
        const uint32_t set = __ballot_sync(0xffffffffu, (id[u] >> b) & 1);
        same &= ((id[u] >> b) & 1) ? set : ~set;
      }
      const bool in = id[u] < E;
      const int at = in ? mine[id[u]] : 0;
      __syncwarp();
      if (in) {
        order[at + __popc(same & ((1u << lane) - 1u))] = i0 + 32 * u + lane;
        if (lane == __ffs(same) - 1) mine[id[u]] = at + __popc(same);
      }
      __syncwarp();
    }
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

__global__ void __launch_bounds__(512) plan_kernel(const int32_t* __restrict__ ids, int S, int E,
                                                    int32_t* __restrict__ offsets,
                                                    int32_t* __restrict__ order) {
  grid_dep_wait();
  grid_dep_launch();
  extern __shared__ int s_plan[];
  plan_experts_cta(ids, S, E, offsets, order, plan_shared(s_plan, E, blockDim.x >> 5),
                   (int)blockIdx.x, (int)gridDim.x);
}

// Routing and grouping of a few tokens in one CTA: a decode step is bound by its launches.
template <int DT, int EPL, bool GROUPS>
__global__ void __launch_bounds__(512) route_plan_kernel(const RouteArgs a, int32_t* offsets,
                                                         int32_t* order) {
  grid_dep_wait();
  grid_dep_launch();
  extern __shared__ double s_v[];   // [warps][E] with groups; the counting sort's arrays after
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  route_tokens<DT, EPL, GROUPS>(a, warp, warps, 1, s_v + (GROUPS ? (size_t)warp * a.E : 0), lane);
  __syncthreads();   // the ids in global memory are this CTA's own writes
  plan_experts_cta(a.ids, a.T * a.k, a.E, offsets, order,
                   plan_shared(reinterpret_cast<int*>(s_v), a.E, warps), 0, 1);
}

}  // namespace apex
