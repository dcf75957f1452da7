// gemm_f8_block.cuh -- the block-scaled FP8 GEMM for many tokens, dense and over experts.
//
//   Y[m,n] = sum_g P_g[m,n] * (sa[m,g] * sw[n/128,g]),   P_g = sum_{k in 128-wide group g} a*w
//
// with E4M3 operands (f8_block.cuh).  The tensor cores form P_g in fp32 (tcgen05.mma
// kind::f8f6f4); one weight scale serves 128 outputs, so with tokens in the tensor-memory
// lanes a thread multiplies its token's whole row of partials by one number: one packed fma
// per two partials, half of what per-row weight scales cost (gemm_f8.cuh).
//
// Kinds:
//   FB_DENSE  Y[M][N] = A . W^T.
//   FB_UP     for rows grouped by expert (slots), row of slot s = token order[s] / k: the
//             products with the expert's gate and up matrices, h = silu(gate) * up, quantized
//             in groups of 128 as the next product's operand.  A tile is 128 rows x 128
//             columns of h: its weight operand is 128 gate rows above 128 up rows.
//   FB_DOWN   h . W^T of each slot's expert, written to row order[s] (token-major).
// FB_UP fetches its scattered token rows by TMA row gathers (four rows each), so no permuted
// copy of the activations is made.
//
// Tile: 128 tokens (MMA M) x BN weight rows (MMA N), one K-group per pipeline stage, both
// operands by TMA with 128-byte swizzle; the group's partial goes to one of 512 / BN
// tensor-memory slots, which the epilogue drains while the next groups' MMAs fill the others.
// Roles (384 threads, one persistent CTA per SM): warp 0 TMA, warp 1 MMA, warps 4..11
// epilogue (warp w: lanes 32*(w%4).., half (w-4)/4 of the columns).
#pragma once
#include <cuda.h>
#include <stdint.h>

#include "f8_block.cuh"
#include "ptx.cuh"

namespace apex {

enum FBKind : int { FB_DENSE = 0, FB_UP = 1, FB_DOWN = 2 };

struct FBArgs {
  int M, N, K;          // rows (dense), outputs, inner size
  int G, NB;            // ceil(K / 128), ceil(N / 128)
  int tiles_m, tiles_n; // dense: token tiles; all: column tiles
  int P;                // persistent CTAs
  // experts (FB_UP, FB_DOWN): slots = T * k rows at most, grouped by expert
  int E, slots, top_k;
  const int32_t* offsets;   // [E + 1]
  const int32_t* order;     // [slots]
  const float* sa;          // [rows][G]
  const float* sw;          // [E (x 2 for FB_UP)][NB][G]
  void* y;                  // [rows][N]
  uint8_t* hq;              // FB_UP: codes [slots][N] and scales [slots][NB]
  float* hs;
  int s_vec;                // scale rows readable as 16-byte blocks of 4 groups
  int y_vec;                // output rows writable as 16-byte vectors
  unsigned long long wait_ns;
};

constexpr int kMaxExperts = 512;

template <int BN>
struct FBCfg {
  static constexpr int BM = 128;
  static constexpr int A_BYTES = BM * 128;
  static constexpr int B_BYTES = BN * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int NS = BN == 256 ? 4 : 6;
  static constexpr int SLOTS = 512 / BN;
  static constexpr int EPI_WARPS = 8;
  static constexpr int THREADS = 128 + 32 * EPI_WARPS;
  // 384 x 168 registers at launch; the first warpgroup keeps 40, the epilogue takes 232
  static constexpr int REGS_CTRL = 40, REGS_EPI = 232;
  static_assert(128 * REGS_CTRL + 256 * REGS_EPI <= THREADS * 168, "register pool");
  static constexpr int CPT = BN / 2;   // partials per epilogue thread
  static constexpr int OFF_CUM = NS * STAGE;                       // [kMaxExperts + 1] ints
  static constexpr int OFF_AMAX = OFF_CUM + (kMaxExperts + 4) * 4;  // [2][2][128] words
  static constexpr int OFF_BAR = OFF_AMAX + 2 * 2 * 128 * 4;
  static constexpr int NBAR = 2 * NS + 2 * SLOTS + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

// The number of rows of expert e, clamped so that no offsets array leads out of the slots.
__device__ __forceinline__ int expert_rows(const int32_t* offsets, int e, int slots, int* first) {
  const int a = max(0, min(__ldg(offsets + e), slots));
  const int b = max(0, min(__ldg(offsets + e + 1), slots));
  *first = a;
  return max(0, b - a);
}

// cum[e] = tiles of BM rows of the experts before e (cum[E]: all of them), by one warp.
__device__ __forceinline__ void expert_tiles_scan(const int32_t* offsets, int E, int slots,
                                                  int bm, int* cum, int lane) {
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    int first, n = 0;
    if (e0 + lane < E) n = (expert_rows(offsets, e0 + lane, slots, &first) + bm - 1) / bm;
    int v = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (e0 + lane < E) cum[e0 + lane] = carry + v - n;
    carry += __shfl_sync(0xffffffffu, v, 31);
    // more tiles than the slots can fill: offsets that do not ascend.  No tile is computed.
    if (carry > slots / bm + E) {
      carry = 0;
      break;
    }
  }
  if (lane == 0) cum[E] = carry;
}

struct ExpertTile {
  int e;      // expert (0 when dense)
  int row0;   // first row / slot
  int rows;   // rows of the tile that exist
  int tn;     // column tile
};

// Tile t of an expert grid: experts in order; within one, its row tiles fastest, so that CTAs
// running together share the expert's weight tiles while they are in L2.
__device__ __forceinline__ ExpertTile expert_tile(const int32_t* offsets, const int* cum, int E,
                                                  int slots, int tiles_n, int bm, int t) {
  int lo = 0, hi = E;   // cum[lo] * tiles_n <= t < cum[hi] * tiles_n
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cum[mid] * tiles_n <= t) lo = mid; else hi = mid;
  }
  ExpertTile x;
  const int mt = cum[lo + 1] - cum[lo];
  const int local = t - cum[lo] * tiles_n;
  int first;
  const int n = expert_rows(offsets, lo, slots, &first);
  const int tm = local % mt;
  x.e = lo;
  x.tn = local / mt;
  x.row0 = first + tm * bm;
  x.rows = min(bm, n - tm * bm);
  return x;
}

// Scales of groups g0..g0+3 of one row (0 past G).
__device__ __forceinline__ float4 scales4(const float* row, int g0, int G, bool vec) {
  if (vec) return __ldg(reinterpret_cast<const float4*>(row + g0));
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (g0 < G) v.x = __ldg(row + g0);
  if (g0 + 1 < G) v.y = __ldg(row + g0 + 1);
  if (g0 + 2 < G) v.z = __ldg(row + g0 + 2);
  if (g0 + 3 < G) v.w = __ldg(row + g0 + 3);
  return v;
}

__device__ __forceinline__ float4 mul4(float4 a, float4 b) {
  return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}
__device__ __forceinline__ float at4(const float4& v, int j) {
  return j < 2 ? (j == 0 ? v.x : v.y) : (j == 2 ? v.z : v.w);
}

__device__ __forceinline__ float silu_mul(float g, float u) {
  return __fdividef(g, 1.0f + __expf(-g)) * u;
}

template <int BN, int KIND, int DT>
__global__ void __launch_bounds__(FBCfg<BN>::THREADS, 1)
    f8_block_gemm_kernel(const __grid_constant__ CUtensorMap tmA,
                         const __grid_constant__ CUtensorMap tmB, const FBArgs args) {
  using C = FBCfg<BN>;
  using D = DTraits<DT>;
  constexpr bool EXPERTS = KIND != FB_DENSE;
  static_assert(KIND != FB_UP || BN == 256, "gate and up halves of 128");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  int* s_cum = reinterpret_cast<int*>(smem + C::OFF_CUM);
  uint32_t* s_amax = reinterpret_cast<uint32_t*>(smem + C::OFF_AMAX);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* full = bars;                 // stage loaded (TMA bytes)
  uint64_t* empty = full + C::NS;        // stage read by its MMAs (commit)
  uint64_t* tfull = empty + C::NS;       // slot holds a finished partial (commit)
  uint64_t* tempty = tfull + C::SLOTS;   // slot read out (one arrival per epilogue warp)
  uint64_t* mma_done = tempty + C::SLOTS;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  int* s_abort = reinterpret_cast<int*>(smem + C::OFF_MISC + 4);
  int* s_never = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint64_t lim = args.wait_ns;
  const int G = args.G;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), 1);
    }
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(smem_u32(&tfull[i]), 1);
      mbar_init(smem_u32(&tempty[i]), C::EPI_WARPS);
    }
    mbar_init(smem_u32(mma_done), 1);
    *s_abort = 0;
    *s_never = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), 512);
    tmem_relinquish();
  }
  if constexpr (EXPERTS) {
    grid_dep_wait();   // the offsets
    if (warp == 2) expert_tiles_scan(args.offsets, args.E, args.slots, C::BM, s_cum, lane);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch();
  const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(s_tmem);
  volatile int* abort_flag = s_abort;
  volatile int* never = s_never;
  const int T = EXPERTS ? s_cum[args.E] * args.tiles_n : args.tiles_m * args.tiles_n;

  // token tiles fastest: a weight tile streams from HBM once and serves every token tile
  auto tile_of = [&](int t) {
    if constexpr (EXPERTS) {
      return expert_tile(args.offsets, s_cum, args.E, args.slots, args.tiles_n, C::BM, t);
    } else {
      ExpertTile x;
      x.e = 0;
      x.tn = t / args.tiles_m;
      x.row0 = (t % args.tiles_m) * C::BM;
      x.rows = min(C::BM, args.M - x.row0);
      return x;
    }
  };

  if (warp < 4) {
    regs_dec<C::REGS_CTRL>();
    if (warp == 0) {
      // ---------------------------------------------------------- TMA producer
      if constexpr (!EXPERTS) grid_dep_wait();
      int it = 0, last = -1;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < T; t += args.P) {
        const ExpertTile x = tile_of(t);
        int r[4] = {0, 0, 0, 0};   // FB_UP: the tokens of this lane's four rows
        if constexpr (KIND == FB_UP) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int s = x.row0 + min(4 * lane + i, x.rows - 1);   // past the end: the last row
            const int f = __ldg(args.order + s);
            r[i] = f >= 0 && f < args.slots ? f / args.top_k : 0;
          }
        }
        for (int g = 0; g < G; ++g, ++it) {
          const int st = it % C::NS;
          ok = mbar_wait(smem_u32(&empty[st]), ((uint32_t)(it / C::NS) & 1u) ^ 1u, lim, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t fb = smem_u32(&full[st]);
          const uint32_t a_dst = smem_u32(smem + st * C::STAGE);
          const uint32_t b_dst = a_dst + C::A_BYTES;
          if (lane == 0) mbar_arrive_expect_tx(fb, C::STAGE);
          __syncwarp();
          if constexpr (KIND == FB_UP) {
            tma_gather4(a_dst + lane * 512, &tmA, fb, g * 128, r[0], r[1], r[2], r[3]);
          }
          if (lane == 0) {
            if constexpr (KIND != FB_UP) tma_load_2d(a_dst, &tmA, fb, g * 128, x.row0);
            if constexpr (KIND == FB_UP) {
              tma_load_3d(b_dst, &tmB, fb, g * 128, x.tn * 128, 2 * x.e);
              tma_load_3d(b_dst + 128 * 128, &tmB, fb, g * 128, x.tn * 128, 2 * x.e + 1);
            } else {
#pragma unroll
              for (int h = 0; h < BN / 128; ++h)
                tma_load_3d(b_dst + h * 128 * 128, &tmB, fb, g * 128, x.tn * BN + h * 128, x.e);
            }
          }
          __syncwarp();
          last = it;
        }
      }
      // never leave the CTA with bulk copies in flight
      for (int s = (last - C::NS + 1 > 0 ? last - C::NS + 1 : 0); s <= last; ++s)
        mbar_wait(smem_u32(&full[s % C::NS]), (uint32_t)(s / C::NS) & 1u, lim, never);
      __syncwarp();
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc = idesc_e4m3(C::BM, BN);
      int it = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < T; t += args.P) {
        for (int g = 0; g < G; ++g, ++it) {
          const int st = it % C::NS, sl = it % C::SLOTS;
          ok = mbar_wait2(smem_u32(&full[st]), (uint32_t)(it / C::NS) & 1u, smem_u32(&tempty[sl]),
                          ((uint32_t)(it / C::SLOTS) & 1u) ^ 1u, lim, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          if (lane == 0) {
            const uint32_t a_at = smem_u32(smem + st * C::STAGE);
            const uint64_t a0 = smem_desc_k_sw128(a_at);
            const uint64_t b0 = smem_desc_k_sw128(a_at + C::A_BYTES);
            const uint32_t d = tbase + sl * BN;
#pragma unroll
            for (int j = 0; j < 4; ++j)   // 32 codes of K per MMA (+2 in 16-byte units)
              umma_f8_ss(d, a0 + (uint64_t)(2 * j), b0 + (uint64_t)(2 * j), idesc, j > 0 ? 1u : 0u);
            umma_commit(smem_u32(&empty[st]));
            umma_commit(smem_u32(&tfull[sl]));
          }
          __syncwarp();
        }
      }
      if (lane == 0) umma_commit(smem_u32(mma_done));
      __syncwarp();
      mbar_wait(smem_u32(mma_done), 0u, lim, never);
      __syncwarp();
    }
  } else {
    regs_inc<C::REGS_EPI>();
    // ------------------------------------------------------------ epilogue
    if constexpr (!EXPERTS) grid_dep_wait();
    const int lq = warp & 3;                  // tensor-memory lane quarter of this warp
    const int half = (warp - 4) >> 2;
    const int row = 32 * lq + lane;           // token of the tile
    const uint32_t t_lane = (uint32_t)(32 * lq) << 16;
    const bool s_vec = args.s_vec != 0;
    constexpr int NCH = C::CPT / 32;
    // tensor-memory column of this thread's 32-column chunk cc: for FB_UP its 64 gate
    // columns, then the 64 up columns of the same outputs
    auto chunk_col = [&](int cc) {
      if constexpr (KIND == FB_UP) return (cc < 2 ? 64 * half + 32 * cc : 128 + 64 * half + 32 * (cc - 2));
      else return half * C::CPT + 32 * cc;
    };
    float2 acc[C::CPT / 2];
    bool ok = true;
    int it = 0;
    uint32_t par = 0;
    for (int t = blockIdx.x; ok && t < T; t += args.P, par ^= 1u) {
      const ExpertTile x = tile_of(t);
      const bool live = row < x.rows;
      const int s = x.row0 + (live ? row : 0);
      int f = 0;   // this row's flat (token, choice) index
      if constexpr (EXPERTS) {
        f = __ldg(args.order + s);
        if (f < 0 || f >= args.slots) f = -1;
      }
      const int a_row = KIND == FB_UP ? (f < 0 ? 0 : f / args.top_k) : s;
      const float* sa = args.sa + (size_t)a_row * G;
      // the weight blocks of this thread's columns (clamped: columns past N are not written)
      const int nb0 = KIND == FB_UP ? x.tn : min((x.tn * BN + half * C::CPT) / 128, args.NB - 1);
      const float* sw0 = args.sw + ((size_t)(KIND == FB_UP ? 2 * x.e : x.e) * args.NB + nb0) * G;
      const float* sw1 = sw0 + (size_t)args.NB * G;   // FB_UP: the up matrix
#pragma unroll
      for (int e = 0; e < C::CPT / 2; ++e) acc[e] = make_float2(0.0f, 0.0f);
      float4 sa_n = scales4(sa, 0, G, s_vec), w0_n = scales4(sw0, 0, G, s_vec), w1_n = w0_n;
      if constexpr (KIND == FB_UP) w1_n = scales4(sw1, 0, G, s_vec);
      for (int gb = 0; ok && gb < G; gb += 4) {
        const float4 c0 = mul4(sa_n, w0_n);
        const float4 c1 = KIND == FB_UP ? mul4(sa_n, w1_n) : c0;
        if (gb + 4 < G) {   // the next four groups' scales are in flight meanwhile
          sa_n = scales4(sa, gb + 4, G, s_vec);
          w0_n = scales4(sw0, gb + 4, G, s_vec);
          if constexpr (KIND == FB_UP) w1_n = scales4(sw1, gb + 4, G, s_vec);
        }
        const int je = min(4, G - gb);
        for (int j = 0; j < je; ++j, ++it) {
          const int sl = it % C::SLOTS;
          ok = mbar_wait(smem_u32(&tfull[sl]), (uint32_t)(it / C::SLOTS) & 1u, lim, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint32_t td = tbase + t_lane + sl * BN;
          const float k0 = at4(c0, j), k1 = at4(c1, j);
          uint32_t p[2][32];
          tmem_ld32_nowait(td + chunk_col(0), p[0]);
          tmem_ld_wait32(p[0]);
#pragma unroll
          for (int cc = 0; cc < NCH; ++cc) {
            uint32_t* pc = p[cc & 1];
            if (cc + 1 < NCH) tmem_ld32_nowait(td + chunk_col(cc + 1), p[(cc + 1) & 1]);
            const float kk = KIND == FB_UP && cc >= 2 ? k1 : k0;
            const float2 k2 = make_float2(kk, kk);
#pragma unroll
            for (int q = 0; q < 16; ++q)
              acc[cc * 16 + q] = __ffma2_rn(
                  make_float2(__uint_as_float(pc[2 * q]), __uint_as_float(pc[2 * q + 1])), k2,
                  acc[cc * 16 + q]);
            if (cc + 1 < NCH) tmem_ld_wait32(p[(cc + 1) & 1]);
            if (cc == NCH - 2) {   // every load of the slot has completed
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(&tempty[sl]));
            }
          }
        }
      }
      if constexpr (KIND == FB_UP) {
        // h of this thread's 64 columns, the group's maximum with the thread that holds the
        // row's other 64, then the codes
        uint32_t mx = 0;
        float h[64];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          h[2 * e] = silu_mul(acc[e].x, acc[32 + e].x);
          h[2 * e + 1] = silu_mul(acc[e].y, acc[32 + e].y);
        }
        const int n0 = x.tn * 128 + 64 * half;
#pragma unroll
        for (int e = 0; e < 64; ++e) mx = max(mx, abs_bits(h[e]));   // columns past N are 0
        uint32_t* am = s_amax + par * 256;
        am[half * 128 + row] = mx;
        ok = !bar_red_or(1, 256, !ok);   // one decision for all epilogue warps
        if (ok && live) {
          mx = max(mx, am[(half ^ 1) * 128 + row]);
          const F8Scale q = f8_scale(mx);
          uint8_t* dst = args.hq + (size_t)s * args.N + n0;
#pragma unroll
          for (int e = 0; e < 64; e += 16) {   // N % 16 == 0
            if (n0 + e < args.N) {
              float v0[8], v1[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                v0[i] = h[e + i];
                v1[i] = h[e + 8 + i];
              }
              const uint2 a = f8_codes8(v0, q), b = f8_codes8(v1, q);
              *reinterpret_cast<uint4*>(dst + e) = make_uint4(a.x, a.y, b.x, b.y);
            }
          }
          if (half == 0) args.hs[(size_t)s * args.NB + x.tn] = q.s;
        }
      } else {
        const int n0 = x.tn * BN + half * C::CPT;
        const int out_row = KIND == FB_DOWN ? f : s;
        if (ok && live && out_row >= 0) {
          typename D::T* dst = static_cast<typename D::T*>(args.y) + (size_t)out_row * args.N + n0;
          if (args.y_vec && n0 + C::CPT <= args.N) {
#pragma unroll
            for (int e = 0; e < C::CPT / 2; e += 4)
              *reinterpret_cast<uint4*>(dst + 2 * e) = make_uint4(
                  D::pack(acc[e].x, acc[e].y), D::pack(acc[e + 1].x, acc[e + 1].y),
                  D::pack(acc[e + 2].x, acc[e + 2].y), D::pack(acc[e + 3].x, acc[e + 3].y));
          } else {
#pragma unroll
            for (int e = 0; e < C::CPT; ++e) {
              const float v = (e & 1) ? acc[e / 2].y : acc[e / 2].x;
              if (n0 + e < args.N) dst[e] = D::one(v);
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

}  // namespace apex
