// gemm_f8_small.cuh -- the block-scaled FP8 GEMM for few tokens, dense and over experts: the
// kinds, operands and results of gemm_f8_block.cuh.
//
// FB_UP takes slot s's row of token order[s] / k itself, by TMA row gathers; FB_DOWN writes row
// order[s], in fp32.
//
// Bound: the weights' stream from HBM.  The 128 tensor-memory lanes hold weight rows and the
// tokens are the MMA's N (BT = 16 or 32), so a tile wastes little on absent tokens.  A
// pipeline stage is one K-group of 128 weight rows (16 KB) and its tokens; for FB_UP the gate
// and up rows of an output block alternate as stages.  Two CTAs share an SM, each with its ring
// of stages, so that one streams while the other starts or ends.
//
// K is split over the S CTAs of a thread-block cluster when there are too few tiles: every
// CTA sends its fp32 sums of BT / S tokens to each of the others (st.async, counted on an
// mbarrier), and adds the S parts of its own tokens in the order of the ranks.
//
// early: the launch follows the activations' quantizer (or FB_UP) of the same call, which
// lets its dependents start only after everything before it has finished.  Weights, offsets
// and order are then complete, and the first stages' weights are fetched while it still runs.
// Measured: 8192 x 8192, 1 and 16 tokens, with the quantizer: 16.8 and 18.0 us (67 MB: 10.3 us at
// the copy rate); 64 experts of 2048 x 1024, 16 tokens, the whole MLP: 68 us (297 MB: 45 us).
// Roles (192 threads): warp 0 TMA, warp 1 MMA, warps 2..5 epilogue (lanes 32 * (warp % 4)..).
#pragma once
#include <cuda.h>
#include <stdint.h>

#include "f8_block.cuh"
#include "gemm_f8_block.cuh"
#include "ptx.cuh"

namespace apex {

struct FSArgs {
  FBArgs b;
  const int32_t* order;   // [slots] (experts)
  int S;       // CTAs of a tile's cluster (1: no split; more: one tile per cluster)
  int early;
};

template <int BT, int KIND>
struct FSCfg {
  static constexpr int HALVES = KIND == FB_UP ? 2 : 1;
  static constexpr int CTAS_PER_SM = 2;
  static constexpr int W_BYTES = 128 * 128;
  static constexpr int X_BYTES = BT * 128;
  static constexpr int STAGE = W_BYTES + X_BYTES;
  static constexpr int RECV = HALVES * BT * 128 * 4;    // the cluster's sums of this CTA's tokens
  static constexpr int SC = 4 * 2 * 4 * BT * 4;         // [warp][2][4 groups][BT] token scales
  static constexpr int CUM = KIND == FB_DENSE ? 0 : (kMaxExperts + 4) * 4;
  static constexpr int FIXED = RECV + SC + CUM + 4 * BT * 4 + 512 + 1024;
  static constexpr int BUDGET = 113 * 1024;
  static constexpr int NS = (BUDGET - FIXED) / STAGE < 8 ? (BUDGET - FIXED) / STAGE : 8;
  static constexpr int SLOTS = 256 / BT < 8 ? 256 / BT : 8;   // partials of BT columns
  static constexpr int TMEM_COLS = SLOTS * BT;
  static constexpr int THREADS = 192;
  static constexpr int OFF_RECV = NS * STAGE;
  static constexpr int OFF_SC = OFF_RECV + RECV;
  static constexpr int OFF_CUM = OFF_SC + SC;
  static constexpr int OFF_MAX = OFF_CUM + CUM;                // [4][BT] words
  static constexpr int OFF_BAR = OFF_MAX + 4 * BT * 4;
  static constexpr int NBAR = 2 * NS + 2 * SLOTS + 2;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static_assert(NS >= 3, "a ring of stages");
  static_assert(SMEM * CTAS_PER_SM <= 226 * 1024, "shared memory budget");
  // Two CTAs of these kernels fit an SM's tensor memory, and no other kernel here that
  // allocates some fits beside one in shared memory (171 KB at least): no CTA waits for tensor
  // memory that a CTA of another cluster holds while it waits for its own.
  static_assert(TMEM_COLS * CTAS_PER_SM <= 512, "tensor memory budget");
};

__device__ __forceinline__ void st_async_v2(uint32_t raddr, float a, float b, uint32_t rbar) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
          raddr),
      "f"(a), "f"(b), "r"(rbar)
      : "memory");
}

template <int BT>
__device__ __forceinline__ void tmem_ld_tokens(uint32_t taddr, uint32_t (&v)[BT]) {
  if constexpr (BT == 16) {
    tmem_ld16_nowait(taddr, v);
    tmem_ld_wait16(v);
  } else {
    static_assert(BT == 32, "16 or 32 tokens");
    tmem_ld32_nowait(taddr, v);
    tmem_ld_wait32(v);
  }
}

template <int BT, int KIND, int DT>
__global__ void __launch_bounds__(192, FSCfg<BT, KIND>::CTAS_PER_SM)
    f8_small_gemm_kernel(const __grid_constant__ CUtensorMap tmW,
                         const __grid_constant__ CUtensorMap tmX, const FSArgs fs) {
  using C = FSCfg<BT, KIND>;
  using D = DTraits<DT>;
  constexpr bool EXPERTS = KIND != FB_DENSE;
  constexpr int HALVES = C::HALVES;
  const FBArgs& args = fs.b;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* s_recv = reinterpret_cast<float*>(smem + C::OFF_RECV);
  int* s_cum = reinterpret_cast<int*>(smem + C::OFF_CUM);
  uint32_t* s_max = reinterpret_cast<uint32_t*>(smem + C::OFF_MAX);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* full = bars;
  uint64_t* empty = full + C::NS;
  uint64_t* tfull = empty + C::NS;
  uint64_t* tempty = tfull + C::SLOTS;
  uint64_t* mma_done = tempty + C::SLOTS;
  uint64_t* rbar = mma_done + 1;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  int* s_abort = reinterpret_cast<int*>(smem + C::OFF_MISC + 4);
  int* s_never = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint64_t lim = args.wait_ns;
  const int S = fs.S;
  const int rank = S > 1 ? (int)(blockIdx.x % (unsigned)S) : 0;
  const int g0 = (int)((long long)args.G * rank / S), g1 = (int)((long long)args.G * (rank + 1) / S);
  const int units = (g1 - g0) * HALVES;   // stages of one tile

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), 1);
    }
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(smem_u32(&tfull[i]), 1);
      mbar_init(smem_u32(&tempty[i]), 4);
    }
    mbar_init(smem_u32(mma_done), 1);
    mbar_init(smem_u32(rbar), 1);
    *s_abort = 0;
    *s_never = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), C::TMEM_COLS);
    tmem_relinquish();
  }
  if constexpr (EXPERTS) {
    if (!fs.early) grid_dep_wait();   // the offsets
    if (warp == 2) expert_tiles_scan(args.offsets, args.E, args.slots, BT, s_cum, lane);
  }
  tc_fence_before();
  __syncthreads();
  if (S > 1) {   // every CTA's barriers exist before anyone sends to them
    cluster_arrive();
    cluster_wait();
  }
  tc_fence_after();
  const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(s_tmem);
  volatile int* abort_flag = s_abort;
  volatile int* never = s_never;
  const int T = EXPERTS ? s_cum[args.E] * args.tiles_n : args.tiles_m * args.tiles_n;
  const int t_first = (int)(blockIdx.x / (unsigned)S), t_step = S > 1 ? T : args.P;

  auto tile_of = [&](int t) {
    if constexpr (EXPERTS) {
      return expert_tile(args.offsets, s_cum, args.E, args.slots, args.tiles_n, BT, t);
    } else {
      ExpertTile x;
      x.e = 0;
      x.tn = t / args.tiles_m;   // token tiles fastest: they share the weight tile in L2
      x.row0 = (t % args.tiles_m) * BT;
      x.rows = min(BT, args.M - x.row0);
      return x;
    }
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    auto load_w = [&](const ExpertTile& x, int u, int st) {
      const int g = g0 + u / HALVES;
      tma_load_3d(smem_u32(smem + st * C::STAGE), &tmW, smem_u32(&full[st]), g * 128, x.tn * 128,
                  x.e * HALVES + u % HALVES);
    };
    int pre = 0;
    if (fs.early && t_first < T) {
      const ExpertTile x = tile_of(t_first);
      pre = min(C::NS, units);
      if (elect_one()) {
        for (int u = 0; u < pre; ++u) {
          mbar_arrive_expect_tx(smem_u32(&full[u]), C::STAGE);
          load_w(x, u, u);
        }
      }
      __syncwarp();
    }
    grid_dep_wait();
    int it = 0, last = -1;
    bool ok = true;
    for (int t = t_first; ok && t < T; t += t_step) {
      const ExpertTile x = tile_of(t);
      int r[4] = {0, 0, 0, 0};
      if constexpr (KIND == FB_UP) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int f = __ldg(fs.order + x.row0 + min(4 * lane + i, x.rows - 1));
          r[i] = f >= 0 && f < args.slots ? f / args.top_k : 0;
        }
      }
      for (int u = 0; u < units; ++u, ++it) {
        const int st = it % C::NS;
        ok = mbar_wait_warp(smem_u32(&empty[st]), ((uint32_t)(it / C::NS) & 1u) ^ 1u, lim, abort_flag);
        if (!ok) break;
        const uint32_t fb = smem_u32(&full[st]);
        const uint32_t x_dst = smem_u32(smem + st * C::STAGE + C::W_BYTES);
        const int g = g0 + u / HALVES;
        if (elect_one() && it >= pre) {
          mbar_arrive_expect_tx(fb, C::STAGE);
          load_w(x, u, st);
        }
        __syncwarp();
        if constexpr (KIND == FB_UP) {
          if (lane < BT / 4)
            tma_gather4(x_dst + lane * 512, &tmX, fb, g * 128, r[0], r[1], r[2], r[3]);
        } else {
          if (elect_one()) tma_load_2d(x_dst, &tmX, fb, g * 128, x.row0);
        }
        __syncwarp();
        last = it;
      }
    }
    // never leave the CTA with bulk copies in flight: the issued stages' bytes arrive (a stage
    // whose weights alone were fetched, after a wait that gave up, cannot complete: its tokens
    // are fetched now)
    for (int it2 = last + 1; it2 < pre; ++it2) {
      if (elect_one() && KIND != FB_UP)
        tma_load_2d(smem_u32(smem + it2 * C::STAGE + C::W_BYTES), &tmX, smem_u32(&full[it2]), 0, 0);
      if (KIND == FB_UP && lane < BT / 4)
        tma_gather4(smem_u32(smem + it2 * C::STAGE + C::W_BYTES) + lane * 512, &tmX,
                    smem_u32(&full[it2]), 0, 0, 0, 0, 0);
      last = it2;
    }
    for (int s = (last - C::NS + 1 > 0 ? last - C::NS + 1 : 0); s <= last; ++s)
      mbar_wait(smem_u32(&full[s % C::NS]), (uint32_t)(s / C::NS) & 1u, lim, never);
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    grid_dep_wait();   // (the wait limit counts from here, not from the grids before)
    constexpr uint32_t idesc = idesc_e4m3(128, BT);
    int it = 0;
    bool ok = true;
    for (int t = t_first; ok && t < T; t += t_step) {
      for (int u = 0; u < units; ++u, ++it) {
        const int st = it % C::NS, sl = it % C::SLOTS;
        ok = mbar_wait2_warp(smem_u32(&full[st]), (uint32_t)(it / C::NS) & 1u, smem_u32(&tempty[sl]),
                             ((uint32_t)(it / C::SLOTS) & 1u) ^ 1u, lim, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t at = smem_u32(smem + st * C::STAGE);
          const uint64_t w0 = smem_desc_k_sw128(at);
          const uint64_t x0 = smem_desc_k_sw128(at + C::W_BYTES);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            umma_f8_ss(tbase + sl * BT, w0 + (uint64_t)(2 * j), x0 + (uint64_t)(2 * j), idesc,
                       j > 0 ? 1u : 0u);
          umma_commit(smem_u32(&empty[st]));
          umma_commit(smem_u32(&tfull[sl]));
        }
        __syncwarp();
      }
    }
    if (elect_one()) umma_commit(smem_u32(mma_done));
    __syncwarp();
    mbar_wait(smem_u32(mma_done), 0u, lim, never);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    grid_dep_wait();
    grid_dep_launch();   // dependents start after everything before this grid has finished
    const int lq = warp & 3;
    const int row = 32 * lq + lane;           // weight row of the tile
    const uint32_t t_lane = (uint32_t)(32 * lq) << 16;
    const bool s_vec = args.s_vec != 0;
    constexpr int TPL = (BT + 31) / 32;       // tokens whose scales a lane loads
    float* sc = reinterpret_cast<float*>(smem + C::OFF_SC) + lq * (2 * 4 * BT);
    float2 acc[HALVES][BT / 2];
    bool ok = true;
    int it = 0;
    uint32_t buf = 0;
    for (int t = t_first; ok && t < T; t += t_step) {
      const ExpertTile x = tile_of(t);
      // this lane's tokens' scale rows (null: no such token)
      const float* sa[TPL];
#pragma unroll
      for (int i = 0; i < TPL; ++i) {
        const int tok = lane + 32 * i;
        sa[i] = nullptr;
        if (tok < BT && tok < x.rows) {
          int r = x.row0 + tok;
          if constexpr (KIND == FB_UP) {
            const int f = __ldg(fs.order + r);
            r = f >= 0 && f < args.slots ? f / args.top_k : 0;
          }
          sa[i] = args.sa + (size_t)r * args.G;
        }
      }
      const float* sw = args.sw + ((size_t)x.e * HALVES * args.NB + x.tn) * args.G;
      auto load_scales = [&](int g, float4 (&a4)[TPL], float4 (&w4)[HALVES]) {
        const bool v = s_vec && (g & 3) == 0;
#pragma unroll
        for (int i = 0; i < TPL; ++i)
          a4[i] = sa[i] ? scales4(sa[i], g, args.G, v) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int h = 0; h < HALVES; ++h) w4[h] = scales4(sw + (size_t)h * args.NB * args.G, g, args.G, v);
      };
#pragma unroll
      for (int h = 0; h < HALVES; ++h)
#pragma unroll
        for (int e = 0; e < BT / 2; ++e) acc[h][e] = make_float2(0.0f, 0.0f);
      float4 an[TPL], wn[HALVES];
      load_scales(g0, an, wn);
      for (int gb = g0; ok && gb < g1; gb += 4, buf ^= 1u) {
        // this block's token scales to shared memory (the warp's own buffer), the next one's
        // into registers
        float* s4 = sc + buf * (4 * BT);
        float4 w4[HALVES];
#pragma unroll
        for (int i = 0; i < TPL; ++i) {
          const int tok = lane + 32 * i;
          if (tok < BT) {
            s4[tok] = an[i].x;
            s4[BT + tok] = an[i].y;
            s4[2 * BT + tok] = an[i].z;
            s4[3 * BT + tok] = an[i].w;
          }
        }
#pragma unroll
        for (int h = 0; h < HALVES; ++h) w4[h] = wn[h];
        __syncwarp();
        if (gb + 4 < g1) load_scales(gb + 4, an, wn);
        const int je = min(4, g1 - gb);
        for (int j = 0; j < je && ok; ++j) {
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
            const int sl = it % C::SLOTS;
            ok = ok && mbar_wait(smem_u32(&tfull[sl]), (uint32_t)(it / C::SLOTS) & 1u, lim, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
              tc_fence_after();
              uint32_t p[BT];
              tmem_ld_tokens<BT>(tbase + t_lane + sl * BT, p);
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(&tempty[sl]));
              const float w = at4(w4[h], j);
              const float2 w2 = make_float2(w, w);
              const float4* c4 = reinterpret_cast<const float4*>(s4 + j * BT);
#pragma unroll
              for (int q = 0; q < BT / 4; ++q) {
                const float4 c = c4[q];
                acc[h][2 * q] = __ffma2_rn(
                    make_float2(__uint_as_float(p[4 * q]), __uint_as_float(p[4 * q + 1])),
                    __fmul2_rn(make_float2(c.x, c.y), w2), acc[h][2 * q]);
                acc[h][2 * q + 1] = __ffma2_rn(
                    make_float2(__uint_as_float(p[4 * q + 2]), __uint_as_float(p[4 * q + 3])),
                    __fmul2_rn(make_float2(c.z, c.w), w2), acc[h][2 * q + 1]);
              }
            }
            ++it;
          }
        }
      }
      // the cluster's exchange: this CTA finishes tokens rank * W .. + W - 1
      const int W = BT / S;            // a power of two, 2 at least
      const int lw = __ffs(W) - 1;
      const int tb = rank * W;
      if (S > 1) {
        if (row == 0) {
          const int mine = max(0, min(W, x.rows - tb));
          mbar_arrive_expect_tx(smem_u32(rbar), (uint32_t)(S * HALVES * ((mine + 1) / 2) * 128 * 8));
        }
        if (ok) {
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
#pragma unroll
            for (int e = 0; e < BT / 2; ++e) {
              if (2 * e < x.rows) {   // pairs with a token
                const int to = (2 * e) >> lw, at = e - to * (W / 2);
                const uint32_t off =
                    (uint32_t)((((rank * HALVES + h) * (W / 2) + at) * 128 + row) * 8);
                st_async_v2(cluster_map(smem_u32(s_recv) + off, (uint32_t)to), acc[h][e].x,
                            acc[h][e].y, cluster_map(smem_u32(rbar), (uint32_t)to));
              }
            }
          }
        }
        ok = mbar_wait_cluster(smem_u32(rbar), 0u, lim, abort_flag) && ok;
        ok = __all_sync(0xffffffffu, ok);
        const float2* rv = reinterpret_cast<const float2*>(s_recv);
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
#pragma unroll
          for (int e = 0; e < BT / 4; ++e) {   // W <= BT / 2 tokens
            if (ok && 2 * e < W && tb + 2 * e < x.rows) {
              float2 v = make_float2(0.0f, 0.0f);
              for (int src = 0; src < S; ++src) {
                const float2 p = rv[((src * HALVES + h) * (W / 2) + e) * 128 + row];
                v.x += p.x;
                v.y += p.y;
              }
              acc[h][e] = v;
            }
          }
        }
      }
      const int n = x.tn * 128 + row;
      const int count = min(W, x.rows - tb);   // this CTA's tokens
      if constexpr (KIND == FB_UP) {
#pragma unroll
        for (int e = 0; e < BT / 2; ++e) {
          acc[0][e].x = silu_mul(acc[0][e].x, acc[1][e].x);
          acc[0][e].y = silu_mul(acc[0][e].y, acc[1][e].y);
        }
#pragma unroll
        for (int e = 0; e < BT; ++e) {
          if (e < count) {
            const uint32_t m = __reduce_max_sync(
                0xffffffffu, abs_bits((e & 1) ? acc[0][e / 2].y : acc[0][e / 2].x));
            if (lane == 0) s_max[lq * BT + e] = m;
          }
        }
        ok = !bar_red_or(1, 128, !ok);
        if (ok) {
#pragma unroll
          for (int e = 0; e < BT; ++e) {
            if (e < count) {
              const F8Scale q = f8_scale(max(max(s_max[e], s_max[BT + e]),
                                             max(s_max[2 * BT + e], s_max[3 * BT + e])));
              const float h = (e & 1) ? acc[0][e / 2].y : acc[0][e / 2].x;
              const float v = f8_quotient(h, q);
              const size_t slot = (size_t)(x.row0 + tb + e);
              if (n < args.N) args.hq[slot * args.N + n] = (uint8_t)f8_pair(v, 0.0f);
              if (row == 0) args.hs[slot * args.NB + x.tn] = q.s;
            }
          }
        }
        bar_red_or(1, 128, false);   // s_max is free for the next tile
      } else {
        if (ok) {
#pragma unroll
          for (int e = 0; e < BT; ++e) {
            if (e < count && n < args.N) {
              int r = x.row0 + tb + e;
              if constexpr (KIND == FB_DOWN) {
                r = __ldg(fs.order + r);
                if (r >= args.slots) r = -1;
              }
              const float v = (e & 1) ? acc[0][e / 2].y : acc[0][e / 2].x;
              if (r >= 0) {
                if constexpr (KIND == FB_DOWN) static_cast<float*>(args.y)[(size_t)r * args.N + n] = v;
                else static_cast<typename D::T*>(args.y)[(size_t)r * args.N + n] = D::one(v);
              }
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
    tmem_dealloc(tbase, C::TMEM_COLS);
  }
  if (S > 1) {   // no CTA leaves while another may still send to it
    cluster_arrive_relaxed();
    cluster_wait();
  }
}

}  // namespace apex
