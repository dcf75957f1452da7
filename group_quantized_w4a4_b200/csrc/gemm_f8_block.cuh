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
//   FB_UP     for rows grouped by expert (slots): the products with the expert's gate and up
//             matrices, h = silu(gate) * up, quantized in groups of 128 as the next product's
//             operand.  A tile is 128 columns of h: its weight operand is 128 gate rows above
//             128 up rows.  The rows are slots: f8_permute_kernel has copied each token's
//             codes to the slots of its choices (fetching scattered rows here by TMA gathers of
//             four took 1.5 us a K-group, three times the products).
//   FB_DOWN   h . W^T of each slot's expert, by slot, in fp32: a token's weights multiply its
//             choices' rows before the one rounding, and a row alone may leave fp16's range or
//             cancel against another (16-bit rows: inf for 0.1 * 70000, and 1.4 times the error).
//
// Tile: 128 tokens (MMA M) x BN weight rows (MMA N), one K-group per pipeline stage, both
// operands by TMA with 128-byte swizzle; the group's partial goes to one of 512 / BN
// tensor-memory slots, which the epilogue drains while the next groups' MMAs fill the others.
// Roles (384 threads, one persistent CTA per SM): warp 0 TMA, warp 1 MMA, warps 2, 3 scales
// (global memory to a ring in shared memory, four K-groups of the 128 tokens and of the tile's
// two weight blocks at a time, and which tile they are of), warps 4..11 epilogue (warp w: lanes
// 32*(w%4).., half (w-4)/4 of the columns).  With its 128 accumulators and 64 partials in
// flight an epilogue thread has no registers for scales on their way from memory: loaded
// there, every fourth group waited 1,100 cycles for them.
//
// Bound: the partials' way out of tensor memory and the fma on each; the tensor pipe is 59 %
// busy.  Measured: 4096 x 8192 x 8192 248 us (2.2 PFLOP/s; a library product with one scale a
// tensor 190), one call with the quantizer and a cold L2 286, 328 in an unbroken loop under the
// power cap.  CTA pairs with 256 x 256 tiles took the same time and left more of a ragged tile
// empty.  Experts, 32768 rows through 64 of 2048 x 1024: UP 206 us; DOWN 136 (116 with 16-bit rows:
// 134 MB less to write, and no buffers to wait for).
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
  const float* sa;          // [rows][G]
  const float* sw;          // [E (x 2 for FB_UP)][NB][G]
  void* y;                  // [rows][N], 16-bit; FB_DOWN: fp32
  uint8_t* hq;              // FB_UP: codes [slots][N] and scales [slots][NB]
  float* hs;
  int s_vec;                // scale rows readable as 16-byte blocks of 4 groups
  int y_map;                // rows of y are 16-byte multiples: tmY describes them
  unsigned long long wait_ns;
};

constexpr int kMaxExperts = 512;

template <int BN>
struct FBCfg {
  static constexpr int BM = 128;
  static constexpr int A_BYTES = BM * 128;
  static constexpr int B_BYTES = BN * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int NS = 168 * 1024 / STAGE;
  static constexpr int SLOTS = 512 / BN;
  static constexpr int EPI_WARPS = 8;
  static constexpr int THREADS = 128 + 32 * EPI_WARPS;
  // 384 x 168 registers at launch; the first warpgroup keeps 56, the epilogue takes 224
  static constexpr int REGS_CTRL = 56, REGS_EPI = 224;
  static_assert(128 * REGS_CTRL + 256 * REGS_EPI <= THREADS * 168, "register pool");
  static constexpr int CPT = BN / 2;   // partials per epilogue thread
  static constexpr int SR = 4;                     // ring of scale blocks (4 K-groups each)
  static constexpr int SC_BLOCK = (128 + 2) * 16;  // [128 tokens, 2 weight blocks][4 groups]
  static constexpr int ST_WARP = CPT * 64;         // a warp's 32 rows of outputs on their way
  static constexpr int OFF_ST = NS * STAGE;
  static constexpr int OFF_SC = OFF_ST + EPI_WARPS * ST_WARP;
  static constexpr int OFF_CUM = OFF_SC + SR * SC_BLOCK;           // [kMaxExperts + 1] ints
  static constexpr int OFF_AMAX = OFF_CUM + (kMaxExperts + 4) * 4;  // [2][2][128] words
  static constexpr int TR = 8;                     // ring of tile descriptions, 16 bytes each
  static constexpr int OFF_TILE = OFF_AMAX + 2 * 2 * 128 * 4;
  static constexpr int OFF_BAR = OFF_TILE + TR * 16;
  static_assert(TR > SR, "a tile has at least one scale block");
  static constexpr int NBAR = 2 * NS + 2 * SLOTS + 1 + 2 * SR;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static_assert(OFF_BAR % 8 == 0 && SMEM <= 227 * 1024, "shared memory budget");
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

__device__ __forceinline__ float at4(const float4& v, int j) {
  return j < 2 ? (j == 0 ? v.x : v.y) : (j == 2 ? v.z : v.w);
}

// g * sigmoid(g) * u.  With t = exp(-|g|) <= 1, sigmoid is 1 / (1 + t) or t / (1 + t): nothing
// overflows, and the divisor in [1, 2] has a reciprocal within an ulp.  (1 / (1 + exp(-g)) by the
// same reciprocal is 0 below g = -87.3, and the fast exponential's error grows with |g|.)
__device__ __forceinline__ float silu_mul(float g, float u) {
  const float t = expf(-fabsf(g));
  return g * ((g < 0.0f ? t : 1.0f) * rcp_approx(1.0f + t)) * u;
}

// Every token's codes and scales to the slots of its choices: slot s gets row order[s] / k, and
// slot_of[order[s]] = s.
// Bound: the copy itself, a byte read (from L2, k times) and written per element.  A warp per
// slot (32768 slots of 2048: 19 us).
__global__ void __launch_bounds__(256) f8_permute_kernel(const uint8_t* __restrict__ codes,
                                                         const float* __restrict__ scales,
                                                         const int32_t* __restrict__ order,
                                                         int slots, int top_k, int K, int G,
                                                         uint8_t* __restrict__ to_codes,
                                                         float* __restrict__ to_scales,
                                                         int32_t* __restrict__ slot_of) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int chunks = K / 16;
  for (int s = blockIdx.x * 8 + (threadIdx.x >> 5); s < slots; s += gridDim.x * 8) {
    const int f = __ldg(order + s);
    uint4* dst = reinterpret_cast<uint4*>(to_codes + (size_t)s * K);
    if (f < 0 || f >= slots) {
      // no choice: zeros, for a tile that ends among such slots (NaNs that memory happened to
      // hold would take the rounding's rare path there, 20 us of a tile's time)
      for (int c = lane; c < chunks; c += 32) dst[c] = make_uint4(0u, 0u, 0u, 0u);
      continue;
    }
    const int t = f / top_k;
    if (lane == 0) slot_of[f] = s;
    const uint4* src = reinterpret_cast<const uint4*>(codes + (size_t)t * K);
    for (int c0 = 0; c0 < chunks; c0 += 128) {   // four loads in flight
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c0 + 32 * i + lane < chunks) v[i] = __ldg(src + c0 + 32 * i + lane);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c0 + 32 * i + lane < chunks) dst[c0 + 32 * i + lane] = v[i];
    }
    for (int g = lane; g < G; g += 32) to_scales[(size_t)s * G + g] = __ldg(scales + (size_t)t * G + g);
  }
}

template <int BN, int KIND, int DT>
__global__ void __launch_bounds__(FBCfg<BN>::THREADS, 1)
    f8_block_gemm_kernel(const __grid_constant__ CUtensorMap tmA,
                         const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap tmY, const FBArgs args) {
  using C = FBCfg<BN>;
  using D = DTraits<DT>;
  constexpr bool EXPERTS = KIND != FB_DENSE;
  static_assert(KIND != FB_UP || BN == 256, "gate and up halves of 128");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  int* s_cum = reinterpret_cast<int*>(smem + C::OFF_CUM);
  uint32_t* s_amax = reinterpret_cast<uint32_t*>(smem + C::OFF_AMAX);
  int4* s_tile = reinterpret_cast<int4*>(smem + C::OFF_TILE);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* full = bars;                 // stage loaded (TMA bytes)
  uint64_t* empty = full + C::NS;        // stage read by its MMAs (commit)
  uint64_t* tfull = empty + C::NS;       // slot holds a finished partial (commit)
  uint64_t* tempty = tfull + C::SLOTS;   // slot read out (one arrival per epilogue warp)
  uint64_t* mma_done = tempty + C::SLOTS;
  uint64_t* sfull = mma_done + 1;        // scale block written (every scale thread)
  uint64_t* sempty = sfull + C::SR;      // scale block read (one arrival per epilogue warp)
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
    for (int i = 0; i < C::SR; ++i) {
      mbar_init(smem_u32(&sfull[i]), 64);
      mbar_init(smem_u32(&sempty[i]), C::EPI_WARPS);
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
        for (int g = 0; g < G; ++g, ++it) {
          const int st = it % C::NS;
          ok = mbar_wait_warp(smem_u32(&empty[st]), ((uint32_t)(it / C::NS) & 1u) ^ 1u, lim, abort_flag);
          if (!ok) break;
          const uint32_t fb = smem_u32(&full[st]);
          const uint32_t a_dst = smem_u32(smem + st * C::STAGE);
          const uint32_t b_dst = a_dst + C::A_BYTES;
          if (elect_one()) {
            mbar_arrive_expect_tx(fb, C::STAGE);
            tma_load_2d(a_dst, &tmA, fb, g * 128, x.row0);
#pragma unroll
            for (int h = 0; h < BN / 128; ++h) {
              // FB_UP: 128 gate rows, then the 128 up rows of the same outputs
              const int n = KIND == FB_UP ? x.tn * 128 : x.tn * BN + h * 128;
              const int z = KIND == FB_UP ? 2 * x.e + h : x.e;
              tma_load_3d(b_dst + h * 128 * 128, &tmB, fb, g * 128, n, z);
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
      grid_dep_wait();   // (the wait limit counts from here, not from the grids before)
      constexpr uint32_t idesc = idesc_e4m3(C::BM, BN);
      int it = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < T; t += args.P) {
        for (int g = 0; g < G; ++g, ++it) {
          const int st = it % C::NS, sl = it % C::SLOTS;
          ok = mbar_wait2_warp(smem_u32(&full[st]), (uint32_t)(it / C::NS) & 1u,
                               smem_u32(&tempty[sl]), ((uint32_t)(it / C::SLOTS) & 1u) ^ 1u, lim,
                               abort_flag);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
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
      if (elect_one()) umma_commit(smem_u32(mma_done));
      __syncwarp();
      mbar_wait(smem_u32(mma_done), 0u, lim, never);
      __syncwarp();
    } else {
      // ---------------------------------------------------------- scales
      if constexpr (!EXPERTS) grid_dep_wait();
      const int i0 = threadIdx.x - 64;          // rows i0 and i0 + 64 of the tile's 128
      const bool s_vec = args.s_vec != 0;
      int sb = 0, tno = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < T; t += args.P, ++tno) {
        const ExpertTile x = tile_of(t);
        const float* sa[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = i0 + 64 * i;
          sa[i] = nullptr;
          if (r < x.rows) sa[i] = args.sa + (size_t)(x.row0 + r) * G;
        }
        // the tile's weight blocks: of its two column halves, or FB_UP's gate and up (clamped:
        // columns past N are not written)
        const float* sw = nullptr;
        if (i0 < 2) {
          if constexpr (KIND == FB_UP) sw = args.sw + ((size_t)(2 * x.e + i0) * args.NB + x.tn) * G;
          else sw = args.sw + ((size_t)x.e * args.NB + min((x.tn * BN + i0 * C::CPT) / 128, args.NB - 1)) * G;
        }
        for (int gb = 0; gb < G; gb += 4, ++sb) {
          const int b = sb % C::SR;
          float4 v[2], w = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            v[i] = sa[i] ? scales4(sa[i], gb, G, s_vec) : make_float4(0.f, 0.f, 0.f, 0.f);
          if (sw) w = scales4(sw, gb, G, s_vec);
          ok = mbar_wait_warp(smem_u32(&sempty[b]), ((uint32_t)(sb / C::SR) & 1u) ^ 1u, lim, abort_flag);
          if (!ok) break;
          float4* blk = reinterpret_cast<float4*>(smem + C::OFF_SC + b * C::SC_BLOCK);
          blk[i0] = v[0];
          blk[i0 + 64] = v[1];
          if (i0 < 2) blk[128 + i0] = w;
          // (the scale blocks are at most SR ahead of the epilogue, so the tile's place is free)
          if (i0 == 0 && gb == 0) s_tile[tno % C::TR] = make_int4(x.e, x.row0, x.rows, x.tn);
          mbar_arrive(smem_u32(&sfull[b]));
        }
      }
    }
  } else {
    regs_inc<C::REGS_EPI>();
    // ------------------------------------------------------------ epilogue
    if constexpr (!EXPERTS) grid_dep_wait();
    const int lq = warp & 3;                  // tensor-memory lane quarter of this warp
    const int half = (warp - 4) >> 2;
    const int row = 32 * lq + lane;           // token of the tile
    const uint32_t t_lane = (uint32_t)(32 * lq) << 16;
    constexpr int NCH = C::CPT / 32;
    // tensor-memory column of this thread's 32-column chunk cc: for FB_UP its 64 gate
    // columns, then the 64 up columns of the same outputs
    auto chunk_col = [&](int cc) {
      if constexpr (KIND == FB_UP) return (cc < 2 ? 64 * half + 32 * cc : 128 + 64 * half + 32 * (cc - 2));
      else return half * C::CPT + 32 * cc;
    };
    float2 acc[C::CPT / 2];
    bool ok = true;
    int it = 0, sb = 0, tno = 0;
    for (int t = blockIdx.x; ok && t < T; t += args.P, ++tno) {
      // the tile's first scale block comes with its description
      ok = mbar_wait_warp(smem_u32(&sfull[sb % C::SR]), (uint32_t)(sb / C::SR) & 1u, lim, abort_flag);
      const int4 xd = ok ? s_tile[tno % C::TR] : make_int4(0, 0, 0, 0);
      const int x_row0 = xd.y, x_rows = xd.z, x_tn = xd.w;
      const bool live = row < x_rows;
      const int s = x_row0 + (live ? row : 0);
#pragma unroll
      for (int e = 0; e < C::CPT / 2; ++e) acc[e] = make_float2(0.0f, 0.0f);
      // The partials come in chunks of 32 columns, the next one's load in flight while one is
      // used.  (Asking for the next group's first chunk before this group's last fmas was
      // slower, 0.54 against 0.45 us a K-group, and so was handing the slot back by a
      // predicated arrive of the whole warp instead of one elected lane's, 0.56 us.)
      uint32_t p[2][32];
      float4 c0, c1;   // sa * sw of the four groups of the block (FB_UP: c1 of the up matrix)
      auto block_bar = [&]() { return smem_u32(&sfull[sb % C::SR]); };
      auto block_par = [&]() { return (uint32_t)(sb / C::SR) & 1u; };
      auto load_block = [&]() {
        const float4* blk = reinterpret_cast<const float4*>(smem + C::OFF_SC + (sb % C::SR) * C::SC_BLOCK);
        const float4 a = blk[row], w0 = blk[128 + (KIND == FB_UP ? 0 : half)];
        c0 = make_float4(a.x * w0.x, a.y * w0.y, a.z * w0.z, a.w * w0.w);
        if constexpr (KIND == FB_UP) {
          const float4 w1 = blk[129];
          c1 = make_float4(a.x * w1.x, a.y * w1.y, a.z * w1.z, a.w * w1.w);
        }
        __syncwarp();
        if (elect_one()) mbar_arrive(smem_u32(&sempty[sb % C::SR]));
        ++sb;
      };
      auto load_chunk = [&](int i, int cc) {   // group number i's chunk cc
        tmem_ld32_nowait(tbase + t_lane + (i % C::SLOTS) * BN + chunk_col(cc), p[cc & 1]);
      };
      auto wait_group = [&]() {
        const bool r = mbar_wait_warp(smem_u32(&tfull[it % C::SLOTS]), (uint32_t)(it / C::SLOTS) & 1u, lim, abort_flag);
        tc_fence_after();
        return r;
      };
      if (ok) load_block();
      for (int g = 0; ok && g < G; ++g) {
        const int sl = it % C::SLOTS;
        const int j = g & 3;
        const float k0 = at4(c0, j), k1 = KIND == FB_UP ? at4(c1, j) : k0;
        auto fma_chunk = [&](int cc) {
          const uint32_t* pc = p[cc & 1];
          const float kk = KIND == FB_UP && cc >= 2 ? k1 : k0;
          const float2 k2 = make_float2(kk, kk);
#pragma unroll
          for (int q = 0; q < 16; ++q)
            acc[cc * 16 + q] = __ffma2_rn(
                make_float2(__uint_as_float(pc[2 * q]), __uint_as_float(pc[2 * q + 1])), k2,
                acc[cc * 16 + q]);
        };
        ok = wait_group();
        if (!ok) break;
        load_chunk(it, 0);
        tmem_ld_wait32(p[0]);
#pragma unroll
        for (int cc = 0; cc < NCH; ++cc) {
          if (cc + 1 < NCH) load_chunk(it, cc + 1);
          fma_chunk(cc);
          if (cc + 1 < NCH) tmem_ld_wait32(p[(cc + 1) & 1]);
          if (cc == NCH - 2) {   // every load of the slot has completed
            tc_fence_before();
            __syncwarp();
            if (elect_one()) mbar_arrive(smem_u32(&tempty[sl]));
          }
        }
        ++it;
        if (j == 3 && g + 1 < G) {
          ok = mbar_wait_warp(block_bar(), block_par(), lim, abort_flag);
          if (ok) load_block();
        }
      }
      // The tile's outputs go through the warp's own shared memory (16-byte chunks permuted as
      // the 128-byte, FB_UP: 64-byte, swizzle of the output's map) and leave by bulk stores,
      // which drain while the next tile is computed: the CTAs finish their tiles together, and
      // plain stores of 64 KB from each then took 3,300 to 4,200 cycles, a quarter of a tile of
      // eight K-groups.  Rows of the last, partly filled tile of an expert, which other rows
      // follow, are stored one by one, and so are outputs no map can describe.
      uint8_t* stage = smem + C::OFF_ST + (warp - 4) * C::ST_WARP;
      if constexpr (KIND != FB_DOWN) {
        if (elect_one()) bulk_wait_read();   // the last tile's
        __syncwarp();
      }
      const bool whole = 32 * lq + 32 <= x_rows;
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
        const int n0 = x_tn * 128 + 64 * half;
#pragma unroll
        for (int e = 0; e < 64; ++e) mx = max(mx, abs_bits(h[e]));   // columns past N are 0
        uint32_t* am = s_amax + (tno & 1) * 256;
        am[half * 128 + row] = mx;
        ok = !bar_red_or(1, 256, !ok);   // one decision for all epilogue warps
        if (ok) {
          mx = max(mx, am[(half ^ 1) * 128 + row]);
          const F8Scale q = f8_scale(mx);
#pragma unroll
          for (int e = 0; e < 64; e += 16) {
            float v0[8], v1[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              v0[i] = h[e + i];
              v1[i] = h[e + 8 + i];
            }
            const uint2 a = f8_codes8<true>(v0, q), b = f8_codes8<true>(v1, q);
            *reinterpret_cast<uint4*>(stage + lane * 64 + (((e >> 4) ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(a.x, a.y, b.x, b.y);
          }
          if (half == 0 && live) args.hs[(size_t)s * args.NB + x_tn] = q.s;
          if (whole) {
            fence_proxy_async_smem();
            __syncwarp();
            if (elect_one() && n0 < args.N) {
              tma_store_2d(&tmY, smem_u32(stage), n0, x_row0 + 32 * lq);
              bulk_commit();
            }
          } else {
            __syncwarp();
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              const int r = i * 8 + (lane >> 2), c = lane & 3;
              if (32 * lq + r < x_rows && n0 + c * 16 < args.N)   // N % 16 == 0
                *reinterpret_cast<uint4*>(args.hq + (size_t)(x_row0 + 32 * lq + r) * args.N + n0 + c * 16) =
                    *reinterpret_cast<const uint4*>(stage + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
            }
            __syncwarp();
          }
        }
      } else if constexpr (KIND == FB_DOWN) {
        // fp32 rows, 32 columns at a time through two buffers in turn: every part, stored by bulk
        // or not, is one bulk group, so all but the last group read means that its buffer is free
        if (ok) {
          const int n0 = x_tn * BN + half * C::CPT;
          float* y = static_cast<float*>(args.y);
#pragma unroll
          for (int b = 0; b < C::CPT / 32; ++b) {
            uint8_t* buf = stage + (b & 1) * 4096;
            const int n = n0 + 32 * b;
            if (elect_one()) bulk_wait_read_but1();
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float2 lo = acc[b * 16 + 2 * c], hi = acc[b * 16 + 2 * c + 1];
              *reinterpret_cast<float4*>(buf + lane * 128 + ((c ^ (lane & 7)) << 4)) =
                  make_float4(lo.x, lo.y, hi.x, hi.y);
            }
            if (whole) {
              fence_proxy_async_smem();
              __syncwarp();
              if (elect_one()) {
                if (n < args.N) tma_store_2d(&tmY, smem_u32(buf), n, x_row0 + 32 * lq);
                bulk_commit();
              }
            } else {   // an expert's last rows: N % 16 == 0, 16-byte rows
              __syncwarp();
#pragma unroll 1
              for (int i = 0; i < 8; ++i) {   // 4 rows each
                const int r = i * 4 + (lane >> 3), c = lane & 7;
                if (32 * lq + r < x_rows && n + 4 * c < args.N)
                  *reinterpret_cast<float4*>(y + (size_t)(x_row0 + 32 * lq + r) * args.N + n + 4 * c) =
                      *reinterpret_cast<const float4*>(buf + r * 128 + ((c ^ (r & 7)) << 4));
              }
              if (elect_one()) bulk_commit();
              __syncwarp();
            }
          }
        }
      } else if (ok) {
#pragma unroll
        for (int pass = 0; pass < C::CPT / 64; ++pass)
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float2* a = acc + pass * 32 + c * 4;
            *reinterpret_cast<uint4*>(stage + pass * 4096 + lane * 128 + ((c ^ (lane & 7)) << 4)) =
                make_uint4(D::pack(a[0].x, a[0].y), D::pack(a[1].x, a[1].y),
                           D::pack(a[2].x, a[2].y), D::pack(a[3].x, a[3].y));
          }
        const int n0 = x_tn * BN + half * C::CPT;
        if (args.y_map) {
          fence_proxy_async_smem();
          __syncwarp();
          if (elect_one() && 32 * lq < x_rows) {
#pragma unroll
            for (int pass = 0; pass < C::CPT / 64; ++pass)
              if (n0 + pass * 64 < args.N)
                tma_store_2d(&tmY, smem_u32(stage + pass * 4096), n0 + pass * 64, x_row0 + 32 * lq);
            bulk_commit();
          }
        } else {
          // rows of any alignment: a row's 64 columns at a time, in words of two columns where
          // the row lies on words, else in words of two lanes' columns (330 x 5676 x 1520
          // 10.8 us, 8.7 with 5680 columns and the bulk stores; eight 2-byte stores a lane 16.7)
          __syncwarp();
          const int rows = min(32, x_rows - 32 * lq);
#pragma unroll
          for (int pass = 0; pass < C::CPT / 64; ++pass) {
            const int n = n0 + pass * 64 + 2 * lane;
#pragma unroll 4
            for (int r = 0; r < rows; ++r) {
              const uint32_t w = *reinterpret_cast<const uint32_t*>(
                  stage + pass * 4096 + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
              const uint32_t next = __shfl_down_sync(0xffffffffu, w, 1);
              uint16_t* dst = static_cast<uint16_t*>(args.y) + (size_t)(x_row0 + 32 * lq + r) * args.N + n;
              if ((reinterpret_cast<uintptr_t>(dst) & 2u) == 0) {   // the same for all lanes
                if (n + 1 < args.N) *reinterpret_cast<uint32_t*>(dst) = w;
                else if (n < args.N) dst[0] = (uint16_t)w;
              } else {
                if (lane == 0 && n < args.N) dst[0] = (uint16_t)w;
                if (lane < 31 && n + 2 < args.N)
                  *reinterpret_cast<uint32_t*>(dst + 1) = __funnelshift_r(w, next, 16);
                else if (n + 1 < args.N) dst[1] = (uint16_t)(w >> 16);
              }
            }
          }
          __syncwarp();
        }
      }
    }
    if (elect_one()) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

}  // namespace apex
