// fp8_block_host.cuh -- host side of the block-scaled FP8, expert and block-norm entry points:
// argument checks, tensor maps, launches.  Included by apex_w4a4.cu, whose helpers it uses.
#pragma once

namespace {

using apex::FBArgs;
using apex::FBCfg;

bool is_16bit(int32_t dt) { return dt == APEX_DTYPE_F16 || dt == APEX_DTYPE_BF16; }
bool is_float(int32_t dt) { return is_16bit(dt) || dt == APEX_DTYPE_F32; }
size_t pad256(size_t n) { return (n + 255) & ~(size_t)255; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kMaxBlockDim = 1 << 20;   // largest N, K, H of these entry points
constexpr int64_t kMaxSlots = 1 << 30;

apex_status_t launched(cudaError_t e) {
  if (e != cudaSuccess) {
    (void)cudaGetLastError();   // reported here, not by the caller's next call
    return APEX_ERR_CUDA;
  }
  return APEX_OK;
}

// 3-D map over E4M3 codes [Z][rows][K]; box = 128 codes x box_rows rows of one matrix, 128-byte
// swizzle; rows and columns outside a matrix read as zeros.
bool make_codes3_map(CUtensorMap* map, const void* base, int64_t Z, int64_t rows, int64_t K,
                     int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)rows, (cuuint64_t)Z};
  cuuint64_t strides[2] = {(cuuint64_t)K, (cuuint64_t)(K * rows)};
  cuuint32_t box[3] = {128u, (cuuint32_t)box_rows, 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// 2-D map over outputs [rows][cols] of `size`-byte elements (codes, 16-bit values or fp32), written
// in boxes of 32 rows x box_cols columns from shared memory with that many bytes' swizzle.
bool make_out_map(CUtensorMap* map, void* base, int64_t rows, int64_t cols, int size,
                  int box_cols) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(cols * size)};
  cuuint32_t box[2] = {(cuuint32_t)box_cols, 32u};
  cuuint32_t estr[2] = {1u, 1u};
  const CUtensorMapDataType type = size == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : size == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16
                                               : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  CUresult r = fn(map, type, 2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  box_cols * size == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

template <typename F>
cudaError_t set_smem(F kern, int bytes, int* attr_dev) {   // once per device and kernel
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (*attr_dev != dev) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) *attr_dev = dev;
  }
  return e;
}

// Launches over `tiles` tiles (an upper bound for experts), one persistent CTA per SM at most.
template <int BN, int KIND, int DT>
apex_status_t launch_fb(const void* a_codes, int64_t a_rows, const void* w_codes, int64_t Z,
                        FBArgs a, int64_t tiles, cudaStream_t s) {
  using C = FBCfg<BN>;
  auto kern = apex::f8_block_gemm_kernel<BN, KIND, DT>;
  static thread_local int attr_dev = -1;
  if (set_smem(kern, C::SMEM, &attr_dev) != cudaSuccess) return launched(cudaErrorUnknown);
  CUtensorMap ma, mb, my;
  if (!make_expanded_map(&ma, a_codes, a_rows, a.K, 128) ||
      !make_codes3_map(&mb, w_codes, Z, a.N, a.K, 128))
    return APEX_ERR_CUDA;
  if (KIND == apex::FB_UP) {
    if (!make_out_map(&my, a.hq, a_rows, a.N, 1, 64)) return APEX_ERR_CUDA;
  } else if (KIND == apex::FB_DOWN) {
    if (!make_out_map(&my, a.y, a_rows, a.N, 4, 32)) return APEX_ERR_CUDA;
  } else if (a.y_map) {
    if (!make_out_map(&my, a.y, a_rows, a.N, 2, 64)) return APEX_ERR_CUDA;
  } else {
    my = ma;   // never used
  }
  const int64_t most = dev_info().sms;
  a.P = (int)(tiles < most ? tiles : most);
  return launched(launch_pdl(kern, (unsigned)a.P, C::THREADS, (size_t)C::SMEM, s, ma, mb, my, a));
}

template <int DT>
cudaError_t f8_quantize_t(const void* x, int64_t M, int64_t K, void* codes, void* scales,
                          cudaStream_t s) {
  const int G = (int)ceil_div(K, 128);
  const int g_shift = (G & (G - 1)) == 0 ? __builtin_ctz((unsigned)G) : -1;
  int64_t blocks = ceil_div(M * G, 8);
  const int64_t cap = (int64_t)dev_info().sms * 32;
  if (blocks > cap) blocks = cap;
  return launch_pdl(apex::f8_quantize_act_kernel<DT>, (unsigned)blocks, 128, 0, s, x, (int)M,
                    (int)K, G, g_shift, static_cast<uint8_t*>(codes),
                    static_cast<float*>(scales));
}

apex_status_t check_f8_dims(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || K % 16) return APEX_ERR_INVALID_ARG;
  if (M > kMaxSlots || N > kMaxBlockDim || K > kMaxBlockDim) return APEX_ERR_UNSUPPORTED;
  if (M * ceil_div(K, 128) >= (1ll << 31)) return APEX_ERR_UNSUPPORTED;
  return APEX_OK;
}

FBArgs fb_args(int64_t M, int64_t N, int64_t K, const void* sa, const void* sw) {
  FBArgs a;
  memset(&a, 0, sizeof(a));
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.G = (int)ceil_div(K, 128);
  a.NB = (int)ceil_div(N, 128);
  a.sa = static_cast<const float*>(sa);
  a.sw = static_cast<const float*>(sw);
  a.s_vec = a.G % 4 == 0 && aligned(sa, 16) && aligned(sw, 16);
  a.wait_ns = g_wait_limit_ns;
  return a;
}

// ------------------------------------------------------------------ few tokens

// The few-token kernel runs up to this many tokens (dense; 8192 x 8192: 32 tokens 18.0 us against
// 23.9, but 48 tokens 25.1 against 24.2; 5000 x 2064: 32 tokens 8.8 against 9.2, 48 tokens 14.1
// against 9.2), or this many rows of an expert on average (64 experts of 2048 x 1024: 8 rows 86 us
// against 95, 12 rows 101 against 96).
constexpr int64_t kSmallTokens = 32;
constexpr int64_t kSmallRows = 10;

template <int BT, int KIND, int DT>
apex_status_t launch_fs(const CUtensorMap& mw, const CUtensorMap& mx, const FBArgs& b,
                        const int32_t* order, int64_t tiles, bool early, cudaStream_t s) {
  using C = apex::FSCfg<BT, KIND>;
  auto kern = apex::f8_small_gemm_kernel<BT, KIND, DT>;
  static thread_local int attr_dev = -1;
  if (set_smem(kern, C::SMEM, &attr_dev) != cudaSuccess) return launched(cudaErrorUnknown);
  apex::FSArgs a;
  a.b = b;
  a.order = order;
  a.early = early ? 1 : 0;
  // K split over a cluster while that leaves every CTA two groups and all CTAs resident
  const int64_t room = (int64_t)dev_info().sms * C::CTAS_PER_SM;
  a.S = 1;
  while (a.S < 8 && tiles * a.S * 2 <= room && b.G >= a.S * 4) a.S *= 2;
  a.b.P = (int)(a.S > 1 ? tiles * a.S : (tiles < room ? tiles : room));
  return launched(launch_pdl_cl(kern, (unsigned)a.b.P, (unsigned)C::THREADS, (size_t)C::SMEM, s,
                                (unsigned)a.S, mw, mx, a));
}

template <int DT>
apex_status_t fb_dense_t(int64_t M, int64_t N, int64_t K, const void* a_codes, const void* w_codes,
                         FBArgs a, bool early, cudaStream_t s) {
  const int sms = dev_info().sms;
  if (M <= kSmallTokens) {
    const int bt = M <= 16 ? 16 : 32;
    CUtensorMap ma, mb;
    if (!make_codes3_map(&mb, w_codes, 1, N, K, 128) || !make_expanded_map(&ma, a_codes, M, K, bt))
      return APEX_ERR_CUDA;
    a.tiles_m = (int)ceil_div(M, bt);
    a.tiles_n = a.NB;
    const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
    return bt == 16 ? launch_fs<16, apex::FB_DENSE, DT>(mb, ma, a, nullptr, tiles, early, s)
                    : launch_fs<32, apex::FB_DENSE, DT>(mb, ma, a, nullptr, tiles, early, s);
  }
  if (ceil_div(M, 128) * ceil_div(N, 128) >= (1ll << 31) - sms) return APEX_ERR_UNSUPPORTED;
  // 128 x 256 tiles or 128 x 128: the wider ones take about 1.6 times as long (0.48 and 0.3 us a
  // K-group), so whichever finishes its rounds over the SMs first (512 x 8192 x 8192: 39 against
  // 50 us, 256 x 8192 x 8192: 37 against 26)
  a.tiles_m = (int)ceil_div(M, 128);
  const int64_t wide = a.tiles_m * ceil_div(N, 256), narrow = a.tiles_m * ceil_div(N, 128);
  if (8 * ceil_div(wide, sms) <= 5 * ceil_div(narrow, sms)) {
    a.tiles_n = (int)ceil_div(N, 256);
    return launch_fb<256, apex::FB_DENSE, DT>(a_codes, M, w_codes, 1, a, wide, s);
  }
  a.tiles_n = (int)ceil_div(N, 128);
  return launch_fb<128, apex::FB_DENSE, DT>(a_codes, M, w_codes, 1, a, narrow, s);
}

// early: the activations' quantizer of the same call is the launch before this one.  It may fetch
// weights ahead of its wait because that launch, whatever it is, must release its dependents only
// after its own wait, when all before it has ended: the quantizer and the few-token GEMM do, the
// dense many-token GEMM does not.
apex_status_t fb_dense(int64_t M, int64_t N, int64_t K, const void* a_codes, const void* a_scales,
                       const void* w_codes, const void* w_scales, int32_t dtype, void* y,
                       bool early, cudaStream_t s) {
  FBArgs a = fb_args(M, N, K, a_scales, w_scales);
  a.y = y;
  a.y_map = N % 8 == 0 && aligned(y, 16);
  return dtype == APEX_DTYPE_F16 ? fb_dense_t<apex::DT_F16>(M, N, K, a_codes, w_codes, a, early, s)
                                 : fb_dense_t<apex::DT_BF16>(M, N, K, a_codes, w_codes, a, early, s);
}

// Few rows for each expert: the few-token kernel, which gathers FB_UP's rows of tokens itself.
bool moe_small(int64_t S, int64_t E) { return S <= (S < E ? S : E) * kSmallRows; }

// FB_UP or FB_DOWN over the experts' rows, by the few-token kernel or the other one.  `rows`:
// of the activations' codes; the launch before this one is the one that writes them.
template <int KIND, int DT>
apex_status_t fb_experts(const void* codes, int64_t rows, const void* w_codes, FBArgs a,
                         const int32_t* order, cudaStream_t s) {
  const int64_t S = a.slots, N = a.N, K = a.K;
  const int64_t Z = (KIND == apex::FB_UP ? 2 : 1) * (int64_t)a.E;
  const int64_t experts = S < a.E ? S : a.E;
  // at most: one partly filled tile for each expert that has rows, and the full ones
  auto most_tiles = [&](int64_t bm, int64_t tiles_n) { return (experts + S / bm) * tiles_n; };
  if (most_tiles(16, a.NB) >= (1ll << 31) - 4096) return APEX_ERR_UNSUPPORTED;
  if (moe_small(S, a.E)) {
    CUtensorMap ma, mb;
    if (!make_codes3_map(&mb, w_codes, Z, N, K, 128) ||
        !make_expanded_map(&ma, codes, rows, K, KIND == apex::FB_UP ? 1 : 16))
      return APEX_ERR_CUDA;
    a.tiles_n = a.NB;
    return launch_fs<16, KIND, DT>(mb, ma, a, order, most_tiles(16, a.NB), true, s);
  }
  a.tiles_n = KIND == apex::FB_UP ? a.NB : (int)ceil_div(N, 256);
  return launch_fb<256, KIND, DT>(codes, rows, w_codes, Z, a, most_tiles(128, a.tiles_n), s);
}

struct MoeWork {   // byte offsets into the workspace of apex_moe_mlp_fp8_block
  size_t xq, xs, pq, ps, slot, hq, hs, y, total;
};
MoeWork moe_work(int64_t T, int64_t E, int64_t k, int64_t H, int64_t I) {
  MoeWork w;
  const size_t S = (size_t)T * (size_t)k;
  w.xq = 0;
  w.xs = w.xq + pad256((size_t)T * H);
  w.pq = w.xs + pad256((size_t)T * ceil_div(H, 128) * 4);
  // the tokens' rows by slot and the flat indices' slots, where rows are not gathered
  const bool small = moe_small((int64_t)S, E);
  w.ps = w.pq + (small ? 0 : pad256(S * H));
  w.slot = w.ps + (small ? 0 : pad256(S * ceil_div(H, 128) * 4));
  w.hq = w.slot + (small ? 0 : pad256(S * 4));
  w.hs = w.hq + pad256(S * I);
  w.y = w.hs + pad256(S * ceil_div(I, 128) * 4);
  w.total = w.y + pad256(S * H * 4);
  return w;
}

apex_status_t check_moe(int64_t T, int32_t E, int32_t k, int64_t H, int64_t I) {
  if (T <= 0 || E <= 0 || k <= 0 || H <= 0 || I <= 0 || H % 16 || I % 16)
    return APEX_ERR_INVALID_ARG;
  if (E > APEX_MAX_EXPERTS || k > APEX_MAX_TOP_K || H > kMaxBlockDim || I > kMaxBlockDim ||
      T > kMaxSlots)
    return APEX_ERR_UNSUPPORTED;
  if (T * k >= kMaxSlots || T * k * ceil_div(H > I ? H : I, 128) >= (1ll << 31))
    return APEX_ERR_UNSUPPORTED;
  return APEX_OK;
}

// ------------------------------------------------------------------ routing

// Up to this many tokens, one for each warp, one CTA of 16 warps routes and groups them: one launch
// instead of two (in a graph, 16 tokens: 64 experts 5.4 us against 5.9, 256 in 8 groups 8.8 against
// 8.2 and a launch of the host's less; 32 tokens: 7.7 against 5.9, 13.7 against 8.3).
constexpr int64_t kRoutePlanTokens = 16;
constexpr int kRoutePlanWarps = 16;
// Four neighbouring tokens a warp from here on (64 experts: 4096 tokens 6.0 us against 6.3, 8192 7.4
// against 9.2; 256 in 8 groups with a bias: 4096 16.1 against 14.0, 8192 22.3 against 22.4, 16384
// 33.8 against 37.9).
constexpr int64_t kRouteBatchTokens = 8192;
// Grouping: one CTA of 8 warps, a cluster of 8 such, a cluster of 16 CTAs of 16 warps.  With 512
// choices they take 3.6, 4.1 and 5.1 us; with 1600 5.2, 4.4 and 5.1; with 8000 14.9, 5.7 and 5.7;
// with 131072 214, 31 and 12.7 (8 CTAs of 16 warps: 20.5).
constexpr int64_t kPlanCtaChoices = 768;
constexpr int64_t kPlanClusterChoices = 8192;
constexpr int kPlanWarps = 16;

apex_status_t route_args(apex::RouteArgs* a, const void* logits, int32_t dtype, int64_t T,
                         int32_t E, int32_t k, int32_t score, const void* bias_f32,
                         int32_t groups, int32_t topk_groups, int32_t renormalize, float scale,
                         const void* mask_u8, void* weights_f32, void* ids_i32) {
  if (!logits || !weights_f32 || !ids_i32 || T <= 0 || E <= 0 || k <= 0 || groups <= 0 ||
      topk_groups <= 0 || topk_groups > groups || E % groups)
    return APEX_ERR_INVALID_ARG;
  const bool group_max = (score & APEX_GROUP_MAX) != 0;
  score &= ~APEX_GROUP_MAX;
  if (score != APEX_SCORE_SOFTMAX && score != APEX_SCORE_SIGMOID) return APEX_ERR_INVALID_ARG;
  if (k > topk_groups * (E / groups)) return APEX_ERR_INVALID_ARG;
  if (!is_float(dtype) || E > APEX_MAX_EXPERTS || k > APEX_MAX_TOP_K || groups > 32 ||
      T >= kMaxSlots || T * (int64_t)k >= kMaxSlots)
    return APEX_ERR_UNSUPPORTED;
  if (!aligned(logits, dtype == APEX_DTYPE_F32 ? 4 : 2) || !aligned(bias_f32, 4) ||
      !aligned(weights_f32, 4) || !aligned(ids_i32, 4))
    return APEX_ERR_ALIGNMENT;
  a->logits = logits;
  a->bias = static_cast<const float*>(bias_f32);
  a->mask = static_cast<const uint8_t*>(mask_u8);
  a->T = (int)T;
  a->E = E;
  a->k = k;
  a->G = groups;
  a->TG = topk_groups;
  a->sigmoid = score == APEX_SCORE_SIGMOID;
  a->renorm = renormalize != 0;
  a->group_max = group_max;
  a->scale = scale;
  a->ids = static_cast<int32_t*>(ids_i32);
  a->weights = static_cast<float*>(weights_f32);
  return APEX_OK;
}

template <int DT, int EPL, bool GROUPS>
apex_status_t route_launch_t(const apex::RouteArgs& a, int32_t* offsets, int32_t* order,
                             cudaStream_t s) {
  if (offsets) {
    auto kern = apex::route_plan_kernel<DT, EPL, GROUPS>;
    const int warps = kRoutePlanWarps;
    const int route = GROUPS ? warps * a.E * 8 : 0, plan = apex::plan_smem(a.E, warps);
    constexpr int most = kRoutePlanWarps * APEX_MAX_EXPERTS * 8;
    static thread_local int attr_dev = -1;
    if (set_smem(kern, most, &attr_dev) != cudaSuccess) return launched(cudaErrorUnknown);
    return launched(launch_pdl(kern, 1u, 32u * warps, (size_t)(route > plan ? route : plan), s, a,
                               offsets, order));
  }
  // many tokens: four neighbours a warp, whose weights (64-bit exponentials and quotients) are
  // then computed together
  const int batch = a.k <= 8 && a.T >= kRouteBatchTokens ? 4 : 1;
  int64_t blocks = ceil_div(a.T, apex::kRouteWarps * batch);
  const int64_t cap = (int64_t)dev_info().sms * 16;
  if (blocks > cap) blocks = cap;
  return launched(launch_pdl(apex::route_kernel<DT, EPL, GROUPS>, (unsigned)blocks,
                             32 * apex::kRouteWarps,
                             GROUPS ? (size_t)apex::kRouteWarps * a.E * 8 : 0, s, a, batch));
}

template <int DT, int EPL>
apex_status_t route_launch_g(const apex::RouteArgs& a, int32_t* offsets, int32_t* order,
                             cudaStream_t s) {
  return a.G > 1 ? route_launch_t<DT, EPL, true>(a, offsets, order, s)
                 : route_launch_t<DT, EPL, false>(a, offsets, order, s);
}

template <int DT>
apex_status_t route_launch_e(const apex::RouteArgs& a, int32_t* offsets, int32_t* order,
                             cudaStream_t s) {
  if (a.E <= 64) return route_launch_g<DT, 2>(a, offsets, order, s);
  if (a.E <= 128) return route_launch_g<DT, 4>(a, offsets, order, s);
  if (a.E <= 256) return route_launch_g<DT, 8>(a, offsets, order, s);
  return route_launch_g<DT, 16>(a, offsets, order, s);
}

apex_status_t route_launch(const apex::RouteArgs& a, int32_t dtype, int32_t* offsets,
                           int32_t* order, cudaStream_t s) {
  if (dtype == APEX_DTYPE_F16) return route_launch_e<apex::DT_F16>(a, offsets, order, s);
  if (dtype == APEX_DTYPE_BF16) return route_launch_e<apex::DT_BF16>(a, offsets, order, s);
  return route_launch_e<apex::DT_F32>(a, offsets, order, s);
}

apex_status_t check_plan(const void* ids, int64_t T, int32_t k, int32_t E, const void* offsets,
                         const void* order) {
  if (!ids || !offsets || !order || T <= 0 || k <= 0 || E <= 0) return APEX_ERR_INVALID_ARG;
  if (E > APEX_MAX_EXPERTS || k > APEX_MAX_TOP_K || T >= kMaxSlots || T * (int64_t)k >= kMaxSlots)
    return APEX_ERR_UNSUPPORTED;
  if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(order, 4)) return APEX_ERR_ALIGNMENT;
  return APEX_OK;
}

// Whether clusters of that many CTAs of the grouping kernel can run on the current device (above 8
// is a kernel's own choice).
bool plan_cluster_fits(int ctas) {
  if (cudaFuncSetAttribute(apex::plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
      cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(32u * kPlanWarps);
  cfg.dynamicSmemBytes = (size_t)apex::plan_smem(APEX_MAX_EXPERTS, kPlanWarps);
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)ctas;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, apex::plan_kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return n > 0;
}

apex_status_t plan_launch(const int32_t* ids, int64_t S, int32_t E, int32_t* offsets,
                          int32_t* order, cudaStream_t s) {
  static thread_local int attr_dev = -1;
  static thread_local bool wide = false;   // clusters of 16 run here (not on every part of a GPU)
  const int before = attr_dev;
  if (set_smem(apex::plan_kernel, apex::plan_smem(APEX_MAX_EXPERTS, kPlanWarps), &attr_dev) !=
      cudaSuccess)
    return launched(cudaErrorUnknown);
  if (attr_dev != before) wide = plan_cluster_fits(apex::kPlanClusterMax);
  const unsigned ctas = S <= kPlanCtaChoices                ? 1u
                        : S <= kPlanClusterChoices || !wide ? 8u
                                                            : (unsigned)apex::kPlanClusterMax;
  const int warps = S <= kPlanClusterChoices ? 8 : kPlanWarps;
  return launched(launch_pdl_cl(apex::plan_kernel, ctas, 32u * warps,
                                (size_t)apex::plan_smem(E, warps), s, ctas, ids, (int)S, (int)E,
                                offsets, order));
}

}  // namespace

extern "C" {

apex_status_t apex_quantize_act_fp8_block(const void* x, int32_t dtype, int64_t M, int64_t K,
                                          void* codes, void* scales_f32, void* stream) {
  if (!x || !codes || !scales_f32) return APEX_ERR_INVALID_ARG;
  if (!is_16bit(dtype)) return APEX_ERR_UNSUPPORTED;
  apex_status_t st = check_f8_dims(M, 1, K);
  if (st != APEX_OK) return st;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales_f32, 4)) return APEX_ERR_ALIGNMENT;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launched(dtype == APEX_DTYPE_F16
                      ? f8_quantize_t<apex::DT_F16>(x, M, K, codes, scales_f32, s)
                      : f8_quantize_t<apex::DT_BF16>(x, M, K, codes, scales_f32, s));
}

apex_status_t apex_pack_weights_fp8_block(const void* w, int32_t dtype, int64_t E, int64_t N,
                                          int64_t K, void* codes, void* scales_f32, void* stream) {
  if (!w || !codes || !scales_f32 || E <= 0) return APEX_ERR_INVALID_ARG;
  if (!is_float(dtype)) return APEX_ERR_UNSUPPORTED;
  apex_status_t st = check_f8_dims(1, N, K);
  if (st != APEX_OK) return st;
  if (!aligned(w, 16) || !aligned(codes, 16) || !aligned(scales_f32, 4)) return APEX_ERR_ALIGNMENT;
  const int G = (int)ceil_div(K, 128), NB = (int)ceil_div(N, 128);
  if (E > (1ll << 20) || (int64_t)G * NB * E >= (1ll << 31)) return APEX_ERR_UNSUPPORTED;
  const unsigned blocks = (unsigned)((int64_t)G * NB * E);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto run = [&](auto kern) {
    return launched(launch_pdl(kern, blocks, 256, 0, s, w, (int)N, (int)K, G, NB,
                               static_cast<uint8_t*>(codes), static_cast<float*>(scales_f32)));
  };
  if (dtype == APEX_DTYPE_F16) return run(apex::f8_pack_weights_kernel<apex::DT_F16>);
  if (dtype == APEX_DTYPE_BF16) return run(apex::f8_pack_weights_kernel<apex::DT_BF16>);
  return run(apex::f8_pack_weights_kernel<apex::DT_F32>);
}

apex_status_t apex_gemm_fp8_block(int64_t M, int64_t N, int64_t K, const void* a_codes,
                                  const void* a_scales, const void* w_codes, const void* w_scales,
                                  int32_t dtype, void* y, void* stream) {
  if (!a_codes || !a_scales || !w_codes || !w_scales || !y) return APEX_ERR_INVALID_ARG;
  if (!is_16bit(dtype)) return APEX_ERR_UNSUPPORTED;
  apex_status_t st = check_f8_dims(M, N, K);
  if (st != APEX_OK) return st;
  if (!aligned(a_codes, 16) || !aligned(w_codes, 16) || !aligned(a_scales, 4) ||
      !aligned(w_scales, 4) || !aligned(y, 2))
    return APEX_ERR_ALIGNMENT;
  return fb_dense(M, N, K, a_codes, a_scales, w_codes, w_scales, dtype, y, false,
                  static_cast<cudaStream_t>(stream));
}

size_t apex_linear_fp8_block_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (check_f8_dims(M, N, K) != APEX_OK) return 0;
  return pad256((size_t)M * K) + pad256((size_t)M * ceil_div(K, 128) * 4);
}

apex_status_t apex_linear_fp8_block(int64_t M, int64_t N, int64_t K, const void* x, int32_t dtype,
                                    const void* w_codes, const void* w_scales, void* y,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  if (!x || !w_codes || !w_scales || !y || !workspace) return APEX_ERR_INVALID_ARG;
  if (!is_16bit(dtype)) return APEX_ERR_UNSUPPORTED;
  apex_status_t st = check_f8_dims(M, N, K);
  if (st != APEX_OK) return st;
  if (!aligned(x, 16) || !aligned(w_codes, 16) || !aligned(w_scales, 4) || !aligned(y, 2) ||
      !aligned(workspace, 256))
    return APEX_ERR_ALIGNMENT;
  if (workspace_bytes < apex_linear_fp8_block_workspace_size(M, N, K)) return APEX_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  void* sc = ws + pad256((size_t)M * K);
  st = apex_quantize_act_fp8_block(x, dtype, M, K, ws, sc, stream);
  if (st != APEX_OK) return st;
  return fb_dense(M, N, K, ws, sc, w_codes, w_scales, dtype, y, true,
                  static_cast<cudaStream_t>(stream));
}

apex_status_t apex_route_experts(const void* logits, int32_t dtype, int64_t T, int32_t E,
                                 int32_t k, int32_t score, const void* bias_f32, int32_t groups,
                                 int32_t topk_groups, int32_t renormalize, float scale,
                                 const void* mask_u8, void* weights_f32, void* ids_i32,
                                 void* stream) {
  apex::RouteArgs a;
  apex_status_t st = route_args(&a, logits, dtype, T, E, k, score, bias_f32, groups, topk_groups,
                                renormalize, scale, mask_u8, weights_f32, ids_i32);
  if (st != APEX_OK) return st;
  return route_launch(a, dtype, nullptr, nullptr, static_cast<cudaStream_t>(stream));
}

apex_status_t apex_plan_experts(const void* ids_i32, int64_t T, int32_t k, int32_t E,
                                void* offsets_i32, void* order_i32, void* stream) {
  apex_status_t st = check_plan(ids_i32, T, k, E, offsets_i32, order_i32);
  if (st != APEX_OK) return st;
  return plan_launch(static_cast<const int32_t*>(ids_i32), T * k, E,
                     static_cast<int32_t*>(offsets_i32), static_cast<int32_t*>(order_i32),
                     static_cast<cudaStream_t>(stream));
}

apex_status_t apex_route_plan_experts(const void* logits, int32_t dtype, int64_t T, int32_t E,
                                      int32_t k, int32_t score, const void* bias_f32,
                                      int32_t groups, int32_t topk_groups, int32_t renormalize,
                                      float scale, const void* mask_u8, void* weights_f32,
                                      void* ids_i32, void* offsets_i32, void* order_i32,
                                      void* stream) {
  apex::RouteArgs a;
  apex_status_t st = route_args(&a, logits, dtype, T, E, k, score, bias_f32, groups, topk_groups,
                                renormalize, scale, mask_u8, weights_f32, ids_i32);
  if (st == APEX_OK) st = check_plan(ids_i32, T, k, E, offsets_i32, order_i32);
  if (st != APEX_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t* off = static_cast<int32_t*>(offsets_i32);
  int32_t* order = static_cast<int32_t*>(order_i32);
  if (T <= kRoutePlanTokens) return route_launch(a, dtype, off, order, s);
  st = route_launch(a, dtype, nullptr, nullptr, s);
  if (st != APEX_OK) return st;
  return plan_launch(a.ids, T * k, E, off, order, s);
}

size_t apex_moe_mlp_fp8_block_workspace_size(int64_t T, int32_t E, int32_t k, int64_t H,
                                             int64_t I) {
  if (check_moe(T, E, k, H, I) != APEX_OK) return 0;
  return moe_work(T, E, k, H, I).total;
}

apex_status_t apex_moe_mlp_fp8_block(int64_t T, int32_t E, int32_t k, int64_t H, int64_t I,
                                     const void* x, int32_t dtype, const void* weights_f32,
                                     const void* ids_i32, const void* offsets_i32,
                                     const void* order_i32, const void* w13_codes,
                                     const void* w13_scales, const void* w2_codes,
                                     const void* w2_scales, void* y, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  if (!x || !weights_f32 || !ids_i32 || !offsets_i32 || !order_i32 || !w13_codes || !w13_scales ||
      !w2_codes || !w2_scales || !y || !workspace)
    return APEX_ERR_INVALID_ARG;
  if (!is_16bit(dtype)) return APEX_ERR_UNSUPPORTED;
  apex_status_t st = check_moe(T, E, k, H, I);
  if (st != APEX_OK) return st;
  if (!aligned(x, 16) || !aligned(w13_codes, 16) || !aligned(w2_codes, 16) || !aligned(y, 16) ||
      !aligned(workspace, 256) || !aligned(weights_f32, 4) || !aligned(ids_i32, 4) ||
      !aligned(offsets_i32, 4) || !aligned(order_i32, 4) || !aligned(w13_scales, 4) ||
      !aligned(w2_scales, 4))
    return APEX_ERR_ALIGNMENT;
  const MoeWork w = moe_work(T, E, k, H, I);
  if (workspace_bytes < w.total) return APEX_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  st = apex_quantize_act_fp8_block(x, dtype, T, H, ws + w.xq, ws + w.xs, stream);
  if (st != APEX_OK) return st;

  const int64_t S = T * k;
  auto with_experts = [&](FBArgs a) {
    a.E = E;
    a.slots = (int)S;
    a.top_k = k;
    a.offsets = static_cast<const int32_t*>(offsets_i32);
    return a;
  };
  const int32_t* order = static_cast<const int32_t*>(order_i32);
  const bool small = moe_small(S, E);
  if (!small) {
    st = launched(launch_pdl(apex::f8_permute_kernel, grid_for(S * 32, 256, 8), 256, 0, s,
                             (const uint8_t*)(ws + w.xq), (const float*)(ws + w.xs),
                             order, (int)S, (int)k, (int)H, (int)ceil_div(H, 128), ws + w.pq,
                             reinterpret_cast<float*>(ws + w.ps),
                             reinterpret_cast<int32_t*>(ws + w.slot)));
    if (st != APEX_OK) return st;
  }
  FBArgs up = with_experts(fb_args(small ? T : S, I, H, ws + (small ? w.xs : w.ps), w13_scales));
  up.hq = ws + w.hq;
  up.hs = reinterpret_cast<float*>(ws + w.hs);
  st = fb_experts<apex::FB_UP, apex::DT_BF16>(ws + (small ? w.xq : w.pq), small ? T : S, w13_codes,
                                              up, order, s);
  if (st != APEX_OK) return st;

  FBArgs down = with_experts(fb_args(S, H, I, ws + w.hs, w2_scales));
  down.y = ws + w.y;
  const bool f16 = dtype == APEX_DTYPE_F16;
  st = fb_experts<apex::FB_DOWN, apex::DT_F32>(ws + w.hq, S, w2_codes, down, order, s);
  if (st != APEX_OK) return st;

  const unsigned blocks = grid_for(T * (H / 8), 256, 16);
  const int32_t* slot_of = small ? nullptr : reinterpret_cast<const int32_t*>(ws + w.slot);
  return launched(f16 ? launch_pdl(apex::combine_kernel<apex::DT_F16>, blocks, 256, 0, s,
                                   (const float*)(ws + w.y), static_cast<const float*>(weights_f32),
                                   static_cast<const int32_t*>(ids_i32), slot_of, (int)T, (int)H,
                                   (int)k, (int)E, y)
                      : launch_pdl(apex::combine_kernel<apex::DT_BF16>, blocks, 256, 0, s,
                                   (const float*)(ws + w.y), static_cast<const float*>(weights_f32),
                                   static_cast<const int32_t*>(ids_i32), slot_of, (int)T, (int)H,
                                   (int)k, (int)E, y));
}

apex_status_t apex_block_norm(const void* x, int32_t dtype, int64_t T, int64_t H,
                              const void* residual, const void* post_weight, const void* gate,
                              int64_t gate_rows, float alpha, const void* pre_weight, float eps,
                              float weight_offset, void* h, void* y, void* y_codes,
                              void* y_scales_f32, void* stream) {
  if (!x || T <= 0 || H <= 0 || H % 8 || !(eps >= 0.0f)) return APEX_ERR_INVALID_ARG;
  if (!h && !y && !y_codes) return APEX_ERR_INVALID_ARG;
  if ((y || y_codes) && !pre_weight) return APEX_ERR_INVALID_ARG;
  if (y_codes && (!y_scales_f32 || H % 16)) return APEX_ERR_INVALID_ARG;
  if (gate && (gate_rows <= 0 || T % gate_rows)) return APEX_ERR_INVALID_ARG;
  if (!is_16bit(dtype) || H > 32768 || T >= (1ll << 31)) return APEX_ERR_UNSUPPORTED;
  for (const void* p : {x, residual, post_weight, gate, pre_weight, (const void*)h,
                        (const void*)y, (const void*)y_codes})
    if (!aligned(p, 16)) return APEX_ERR_ALIGNMENT;
  if (!aligned(y_scales_f32, 4)) return APEX_ERR_ALIGNMENT;
  apex::NormArgs a;
  a.x = x;
  a.residual = residual;
  a.post = post_weight;
  a.gate = gate;
  a.pre = (y || y_codes) ? pre_weight : nullptr;
  a.T = (int)T;
  a.H = (int)H;
  a.G = (int)ceil_div(H, 128);
  a.rows_per_gate = gate ? (int)(T / gate_rows) : 1;
  a.alpha = alpha;
  a.eps = eps;
  a.off = weight_offset;
  a.h = h;
  a.y = y;
  a.codes = static_cast<uint8_t*>(y_codes);
  a.scales = static_cast<float*>(y_scales_f32);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto run = [&](auto kern, int nc) {
    const unsigned threads = (unsigned)(ceil_div(ceil_div(H, 8 * nc), 32) * 32);
    return launched(launch_pdl(kern, (unsigned)T, threads, 0, s, a));
  };
  auto by_width = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    // CTAs of at most 256 threads, four of which share an SM, once there are two tokens for each
    // SM, or one chunk a thread.  In a graph, with post-norm and residual, h, y and codes: 4096 x
    // 8192 53 us against 96, 4096 x 4096 29 against 36; 296 tokens of 8192 6.4 against 6.8, of 4096
    // 4.1 against 4.4, of 2048 3.6 against 3.0 (592: 4.1 against 4.4); 148 of 8192 5.4 against 3.9.
    const bool many = T >= 2 * (int64_t)dev_info().sms;
    if (many && H <= 4096) return run(apex::block_norm_kernel<DT, 2, 256, 4>, 2);
    if (many && H <= 8192) return run(apex::block_norm_kernel<DT, 4, 256, 4>, 4);
    if (H <= 8192) return run(apex::block_norm_kernel<DT, 1, 1024, 1>, 1);
    if (H <= 16384) return run(apex::block_norm_kernel<DT, 2, 1024, 1>, 2);
    return run(apex::block_norm_kernel<DT, 4, 1024, 1>, 4);
  };
  return dtype == APEX_DTYPE_F16 ? by_width(std::integral_constant<int, apex::DT_F16>{})
                                 : by_width(std::integral_constant<int, apex::DT_BF16>{});
}

}  // extern "C"
