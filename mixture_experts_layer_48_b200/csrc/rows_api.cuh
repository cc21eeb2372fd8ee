// Host side of the operators around the layer (include/moe.h, "Training and the block around the
// layer"): argument checks, kernel variants and launches.  Included once, by moe_api.cu, whose
// handle, launch helpers and TMA encoder it uses.
#pragma once

namespace {

constexpr int kMaxKN = 32768;         // K and N of the grouped products (gate/up: N = 2I)
constexpr int kMaxRows = 1 << 28;     // rows of one call
constexpr int kColsSmallRows = 32;    // rows per tile of the few-row kernels
constexpr int kColsRows = 128;

bool on_device(const moe_ctx* c) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return dev == c->device;
}

// Arrays that kernels read one element at a time: offsets, per-row weights and norms.
bool all_aligned4(std::initializer_list<const void*> ps) {  // null passes
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return false;
  return true;
}
bool all_aligned16(std::initializer_list<const void*> ps) {  // null passes
  for (const void* p : ps)
    if (!aligned16(p)) return false;
  return true;
}

// bf16 rows [rows, cols], or planes [planes, rows, cols], with a [box_rows, 64] box and the
// 128-byte swizzle.  Encoded for every call: the map holds nothing but the call's own arguments.
bool encode_rows(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  return encode_2d(m, base, rows, cols, box_rows, kGrBK, CU_TENSOR_MAP_SWIZZLE_128B, true);
}
bool encode_planes(CUtensorMap* m, const void* base, uint64_t planes, uint64_t rows, uint64_t cols,
                   uint32_t box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {cols, rows, planes};
  cuuint64_t strides[2] = {cols * 2, rows * cols * 2};
  cuuint32_t box[3] = {(cuuint32_t)kGrBK, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launch with programmatic dependent launch on clusters of `cluster` CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                               int cluster, cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Whether the kernel may take `bytes` of dynamic shared memory on the handle's device: asked for at
// the handle's first use of the kernel (for all of them in moe_create it took 0.3 s of loading).
template <typename... A>
bool ready(moe_ctx* c, void (*kernel)(A...), size_t bytes) {
  const void* f = reinterpret_cast<const void*>(kernel);
  for (int i = 0; i < c->n_ready; ++i)
    if (c->ready[i] == f) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
    return false;
  if (c->n_ready < moe_ctx::kMaxReady) c->ready[c->n_ready++] = f;
  return true;
}

// Clusters of 2, 4 and 8 CTAs of the few-row kernel (one CTA per SM) that fit the GPU at once: a
// cluster lies inside one GPC, whose SM count need not be a multiple of its size.
bool query_clusters(moe_ctx* c) {
  if (c->max_clusters[0] > 0) return true;
  auto kernel = grouped_cols_kernel<kColsSmallRows, 1, false, false>;
  const size_t smem = ColsCfg<kColsSmallRows, 1>::kSmem;
  int out[3];
  if (!ready(c, kernel, smem)) return false;
  for (int i = 0; i < 3; ++i) {
    const int size = 2 << i;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c->num_sms / size * size);
    cfg.blockDim = dim3(ColsCfg<kColsSmallRows, 1>::kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&out[i], kernel, &cfg) != cudaSuccess || out[i] < 1)
      return false;
  }
  for (int i = 0; i < 3; ++i) c->max_clusters[i] = out[i];
  return true;
}

// Which kernel multiplies a call's rows, from sizes the host knows (the segments stay on the
// device): the one with the smallest estimate.
struct GroupedPlan {
  enum Kind { kColsSmall, kColsWide, kRows } kind;
  int split;    // CTAs per cluster that share a tile's reduction
};

// Estimate in us of `tiles` tiles on `slots` CTAs (or pairs) at a time, `stages` stages each: a
// stage takes at least `stage_us`, or as long as HBM needs for the weight bytes that all slots
// load in it; `tile_us` more per tile.
double grouped_us(long long tiles, int slots, double stages, double stage_us, double hbm_bytes,
                  double tile_us) {
  const double us_per_byte = 1.0 / 6.5e6;
  const long long full = tiles / slots, rem = tiles % slots;
  auto round = [&](double n) {
    return stages * std::max(stage_us, n * hbm_bytes * us_per_byte) + tile_us;
  };
  return full * round(slots) + (rem ? round((double)rem) : 0.0);
}

// The constants are fitted to 176 measured calls (1..128 experts of 2..640 rows, four weight
// shapes; bf16, graph replay): the choice costs 0.4 % over the best kernel of each, 12 % at worst.
// It sees the mean rows of an expert only; on skewed calls (32 experts, 64..2048 tokens of 4 choices,
// popularity falling as rank^-0.5 .. rank^-1.5) it costs up to 4 %, mostly under 0.5 %.
// Some of them, us as 128-column tiles / split in two / in four / 256-column tiles / pairs:
//   1 expert of 4 rows, 2880 x 2880          18.0 / 11.7 / 8.8 / 22.7 / 19.0
//   8 experts of 4 rows, 2880 x 2880         36.7 / 30.5 / 31.1 / 25.6 / 35.6
//   8 experts of 4 rows, 2880 x 5760         52.7 / 46.6 / 50.8 / 54.8 / 52.3
//   32 experts of 128 rows, 2880 x 2880      256 columns 97, pairs 122
//   32 experts of 192 rows, 2880 x 2880      256 columns 195, pairs 123
GroupedPlan plan_grouped(const moe_ctx* c, int R, int Kred, int Ncols) {
  const int nk = (Kred + kGrBK - 1) / kGrBK;
  const int busy = std::min(R, c->E);                // experts that can hold rows
  const int mean = (R + busy - 1) / busy;
  auto chunks = [&](int rows) { return (long long)(mean + rows - 1) / rows; };
  auto blocks = [&](int cols) { return (long long)(Ncols + cols - 1) / cols; };
  GroupedPlan best{GroupedPlan::kRows, 1};
  double us = grouped_us(busy * chunks(256) * blocks(256), c->num_sms / 2, nk, 0.36, 0.0, 0.8);
  auto consider = [&](GroupedPlan p, double t) {
    if (t < us) {
      best = p;
      us = t;
    }
  };
  // a weight block is read from HBM once for all chunks of its expert
  consider({GroupedPlan::kColsWide, 1},
           grouped_us(busy * chunks(kColsRows) * blocks(256), c->num_sms, nk,
                      0.40 + 0.15 * std::min(mean, kColsRows) / kColsRows,
                      32768.0 / chunks(kColsRows), 0.1));
  if (mean <= 4 * kColsSmallRows)
    for (int s = 1; s <= 4; s *= 2) {
      const int slots = s == 1 ? c->num_sms : c->max_clusters[s / 4];
      consider({GroupedPlan::kColsSmall, s},
               grouped_us(busy * chunks(kColsSmallRows) * blocks(128), slots, (double)nk / s, 0.34,
                          s * 16384.0 / chunks(kColsSmallRows),
                          0.3 + 0.03 * std::min(mean, kColsSmallRows) + (s > 1 ? 0.4 : 0.0)));
    }
  return best;
}

// CTA pairs that share a weight-gradient tile: 1 while the tiles fill the GPU or the segments are
// short.  A stage of 64 rows takes about 0.42 us; an exchange about 4.
int plan_wgrad(const moe_ctx* c, int R, int K, int N) {
  const long long tiles = (long long)c->E * ((K + 255) / 256) * ((N + 255) / 256);
  const double stages = std::max(1.0, (double)R / c->E / kGrBK);
  int best = 1;
  double us = grouped_us(tiles, c->num_sms / 2, stages, 0.42, 0.0, 0.0);
  for (int pairs = 2; pairs <= 4; pairs *= 2) {
    const double t = grouped_us(tiles, c->max_clusters[pairs / 2], stages / pairs, 0.42, 0.0, 4.0);
    if (t < us) {
      us = t;
      best = pairs;
    }
  }
  return best;
}

template <int ROWS, int NM, bool TRANS, bool F32>
cudaError_t launch_cols(moe_ctx* c, int split, const GroupedArgs& a, const CUtensorMap& wmap,
                        const CUtensorMap& xmap, cudaStream_t st) {
  auto kernel = grouped_cols_kernel<ROWS, NM, TRANS, F32>;
  const size_t smem = ColsCfg<ROWS, NM>::kSmem;
  if (!ready(c, kernel, smem)) return cudaErrorInvalidConfiguration;
  const int clusters = split == 1 ? c->num_sms : c->max_clusters[split / 4];  // 2, 4 -> 0, 1
  return launch_pdl_cluster(kernel, dim3(clusters * split), dim3(ColsCfg<ROWS, NM>::kThreads), smem, split, st, a,
                            wmap, xmap, split);
}

template <bool TRANS, bool F32>
moe_status run_grouped(moe_ctx* c, const GroupedArgs& a, const void* W, const void* x, int K, int N,
                       cudaStream_t st) {
  if (!query_clusters(c)) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  const GroupedPlan p = plan_grouped(c, a.R, a.Kred, a.Ncols);
  const uint32_t box = p.kind == GroupedPlan::kRows       ? kPairHalf
                       : p.kind == GroupedPlan::kColsWide ? ColsCfg<kColsRows, 2>::kRowBox
                                                          : ColsCfg<kColsSmallRows, 1>::kRowBox;
  CUtensorMap wmap, xmap;
  // weight boxes 64 columns wide; transposed: 128 rows (columns of the result), else a stage's
  const int wrows = TRANS ? 128 : p.kind == GroupedPlan::kColsSmall ? ColsCfg<kColsSmallRows, 1>::kK : kGrBK;
  if (!encode_planes(&wmap, W, c->E, K, N, wrows) ||
      !encode_rows(&xmap, x, a.R, a.Kred, box))
    return MOE_ERR_CUDA;
  return launch(c, -1, st, [&] {
    switch (p.kind) {
      case GroupedPlan::kColsSmall:
        return launch_cols<kColsSmallRows, 1, TRANS, F32>(c, p.split, a, wmap, xmap, st);
      case GroupedPlan::kColsWide:
        return launch_cols<kColsRows, 2, TRANS, F32>(c, p.split, a, wmap, xmap, st);
      default:
        if (!ready(c, grouped_rows_kernel<TRANS, F32>, kPairSmem)) return cudaErrorInvalidConfiguration;
        return launch_pdl(grouped_rows_kernel<TRANS, F32>, dim3(c->num_sms / 2 * 2),
                          dim3(kPairThreads), (size_t)kPairSmem, st, a, wmap, xmap);
    }
  });
}

bool grouped_shape_ok(const moe_ctx* c, int R, int K, int N, moe_dtype out_type) {
  return R >= 0 && R <= kMaxRows && K >= 8 && K <= kMaxKN && K % 8 == 0 && N >= 8 && N <= kMaxKN &&
         N % 8 == 0 && (out_type == MOE_BF16 || out_type == MOE_F32);
}

// ---- row kernels: threads per row from the row's length ------------------------------------------
// f(TPR, VPT) for a row of n4 vectors: the fewest threads (up to 512) that hold it with three
// vectors each, two where they suffice.  Rows beyond that take more vectors.
template <typename F>
moe_status by_row_length(int n4, F&& f) {
  using std::integral_constant;
  auto pick = [&](auto tpr, auto vpt) { return f(tpr, vpt); };
#define MOE_ROW(tpr, vpt) \
  if (n4 <= tpr * vpt) return pick(integral_constant<int, tpr>{}, integral_constant<int, vpt>{})
  MOE_ROW(32, 1);
  MOE_ROW(32, 2);
  MOE_ROW(32, 3);
  MOE_ROW(64, 2);
  MOE_ROW(64, 3);
  MOE_ROW(128, 2);
  MOE_ROW(128, 3);
  MOE_ROW(256, 2);
  MOE_ROW(256, 3);
  MOE_ROW(512, 2);
  MOE_ROW(512, 3);
  MOE_ROW(512, 4);
  MOE_ROW(512, 6);
#undef MOE_ROW
  return pick(integral_constant<int, 512>{}, integral_constant<int, 8>{});
}

template <typename F>
moe_status by_types(moe_dtype resid_type, moe_dtype y_type, F&& f) {
  if (resid_type == MOE_F32)
    return y_type == MOE_F32 ? f(float{}, float{}) : f(float{}, uint16_t{});
  return y_type == MOE_F32 ? f(uint16_t{}, float{}) : f(uint16_t{}, uint16_t{});
}

bool dtype_ok(moe_dtype t) { return t == MOE_BF16 || t == MOE_F32; }

// Ring of a staged norm: blocks per SM and stages.  As many blocks, then stages, as fit an SM's
// shared memory with two stages each; one stage where two of one block do not fit.
struct RowPlan {
  int blocks, stages;
};
constexpr int kRowRingBytes = 224 * 1024;          // of one block (and its attribute)
RowPlan plan_rows(int stage_bytes, int max_blocks) {
  const int budget = 228 * 1024, fixed = 1536;   // an SM's; a block's reserve and static part
  RowPlan best{1, 1};
  for (int b = 1; b <= max_blocks; ++b)
    for (int s = 2; s <= kRowRingMax; ++s)
      if ((long long)s * stage_bytes <= kRowRingBytes &&
          b * ((long long)s * stage_bytes + fixed) <= budget)
        best = {b, s};
  return best;
}

// What every norm kernel gets from the handle.
NormArgs norm_args(const moe_ctx* c, int T, float scale) {
  NormArgs a{};
  a.T = T;
  a.H = c->H;
  a.scale = scale;
  a.lose_row = c->norm_lose_row;
  a.status = c->d_status;
  return a;
}

// Persistent blocks of a call.
template <int TPR, int VPT>
int row_grid(const moe_ctx* c, int T, int blocks) {
  const long long need = ((long long)T + RowCfg<TPR, VPT>::kRows - 1) / RowCfg<TPR, VPT>::kRows;
  return (int)std::min<long long>(need, (long long)c->num_sms * blocks);
}

// Most partial rows that a column sum of T rows can have.
int norm_backward_parts(const moe_ctx* c, int T) {
  int parts = 0;
  by_row_length(c->H / 4, [&](auto tpr, auto vpt) {
    constexpr int TPR = decltype(tpr)::value, VPT = decltype(vpt)::value;
    parts = row_grid<TPR, VPT>(c, T, norm_backward_blocks<TPR, VPT>()) * RowCfg<TPR, VPT>::kRows;
    return MOE_OK;
  });
  return parts;
}

// The staged kernels hold their vectors (and the backward one its sums) in registers: up to four
// vectors a thread.  The forward kernel is staged while it reads at most 6 bytes an element (8189
// rows of 2880, bf16 residual: 17.7 us staged, 23.0 not, without a block; 41.8 and 46.5 with an
// fp32 block output; an fp32 residual and block output, 32768 rows: 215 and 193).
template <int VPT>
constexpr bool norm_staged() { return VPT <= 4; }

}  // namespace

extern "C" {

moe_status moe_grouped_matmul(moe_t c, int R, int K, int N, int transpose, const int32_t* offsets,
                              const void* x_rows_bf16, const void* W_bf16, void* out,
                              moe_dtype out_type, moe_stream_t stream) {
  if (!c || !grouped_shape_ok(c, R, K, N, out_type)) return MOE_ERR_ARG;
  if (R == 0) return MOE_OK;
  if (!offsets || !x_rows_bf16 || !W_bf16 || !out) return MOE_ERR_ARG;
  if (!all_aligned4({offsets}) || !all_aligned16({x_rows_bf16, W_bf16, out}) || !on_device(c))
    return MOE_ERR_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  GroupedArgs a{};
  a.offsets = offsets;
  a.E = c->E;
  a.R = R;
  a.Kred = transpose ? N : K;
  a.Ncols = transpose ? K : N;
  a.out = out;
  a.status = c->d_status;
  if (transpose)
    return out_type == MOE_F32 ? run_grouped<true, true>(c, a, W_bf16, x_rows_bf16, K, N, st)
                               : run_grouped<true, false>(c, a, W_bf16, x_rows_bf16, K, N, st);
  return out_type == MOE_F32 ? run_grouped<false, true>(c, a, W_bf16, x_rows_bf16, K, N, st)
                             : run_grouped<false, false>(c, a, W_bf16, x_rows_bf16, K, N, st);
}

moe_status moe_grouped_wgrad(moe_t c, int R, int K, int N, const int32_t* offsets,
                             const void* x_rows_bf16, const void* dy_rows_bf16, void* dW,
                             moe_dtype out_type, moe_stream_t stream) {
  if (!c || !grouped_shape_ok(c, R, K, N, out_type)) return MOE_ERR_ARG;
  if (!dW || !aligned16(dW) || !on_device(c)) return MOE_ERR_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (R == 0) {
    const size_t bytes = (size_t)c->E * K * N * (out_type == MOE_F32 ? 4 : 2);
    return cudaMemsetAsync(dW, 0, bytes, st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  if (!offsets || !x_rows_bf16 || !dy_rows_bf16 ||
      !all_aligned4({offsets}) || !all_aligned16({x_rows_bf16, dy_rows_bf16}))
    return MOE_ERR_ARG;
  GroupedArgs a{};
  a.offsets = offsets;
  a.E = c->E;
  a.R = R;
  a.Ncols = N;
  a.M = K;
  a.out = dW;
  a.status = c->d_status;
  CUtensorMap xmap, dymap;
  if (!encode_rows(&xmap, x_rows_bf16, R, K, kGrBK) || !encode_rows(&dymap, dy_rows_bf16, R, N, kGrBK))
    return MOE_ERR_CUDA;
  if (!query_clusters(c)) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  const bool f32 = out_type == MOE_F32;
  const int pairs = plan_wgrad(c, R, K, N);
  const int tiles = c->E * ((K + 255) / 256) * ((N + 255) / 256);
  const int grid = pairs > 1 ? tiles * 2 * pairs : c->num_sms / 2 * 2;
  auto kernel = grouped_wgrad_kernel<true, false, true>;
  if (pairs > 1) kernel = f32 ? grouped_wgrad_kernel<true, true, true> : grouped_wgrad_kernel<false, true, true>;
  else if (!f32) kernel = R > kGrPieceRowsBf16 ? grouped_wgrad_kernel<false, false, true>
                                               : grouped_wgrad_kernel<false, false, false>;
  return launch(c, -1, st, [&] {
    if (!ready(c, kernel, kPairSmem)) return cudaErrorInvalidConfiguration;
    return launch_pdl_cluster(kernel, dim3(grid), dim3(kWgradThreads), (size_t)kPairSmem, 2 * pairs,
                              st, a, xmap, dymap, pairs);
  });
}

moe_status moe_swiglu(moe_t c, int R, const void* gu_bf16, const float* row_w, void* h_bf16,
                      moe_stream_t stream) {
  if (!c || R < 0 || R > kMaxRows) return MOE_ERR_ARG;
  if (R == 0) return MOE_OK;
  if (!gu_bf16 || !h_bf16 || !all_aligned4({row_w}) || !all_aligned16({gu_bf16, h_bf16}) ||
      !on_device(c))
    return MOE_ERR_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const long long blocks = ((long long)R * (c->I / 8) + 255) / 256;
  return launch(c, -1, st, [&] {
    return launch_pdl(swiglu_rows_kernel, dim3((unsigned)std::min<long long>(blocks, 1 << 30)),
                      dim3(256), 0, st, static_cast<const uint16_t*>(gu_bf16), row_w,
                      static_cast<uint16_t*>(h_bf16), R, c->I);
  });
}

moe_status moe_swiglu_backward(moe_t c, int R, const void* dh_bf16, const void* gu_bf16,
                               const float* row_w, void* dgu_bf16, float* drow_w,
                               moe_stream_t stream) {
  if (!c || R < 0 || R > kMaxRows) return MOE_ERR_ARG;
  if (R == 0) return MOE_OK;
  if (!dh_bf16 || !gu_bf16 || !dgu_bf16 || (drow_w && !row_w) ||
      !all_aligned4({row_w, drow_w}) || !all_aligned16({dh_bf16, gu_bf16, dgu_bf16}) ||
      !on_device(c))
    return MOE_ERR_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return by_row_length(c->I / 8, [&](auto tpr, auto vpt) {   // vectors of 8
    constexpr int TPR = decltype(tpr)::value, VPT = decltype(vpt)::value;
    const int rows = RowCfg<TPR, VPT>::kRows;
    return launch(c, -1, st, [&] {
      return launch_pdl(swiglu_rows_backward_kernel<TPR, VPT>, dim3((R + rows - 1) / rows),
                        dim3(RowCfg<TPR, VPT>::kThreads), 0, st,
                        static_cast<const uint16_t*>(dh_bf16),
                        static_cast<const uint16_t*>(gu_bf16), row_w,
                        static_cast<uint16_t*>(dgu_bf16), drow_w, R, c->I);
    });
  });
}

moe_status moe_block_norm(moe_t c, int T, moe_dtype resid_type, moe_dtype y_type, const void* resid,
                          const void* y, const float* w_post, const float* gate, float scale,
                          const float* w_next, float eps, void* resid_out, void* x_bf16,
                          float* rstd_post, float* rstd_next, moe_stream_t stream) {
  if (!c || T < 0 || T > kMaxT || !dtype_ok(resid_type) || !dtype_ok(y_type)) return MOE_ERR_ARG;
  if (!(eps > 0.f) || !std::isfinite(eps) || !std::isfinite(scale)) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!resid || (y != nullptr) != (resid_out != nullptr)) return MOE_ERR_ARG;
  if (!y && (w_post || gate || !w_next)) return MOE_ERR_ARG;
  if ((w_post != nullptr) != (rstd_post != nullptr)) return MOE_ERR_ARG;
  if ((w_next != nullptr) != (x_bf16 != nullptr) || (w_next != nullptr) != (rstd_next != nullptr))
    return MOE_ERR_ARG;
  if (!all_aligned4({rstd_post, rstd_next}) ||
      !all_aligned16({resid, y, w_post, gate, w_next, resid_out, x_bf16}) || !on_device(c))
    return MOE_ERR_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  NormArgs a = norm_args(c, T, scale);
  a.eps = eps;
  a.resid = resid;
  a.y = y;
  a.w_post = w_post;
  a.gate = gate;
  a.w_next = w_next;
  a.resid_out = resid_out;
  a.x = static_cast<uint16_t*>(x_bf16);
  a.rstd_post = rstd_post;
  a.rstd_next = rstd_next;
  return by_row_length(c->H / 4, [&](auto tpr, auto vpt) {
    constexpr int TPR = decltype(tpr)::value, VPT = decltype(vpt)::value;
    return by_types(resid_type, y_type, [&](auto rt, auto yt) {
      using RT = decltype(rt);
      using YT = decltype(yt);
      const int rows = RowCfg<TPR, VPT>::kRows;
      if (norm_staged<VPT>() && sizeof(RT) + (y ? sizeof(YT) : 0) <= 6) {
        a.stage_bytes = rows * c->H * (int)(sizeof(RT) + (y ? sizeof(YT) : 0));
        const RowPlan p = plan_rows(a.stage_bytes, norm_forward_blocks<TPR, VPT>());
        a.stages = p.stages;
        return launch(c, -1, st, [&] {
          auto kernel = block_norm_kernel<TPR, VPT, RT, YT, norm_staged<VPT>()>;
          if (!ready(c, kernel, kRowRingBytes)) return cudaErrorInvalidConfiguration;
          return launch_pdl(kernel, dim3(row_grid<TPR, VPT>(c, T, p.blocks)),
                            dim3(RowCfg<TPR, VPT>::kThreads), (size_t)a.stages * a.stage_bytes, st,
                            a);
        });
      }
      return launch(c, -1, st, [&] {
        return launch_pdl(block_norm_kernel<TPR, VPT, RT, YT, false>,
                          dim3((T + rows - 1) / rows), dim3(RowCfg<TPR, VPT>::kThreads), 0, st, a);
      });
    });
  });
}

moe_status moe_selftest_norm_timeout(moe_t c, int from_row) {
  if (!c) return MOE_ERR_ARG;
  c->norm_lose_row = from_row < 0 ? INT_MAX : from_row;
  return MOE_OK;
}

size_t moe_block_norm_workspace_bytes(moe_t c, int T) {
  if (!c || T < 0 || T > kMaxT) return 0;
  // two partial sums (the norm before, the norm after and the gate) of H columns each
  return 2 * sizeof(float) * (size_t)std::max(1, norm_backward_parts(c, T)) * c->H;
}

moe_status moe_block_norm_backward(moe_t c, int T, moe_dtype resid_type, moe_dtype y_type,
                                   moe_dtype dy_type, const void* dresid, const void* dx_bf16,
                                   const void* resid, const void* y, const float* rstd_post,
                                   const float* rstd_next, const float* w_post, const float* gate,
                                   float scale, const float* w_next, void* dresid_out, void* dy,
                                   float* dw_post, float* dgate, float* dw_next, void* workspace,
                                   size_t ws_bytes, moe_stream_t stream) {
  if (!c || T < 0 || T > kMaxT || !dtype_ok(resid_type) || !dtype_ok(y_type) || !dtype_ok(dy_type))
    return MOE_ERR_ARG;
  if (!std::isfinite(scale)) return MOE_ERR_ARG;
  const bool next = w_next != nullptr, post = w_post != nullptr, gated = gate != nullptr;
  if (next != (dw_next != nullptr) || post != (dw_post != nullptr) || gated != (dgate != nullptr))
    return MOE_ERR_ARG;
  if (T > 0) {
    if (next != (dx_bf16 != nullptr) || next != (rstd_next != nullptr) || (next && !resid))
      return MOE_ERR_ARG;
    if (post != (rstd_post != nullptr) || ((post || gated) && (!y || !dy))) return MOE_ERR_ARG;
    if (!dresid_out || (!next && !dy) || (!next && !dresid)) return MOE_ERR_ARG;
  }
  if (!all_aligned4({rstd_post, rstd_next, dw_post, dgate, dw_next}) ||
      !all_aligned16({dresid, dx_bf16, resid, y, w_post, gate, w_next, dresid_out, dy}) ||
      !on_device(c))
    return MOE_ERR_ARG;
  const bool sums = next || post || gated;
  if (sums && (!workspace || !aligned16(workspace) || ws_bytes < moe_block_norm_workspace_bytes(c, T)))
    return MOE_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  float* part_x = next ? static_cast<float*>(workspace) : nullptr;
  float* part_y = post || gated ? static_cast<float*>(workspace) +
                                      (size_t)norm_backward_parts(c, T) * c->H
                                : nullptr;
  int parts = 0;   // partial rows that this call writes
  if (T > 0) {
    NormArgs a = norm_args(c, T, scale);
    a.resid = resid;
    a.y = post || gated ? y : nullptr;
    a.w_post = w_post;
    a.gate = gate;
    a.w_next = w_next;
    a.dresid = dresid;
    a.dx = static_cast<const uint16_t*>(dx_bf16);
    a.c_rstd_post = rstd_post;
    a.c_rstd_next = rstd_next;
    a.dresid_out = dresid_out;
    a.dy = dy;
    a.dy_f32 = dy_type == MOE_F32;
    a.part_x = part_x;
    a.part_y = part_y;
    MOE_TRY(by_row_length(c->H / 4, [&](auto tpr, auto vpt) {
      constexpr int TPR = decltype(tpr)::value, VPT = decltype(vpt)::value;
      using C = RowCfg<TPR, VPT>;
      return by_types(resid_type, y_type, [&](auto rt, auto yt) {
        using RT = decltype(rt);
        using YT = decltype(yt);
        RowPlan p{norm_backward_blocks<TPR, VPT>(), 0};
        if (norm_staged<VPT>()) {
          a.stage_bytes = C::kRows * c->H * (int)(2 * sizeof(RT) + 2 + (a.y ? sizeof(YT) : 0));
          p = plan_rows(a.stage_bytes, p.blocks);
          a.stages = p.stages;
        }
        const int grid = row_grid<TPR, VPT>(c, T, p.blocks);
        parts = grid * C::kRows;
        return launch(c, -1, st, [&] {
          auto kernel = block_norm_backward_kernel<TPR, VPT, RT, YT, norm_staged<VPT>()>;
          if (a.stages && !ready(c, kernel, kRowRingBytes)) return cudaErrorInvalidConfiguration;
          return launch_pdl(kernel, dim3(grid), dim3(C::kThreads), (size_t)a.stages * a.stage_bytes, st, a);
        });
      });
    }));
  }
  if (!sums) return MOE_OK;
  return launch(c, -1, st, [&] {
    return launch_pdl(block_norm_colsum_kernel, dim3((c->H + 31) / 32, 2), dim3(1024), 0, st,
                      (const float*)part_x, (const float*)part_y, parts, c->H, scale, gate, w_post,
                      dw_next, dw_post, dgate);
  });
}

}  // extern "C"
