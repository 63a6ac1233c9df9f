// Host side of the few-row bf16 products.
#include "gemm_few.cuh"

#include <atomic>
#include <cstring>

#include "cluster_fit.cuh"

namespace tpmlp {
namespace {

template <int BT, int MATS>
cudaError_t run_few(GemmFewParams& p, const GemmFewLaunch& g, const DeviceCtx& ctx, cudaStream_t s) {
  using S = GemmFewShape<BT, MATS>;
  auto kern = k_gemm_few<BT, MATS>;
  static std::atomic<unsigned long long> set[64] = {};
  const cudaError_t e = raise_smem_once(kern, S::kSmem, ctx, set);
  if (e != cudaSuccess) return e;
  p.box_rows = g.M;  // copies of the rows there are: zero rows behind them would cost more than real ones
  bool ok = encode_tile_map(&p.tmX, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, g.x, g.K, g.M, g.K, kBK, p.box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
  for (int i = 0; i < MATS; ++i)
    ok = ok && encode_tile_map(&p.tmW[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, g.w[i], g.N, g.K, g.N, 64, kBK, CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok) return cudaErrorInvalidValue;
  const int tiles = (g.N + kFewCols - 1) / kFewCols;
  const int ranks = few_ranks<S>(tiles, p.k_blocks, kFewRanks, ctx);
  p.ranks = ranks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks * tiles);
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = ranks;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = ranks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int MATS>
cudaError_t launch(const GemmFewLaunch& g, const DeviceCtx& ctx, cudaStream_t s) {
  GemmFewParams p;
  memset(&p, 0, sizeof(p));
  p.M = g.M;
  p.N = g.N;
  p.k_blocks = (g.K + kBK - 1) / kBK;
  p.act = g.act;
  p.early_weights = g.early_weights ? 1 : 0;
  p.out = g.out;
  for (int i = 0; i < 2; ++i) {
    p.bias[i] = g.bias[i];
    p.pre[i] = g.pre[i];
  }
  p.err = ctx.err;
  p.timeout_ns = ctx.timeout_ns;
  return g.M <= 16   ? run_few<16, MATS>(p, g, ctx, s)
         : g.M <= 32 ? run_few<32, MATS>(p, g, ctx, s)
         : g.M <= 64 ? run_few<64, MATS>(p, g, ctx, s)
                     : run_few<128, MATS>(p, g, ctx, s);
}

}  // namespace

cudaError_t gemm_few_bounds_status(unsigned int* count, unsigned int* site) {
#ifdef TPMLP_DEBUG_BOUNDS
  return bounds_read_and_clear(count, site);
#else
  *count = *site = 0;
  return cudaSuccess;
#endif
}

cudaError_t launch_gemm_few(const GemmFewLaunch& g, const DeviceCtx& ctx, cudaStream_t s) {
  if (g.M < 1 || g.M > kFewRows || g.K < 1) return cudaErrorInvalidValue;
  return g.w[1] != nullptr ? launch<2>(g, ctx, s) : launch<1>(g, ctx, s);
}

}  // namespace tpmlp
