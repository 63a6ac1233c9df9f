// Matrix products of block-scaled 8-bit operands:
//   C[m, n] = sum_kb sA[kb, m] sB[kb, n] sum_{k in block kb} A8[m, k] B8[n, k]  (+ bias[n]).
// The sum over a block of 128 is scaled as a whole and added to an fp32 accumulator.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <atomic>
#include <climits>
#include <cstring>

#include "gemm_block_few.cuh"

namespace tpmlp {
namespace {

// Largest number of co-resident clusters of `kern` on the current device (cached per device).
template <typename K>
int max_clusters(K kern, int cluster, int smem, int threads, std::atomic<int>* cache) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  const int known = cache[dev & 63].load(std::memory_order_relaxed);
  if (known > 0) return known;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) n = 1;
  cache[dev & 63].store(n, std::memory_order_relaxed);
  return n;
}

template <int OUT, bool BVEC>
cudaError_t run_pair(const GemmBlockParams& p, const DeviceCtx& ctx, cudaStream_t s) {
  using S = BlockPairShape<BVEC>;
  auto kern = k_gemm_block_pair<OUT, BVEC>;
  static std::atomic<int> cache[64] = {};
  static std::atomic<unsigned long long> set[64] = {};
  const cudaError_t e = raise_smem_once(kern, S::kSmem, ctx, set);
  if (e != cudaSuccess) return e;
  const int pairs = max_clusters(kern, 2, S::kSmem, S::kThreads, cache);
  const int tiles = p.m_blocks * p.n_blocks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (tiles < pairs ? tiles : pairs));
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// Stands for the few-row kernel in occupancy queries and is never launched: for a kernel that uses tensor memory the
// query answers one block an SM, while two are resident (their TMEM is half of it each).
__global__ void __launch_bounds__(320) k_slot() {}

// Clusters of `ranks` CTAs of the BT kernel that the device holds at once.  (Clusters of eight with a CTA an SM leave a
// fifth of the SMs unused: 15 fit, 120 CTAs of 152.)
template <int BT>
int few_clusters(int ranks, const DeviceCtx& ctx) {
  using S = BlockFewShape<BT, true>;  // the larger of the two
  static std::atomic<int> cache[4][64] = {};
  static std::atomic<unsigned long long> set[64] = {};
  if (raise_smem_once(k_slot, 227 * 1024, ctx, set) != cudaSuccess) return 1;
  const int slot = ranks == 1 ? 0 : ranks == 2 ? 1 : ranks == 4 ? 2 : 3;
  return max_clusters(k_slot, ranks, S::kSmem, S::kThreads, cache[slot]);
}

// CTAs that share a tile's k-blocks: as many (a power of two up to 8) as the device holds for all tiles at once, which
// keeps the most bytes in flight, with two k-blocks each at least.
template <int BT>
int few_ranks(long long tiles, int k_blocks, const DeviceCtx& ctx) {
  int ranks = 1;
  while (ranks < kFewMaxRanks && 4 * ranks <= k_blocks && tiles <= few_clusters<BT>(2 * ranks, ctx)) ranks *= 2;
  return ranks;
}

// Which kernel: up to 128 rows the one that streams B once.  Above, whichever has fewer k-blocks one after the other, and
// at as many the same: a pair's k-block (256 x 256) takes about 0.41 us (0.65 with column scales) and a 128 x 128 one 0.37
// (0.41), measured on GB300 with tiles for a single wave (M = 256, N = 8192, K = 8192: 30.2 us on pairs, 27.1 with this rule;
// with column scales 45.3 and 30.2.  M = 300, N = 4096, K = 4096: 17.0 and 15.2 us.  M = 640: 17.3 us on pairs, 29.1 in two
// waves of the other).  The counts alone are compared: where three waves of the small kernel with column scales (1.23 us a
// k-block) meet two of pairs (1.30), pairs are taken.
bool few_rows(const GemmBlockLaunch& g, int k_blocks, const DeviceCtx& ctx) {
  const int sms = ctx.sm_count;
  if (g.M <= 128) return true;
  const long long few_tiles = static_cast<long long>((g.M + 127) / 128) * ((g.N + 127) / 128);
  if (few_tiles > 4ll * sms) return false;
  const long long ranks = few_ranks<128>(few_tiles, k_blocks, ctx);
  const long long few = (few_tiles * ranks + sms - 1) / sms * ((k_blocks + ranks - 1) / ranks);
  const long long pairs = sms / 2, pair_tiles = static_cast<long long>((g.M + 255) / 256) * ((g.N + 255) / 256);
  const long long pair = (pair_tiles + pairs - 1) / pairs * k_blocks;
  return few <= pair;
}

template <int BT, int OUT, bool BVEC>
cudaError_t run_few(GemmBlockParams p, const DeviceCtx& ctx, cudaStream_t s) {
  using S = BlockFewShape<BT, BVEC>;
  auto kern = k_gemm_block_few<BT, OUT, BVEC>;
  static std::atomic<unsigned long long> set[64] = {};
  const cudaError_t e = raise_smem_once(kern, S::kSmem, ctx, set);
  if (e != cudaSuccess) return e;
  const int tiles = (p.g.N + 127) / 128, row_tiles = (p.g.M + BT - 1) / BT;
  const int ranks = few_ranks<BT>(static_cast<long long>(tiles) * row_tiles, p.k_blocks, ctx);
  p.ranks = ranks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks * tiles, row_tiles);
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

template <int BT>
cudaError_t launch_few(GemmBlockParams& p, const DeviceCtx& ctx, cudaStream_t s) {
  const GemmBlockLaunch& g = p.g;
  p.box_rows = g.M < BT ? g.M : BT;
  bool ok = encode_tile_map(&p.tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.a, g.K, g.M, g.K, 128, p.box_rows, CU_TENSOR_MAP_SWIZZLE_128B) &&
            encode_tile_map(&p.tmB, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.b, g.K, g.N, g.K, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) &&
            encode_tile_map(&p.tmSA, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, g.a_scales, p.m_pad, p.k_blocks, p.m_pad, BT, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (g.b_block_rows == 1)
    ok = ok && encode_tile_map(&p.tmSB, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, g.b_scales, p.n_pad, p.k_blocks, p.n_pad, 128, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (!ok) return cudaErrorInvalidValue;
  if (g.hq != nullptr) return run_few<BT, kOutGelu8, false>(p, ctx, s);  // weights have 128-row tiles
  if (g.b_block_rows == 1) return g.c_fp32 ? run_few<BT, kOutFp32, true>(p, ctx, s) : run_few<BT, kOutBf16, true>(p, ctx, s);
  return g.c_fp32 ? run_few<BT, kOutFp32, false>(p, ctx, s) : run_few<BT, kOutBf16, false>(p, ctx, s);
}

}  // namespace

cudaError_t gemm_block_bounds_status(unsigned int* count, unsigned int* site) {
#ifdef TPMLP_DEBUG_BOUNDS
  return bounds_read_and_clear(count, site);
#else
  *count = *site = 0;
  return cudaSuccess;
#endif
}

cudaError_t launch_gemm_block(const GemmBlockLaunch& g, const DeviceCtx& ctx, cudaStream_t s) {
  GemmBlockParams p;
  memset(&p, 0, sizeof(p));
  p.g = g;
  p.m_pad = pad128(g.M);
  p.n_pad = pad128(g.N);
  p.k_blocks = (g.K + kBlock - 1) / kBlock;
  p.err = ctx.err;
  p.timeout_ns = ctx.timeout_ns;
  if (few_rows(g, p.k_blocks, ctx))
    // the narrowest tile that holds the rows: sixteen columns more are about 0.5 us (40 rows, N = 16384, K = 4096: 15.6 us
    // in 48 columns, 16.3 in 64)
    return g.M <= 16   ? launch_few<16>(p, ctx, s)
           : g.M <= 32 ? launch_few<32>(p, ctx, s)
           : g.M <= 48 ? launch_few<48>(p, ctx, s)
           : g.M <= 64 ? launch_few<64>(p, ctx, s)
                       : launch_few<128>(p, ctx, s);
  if (static_cast<long long>((g.M + 255) / 256) * ((g.N + 255) / 256) > INT_MAX) return cudaErrorNotSupported;
  p.m_blocks = (g.M + 255) / 256;
  p.n_blocks = (g.N + 255) / 256;
  // the factor of a division by d for dividends below 2^31: floor(2^32 (2^s - d) / d) + 1 with 2^s >= d
  const unsigned long long d = static_cast<unsigned long long>(kGroupM) * p.n_blocks;
  while ((1ull << p.group_shift) < d) ++p.group_shift;
  p.group_factor = static_cast<uint32_t>((((1ull << p.group_shift) - d) << 32) / d + 1);
  bool ok = encode_tile_map(&p.tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.a, g.K, g.M, g.K, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) &&
            encode_tile_map(&p.tmB, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.b, g.K, g.N, g.K, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  ok = ok && encode_tile_map(&p.tmSA, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, g.a_scales, p.m_pad, p.k_blocks, p.m_pad, 128, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (g.b_block_rows == 1)
    ok = ok && encode_tile_map(&p.tmSB, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, g.b_scales, p.n_pad, p.k_blocks, p.n_pad, 256, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (g.c != nullptr && g.c_fp32)
    ok = ok && encode_tile_map(&p.tmC, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, g.c, g.N, g.M, g.ldc, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B);
  else if (g.c != nullptr)
    ok = ok && encode_tile_map(&p.tmC, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, g.c, g.N, g.M, g.ldc, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  if (g.pre != nullptr)
    ok = ok && encode_tile_map(&p.tmC, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, g.pre, g.N, g.M, g.N, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  if (g.hq != nullptr)
    ok = ok && encode_tile_map(&p.tmH, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.hq, g.N, g.M, g.N, 128, 32, CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok) return cudaErrorInvalidValue;
  if (g.hq != nullptr) return run_pair<kOutGelu8, false>(p, ctx, s);  // weights have 128-row tiles
  if (g.b_block_rows == 1) return g.c_fp32 ? run_pair<kOutFp32, true>(p, ctx, s) : run_pair<kOutBf16, true>(p, ctx, s);
  return g.c_fp32 ? run_pair<kOutFp32, false>(p, ctx, s) : run_pair<kOutBf16, false>(p, ctx, s);
}

}  // namespace tpmlp
