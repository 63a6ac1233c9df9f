// Matrix products of block-scaled 8-bit operands:
//   C[m, n] = sum_kb sA[kb, m] sB[kb, n] sum_{k in block kb} A8[m, k] B8[n, k]  (+ bias[n]).
// The sum over a block of 128 is scaled as a whole and added to an fp32 accumulator.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <atomic>
#include <cstring>

#include "gemm_block_pair.cuh"

namespace tpmlp {
namespace {

__device__ __forceinline__ float fp8_value(uint8_t b, int fmt) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, fmt == 0 ? __NV_E4M3 : __NV_E5M2)));
}

// CUDA-core form: a 32 x 128 tile per block of 256 threads; warp w holds rows 4 w .. 4 w + 3, lane l columns
// 4 l .. 4 l + 3, so the 128 columns of a row (one block of the 8-bit output) lie in one warp.
__global__ void __launch_bounds__(256) k_gemm_block_simt(const GemmBlockParams p) {
  __shared__ float sa[32][33];
  __shared__ float sb[128][33];
  const GemmBlockLaunch& g = p.g;
  const int m0 = blockIdx.y * 32, n0 = blockIdx.x * 128;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float acc[4][4] = {}, part[4][4] = {};
  for (int k0 = 0; k0 < g.K; k0 += 32) {
    for (int i = threadIdx.x; i < 32 * 32; i += 256) {
      const int r = i >> 5, k = i & 31;
      sa[r][k] = m0 + r < g.M && k0 + k < g.K ? fp8_value(g.a[static_cast<long long>(m0 + r) * g.K + k0 + k], g.a_fmt) : 0.f;
    }
    for (int i = threadIdx.x; i < 128 * 32; i += 256) {
      const int r = i >> 5, k = i & 31;
      sb[r][k] = n0 + r < g.N && k0 + k < g.K ? fp8_value(g.b[static_cast<long long>(n0 + r) * g.K + k0 + k], g.b_fmt) : 0.f;
    }
    __syncthreads();
    for (int k = 0; k < 32; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[i][j] = fmaf(sa[warp * 4 + i][k], sb[lane * 4 + j][k], part[i][j]);
    __syncthreads();
    if ((k0 & 127) == 96 || k0 + 32 >= g.K) {
      const long long kb = k0 >> 7;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = m0 + warp * 4 + i;
        const float ra = m < g.M ? g.a_scales[kb * p.m_pad + m] : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = n0 + lane * 4 + j;
          const float cb = n >= g.N ? 0.f
                           : g.b_block_rows == 1 ? g.b_scales[kb * p.n_pad + n]
                                                 : g.b_scales[(n >> 7) * static_cast<long long>(p.k_blocks) + kb];
          acc[i][j] = fmaf(ra * cb, part[i][j], acc[i][j]);
          part[i][j] = 0.f;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + warp * 4 + i;
    if (m >= g.M) continue;
    float h[4], amax = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + lane * 4 + j;
      h[j] = 0.f;
      if (n >= g.N) continue;
      float v = acc[i][j];
      if (g.bias != nullptr) v += __bfloat162float(static_cast<const __nv_bfloat16*>(g.bias)[n]);
      if (g.c != nullptr) {
        if (g.c_fp32)
          static_cast<float*>(g.c)[m * g.ldc + n] = v;
        else
          static_cast<__nv_bfloat16*>(g.c)[m * g.ldc + n] = __float2bfloat16_rn(v);
      } else {
        if (g.pre != nullptr) static_cast<__nv_bfloat16*>(g.pre)[static_cast<long long>(m) * g.N + n] = __float2bfloat16_rn(v);
        h[j] = gelu_f(v);
        amax = fmaxf(amax, fabsf(h[j]));
      }
    }
    if (g.hq != nullptr) {
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const BlockScale b = block_scale(amax, 448.f);
      if (n0 + lane * 4 < g.N)
        *reinterpret_cast<uint32_t*>(g.hq + static_cast<long long>(m) * g.N + n0 + lane * 4) = e4m3x4(h[0], h[1], h[2], h[3], b.inv);
      if (lane == 0) g.h_scales[blockIdx.x * p.m_pad + m] = b.scale;
    }
  }
}

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
cudaError_t run_pair(const GemmBlockParams& p, cudaStream_t s) {
  using S = BlockPairShape<BVEC>;
  auto kern = k_gemm_block_pair<OUT, BVEC>;
  static std::atomic<int> cache[64] = {};
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
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

}  // namespace

cudaError_t launch_gemm_block(const GemmBlockLaunch& g, const DeviceCtx& ctx, cudaStream_t s) {
  GemmBlockParams p;
  memset(&p, 0, sizeof(p));
  p.g = g;
  p.m_pad = pad128(g.M);
  p.n_pad = pad128(g.N);
  p.k_blocks = (g.K + kBlock - 1) / kBlock;
  p.err = ctx.err;
  p.timeout_ns = ctx.timeout_ns;
  if (g.M <= 16) {
    const dim3 grid((g.N + 127) / 128, (g.M + 31) / 32);
    k_gemm_block_simt<<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
  }
  p.m_blocks = (g.M + 255) / 256;
  p.n_blocks = (g.N + 255) / 256;
  p.group_m = 8;
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
  if (g.hq != nullptr) return run_pair<kOutGelu8, false>(p, s);  // weights have 128-row tiles
  if (g.b_block_rows == 1) return g.c_fp32 ? run_pair<kOutFp32, true>(p, s) : run_pair<kOutBf16, true>(p, s);
  return g.c_fp32 ? run_pair<kOutFp32, false>(p, s) : run_pair<kOutBf16, false>(p, s);
}

}  // namespace tpmlp
