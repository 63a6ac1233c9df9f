// How many CTAs of a cluster share a tile: as many as the device holds for all tiles at once.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "launch.h"

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

// Stands for a few-row kernel in occupancy queries and is never launched: for a kernel that uses tensor memory the
// query answers one block an SM, while two are resident (their TMEM is half of it each).
__global__ void __launch_bounds__(1024) k_slot() {}

// Clusters of `ranks` (1 to 8) CTAs of a kernel of shape S that the device holds at once.  (Clusters of eight with
// a CTA an SM leave a fifth of the SMs unused: 15 fit, 120 CTAs of 152.)
template <typename S>
int few_clusters(int ranks, const DeviceCtx& ctx) {
  static std::atomic<int> cache[8][64] = {};
  static std::atomic<unsigned long long> set[64] = {};
  if (raise_smem_once(k_slot, 227 * 1024, ctx, set) != cudaSuccess) return 1;
  return max_clusters(k_slot, ranks, S::kSmem, S::kThreads, cache[ranks - 1]);
}

// CTAs that share a tile's k-blocks: as many (a power of two up to max_ranks) as the device holds for all tiles at once,
// which keeps the most bytes in flight, with two k-blocks each at least.
template <typename S>
int few_ranks(long long tiles, int k_blocks, int max_ranks, const DeviceCtx& ctx) {
  int ranks = 1;
  while (ranks < max_ranks && 4 * ranks <= k_blocks && tiles <= few_clusters<S>(2 * ranks, ctx)) ranks *= 2;
  return ranks;
}

// The same, of any number up to max_ranks, for a kernel whose tiles are long: 16 tiles that find no room in clusters of eight
// then take clusters of six, not four.
template <typename S>
int few_ranks_any(long long tiles, int k_blocks, int max_ranks, const DeviceCtx& ctx) {
  int ranks = max_ranks;
  while (ranks > 1 && (2 * ranks > k_blocks || tiles > few_clusters<S>(ranks, ctx))) --ranks;
  return ranks;
}

}  // namespace
}  // namespace tpmlp
