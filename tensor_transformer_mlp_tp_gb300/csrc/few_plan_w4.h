// Split of a product of up to eight tokens with 4-bit weights over blocks and their shared memory (host arithmetic, no CUDA
// types).
#pragma once

namespace tpmlp {

constexpr int kW4Cols = 16, kW4Rows = 64;  // of a tile of codes: 512 bytes

// Two tiles of tokens took 17.3 us for 9 tokens and 21.8 for 16 (K = 4096, N = 16384, groups of 128), the UMMA 15.1 and 15.3
// (14.3 since).
constexpr int kW4FewTokens = 8;
constexpr int kW4FewWarps = 8;    // of a team
constexpr int kW4FewTeams = 2;
constexpr int kW4FewRanks = 4;    // blocks of a cluster at most
constexpr int kW4FewStages = 4;   // copies in flight a team at most
constexpr int kW4FewSmem = 232448;
constexpr int kW4FewSums = kW4FewTokens * kW4Cols;  // of a tile

// Scales and zero points of a warp's part of a chunk, for every row tile or half of one: bytes of a part, of a slot.
constexpr int w4_few_part_bytes(bool zeros) { return zeros ? 48 : 32; }
constexpr int w4_few_slot(bool g32, bool zeros) { return (g32 ? 16 : 8) * w4_few_part_bytes(zeros); }
// Rows of zeros, scales in flight, the tokens' powers of two, barriers.
constexpr int w4_few_fixed(bool g32, bool zeros) {
  return 512 + kW4FewTeams * kW4FewWarps * 4 * w4_few_slot(g32, zeros) + kW4FewWarps * kW4FewTokens * 4 + 256;
}

struct W4FewPlan {
  int ranks, clusters;         // blocks of a cluster; clusters (0: no room for X)
  int chunk, stages, round;    // row tiles a copy; a team's copies in flight; column tiles (of either matrix) between joins
  int x_pitch;                 // bytes of a token's staged row
};

// Blocks of a cluster: the number that leaves the busiest SM the least to read, with room for X, for 64 KB of codes in
// flight (or half of that, if none has room for it), and for two column tiles' sums.  A larger cluster has to save 7% of that
// for its joins (K = 4096, groups of 128, one token; clusters of two that save nothing: 20480 columns 11.7 -> 14.1 us, 24576
// 13.2 -> 15.7).  Clusters of two that read 8% less still lose (12288 columns 10.9 us, single blocks 8.9), so the right share is
// larger; which, was not measured.  fit(r): clusters of r blocks that the device holds at once.
template <typename Fit>
inline W4FewPlan w4_few_plan(int M, int N, int K, int mats, int fixed, Fit fit) {
  W4FewPlan p{};
  const int col_tiles = (N + kW4Cols - 1) / kW4Cols, k_tiles = (K + kW4Rows - 1) / kW4Rows;
  double least = 0;
  for (int ring_least = 65536; ring_least >= 32768 && p.clusters == 0; ring_least /= 2)
    for (int r = 1; r <= kW4FewRanks && k_tiles >= r; r *= 2) {
      const int fits = fit(r);
      const double load = static_cast<double>((col_tiles + fits - 1) / fits) / r;
      const int mine = (k_tiles + r - 1) / r;
      constexpr int tile_bytes = kW4FewWarps * kW4FewSums * 4;
      // (K / 64 row tiles of 128 bytes can pass 32 bits: what has no room is refused before anything is narrowed)
      const long long x_pitch = mine * 128ll + 16, left = kW4FewSmem - fixed - M * x_pitch;
      if (left < ring_least + 2 * tile_bytes || (p.clusters != 0 && load > 0.93 * least)) continue;
      least = load;
      p.ranks = r;
      p.clusters = fits < col_tiles ? fits : col_tiles;
      p.x_pitch = static_cast<int>(x_pitch);
      // a round is all of the cluster's tiles, or as many as leave the ring its part
      const int most = static_cast<int>((left - ring_least) / tile_bytes) / 2 * 2;
      const int all = (col_tiles + p.clusters - 1) / p.clusters * mats;
      p.round = all < most ? all : most;
      const int ring = static_cast<int>(left) - p.round * tile_bytes;
      p.chunk = mine < 64 ? mine : 64;
      while (p.chunk > 16 && ring / (kW4FewTeams * (p.chunk * 512 + 16)) < 2) p.chunk /= 2;
      p.stages = ring / (kW4FewTeams * (p.chunk * 512 + 16));
      if (p.stages > kW4FewStages) p.stages = kW4FewStages;
    }
  return p;
}

}  // namespace tpmlp
