// Products with 4-bit weights and group scales, their quantiser and its inverse.
#include <cuda_bf16.h>

#include <atomic>
#include <climits>
#include <cstring>

#include "cluster_fit.cuh"
#include "debug_bounds.cuh"
#include "gated.cuh"
#include "w4_tc.cuh"

namespace tpmlp {
namespace {

constexpr float kW4Tiny = 7.8886090522101181e-31f;  // 2^-100, the least range a scale is made from
constexpr float kW4Big = 3.3895313892515355e38f;    // bf16's largest number, the largest

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// Up to eight tokens, the m16n8k16 product's columns.  One block an SM, blocks in clusters of `ranks`; a cluster takes
// every so many-th column tile (both matrices of the gated form), its blocks share K, and eight warps share a block's part
// of it; two such teams take turns with the tiles.  One lane of a warp of its own streams the
// codes of one tile after the other into a ring by bulk copies of up to 32 KB, so that the bytes in flight cost neither
// registers nor instructions.  What a weight costs is its unpacking, nine instructions for eight codes.
//
// The products are of fp16 numbers, for the unpacking's sake.  q - z is exact; what a warp reads of a token is brought
// below 2^15 by a power of two, which loses nothing of a value within 2^-32 of the largest there.  A group's sum in fp32 is
// brought back by that power before its scale, as far as the token's values are below one, and behind the warps' sums as far as
// they are above: a scaled sum is no larger than the part of the result that it stands for, so that scales near the largest
// number overflow where the result does.  (One token of 4096 x 16384 9.8 us for 9.8 without that step, gated 15.9 for 15.7,
// K = 16384 with zero points 14.3 for 14.1; in single fp32 instructions instead of pairs 9.9, 16.2, 14.2.)
//
// X is staged once, so that a lane's B registers of a 64-row tile are 32 consecutive bytes, the rows a multiple of 128
// bytes and 16 apart (conflict-free); lanes past the last token read a row of zeros.  The sums of a round of tiles are joined
// in a fixed order, the warps' and then the blocks'.
//
// Measured (groups of 128): one token of 4096 x 16384 9.8 us (3.5 TB/s; 7.0 without the products), 8 tokens 14.4; both
// matrices of the gated form 15.9 (4.4 TB/s; 11.8 without).  Bound by a tile's instructions and the start: 90 warp instructions
// for 64 rows of 16 columns, 36 of which unpack (the others scale, load X, multiply, wait and fetch), issue 53% of the cycles
// in which an SM has the block, 36% of all under ncu; with more columns, where the start counts less, 64% (N = 65536).  Not kept:
// pairs of column tiles that read X once and share a group's scales (10.0 us for one token, 15.6 for 8: fewer warps wait for each
// copy).
constexpr int kWarps = kW4FewWarps;

struct W4FewParams : W4FewPlan {
  W4Launch g;
  int shift;                   // log2 of the group
  unsigned int* err;
  unsigned long long timeout_ns;
};

template <bool G32, bool ZEROS>
struct W4FewShape {
  static constexpr int kTeams = kW4FewTeams;
  static constexpr int kConsumers = 32 * kTeams * kWarps, kThreads = kConsumers + 32;
  static constexpr int kSums = kW4FewSums;
  static constexpr int kParts = G32 ? 16 : 8, kPartBytes = w4_few_part_bytes(ZEROS), kSlot = w4_few_slot(G32, ZEROS);
  static constexpr int kFixed = w4_few_fixed(G32, ZEROS);
  static constexpr int kSmem = kW4FewSmem;
};

// Row m, column col of the output from the sums (equal for a plain product).
template <int MATS>
__device__ __forceinline__ void w4_finish(const W4Launch& g, int m, int col, float first, float last) {
  if (!TPMLP_IN_BOUNDS(static_cast<long long>(m) * g.N + col, static_cast<long long>(g.M) * g.N, kBoundsW4Out)) return;
  float v[2] = {first, last};
#pragma unroll
  for (int k = 0; k < MATS; ++k)
    if (g.w[k].bias != nullptr) v[k] += __bfloat162float(static_cast<const __nv_bfloat16*>(g.w[k].bias)[col]);
  if (MATS == 2) v[0] = act2(g.act, make_float2(v[0], v[0])).x * v[1];
  static_cast<__nv_bfloat16*>(g.y)[static_cast<long long>(m) * g.N + col] = __float2bfloat16_rn(v[0]);
}

template <int THREADS>
__device__ __forceinline__ void consumers_sync() {
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// Two bf16 of X times f, in fp16.
__device__ __forceinline__ uint32_t x_half2(uint32_t pair, float f) {
  const float2 v = unpack_bf16x2(pair);
  const __half2 h = __floats2half2_rn(v.x * f, v.y * f);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int MATS, bool G32, bool ZEROS>
__global__ void __launch_bounds__(W4FewShape<G32, ZEROS>::kThreads, 1) k_gemm_w4_few(const __grid_constant__ W4FewParams p) {
  using S = W4FewShape<G32, ZEROS>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int M = p.g.M, N = p.g.N, K = p.g.K, ranks = p.ranks;
  const int rank = ranks > 1 ? static_cast<int>(cluster_ctarank()) : 0, cluster = static_cast<int>(blockIdx.x) / ranks;
  const int k_tiles = (K + kW4Rows - 1) / kW4Rows;
  const int kt_a = static_cast<int>(static_cast<long long>(k_tiles) * rank / ranks);
  const int kt_n = static_cast<int>(static_cast<long long>(k_tiles) * (rank + 1) / ranks) - kt_a;
  const int chunks = (kt_n + p.chunk - 1) / p.chunk;  // of a column tile
  const int tiles = ((N + kW4Cols - 1) / kW4Cols - cluster + p.clusters - 1) / p.clusters * MATS;

  uint8_t* ring = smem;
  float* red = reinterpret_cast<float*>(ring + S::kTeams * p.stages * p.chunk * 512);  // [tile of the round][warp][token][column]
  uint8_t* zero_row = reinterpret_cast<uint8_t*>(red + p.round * kWarps * S::kSums);
  uint8_t* slot_mem = zero_row + 512;  // [warp][slot]
  uint8_t* sx = slot_mem + S::kTeams * kWarps * 4 * S::kSlot;
  float* tok = reinterpret_cast<float*>(sx + M * p.x_pitch);  // [warp][token]: the power of two to take back
  uint64_t* full = reinterpret_cast<uint64_t*>(tok + kWarps * kW4FewTokens);
  uint64_t* empty = full + S::kTeams * p.stages;
  int* abort_flag = reinterpret_cast<int*>(empty + S::kTeams * p.stages);
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kTeams * p.stages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, kWarps);
    }
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  const WaitCtx wc{abort_flag, p.err, p.timeout_ns};
  griddep_wait();
  griddep_launch_dependents();

  if (warp == S::kTeams * kWarps) {
    // Each team has a ring of its own: a wait tells a phase from the one before it only, and a team that skipped the other's
    // would miss some.
    int stage[S::kTeams] = {};
    uint32_t phase[S::kTeams] = {}, issued = 0, issued_parity = 0;
    bool ok = true;
    for (int round0 = 0; round0 < tiles; round0 += p.round) {
      if (lane == 0) {
        for (int tile0 = round0; ok && tile0 < min(tiles, round0 + p.round); tile0 += S::kTeams)
          for (int c = 0; ok && c < chunks; ++c) {
            const uint32_t bytes = static_cast<uint32_t>(min(p.chunk, kt_n - c * p.chunk)) * 512u;
#pragma unroll
            for (int of = 0; of < S::kTeams; ++of) {
              const int tile = tile0 + of, i = of * p.stages + stage[of];
              if (tile >= tiles) break;
              const uint4* src = p.g.w[MATS == 1 ? 0 : tile & 1].q +
                                 ((cluster + static_cast<long long>(tile / MATS) * p.clusters) * k_tiles + kt_a + c * p.chunk) * 32;
              if (!wait_bounded(empty + i, phase[of] ^ 1u, wc, kSiteW4Producer)) {
                ok = false;
                break;
              }
              mbar_arrive_expect_tx(full + i, bytes);
              bulk_load(ring + i * p.chunk * 512, src, bytes, full + i);
              issued |= 1u << i;
              issued_parity = (issued_parity & ~(1u << i)) | (phase[of] << i);
              if (++stage[of] == p.stages) {
                stage[of] = 0;
                phase[of] ^= 1u;
              }
            }
          }
      }
      __syncwarp();
      if (ranks > 1) {
        cluster_sync_all();
        cluster_sync_all();
      }
    }
    if (lane == 0)  // copies in flight land before the block's shared memory is released
      for (int i = 0; i < S::kTeams * p.stages; ++i)
        if (issued & (1u << i)) wait_drain(full + i, (issued_parity >> i) & 1u, p.timeout_ns);
    return;
  }

  const int team = warp / kWarps, w = warp % kWarps;  // this warp takes the team's tiles, part w of each chunk
  // A warp fetches the scales and zero points of what it reads of a chunk (eight row tiles at most) three chunks ahead into
  // slots of its own, eight columns a lane.
  uint8_t* slots = slot_mem + warp * 4 * S::kSlot;
  int f_tile = team, f_chunk = 0, f_slot = 0, f_col = (cluster + team / MATS * p.clusters) * kW4Cols + 8 * (lane & 1);
  long long f_row = 0;  // of scales, times N
  auto fetch = [&]() {
    if (f_tile < tiles && lane < 2 * S::kParts) {
      if (f_tile < S::kTeams || chunks > 1) {
        const int n = min(p.chunk, kt_n - f_chunk * p.chunk), w0 = n * w / kWarps;
        const int row = (kt_a + f_chunk * p.chunk + w0) * kW4Rows + (G32 ? 32 : 64) * (lane >> 1);
        f_row = static_cast<long long>(min(row, K - 1) >> p.shift) * N;
      }
      const W4Matrix& mat = p.g.w[MATS == 1 ? 0 : f_tile & 1];
      const bool in = f_col < N;
      const long long at = f_row + (in ? f_col : 0);
      uint8_t* dst = slots + f_slot * S::kSlot + (lane >> 1) * S::kPartBytes;
      cp_async<16>(dst + 16 * (lane & 1), static_cast<const __nv_bfloat16*>(mat.scales) + at, in ? 16 : 0);
      if (ZEROS) cp_async<8>(dst + 32 + 8 * (lane & 1), mat.zeros + at, in ? 8 : 0);
    }
    cp_async_commit();
    f_slot = (f_slot + 1) & 3;
    if (++f_chunk == chunks) {
      f_chunk = 0;
      f_tile += S::kTeams;
      f_col += S::kTeams / MATS * p.clusters * kW4Cols;
    }
  };

  // X: part w of every chunk (eight row tiles at most, 32 bytes a lane) of the team's tokens, as it is, then each token
  // scaled by its largest value there and turned into the products' order.
  const __nv_bfloat16* xg = static_cast<const __nv_bfloat16*>(p.g.x);
  auto part_of = [&](int c, int& first, int& pieces) {  // of chunk c: its first row tile in the block's part, 16-byte pieces
    const int n = min(p.chunk, kt_n - c * p.chunk), w0 = n * w / kWarps;
    first = c * p.chunk + w0;
    pieces = (n * (w + 1) / kWarps - w0) * 8;
  };
  for (int c = 0; c < chunks; ++c) {
    int first, pieces;
    part_of(c, first, pieces);
    for (int m = team; m < M; m += S::kTeams)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int piece = lane + 32 * h, k = (kt_a + first) * kW4Rows + piece * 8;
        if (piece < pieces)
          cp_async<16>(sx + m * p.x_pitch + first * 128 + piece * 16, xg + static_cast<long long>(m) * K + (k < K ? k : 0), k < K ? 16 : 0);
      }
  }
  cp_async_commit();
#pragma unroll
  for (int i = 0; i < 3; ++i) fetch();
  if (threadIdx.x < 32) reinterpret_cast<uint4*>(zero_row)[threadIdx.x] = make_uint4(0, 0, 0, 0);
  cp_async_wait<3>();
  __syncwarp();
  for (int m = team; m < M; m += S::kTeams) {
    uint8_t* row = sx + m * p.x_pitch;
    uint32_t largest = 0;  // bits of bf16 without the sign
    for (int c = 0; c < chunks; ++c) {
      int first, pieces;
      part_of(c, first, pieces);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (lane + 32 * h < pieces) {
          const uint4 v = reinterpret_cast<const uint4*>(row + first * 128)[lane + 32 * h];
          largest = __vmaxu2(__vmaxu2(largest, __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu)),
                             __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
        }
    }
    largest = __reduce_max_sync(0xffffffffu, max(largest >> 16, largest & 0xFFFFu));
    // its exponent e (infinities and NaN count as the largest finite values); 2^(14 - e), and 2^(e + 1) back
    const int e = min(max(static_cast<int>(largest >> 7) - 127, -112), 126);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
    if (lane == 0) tok[w * kW4FewTokens + m] = __uint_as_float(static_cast<uint32_t>(127 + e + 1) << 23);
    for (int c = 0; c < chunks; ++c) {
      int first, pieces;
      part_of(c, first, pieces);
      uint4 v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (lane + 32 * h < pieces) v[h] = reinterpret_cast<const uint4*>(row + first * 128)[lane + 32 * h];
      __syncwarp();
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (lane + 32 * h < pieces) {
          uint32_t* dst = reinterpret_cast<uint32_t*>(row + (first + 4 * h + (lane >> 3)) * 128) + (lane & 7);
          dst[0] = x_half2(v[h].x, up);
          dst[8] = x_half2(v[h].y, up);
          dst[16] = x_half2(v[h].z, up);
          dst[24] = x_half2(v[h].w, up);
        }
    }
  }
  // this lane's token: its row, or the zeros, which do not advance
  const uint8_t* x_row = g < M ? sx + g * p.x_pitch + t * 32 : zero_row + t * 32;
  const int x_step = g < M ? 128 : 0;
  consumers_sync<S::kConsumers>();  // both teams' tokens
  // what this lane's two tokens' sums are multiplied with before a scale; the second eight columns' codes come out sixteen times
  // as large (subnormal below 2^-107, where it is still exact)
  const float* tok2 = tok + w * kW4FewTokens + 2 * t;
  const float2 back = make_float2(2 * t < M ? fminf(tok2[0], 1.f) * 0x1p-15f : 0.f, 2 * t + 1 < M ? fminf(tok2[1], 1.f) * 0x1p-15f : 0.f);
  const float2 back16 = make_float2(back.x * 0x1p-4f, back.y * 0x1p-4f);
  int stage = team * p.stages, slot = 0;
  uint32_t phase = 0;
  for (int round0 = 0; round0 < tiles; round0 += p.round) {
    const int nt = min(p.round, tiles - round0);
    float* dst = red + (team * kWarps + w) * S::kSums + 2 * t * 16 + g;
    for (int tile = team; tile < nt; tile += S::kTeams, dst += S::kTeams * kWarps * S::kSums) {
      float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;  // columns g, g + 8 of both tokens
      for (int c = 0; c < chunks; ++c) {
        int first, pieces;
        part_of(c, first, pieces);
        cp_async_wait<2>();
        __syncwarp();  // this chunk's scales are there for all lanes, and the slot before has been read
        const uint8_t* sl = slots + slot * S::kSlot;
        slot = (slot + 1) & 3;
        fetch();
        (void)warp_wait(full + stage, phase, wc, kSiteW4Consumer);
        const uint4* src = reinterpret_cast<const uint4*>(ring + (stage * p.chunk + first - c * p.chunk) * 512) + lane;
        const uint8_t* xs = x_row + first * x_step;
#pragma unroll 4
        for (int i = 0; i < pieces; i += 8, src += 32, xs += x_step) {
          const uint4 q4 = *src;
          const uint32_t q[4] = {q4.x, q4.y, q4.z, q4.w};
          const uint4 b4[2] = {reinterpret_cast<const uint4*>(xs)[0], reinterpret_cast<const uint4*>(xs)[1]};
          constexpr int kSteps = G32 ? 2 : 4;  // of 16 rows, with one scale
#pragma unroll
          for (int j0 = 0; j0 < 4; j0 += kSteps, sl += S::kPartBytes) {
            const float s0 = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(sl)[g]);
            const float s1 = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(sl)[g + 8]);
            const uint32_t z0 = w4_base0(ZEROS ? sl[32 + g] & 15u : 8u), z1 = w4_base1(ZEROS ? sl[40 + g] & 15u : 8u);
            float c4[4] = {};
#pragma unroll
            for (int j = j0; j < j0 + kSteps; ++j) {
              uint32_t a[4];
              w4_unpack(q[j], z0, z1, a);
              const uint4 v = b4[j >> 1];
              const uint32_t b[2] = {j & 1 ? v.z : v.x, j & 1 ? v.w : v.y};
              mma_16816(c4, a, b);
            }
            sum0 = __ffma2_rn(__fmul2_rn(make_float2(c4[0], c4[1]), back), make_float2(s0, s0), sum0);
            sum1 = __ffma2_rn(__fmul2_rn(make_float2(c4[2], c4[3]), back16), make_float2(s1, s1), sum1);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + stage);
        if (++stage == (team + 1) * p.stages) {
          stage = team * p.stages;
          phase ^= 1u;
        }
      }
      dst[0] = sum0.x;
      dst[16] = sum0.y;
      dst[8] = sum1.x;
      dst[24] = sum1.y;
    }
    consumers_sync<S::kConsumers>();
    // the block's sums of tile i (column tile c, matrix k), token m, column n; ranks > 1: into the first warp's place
    for (int c = threadIdx.x; c < nt * M * 16; c += S::kConsumers) {
      const int tile = c / (M * 16), r = c - tile * M * 16, m = r >> 4;
      if (MATS == 2 && ranks == 1 && (tile & 1)) continue;
      float v[MATS];
#pragma unroll
      for (int k = 0; k < MATS; ++k) {
        if (k > 0 && ranks > 1) break;
        const float* at = red + (tile + k) * kWarps * S::kSums + r;
        v[k] = 0.f;
#pragma unroll
        for (int o = 0; o < kWarps; ++o) v[k] = fmaf(at[o * S::kSums], fmaxf(tok[o * kW4FewTokens + m], 1.f), v[k]);
      }
      if (ranks > 1) {
        red[tile * kWarps * S::kSums + r] = v[0];
      } else {
        const int col = (cluster + (round0 + tile) / MATS * p.clusters) * kW4Cols + (r & 15);
        if (col < N) w4_finish<MATS>(p.g, m, col, v[0], v[MATS - 1]);
      }
    }
    __syncwarp();
    if (ranks > 1) {
      cluster_sync_all();
      for (int c = threadIdx.x; c < nt / MATS * M * 16; c += S::kConsumers) {
        const int i = c / (M * 16), r = c - i * M * 16, m = r >> 4;
        const int col = (cluster + (round0 / MATS + i) * p.clusters) * kW4Cols + (r & 15);
        if ((i + m) % ranks != rank || col >= N) continue;
        float v[MATS];
#pragma unroll
        for (int k = 0; k < MATS; ++k) {
          v[k] = 0.f;
          const uint32_t at = smem_u32(red + (i * MATS + k) * kWarps * S::kSums + r);
          for (int o = 0; o < ranks; ++o) v[k] += ld_cluster_f1(mapa_shared(at, static_cast<uint32_t>(o)));
        }
        w4_finish<MATS>(p.g, m, col, v[0], v[MATS - 1]);
      }
      __syncwarp();
      cluster_sync_all();  // the cluster has read this block's sums
    } else {
      consumers_sync<S::kConsumers>();  // the next round overwrites this one's scales and sums
    }
  }
}

template <int MATS, bool G32, bool ZEROS>
cudaError_t run_w4_few(const W4Launch& g, const DeviceCtx& ctx, cudaStream_t s) {
  using S = W4FewShape<G32, ZEROS>;
  auto kern = k_gemm_w4_few<MATS, G32, ZEROS>;
  static std::atomic<unsigned long long> set[64] = {};
  const cudaError_t e = raise_smem_once(kern, S::kSmem, ctx, set);
  if (e != cudaSuccess) return e;
  W4FewParams p{};
  static std::atomic<int> cache[3][64] = {};
  static_cast<W4FewPlan&>(p) = w4_few_plan(g.M, g.N, g.K, MATS, S::kFixed, [&](int r) {
    return r == 1 ? ctx.sm_count : max_clusters(kern, r, S::kSmem, S::kThreads, cache[r / 2]);
  });
  p.g = g;
  p.shift = g.group == 32 ? 5 : g.group == 64 ? 6 : 7;
  p.err = ctx.err;
  p.timeout_ns = ctx.timeout_ns;
  if (p.clusters == 0) return cudaErrorNotSupported;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.ranks * p.clusters);
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = p.ranks;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.ranks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int MATS>
cudaError_t launch_w4_few(const W4Launch& g, const DeviceCtx& ctx, cudaStream_t s) {
  const bool z = g.w[0].zeros != nullptr;
  if (g.group == 32) return z ? run_w4_few<MATS, true, true>(g, ctx, s) : run_w4_few<MATS, true, false>(g, ctx, s);
  return z ? run_w4_few<MATS, false, true>(g, ctx, s) : run_w4_few<MATS, false, false>(g, ctx, s);
}

// 16 bytes that are read once.
__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// The quantiser and its inverse: a block takes 128 rows x 64 columns, a whole number of groups and 4 x 2 tiles, through
// shared memory, rows there 34 words apart: the threads of a tile, which read columns g and rows 2 t, then hit 16 banks.
// Measured, 4096 x 16384 with groups of 128, both ways: 62.9 us for 337 MB (5.4 TB/s); straight from global memory, where a
// tile's reads are 16 bytes of each of 64 rows, 398.  The quantiser is bound by its phases (load, extremes, scales, codes): issue
// 73%, the ALU 59%; eight blocks an SM (32 registers) keep more of them apart: six took 64.2, 71.5 for 63.6 with zero points.
constexpr int kPackRows = 128, kPackCols = 64, kPackPitch = 68;  // elements

// Largest and smallest of every column: four rows a thread as they are loaded, 16 by shuffles, a group's by the thread that
// makes its scale; then a tile's words, a lane's 16 bytes a thread.  A code's quotient is w (1 / s), off by less than 2^-19;
// a quotient of two bf16 numbers is half of an odd number or at least 1/1020 away from one, so that rounding it to multiples
// of 2^-10 first gives the division's code.  Without infinities it is within +-16, so that codes are made in pairs of rows:
// packed fp32, then 16-bit halves.  (A block with an infinity brings quotients to +-16 first.)
template <bool INFINITE, bool ZEROS>
__device__ __forceinline__ void quantize_words(const __nv_bfloat16* tile, const float (&s_inv)[4][kPackCols],
                                               const uint32_t (&s_zero)[4][kPackCols], int kt, int ct, int g, int t, int shift,
                                               uint32_t (&words)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int grp = (kt * kW4Rows + 16 * j) >> shift;
    uint32_t word = 0;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int n = ct * kW4Cols + 8 * c + g;
      const float2 inv = make_float2(s_inv[grp][n], s_inv[grp][n]);
      const uint32_t z2 = ZEROS ? s_zero[grp][n] : 0x00080008u;
      const __nv_bfloat16* src = tile + (kt * kW4Rows + 16 * j + 2 * t) * kPackPitch + n;
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // rows 8 half + 2 t and the next
        float2 y = make_float2(__bfloat162float(src[8 * half * kPackPitch]), __bfloat162float(src[(8 * half + 1) * kPackPitch]));
        if (INFINITE) {
          y = __fmul2_rn(y, inv);
          y = make_float2(fminf(fmaxf(y.x, -16.f), 16.f), fminf(fmaxf(y.y, -16.f), 16.f));
          y = __fadd2_rn(y, make_float2(12288.f, 12288.f));
        } else {
          y = __ffma2_rn(y, inv, make_float2(12288.f, 12288.f));  // multiples of 2^-10 there
        }
        y = __fadd2_rn(y, make_float2(12570624.f, 12570624.f));  // 1.5 2^23 in all: the low halves are the quotient's rint
        const uint32_t q2 = __vadd2(__byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x5410), z2);
        word |= __vimin_s16x2_relu(q2, 0x000F000Fu) << (4 * (c + 2 * half));
      }
    }
    words[j] = word;
  }
}

template <bool ZEROS>
__global__ void __launch_bounds__(256, 8) k_quantize_w4(const __grid_constant__ W4Pack p) {
  __shared__ __align__(16) __nv_bfloat16 tile[kPackRows * kPackPitch];
  __shared__ __nv_bfloat162 low[8][32], high[8][32];  // [16 rows][two columns]; the magnitudes' largest without zero points
  __shared__ float s_inv[4][kPackCols];               // [group of the block][column]
  __shared__ uint32_t s_zero[4][kPackCols];           // twice, in both halves
  const int n0 = blockIdx.x * kPackCols, k0 = blockIdx.y * kPackRows;
  const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(p.w);
  const int c0 = (threadIdx.x & 7) * 8, r0 = (threadIdx.x >> 3) * 4;
  __nv_bfloat162 lo[4], hi[4];
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = k0 + r0 + i < p.K && n0 + c0 < p.N ? ld_stream(reinterpret_cast<const uint4*>(w + static_cast<long long>(k0 + r0 + i) * p.N + n0 + c0))
                                               : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int e = 0; e < 4; ++e) lo[e] = hi[e] = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(u + e);
      u[e] &= __heq2_mask(x, x);  // NaN to zero
      x = *reinterpret_cast<const __nv_bfloat162*>(u + e);
      if (ZEROS) lo[e] = __hmin2(lo[e], x);
      hi[e] = __hmax2(hi[e], ZEROS ? x : __habs2(x));
    }
    uint2* dst = reinterpret_cast<uint2*>(tile + (r0 + i) * kPackPitch + c0);
    dst[0] = make_uint2(u[0], u[1]);
    dst[1] = make_uint2(u[2], u[3]);
  }
  bool infinite = false;
  const __nv_bfloat162 top = __floats2bfloat162_rn(kW4Big, kW4Big);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    infinite |= !__hble2(hi[e], top) || (ZEROS && !__hbge2(lo[e], __hneg2(top)));
#pragma unroll
    for (int o = 8; o < 32; o *= 2) {
      hi[e] = __hmax2(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], o));
      if (ZEROS) lo[e] = __hmin2(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], o));
    }
    if ((threadIdx.x & 31) < 8) {
      high[threadIdx.x >> 5][c0 / 2 + e] = hi[e];
      if (ZEROS) low[threadIdx.x >> 5][c0 / 2 + e] = lo[e];
    }
  }
  infinite = __syncthreads_or(infinite);
  const int shift = 31 - __clz(p.group), groups = kPackRows >> shift, segs = p.group / 16;  // of the block; of a group
  for (int i = threadIdx.x; i < groups * kPackCols; i += blockDim.x) {
    const int c = i % kPackCols, grp = i / kPackCols;
    float least = 0.f, most = 0.f;
    for (int q = grp * segs; q < (grp + 1) * segs; ++q) {
      if (ZEROS) least = fminf(least, __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(low[q])[c]));
      most = fmaxf(most, __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(high[q])[c]));
    }
    const float span = fminf(fmaxf(most - least, kW4Tiny), kW4Big);
    const __nv_bfloat16 s = __float2bfloat16_rn(span / (ZEROS ? 15.f : 7.f));
    const uint32_t z = ZEROS ? static_cast<uint32_t>(fminf(fmaxf(rintf(-least / __bfloat162float(s)), 0.f), 15.f)) : 8u;
    s_inv[grp][c] = 1.f / __bfloat162float(s);
    s_zero[grp][c] = z * 0x00010001u;
    const int col = n0 + c, row = k0 + grp * p.group;
    if (col < p.N && row < p.K) {
      const long long at = static_cast<long long>(row >> shift) * p.N + col;
      if (TPMLP_IN_BOUNDS(at, static_cast<long long>((p.K + p.group - 1) / p.group) * p.N, kBoundsW4Scales)) {
        static_cast<__nv_bfloat16*>(p.scales)[at] = s;
        if (ZEROS) p.zeros[at] = static_cast<uint8_t>(z);
      }
    }
  }
  __syncthreads();
  const int kt = threadIdx.x >> 7, ct = threadIdx.x >> 5 & 3, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n_tile = blockIdx.x * 4 + ct, k_tile = blockIdx.y * 2 + kt;
  const int n_tiles = (p.N + kW4Cols - 1) / kW4Cols, k_tiles = (p.K + kW4Rows - 1) / kW4Rows;
  if (n_tile >= n_tiles || k_tile >= k_tiles) return;
  uint32_t words[4];
  if (infinite) quantize_words<true, ZEROS>(tile, s_inv, s_zero, kt, ct, g, t, shift, words);
  else quantize_words<false, ZEROS>(tile, s_inv, s_zero, kt, ct, g, t, shift, words);
  if (ZEROS && ((k_tile + 1) * kW4Rows > p.K || (n_tile + 1) * kW4Cols > p.N)) {  // places past the matrix hold 8, not z
#pragma unroll
    for (int j = 0; j < 4; ++j)
      for (int b = 0; b < 8; ++b) {
        const int i = b & 3, h = b >> 2;
        if (n_tile * kW4Cols + 8 * (i & 1) + g >= p.N || k_tile * kW4Rows + 16 * j + 8 * (i >> 1) + 2 * t + h >= p.K)
          words[j] = (words[j] & ~(15u << (4 * i + 16 * h))) | 8u << (4 * i + 16 * h);
      }
  }
  const long long at = (static_cast<long long>(n_tile) * k_tiles + k_tile) * 32 + lane;
  if (TPMLP_IN_BOUNDS(at, static_cast<long long>(n_tiles) * k_tiles * 32, kBoundsW4Codes))
    p.q[at] = make_uint4(words[0], words[1], words[2], words[3]);
}

// A thread's 32 codes to bf16 in pairs of rows: (q - z) s is exact before its one rounding.
template <bool ZEROS>
__global__ void __launch_bounds__(256) k_dequantize_w4(const __grid_constant__ W4Pack p) {
  __shared__ __align__(16) __nv_bfloat16 tile[kPackRows * kPackPitch];
  const int n0 = blockIdx.x * kPackCols, k0 = blockIdx.y * kPackRows;
  const int kt = threadIdx.x >> 7, ct = threadIdx.x >> 5 & 3, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n_tile = blockIdx.x * 4 + ct, k_tile = blockIdx.y * 2 + kt;
  const int n_tiles = (p.N + kW4Cols - 1) / kW4Cols, k_tiles = (p.K + kW4Rows - 1) / kW4Rows;
  if (n_tile < n_tiles && k_tile < k_tiles) {
    const uint4 q4 = ld_stream(p.q + (static_cast<long long>(n_tile) * k_tiles + k_tile) * 32 + lane);
    const uint32_t q[4] = {q4.x, q4.y, q4.z, q4.w};
    const int shift = 31 - __clz(p.group), last = ((p.K + p.group - 1) >> shift) - 1;
    __nv_bfloat162 s[2][2];  // [half of the row tile][columns g, g + 8]
    uint32_t base[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = n_tile * kW4Cols + 8 * c + g, grp = min((k_tile * kW4Rows + 32 * h) >> shift, last);
        const long long at = static_cast<long long>(grp) * p.N + min(col, p.N - 1);
        const __nv_bfloat16 v = static_cast<const __nv_bfloat16*>(p.scales)[at];
        s[h][c] = __nv_bfloat162(v, v);
        base[h][c] = w4_base<kW4One>(ZEROS ? p.zeros[at] & 15u : 8u);
      }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t a[4];
      w4_unpack_bf16<kW4One>(q[j], base[j >> 1][0], base[j >> 1][1], a);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(a + i), s[j >> 1][i & 1]);
        __nv_bfloat16* dst = tile + (kt * kW4Rows + 16 * j + 8 * (i >> 1) + 2 * t) * kPackPitch + ct * kW4Cols + 8 * (i & 1) + g;
        dst[0] = v.x;
        dst[kPackPitch] = v.y;
      }
    }
  }
  __syncthreads();
  __nv_bfloat16* w = static_cast<__nv_bfloat16*>(p.w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 32 + (threadIdx.x >> 3), c = (threadIdx.x & 7) * 8;
    const long long at = static_cast<long long>(k0 + r) * p.N + n0 + c;
    if (k0 + r < p.K && n0 + c < p.N && TPMLP_IN_BOUNDS(at + 7, static_cast<long long>(p.K) * p.N, kBoundsW4Weights)) {
      const uint2* src = reinterpret_cast<const uint2*>(tile + r * kPackPitch + c);
      const uint2 a = src[0], b = src[1];
      *reinterpret_cast<uint4*>(w + at) = make_uint4(a.x, a.y, b.x, b.y);
    }
  }
}

}  // namespace

cudaError_t w4_bounds_status(unsigned int* count, unsigned int* site) {
#ifdef TPMLP_DEBUG_BOUNDS
  return bounds_read_and_clear(count, site);
#else
  *count = *site = 0;
  return cudaSuccess;
#endif
}

namespace {

template <int BT, int STEPS, bool ZEROS>
cudaError_t run_w4_tc(W4TcParams& p, const DeviceCtx& ctx, cudaStream_t s) {
  using S = W4TcShape<BT>;
  auto kern = k_gemm_w4_tc<BT, STEPS, ZEROS>;
  static std::atomic<unsigned long long> set[64] = {};
  const cudaError_t e = raise_smem_once(kern, S::kSmem, ctx, set);
  if (e != cudaSuccess) return e;
  const W4Launch& g = p.g;
  p.box_rows = g.M < BT ? g.M : BT;
  if (!encode_tile_map(&p.tmX, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, g.x, g.K, g.M, g.K, kW4Rows, p.box_rows, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const long long words = static_cast<long long>((g.K + kW4Rows - 1) / kW4Rows) * 128;
  for (int i = 0; i < (g.gated ? 2 : 1); ++i)
    if (!encode_tile_map(&p.tmQ[i], CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, g.w[i].q, words, (g.N + kW4Cols - 1) / kW4Cols, words, 256, 8, CU_TENSOR_MAP_SWIZZLE_NONE))
      return cudaErrorInvalidValue;
  const int cols = g.gated ? 128 : 128 * S::kBlocks, blocks = (g.N + cols - 1) / cols, tiles = (g.M + BT - 1) / BT;
  if (tiles > 65535) return cudaErrorNotSupported;
  p.ranks = few_ranks_any<S>(static_cast<long long>(blocks) * tiles, (g.K + kW4TcRows - 1) / kW4TcRows, kW4TcRanks, ctx);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.ranks * blocks, tiles);
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = p.ranks;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.ranks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int BT>
cudaError_t launch_w4_tc(const W4Launch& g, const DeviceCtx& ctx, cudaStream_t s) {
  W4TcParams p;
  memset(&p, 0, sizeof(p));
  p.g = g;
  p.shift = g.group == 32 ? 5 : g.group == 64 ? 6 : 7;
  p.err = ctx.err;
  p.timeout_ns = ctx.timeout_ns;
  const bool z = g.w[0].zeros != nullptr;
  if (g.group == 32) return z ? run_w4_tc<BT, 2, true>(p, ctx, s) : run_w4_tc<BT, 2, false>(p, ctx, s);
  if (g.group == 64) return z ? run_w4_tc<BT, 4, true>(p, ctx, s) : run_w4_tc<BT, 4, false>(p, ctx, s);
  return z ? run_w4_tc<BT, 8, true>(p, ctx, s) : run_w4_tc<BT, 8, false>(p, ctx, s);
}

}  // namespace

cudaError_t launch_gemm_w4(const W4Launch& g, const DeviceCtx& ctx, cudaStream_t s) {
  cudaError_t e = cudaErrorNotSupported;
  if (g.M <= kW4FewTokens) e = g.gated ? launch_w4_few<2>(g, ctx, s) : launch_w4_few<1>(g, ctx, s);
  if (e != cudaErrorNotSupported) return e;  // no room for X there
  if (g.M <= 32) return launch_w4_tc<32>(g, ctx, s);
  // 128 tokens of 128 columns instead of twice 64 of 256 (K = 4096, N = 16384): 65 tokens 23.7 us for 28.7, 128 25.6 for 28.7, 256
  // 49.7 for 57.1.  Of the gated form's two matrices it would take 64 columns each: 256 tokens of 1024 x 4096 14.6 for 13.2.
  return g.M <= 64 || g.gated ? launch_w4_tc<64>(g, ctx, s) : launch_w4_tc<128>(g, ctx, s);
}

cudaError_t launch_quantize_w4(const W4Pack& p, cudaStream_t s) {
  const dim3 grid((p.N + kPackCols - 1) / kPackCols, (p.K + kPackRows - 1) / kPackRows);
  if (p.zeros != nullptr) k_quantize_w4<true><<<grid, 256, 0, s>>>(p);
  else k_quantize_w4<false><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_dequantize_w4(const W4Pack& p, cudaStream_t s) {
  const dim3 grid((p.N + kPackCols - 1) / kPackCols, (p.K + kPackRows - 1) / kPackRows);
  if (p.zeros != nullptr) k_dequantize_w4<true><<<grid, 256, 0, s>>>(p);
  else k_dequantize_w4<false><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace tpmlp
