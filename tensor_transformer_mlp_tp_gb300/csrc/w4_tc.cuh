// Products with 4-bit weights on the UMMA, for more tokens than the m16n8k16 kernel takes: the unpacked weights never touch
// shared memory.
//
// A CTA takes two blocks of 128 columns of W (256 columns, or the same 128 of both matrices of the gated form) as the
// UMMA's rows and up to BT tokens as its columns (128 tokens: one block, plain products only); a cluster of CTAs shares K.
// Warp 0 copies codes and X (TMA boxes), warp 1 issues, sixteen warps unpack: a lane's 16 bytes of a 16 x 64 tile are
// registers in the order of the m16n8k16 product's A operand, which is that of tcgen05.st's 16x128b shape, so tiles go to
// tensor memory by one instruction as the UMMA's A operand.  Codes become bf16 (q - z) 2^-11, exact: a group's
// products with X's largest numbers then sum up below fp32's largest, and 2^11 comes back behind all sums (measured to 2^-130:
// subnormal products and sums are not flushed).  Eight warps scale: the UMMAs of a group make a partial sum in TMEM, a
// thread has those of one column of W, one scale for all of them.  The cluster's sums are joined through distributed
// shared memory in rank order.
//
// Measured, K = 4096, N = 16384, groups of 128: 14.4 us for 17 tokens, 17.5 for 64, 25.4 for 128, 49.7 for 256 (groups of 32
// with zero points: 30.1 for 64); the gated form 22.7 for 16, 29.4 for 64, 114.7 for 256.  A stage (128 rows of 256
// columns) takes about 1100 cycles, of which its 16 UMMAs are 540: in a stage the chain of copy, unpacking, UMMAs and scaling
// binds, no part of it alone (each left out by itself: 1 to 2 us less).  At 64 tokens the 16 stages of a CTA are then 17600
// cycles, half of the time; the other half is start, first copies and the cluster's join.  Eight unpacking warps: 15.2 and
// 18.6; scaling and unpacking by the same warps 22.7; a third buffer of unpacked stages, at 32 tokens: no change.
#pragma once

#include "gated.cuh"
#include "w4.cuh"

namespace tpmlp {

constexpr int kW4TcRanks = 8;  // CTAs of a cluster at most
constexpr int kW4TcRows = 128;  // of W a stage: two row tiles
constexpr float kW4TcBack = 0x1p11f;  // what the unpacked weights are too small by (kW4OneLow)

struct W4TcParams {
  CUtensorMap tmX;      // boxes of 64 x box_rows
  CUtensorMap tmQ[2];   // codes as words, a column tile a row: boxes of two row tiles (256 words) x eight column tiles
  W4Launch g;
  int ranks, box_rows, shift;
  unsigned int* err;
  unsigned long long timeout_ns;
};

template <int BT>
struct W4TcShape {
  static_assert(BT == 32 || BT == 64 || BT == 128, "BT");
  static constexpr int kBlocks = BT == 128 ? 1 : 2;    // of 128 columns of W
  static constexpr int kCodes = kBlocks * 8 * 2 * 512;  // blocks of eight column tiles, two row tiles
  static constexpr int kX = 2 * BT * 128;
  static constexpr int kStage = kCodes + kX;
  static constexpr int kStages = BT == 128 ? 5 : BT == 64 ? 6 : 8;
  static constexpr int kABufs = 2;                     // unpacked stages in TMEM, 64 columns a block
  static constexpr int kD = kABufs * kBlocks * 64;     // partial sums behind them: [buffer][block][BT]
  static constexpr int kAcc = kBlocks * BT / 2;        // sums of a scaling thread: a block's, or half the tokens' of the one
  static constexpr int kTmemCols = 512;
  // A warpgroup copies and issues, four unpack, two scale; their registers, together what the block is launched with (72 a
  // thread): a scaling thread holds up to 64 sums, an unpacking one up to 32 words on their way to tensor memory.
  static constexpr int kUnpackWarps = 16, kScaleWarp = 4 + kUnpackWarps, kWarps = kScaleWarp + 8, kThreads = 32 * kWarps;
  static constexpr int kIssueRegs = 40, kUnpackRegs = 64, kScaleRegs = 104;
  static_assert(128 * kIssueRegs + 32 * kUnpackWarps * kUnpackRegs + 256 * kScaleRegs <= 72 * kThreads, "setmaxnreg split");
  static constexpr int kSlots = 4 * 4 * (8 * 64 + kUnpackWarps * 16);  // scales and zero points in flight: [warp][slot][group]
  static constexpr int kSmem = 1024 + kStages * kStage + kSlots + 256;
  static_assert(kD + 2 * kBlocks * BT <= kTmemCols, "tensor memory");
  static_assert(kStages * kStage >= kBlocks * BT * 128 * 4, "the sums are joined in the ring's memory");
  static_assert(kSmem <= 232448, "shared memory per block");
};

// 16 lanes x 64 columns into TMEM: registers 2 i and 2 i + 1 of lane 4 g + t are column 4 i + t of lanes g and g + 8.
__device__ __forceinline__ void tmem_st_16x64(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// The same of 32 columns.
__device__ __forceinline__ void tmem_st_16x32(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// STEPS: UMMAs (16 rows of W each) of a group.  grid: (cluster size x column blocks, token tiles)
template <int BT, int STEPS, bool ZEROS>
__global__ void __launch_bounds__(W4TcShape<BT>::kThreads, 1) k_gemm_w4_tc(const __grid_constant__ W4TcParams p) {
  using S = W4TcShape<BT>;
  constexpr int STAGES = S::kStages, ABUFS = S::kABufs, BLOCKS = S::kBlocks;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* smem_s = smem + STAGES * S::kStage;
  uint8_t* smem_z = smem_s + 8 * 4 * 4 * 64;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem_s + S::kSlots);
  uint64_t* empty = full + STAGES;
  uint64_t* a_full = empty + STAGES;
  uint64_t* a_empty = a_full + ABUFS;
  uint64_t* tfull = a_empty + ABUFS;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31u;
  const bool gated = BLOCKS == 2 && p.g.gated;
  const int rank = static_cast<int>(cluster_ctarank()), ranks = p.ranks;
  const int N = p.g.N, K = p.g.K;
  const int n0 = static_cast<int>(blockIdx.x) / ranks * (gated ? 128 : 128 * BLOCKS), m0 = static_cast<int>(blockIdx.y) * BT;
  const int k_tiles = (K + kW4Rows - 1) / kW4Rows, all_stages = (k_tiles + 1) / 2;
  const int st0 = static_cast<int>(static_cast<long long>(all_stages) * rank / ranks);
  const int st1 = static_cast<int>(static_cast<long long>(all_stages) * (rank + 1) / ranks);
  const int kt0 = 2 * st0, kts = min(2 * st1, k_tiles) - kt0;  // this CTA's row tiles
  const int parts = (4 * kts + STEPS - 1) / STEPS;             // and groups

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, S::kUnpackWarps + 1);
    }
    for (int i = 0; i < ABUFS; ++i) {
      mbar_init(a_full + i, S::kUnpackWarps);
      mbar_init(a_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull + i, 1);
      mbar_init(tempty + i, 8);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.tmX);
    tma_prefetch_desc(&p.tmQ[0]);
    if (gated) tma_prefetch_desc(&p.tmQ[1]);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();
  const WaitCtx wc{abort_flag, p.err, p.timeout_ns};

  float* red = reinterpret_cast<float*>(smem);
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kIssueRegs));
  if (warp == 0) {
    // up to four boxes a stage (past the matrix's ends they fill zeros): single column tiles by bulk copies of 1 KB, 16 of
    // them, took longer to issue than to multiply
    const uint64_t pol = policy_evict_normal();
    const int tile = n0 / kW4Cols;
    uint32_t issued = 0, issued_parity = 0;
    for (int s = 0; s < st1 - st0; ++s) {
      const int stage = s % STAGES, at = kt0 + 2 * s;  // row tile
      const uint32_t phase = static_cast<uint32_t>(s / STAGES) & 1u;
      if (!warp_wait_spin(empty + stage, phase ^ 1u, wc, kSiteW4TcProducer)) break;
      uint8_t* dst = smem + stage * S::kStage;
      if (lane == 0) {
        mbar_arrive_expect_tx(full + stage, static_cast<uint32_t>(S::kCodes + 2 * p.box_rows * 128));
        for (int b = 0; b < BLOCKS; ++b)
          tma_load_2d(dst + b * 8192, &p.tmQ[gated ? b : 0], full + stage, at * 128, tile + (gated ? 0 : 8 * b), pol);
        for (int r = 0; r < 2; ++r)
          tma_load_2d(dst + S::kCodes + r * (BT * 128), &p.tmX, full + stage, (at + r) * kW4Rows, m0, pol);
      }
      __syncwarp();
      issued |= 1u << stage;
      issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
    }
    if (lane == 0)  // copies in flight land before their memory is used again
      for (int s = 0; s < STAGES; ++s)
        if (issued & (1u << s)) wait_drain(full + s, (issued_parity >> s) & 1u, p.timeout_ns);
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, BT, false, false);
    const bool elected = elect_one();
    bool ok = true;
    for (int st = 0; ok && st < st1 - st0; ++st) {
      const int stage = st % STAGES, abuf = st % ABUFS, steps = 4 * min(2, kts - 2 * st);
      if (!warp_wait_spin(full + stage, static_cast<uint32_t>(st / STAGES) & 1u, wc, kSiteW4TcMmaX) ||
          !warp_wait_spin(a_full + abuf, static_cast<uint32_t>(st / ABUFS) & 1u, wc, kSiteW4TcMmaA))
        break;
      const uint32_t x_base = smem_u32(smem + stage * S::kStage + S::kCodes);
#pragma unroll
      for (int h = 0; h < 8 / STEPS; ++h) {  // groups
        if (h * STEPS >= steps) break;
        const int part = 8 / STEPS * st + h;
        if (!warp_wait_spin(tempty + (part & 1), (static_cast<uint32_t>(part >> 1) & 1u) ^ 1u, wc, kSiteW4TcMmaD)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        if (elected) {
          const uint32_t d = tmem_base + S::kD + (part & 1) * BLOCKS * BT, a = tmem_base + abuf * BLOCKS * 64;
#pragma unroll
          for (int j = h * STEPS; j < (h + 1) * STEPS; ++j) {
            if (j >= steps) break;  // a last, single row tile
            const uint64_t x = sdesc_sw128(x_base + (j >> 2) * (BT * 128) + (j & 3) * 32, 16, 1024);
            umma_bf16_tmem_a(d, a + 8 * j, x, idesc, j % STEPS != 0 ? 1u : 0u);
            if (BLOCKS == 2) umma_bf16_tmem_a(d + BT, a + 64 + 8 * j, x, idesc, j % STEPS != 0 ? 1u : 0u);
          }
          umma_commit(tfull + (part & 1));
        }
        __syncwarp();
      }
      if (!ok) break;
      if (elected) {
        umma_commit(a_empty + abuf);
        umma_commit(empty + stage);
      }
      __syncwarp();
    }
    if (elected) {
      umma_commit(drain);
      wait_drain(drain, 0, p.timeout_ns);
    }
    __syncwarp();
  }
    __syncthreads();
    if (warp == 1) {
      tc_fence_after_sync();
      tmem_dealloc(tmem_base, S::kTmemCols);
    }
    cluster_sync_all();
    cluster_sync_all();
    return;
  }
  if (warp < S::kScaleWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kUnpackRegs));
    // -------------------------------------------------------------------- unpacking
    // a column tile each, or of one block a column tile's row tile
    const int quad = warp & 3, half = (warp >> 2) & 1, upper = (warp - 4) >> 3, g = static_cast<int>(lane) >> 2;
    const int block = BLOCKS == 2 ? upper : 0, row_tile = BLOCKS == 2 ? 0 : upper;
    const int col = n0 + (gated ? 0 : 128 * block) + 32 * quad + 16 * half;  // the first
    const uint8_t* zeros = p.g.w[gated ? block : 0].zeros;
    constexpr int kGroups = 8 / STEPS;  // of a stage
    // Zero points of the tile's columns three stages ahead, by copies that no register waits for: a load among the
    // others makes them wait for it.
    uint8_t* slots = smem_z + (warp - 4) * (4 * kGroups * 16);
    auto fetch = [&](int st) {
      if (ZEROS && st < st1 - st0 && lane < 2 * kGroups) {
        const int row = min((kt0 + 2 * st) * kW4Rows + 16 * STEPS * (static_cast<int>(lane) >> 1), K - 1), at = col + 8 * (static_cast<int>(lane) & 1);
        cp_async<8>(slots + (st & 3) * (kGroups * 16) + lane * 8, zeros + static_cast<long long>(row >> p.shift) * N + (at < N ? at : 0), at < N ? 8 : 0);
      }
      if (ZEROS) cp_async_commit();
    };
#pragma unroll
    for (int u = 0; u < 3; ++u) fetch(u);
    const uint32_t a_lane = tmem_base + (static_cast<uint32_t>(quad * 32 + 16 * half) << 16) + static_cast<uint32_t>(block * 64 + row_tile * 32);
    constexpr int kWords = 4 * BLOCKS;  // of codes a lane, a stage
    for (int st = 0; st < st1 - st0; ++st) {
      const int stage = st % STAGES, abuf = st % ABUFS;
      if (!warp_wait_spin(full + stage, static_cast<uint32_t>(st / STAGES) & 1u, wc, kSiteW4TcUnpack)) break;
      if (ZEROS) {
        cp_async_wait<2>();
        __syncwarp();  // this stage's are there for all lanes, and the slot before has been read
        fetch(st + 3);
      }
      const uint8_t* zs = slots + (st & 3) * (kGroups * 16) + 4 * row_tile / STEPS * 16 + g;
      // (what a second row tile holds behind a last, single one is not multiplied)
      const uint4* src = reinterpret_cast<const uint4*>(smem + stage * S::kStage + (block * 8 + 2 * quad + half) * 1024 + row_tile * 512) + lane;
      uint32_t q[kWords];
#pragma unroll
      for (int r = 0; r < BLOCKS; ++r) {
        const uint4 v = src[r * 32];
        q[4 * r] = v.x;
        q[4 * r + 1] = v.y;
        q[4 * r + 2] = v.z;
        q[4 * r + 3] = v.w;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + stage);
      uint32_t a[4 * kWords];
      uint32_t b0 = w4_base<kW4OneLow>(8u), b1 = b0;
#pragma unroll
      for (int j = 0; j < kWords; ++j) {
        if (ZEROS && j % STEPS == 0) {
          b0 = w4_base<kW4OneLow>(zs[j / STEPS * 16] & 15u);
          b1 = w4_base<kW4OneLow>(zs[j / STEPS * 16 + 8] & 15u);
        }
        w4_unpack_bf16<kW4OneLow>(q[j], b0, b1, a + 4 * j);
      }
      if (!warp_wait_spin(a_empty + abuf, (static_cast<uint32_t>(st / ABUFS) & 1u) ^ 1u, wc, kSiteW4TcUnpackA)) break;
      tc_fence_after_sync();
      if constexpr (BLOCKS == 2) tmem_st_16x64(a_lane + static_cast<uint32_t>(abuf * 128), a);
      else tmem_st_16x32(a_lane + static_cast<uint32_t>(abuf * 64), a);
      tmem_wait_st();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(a_full + abuf);
    }
    __syncthreads();  // the ring is drained: its memory holds the CTA's sums [block][token][128] from here on
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kScaleRegs));
    // -------------------------------------------------------------------- scaling
    const int quad = warp & 3, upper = (warp - S::kScaleWarp) >> 2;
    const int block = BLOCKS == 2 ? upper : 0, token0 = BLOCKS == 2 ? 0 : upper * S::kAcc;
    const int col = n0 + (gated ? 0 : 128 * block) + 32 * quad;  // the quadrant's first
    const uint16_t* scales = static_cast<const uint16_t*>(p.g.w[gated ? block : 0].scales);
    constexpr int kGroups = 8 / STEPS;  // of a stage
    // the quadrant's scales, three stages ahead as the zero points are
    uint8_t* slots = smem_s + (warp - S::kScaleWarp) * (4 * kGroups * 64);
    auto fetch = [&](int st) {
      if (st < st1 - st0 && lane < 4 * kGroups) {
        const int row = min((kt0 + 2 * st) * kW4Rows + 16 * STEPS * (static_cast<int>(lane) >> 2), K - 1), at = col + 8 * (static_cast<int>(lane) & 3);
        cp_async<16>(slots + (st & 3) * (kGroups * 64) + lane * 16, scales + static_cast<long long>(row >> p.shift) * N + (at < N ? at : 0), at < N ? 16 : 0);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int u = 0; u < 3; ++u) fetch(u);
    float acc[S::kAcc] = {};
    const uint32_t d_lane = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(S::kD + block * BT + token0);
    bool ok = true;
    for (int st = 0; ok && st < st1 - st0; ++st) {
      cp_async_wait<2>();
      __syncwarp();
      fetch(st + 3);
      const uint16_t* ss = reinterpret_cast<const uint16_t*>(slots + (st & 3) * (kGroups * 64)) + lane;
#pragma unroll
      for (int h = 0; h < kGroups; ++h) {
        const int part = kGroups * st + h;
        if (part >= parts) break;
        if (!warp_wait_spin(tfull + (part & 1), static_cast<uint32_t>(part >> 1) & 1u, wc, kSiteW4TcScale)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const float s = __uint_as_float(static_cast<uint32_t>(ss[h * 32]) << 16);
#pragma unroll
        for (int c = 0; c < S::kAcc / 16; ++c) {
          uint32_t r[16];
          tmem_load_16cols_async(d_lane + (part & 1) * BLOCKS * BT + c * 16, r);
          tmem_wait_ld(r);
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[c * 16 + j] = fmaf(__uint_as_float(r[j]), s, acc[c * 16 + j]);
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty + (part & 1));
      }
    }
    __syncthreads();
    float* at = red + (block * BT + token0) * 128 + quad * 32 + lane;
#pragma unroll
    for (int j = 0; j < S::kAcc; ++j) at[j * 128] = acc[j];
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kUnpackRegs));
  }
  cluster_sync_all();  // every CTA's sums are written (a cluster of one: a block barrier)
  const int rows = min(BT, p.g.M - m0);
  const uint32_t red_addr = smem_u32(red);
  // a token of a block of columns a warp; the gated form takes both blocks together
  const bool once = gated || BLOCKS == 1;
  for (int i = rank + ranks * (warp - 4); i < (once ? rows : 2 * rows); i += ranks * (S::kWarps - 4)) {
    const int j = once ? i : i >> 1, first = once ? 0 : i & 1;
    const int col = n0 + 128 * first + static_cast<int>(lane) * 4;
    float v[2][4];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (b == 1 && !gated) break;
      float4 q[kW4TcRanks];
#pragma unroll
      for (int r = 0; r < kW4TcRanks; ++r)
        q[r] = r < ranks ? ld_cluster_f4(mapa_shared(red_addr + (((first + b) * BT + j) * 128 + lane * 4) * 4, static_cast<uint32_t>(r)))
                         : make_float4(0.f, 0.f, 0.f, 0.f);
      v[b][0] = v[b][1] = v[b][2] = v[b][3] = 0.f;
#pragma unroll
      for (int r = 0; r < kW4TcRanks; ++r) {  // in rank order
        v[b][0] += q[r].x; v[b][1] += q[r].y; v[b][2] += q[r].z; v[b][3] += q[r].w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v[b][i] *= kW4TcBack;
      const void* bias = p.g.w[b].bias;
      if (bias != nullptr && col < N) {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(bias) + col));
        const float2 lo = unpack_bf16x2(u.x), hi = unpack_bf16x2(u.y);
        v[b][0] += lo.x; v[b][1] += lo.y; v[b][2] += hi.x; v[b][3] += hi.y;
      }
    }
    const long long at = static_cast<long long>(m0 + j) * N + col;
    if (col >= N || !TPMLP_IN_BOUNDS(at + 3, static_cast<long long>(p.g.M) * N, kBoundsW4Out)) continue;
    if (gated) {
      const float2 a = __fmul2_rn(act2(p.g.act, make_float2(v[0][0], v[0][1])), make_float2(v[1][0], v[1][1]));
      const float2 b = __fmul2_rn(act2(p.g.act, make_float2(v[0][2], v[0][3])), make_float2(v[1][2], v[1][3]));
      v[0][0] = a.x; v[0][1] = a.y; v[0][2] = b.x; v[0][3] = b.y;
    }
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.g.y) + at) = make_uint2(pack_bf16x2(v[0][0], v[0][1]), pack_bf16x2(v[0][2], v[0][3]));
  }
  __syncwarp();
  cluster_sync_all();  // the cluster has read this CTA's sums
}

}  // namespace tpmlp
