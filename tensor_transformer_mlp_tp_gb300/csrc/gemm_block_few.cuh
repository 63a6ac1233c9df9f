// The block-scaled product for few rows of A (decoded tokens): every weight byte is read once, so the time is that of
// streaming B.  The operands change sides: a CTA takes 128 rows of B (output columns) as the UMMA's M and up to BT rows
// of A as its N (128 x BT x 32 UMMAs, cta_group::1), and the K blocks are split over a cluster of CTAs, whose fp32 sums
// are joined through distributed shared memory in rank order -- no workspace, no atomics, one launch.
//
// Warp 0 copies (TMA ring), warp 1 issues, the others promote: a thread holds BT (or BT / 2) sums of one output column,
// scaled per k-block by its own row scale of B and the scales of A.  With BT columns a partial sum, several fit in TMEM, so the
// promotion's latency is hidden.  In the end each CTA of the cluster finishes BT / C of the rows: a warp per row, four
// consecutive columns a lane, which makes a 1 x 128 block of an 8-bit output one warp's.
//
// What bounds it: HBM, and a fixed part of about 3 us (set-up, the first bytes, the join).  Measured on GB300: one row,
// N = 4096, K = 16384 (67 MB) 13.3 us, 5.0 TB/s, with 256 CTAs in 32 clusters of eight (15.3 us with four CTAs a tile);
// N = 16384, K = 4096: 13.3 us; 48 rows 15.9 us; 64 rows 16.8 us; 128 rows 20 us (one CTA an SM, 128 x 128 tiles, then the promotion's
// 450 ns a k-block counts).
#pragma once

#include "gemm_block_pair.cuh"

namespace tpmlp {

constexpr int kFewMaxRanks = 8;  // CTAs of a cluster

template <int BT, bool BVEC>
struct BlockFewShape {
  static_assert(BT == 16 || BT == 32 || BT == 48 || BT == 64 || BT == 128, "BT");
  // Two CTAs share an SM up to BT = 64.  (Three with three stages, BT = 16: 13.1 -> 13.7 us; five stages: 13.3.)
  static constexpr int kStages = BT <= 64 ? 4 : 6;
  static constexpr int kWTile = 128 * 128, kTTile = BT * 128;
  static constexpr int kStage = kWTile + kTTile;
  static constexpr int kBufs = BT == 128 ? 2 : 4;  // partial sums in TMEM
  static constexpr int kTmemCols = BT == 48 ? 256 : kBufs * BT;  // allocated in powers of two
  // Promotion warps: four (one a TMEM lane quadrant); eight that halve the columns where a thread would hold 128 sums
  // (at 64 four measure 16.8 us where eight take 17.4: 64 rows, N = 4096, K = 16384).
  static constexpr int kPromoteWarps = BT > 64 ? 8 : 4;
  static constexpr int kCols = BT / (kPromoteWarps / 4);  // of one warp
  static constexpr int kThreads = 64 + 32 * kPromoteWarps;
  // Slots of the k-blocks' scales, rewritten 16 blocks later (see BlockPairShape): the producer is at most kStages
  // blocks ahead of the UMMAs, those at most kBufs ahead of the promotion.
  static constexpr int kScaleSlots = 16;
  static constexpr int kRowFloats = (BT + 31) & -32;  // a copy starts on a 128-byte boundary
  static constexpr int kSlotFloats = kRowFloats + (BVEC ? 128 : 0);
  static constexpr int kStageBytes = kStage + (BT + (BVEC ? 128 : 0)) * 4;  // copied for a k-block of BT rows
  static constexpr int kSmem = 1024 + kStages * kStage + kScaleSlots * kSlotFloats * 4 + 256;
  static_assert(kStages + kBufs + 2 < kScaleSlots, "see kScaleSlots");
  static_assert(kStages * kStage >= BT * 128 * 4, "the sums are joined in the ring's memory");
  static_assert(kSmem <= 232448, "shared memory per block");
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

// grid: (cluster size x column tiles, row tiles).  p.tmA: A [M x K], boxes of 128 bytes x p.box_rows rows, the M there are
// up to BT: with boxes of BT rows the copies' zero rows past A's end cost more than real ones, as if every CTA read one
// line for them (N = 16384, K = 4096: one row 16.3 us, now 13.3; 17 rows 17.5, now 14.6).  The rest of a tile stays unwritten and
// makes columns of partial sums that nothing reads.  p.tmB: B [N x K], 128 bytes x 128 rows; p.tmSA boxes of BT scales,
// p.tmSB (BVEC) of 128.
template <int BT, int OUT, bool BVEC>
__global__ void __launch_bounds__(BlockFewShape<BT, BVEC>::kThreads, BT == 128 ? 1 : 2)
    k_gemm_block_few(const __grid_constant__ GemmBlockParams p) {
  using S = BlockFewShape<BT, BVEC>;
  constexpr int STAGES = S::kStages, BUFS = S::kBufs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sW = smem;
  uint8_t* sT = sW + STAGES * S::kWTile;
  float* scale_ring = reinterpret_cast<float*>(sT + STAGES * S::kTTile);
  uint64_t* full = reinterpret_cast<uint64_t*>(scale_ring + S::kScaleSlots * S::kSlotFloats);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + BUFS;
  uint64_t* drain = tempty + BUFS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31u;
  const int rank = static_cast<int>(cluster_ctarank()), ranks = p.ranks;  // CTAs of the cluster
  const int n0 = static_cast<int>(blockIdx.x) / ranks * 128, m0 = static_cast<int>(blockIdx.y) * BT;
  const int kb0 = static_cast<int>(static_cast<long long>(p.k_blocks) * rank / ranks);
  const int kbs = static_cast<int>(static_cast<long long>(p.k_blocks) * (rank + 1) / ranks) - kb0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int a = 0; a < BUFS; ++a) {
      mbar_init(tfull + a, 1);
      mbar_init(tempty + a, S::kPromoteWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.tmA);
    tma_prefetch_desc(&p.tmB);
    tma_prefetch_desc(&p.tmSA);
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

  // the epilogue's four columns of a lane and their bias, on its way during the product
  const int col = n0 + static_cast<int>(lane) * 4;
  const bool col_in = col < p.g.N;
  float b4[4] = {0.f, 0.f, 0.f, 0.f};
  if (p.g.bias != nullptr && col_in) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.g.bias) + col));
    const float2 lo = unpack_bf16x2(u.x), hi = unpack_bf16x2(u.y);
    b4[0] = lo.x; b4[1] = lo.y; b4[2] = hi.x; b4[3] = hi.y;
  }

  constexpr int CW = S::kCols;
  float2 acc[CW / 2];
  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = policy_evict_normal();
      const uint32_t stage_bytes = S::kStageBytes - (BT - p.box_rows) * 128;
      uint32_t issued = 0, issued_parity = 0;
      for (int b = 0; b < kbs; ++b) {
        const int stage = b % STAGES;
        const uint32_t phase = static_cast<uint32_t>(b / STAGES) & 1u;
        if (!wait_bounded(empty + stage, phase ^ 1u, wc, kSiteBlockProducer)) break;
        mbar_arrive_expect_tx(full + stage, stage_bytes);
        tma_load_2d(sW + stage * S::kWTile, &p.tmB, full + stage, (kb0 + b) * 128, n0, pol);
        tma_load_2d(sT + stage * S::kTTile, &p.tmA, full + stage, (kb0 + b) * 128, m0, pol);
        float* slot = scale_ring + (b & (S::kScaleSlots - 1)) * S::kSlotFloats;
        tma_load_2d(slot, &p.tmSA, full + stage, m0, kb0 + b, pol);
        if (BVEC) tma_load_2d(slot + S::kRowFloats, &p.tmSB, full + stage, n0, kb0 + b, pol);
        issued |= 1u << stage;
        issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
      }
      for (int s = 0; s < STAGES; ++s)  // copies in flight land before their memory is used again
        if (issued & (1u << s)) wait_drain(full + s, (issued_parity >> s) & 1u, p.timeout_ns);
    }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_f8_f32(128, BT, static_cast<uint32_t>(p.g.b_fmt), static_cast<uint32_t>(p.g.a_fmt),
                                        false, false);
    const bool elected = elect_one();
    for (int b = 0; b < kbs; ++b) {
      const int stage = b % STAGES, buf = b % BUFS;
      if (!warp_wait(full + stage, static_cast<uint32_t>(b / STAGES) & 1u, wc, kSiteBlockMmaFull) ||
          !warp_wait(tempty + buf, (static_cast<uint32_t>(b / BUFS) & 1u) ^ 1u, wc, kSiteBlockMmaEmpty))
        break;
      tc_fence_after_sync();
      const uint32_t w_base = smem_u32(sW + stage * S::kWTile), t_base = smem_u32(sT + stage * S::kTTile);
      if (elected) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_f8(tmem_base + buf * BT, sdesc_sw128(w_base + k * 32, 16, 1024), sdesc_sw128(t_base + k * 32, 16, 1024),
                  idesc, k != 0 ? 1u : 0u);
        umma_commit(tfull + buf);
        umma_commit(empty + stage);
      }
      __syncwarp();
    }
    if (elected) {
      umma_commit(drain);
      wait_drain(drain, 0, p.timeout_ns);
    }
  } else {
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const uint32_t trow = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(half * CW);
    const float* sb = p.g.b_scales + (BVEC ? 0 : static_cast<long long>(n0 >> 7) * p.k_blocks + kb0);
    float sb_cur = 0.f, sb_next = 0.f;  // weight scales: lane l holds that of block 32 j + l
    if (!BVEC) {
      if (static_cast<int>(lane) < kbs) sb_cur = __ldg(sb + lane);
      if (32 + static_cast<int>(lane) < kbs) sb_next = __ldg(sb + 32 + lane);
    }
#pragma unroll
    for (int j = 0; j < CW / 2; ++j) acc[j] = make_float2(0.f, 0.f);
    for (int b = 0; b < kbs; ++b) {
      const int buf = b % BUFS;
      if (!warp_wait(tfull + buf, static_cast<uint32_t>(b / BUFS) & 1u, wc, kSiteBlockPromote)) break;
      tc_fence_after_sync();
      constexpr int kChunks = CW / 16, kAhead = kChunks < 3 ? kChunks : 3;  // 16-column loads in flight
      uint32_t r[kAhead][16];
#pragma unroll
      for (int c = 0; c < kAhead; ++c) tmem_load_16cols_async(trow + buf * BT + c * 16, r[c]);
      const float* slot = scale_ring + (b & (S::kScaleSlots - 1)) * S::kSlotFloats;
      const float sr = BVEC ? slot[S::kRowFloats + quad * 32 + lane] : __shfl_sync(0xffffffffu, sb_cur, b & 31);
      const float2 sr2 = make_float2(sr, sr);
      if (!BVEC && (b & 31) == 31) {
        sb_cur = sb_next;
        const int next = b + 33 + static_cast<int>(lane);
        sb_next = next < kbs ? __ldg(sb + next) : 0.f;
      }
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        uint32_t(&v)[16] = r[c % kAhead];
        float2 w[8];  // the chunk's products of scales, while its columns come
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float4 s = *reinterpret_cast<const float4*>(slot + half * CW + c * 16 + 2 * j);
          w[j] = __fmul2_rn(make_float2(s.x, s.y), sr2);
          w[j + 1] = __fmul2_rn(make_float2(s.z, s.w), sr2);
        }
        tmem_wait_ld(v);
        if (c == kChunks - kAhead) {  // every load has returned: the buffer is free before the last sums, not after them
#pragma unroll
          for (int i = 0; i < kAhead; ++i) tmem_wait_ld(r[i]);
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(tempty + buf);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          acc[c * 8 + j] = __ffma2_rn(make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), w[j], acc[c * 8 + j]);
        if (c + kAhead < kChunks) tmem_load_16cols_async(trow + buf * BT + (c + kAhead) * 16, v);
      }
    }
  }
  __syncthreads();  // the ring is drained: its memory holds the CTA's sums [BT][128] from here on
  float* red = reinterpret_cast<float*>(smem);
  if (warp >= 2) {
#pragma unroll
    for (int j = 0; j < CW / 2; ++j) {
      float* at = red + (((warp - 2) >> 2) * CW + 2 * j) * 128 + (warp & 3) * 32 + lane;
      at[0] = acc[j].x;
      at[128] = acc[j].y;
    }
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, S::kTmemCols);
  }
  cluster_sync_all();  // every CTA's sums are written (a cluster of one: a block barrier)
  const uint32_t red_addr = smem_u32(red) + lane * 16;
  const int rows = min(BT, p.g.M - m0);
  for (int j = rank + ranks * warp; j < rows; j += ranks * (S::kThreads / 32)) {
    const int row = m0 + j;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    float4 q[kFewMaxRanks];  // all in flight together, added in rank order
#pragma unroll
    for (int r = 0; r < kFewMaxRanks; ++r)
      q[r] = r < ranks ? ld_cluster_f4(mapa_shared(red_addr + j * 512, static_cast<uint32_t>(r))) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < kFewMaxRanks; ++r) {
      v[0] += q[r].x; v[1] += q[r].y; v[2] += q[r].z; v[3] += q[r].w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += b4[i];
    if constexpr (OUT == kOutFp32) {
      if (col_in) *reinterpret_cast<float4*>(static_cast<float*>(p.g.c) + row * p.g.ldc + col) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      const uint2 u = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      if constexpr (OUT == kOutBf16) {
        if (col_in) *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.g.c) + row * p.g.ldc + col) = u;
      } else {
        const long long at = static_cast<long long>(row) * p.g.N + col;
        if (p.g.pre != nullptr && col_in) *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.g.pre) + at) = u;
        const float2 h0 = gelu2(make_float2(v[0], v[1])), h1 = gelu2(make_float2(v[2], v[3]));
        float amax = col_in ? fmaxf(fmaxf(fabsf(h0.x), fabsf(h0.y)), fmaxf(fabsf(h1.x), fabsf(h1.y))) : 0.f;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const BlockScale b = block_scale(amax, 448.f);
        if (col_in) *reinterpret_cast<uint32_t*>(p.g.hq + at) = e4m3x4(h0.x, h0.y, h1.x, h1.y, b.inv);
        if (lane == 0) p.g.h_scales[(n0 >> 7) * p.m_pad + row] = b.scale;
      }
    }
  }
  cluster_sync_all();  // the cluster has read this CTA's sums
}

}  // namespace tpmlp
