// The block-scaled product for few rows of A (decoded tokens): every weight byte is read once, so the time is that of
// streaming B.  The operands change sides: a CTA takes 128 rows of B (output columns) as the UMMA's M and up to BT rows
// of A as its N (128 x BT x 32 UMMAs, cta_group::1); with 128 rows of A they stay on theirs.  The K blocks are split over
// a cluster of CTAs, whose fp32 sums are joined through distributed shared memory in rank order -- no workspace, no
// atomics, one launch.
//
// Warp 0 copies (TMA ring), warp 1 issues, the others promote: a thread holds BT sums of one output column, scaled per
// k-block by its own row scale of B and the scales of A (BT = 128: 64 sums of one row, or of one column).  With BT columns
// a partial sum, several fit in TMEM, so the promotion's latency is hidden.  In the end each CTA of the cluster finishes
// BT / C of the rows: a warp a few rows at a time, four consecutive columns a lane, which makes a 1 x 128 block of an
// 8-bit output one warp's.
//
// What bounds it: HBM, and a fixed part of about 3 us (set-up, the first bytes, the join).  Measured on GB300: one row,
// N = 4096, K = 16384 (67 MB) 13.2 us, 5.1 TB/s, with 256 CTAs in 32 clusters of eight (15.3 us with four CTAs a tile);
// 48 rows 15.9 us; 64 rows 16.8 us; 128 rows 17.8 us (one CTA an SM; a k-block of operands for all of them is 0.37 us, as
// fast as L2 gives them).  N = 16384, K = 4096: one row 13.3 us, 64 rows 16.3, 128 rows 18.0.
#pragma once

#include <type_traits>

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
  // A's rows as the UMMA's M: a thread's sums are of one row of A, and the scale of all of them in a k-block is one number.
  // With columns of A every lane reads the scales of 64 of them from shared memory: 0.45 us a k-block, now 0.37
  // (128 rows, N = 4096, K = 16384: 20.0 -> 17.9 us).  Column scales would cost the same reads in this order.
  static constexpr bool kRows = BT == 128 && !BVEC;
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
  constexpr bool kRows = S::kRows;
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
  if (p.g.bias != nullptr && col_in && TPMLP_IN_BOUNDS(col + 3, p.g.N, kBoundsBlockBias)) {
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
    const uint32_t fmt_a = static_cast<uint32_t>(p.g.a_fmt), fmt_b = static_cast<uint32_t>(p.g.b_fmt);
    const uint32_t idesc = idesc_f8_f32(128, BT, kRows ? fmt_a : fmt_b, kRows ? fmt_b : fmt_a, false, false);
    const bool elected = elect_one();
    for (int b = 0; b < kbs; ++b) {
      const int stage = b % STAGES, buf = b % BUFS;
      if (!warp_wait(full + stage, static_cast<uint32_t>(b / STAGES) & 1u, wc, kSiteBlockMmaFull) ||
          !warp_wait(tempty + buf, (static_cast<uint32_t>(b / BUFS) & 1u) ^ 1u, wc, kSiteBlockMmaEmpty))
        break;
      tc_fence_after_sync();
      const uint32_t w_base = smem_u32(sW + stage * S::kWTile), t_base = smem_u32(sT + stage * S::kTTile);
      const uint32_t m_base = kRows ? t_base : w_base, n_base = kRows ? w_base : t_base;
      if (elected) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_f8(tmem_base + buf * BT, sdesc_sw128(m_base + k * 32, 16, 1024), sdesc_sw128(n_base + k * 32, 16, 1024),
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
      float sr = BVEC ? slot[S::kRowFloats + quad * 32 + lane] : __shfl_sync(0xffffffffu, sb_cur, b & 31);
      if (kRows) sr *= slot[quad * 32 + lane];
      const float2 sr2 = make_float2(sr, sr);
      if (!BVEC && (b & 31) == 31) {
        sb_cur = sb_next;
        const int next = b + 33 + static_cast<int>(lane);
        sb_next = next < kbs ? __ldg(sb + next) : 0.f;
      }
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        uint32_t(&v)[16] = r[c % kAhead];
        float2 w[kRows ? 1 : 8];  // the chunk's products of scales, while its columns come
        if constexpr (kRows) {
          w[0] = sr2;
        } else {
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const float4 s = *reinterpret_cast<const float4*>(slot + half * CW + c * 16 + 2 * j);
            w[j] = __fmul2_rn(make_float2(s.x, s.y), sr2);
            w[j + 1] = __fmul2_rn(make_float2(s.z, s.w), sr2);
          }
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
          acc[c * 8 + j] = __ffma2_rn(make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), w[kRows ? 0 : j],
                                      acc[c * 8 + j]);
        if (c + kAhead < kChunks) tmem_load_16cols_async(trow + buf * BT + (c + kAhead) * 16, v);
      }
    }
  }
  // The ring is drained: its memory holds the CTA's sums [BT][128] from here on, with kRows the 16-byte pieces of row r at
  // places XOR r % 32 (a row a thread would hit one bank otherwise).
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);
  if (warp >= 2) {
    const int quad = warp & 3, half = (warp - 2) >> 2;
    if constexpr (kRows) {
#pragma unroll
      for (int j = 0; j < CW / 4; ++j)
        *reinterpret_cast<float4*>(red + (quad * 32 + lane) * 128 + ((half * (CW / 4) + j) ^ lane) * 4) =
            make_float4(acc[2 * j].x, acc[2 * j].y, acc[2 * j + 1].x, acc[2 * j + 1].y);
    } else {
#pragma unroll
      for (int j = 0; j < CW / 2; ++j) {
        float* at = red + (half * CW + 2 * j) * 128 + quad * 32 + lane;
        at[0] = acc[j].x;
        at[128] = acc[j].y;
      }
    }
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, S::kTmemCols);
  }
  cluster_sync_all();  // every CTA's sums are written (a cluster of one: a block barrier)
  const uint32_t red_addr = smem_u32(red);
  const int rows = min(BT, p.g.M - m0);
  // Several rows of a warp go through each step together: a read of another SM, the reduction of a block's largest value
  // and the divisions of its scale are long chains (128 rows, N = 16384, K = 4096: 19.9 -> 18.0 us, with GeLU 22.6 -> 20.1).
  const int step = ranks * (S::kThreads / 32);
  auto join = [&](auto rows_const, auto ranks_const) {
    constexpr int R = decltype(rows_const)::value, RANKS = decltype(ranks_const)::value;
    for (int j0 = rank + ranks * warp; j0 < rows; j0 += R * step) {
      float4 q[R][RANKS];
      float v[R][4];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int j = j0 + i * step;
        const uint32_t at = red_addr + j * 512 + (kRows ? lane ^ (j & 31) : lane) * 16;
#pragma unroll
        for (int r = 0; r < RANKS; ++r)
          q[i][r] = r < ranks && j < rows ? ld_cluster_f4(mapa_shared(at, static_cast<uint32_t>(r))) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.f;
#pragma unroll
        for (int r = 0; r < RANKS; ++r) {  // in rank order
          v[i][0] += q[i][r].x; v[i][1] += q[i][r].y; v[i][2] += q[i][r].z; v[i][3] += q[i][r].w;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) v[i][c] += b4[c];
      }
      if constexpr (OUT == kOutGelu8) {
        float2 h[R][2];
        float amax[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
          h[i][0] = gelu2(make_float2(v[i][0], v[i][1]));
          h[i][1] = gelu2(make_float2(v[i][2], v[i][3]));
          amax[i] = col_in ? fmaxf(fmaxf(fabsf(h[i][0].x), fabsf(h[i][0].y)), fmaxf(fabsf(h[i][1].x), fabsf(h[i][1].y))) : 0.f;
        }
        // Each exchange halves the rows that a lane holds: 32 / R lanes end with the largest value of one row and form its
        // scale, R rows' divisions at once.
        int o = 16;
#pragma unroll
        for (int n = R / 2; n >= 1; n /= 2, o /= 2)
#pragma unroll
          for (int i = 0; i < n; ++i) {
            const bool high = lane & o;
            const float keep = high ? amax[i + n] : amax[i], send = high ? amax[i] : amax[i + n];
            amax[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, o));
          }
#pragma unroll
        for (; o >= 1; o /= 2) amax[0] = fmaxf(amax[0], __shfl_xor_sync(0xffffffffu, amax[0], o));
        constexpr int kLanes = 32 / R;
        const BlockScale b = block_scale(amax[0], 448.f);
        const int jl = j0 + static_cast<int>(lane / kLanes) * step;
        if (lane % kLanes == 0 && jl < rows && scale_ok(p, n0 >> 7, m0 + jl))
          p.g.h_scales[(n0 >> 7) * p.m_pad + m0 + jl] = b.scale;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int j = j0 + i * step, row = m0 + j;
          const float inv = __shfl_sync(0xffffffffu, b.inv, i * kLanes);
          const long long at = static_cast<long long>(row) * p.g.N + col;
          if (col_in && j < rows && TPMLP_IN_BOUNDS(at + 3, static_cast<long long>(p.g.M) * p.g.N, kBoundsBlockGemm)) {
            if (p.g.pre != nullptr)
              *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.g.pre) + at) =
                  make_uint2(pack_bf16x2(v[i][0], v[i][1]), pack_bf16x2(v[i][2], v[i][3]));
            *reinterpret_cast<uint32_t*>(p.g.hq + at) = e4m3x4(h[i][0].x, h[i][0].y, h[i][1].x, h[i][1].y, inv);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int j = j0 + i * step;
          if (j >= rows || !col_in) continue;
          const long long at = static_cast<long long>(m0 + j) * p.g.ldc + col;
          if (!TPMLP_IN_BOUNDS(at + 3, (p.g.M - 1) * p.g.ldc + p.g.N, kBoundsBlockGemm)) continue;
          if constexpr (OUT == kOutFp32)
            *reinterpret_cast<float4*>(static_cast<float*>(p.g.c) + at) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
          else
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.g.c) + at) =
                make_uint2(pack_bf16x2(v[i][0], v[i][1]), pack_bf16x2(v[i][2], v[i][3]));
        }
      }
    }
  };
  // as many rows as there are reads in flight for, and one where a warp has no second (with GeLU: 14.2 -> 14.0 us, one row)
  if (OUT == kOutGelu8 && rows <= step) join(std::integral_constant<int, 1>{}, std::integral_constant<int, kFewMaxRanks>{});
  else if (ranks <= 2) join(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
  else join(std::integral_constant<int, 2>{}, std::integral_constant<int, kFewMaxRanks>{});
  cluster_sync_all();  // the cluster has read this CTA's sums
}

}  // namespace tpmlp
