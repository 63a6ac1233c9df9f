// The block-scaled product on CTA pairs (tcgen05, cta_group::2): a cluster of two CTAs computes a 256 x 256 tile of
//   C[m, n] = sum_kb sA[kb, m] sB[kb, n] sum_{k in kb} A8[m, k] B8[n, k].
//
// Each k-block of 128 is summed by the tensor cores into a partial sum in TMEM (four 256 x 256 x 32 UMMAs, the first
// of them overwriting), and eight promotion warps per CTA add it, scaled, to fp32 sums in registers: warp w owns the
// 32 rows of TMEM quadrant w % 4 and 128 of the tile's 256 columns, so a thread keeps 128 sums -- with weight scales, of
// one row: one 1 x 128 block of an 8-bit output, whose amax needs no exchange.  The partial sums are double-buffered
// (2 x 256 TMEM columns), so the UMMAs of k-block i + 1 run while block i is promoted.
//
// Why a whole 256 x 256 tile: with N = 128 an UMMA takes 131 cycles against 163 for N = 256 (measured; shared memory
// feeds both operands and takes the next copies), so four half-width buffers, which would hide the hand-over, lose more.
//
// What bounds it (clock64 on GB300, cycles a k-block): the UMMAs 650; but a buffer is in turn filled (650), committed and
// seen (320), read (370 to 440: eight 16-column loads with the products between them, a packed FMA of three registers
// taking three cycles) and handed back (100 in the even CTA, 230 from the odd one), and two buffers make that 740 to 800.
// A sustained run is at the power limit besides (1360 W at 1.67 GHz).  Measured at 8192 x 4096 x 16384: 370 us in a
// burst, 430 us sustained (2550 TFLOP/s; the per-tensor kernel, which promotes nothing, 306 and 351 us on the same
// codes).  With both operands scaled by rows (BVEC) the products double and the loads are the slower fragment form: 570
// us at 4096 x 16384 x 8192, about 1300 cycles a k-block.
//
// Synchronisation as in the per-tensor pair kernel: full / empty of the TMA ring, tfull / tempty of the partial sums,
// the barriers that count both CTAs in the even one.  All waits are bounded.  An arrive on tempty publishes nothing, so
// it is relaxed: a release at cluster scope waits for the thread's copies in flight and cost half the kernel's time.
#pragma once

#include "block_fp8.cuh"
#include "debug_bounds.cuh"

namespace tpmlp {

struct GemmBlockParams {
  CUtensorMap tmA, tmB;   // [M x K], [N x K] bytes; boxes of 128 bytes x 128 rows
  CUtensorMap tmSA, tmSB; // scales by rows, [k_blocks x m_pad] / [k_blocks x n_pad] fp32, boxes of one k-block
  CUtensorMap tmC;        // C (bf16 / fp32) or the pre-activation (bf16), 32 x 32 boxes
  CUtensorMap tmH;        // 8-bit output, boxes of 128 bytes x 32 rows
  GemmBlockLaunch g;
  int m_blocks, n_blocks, k_blocks;
  int ranks, box_rows;                 // few-row kernel: CTAs of a cluster, rows of a box of A
  uint32_t group_factor, group_shift;  // pair kernel: t / (kGroupM n_blocks) = (umulhi(t, factor) + t) >> shift, t < 2^31
  long long m_pad, n_pad;
  unsigned int* err;
  unsigned long long timeout_ns;
};

constexpr int kGroupM = 8;  // row blocks of a raster group

enum BlockOut : int { kOutBf16 = 0, kOutFp32 = 1, kOutGelu8 = 2 };

template <bool BVEC>
struct BlockPairShape {
  static constexpr int kStages = 4;  // a k-block is 700 to 800 cycles long: five stages measured the same
  static constexpr int kATile = 128 * 128, kBTile = 128 * 128;
  static constexpr int kStage = kATile + kBTile;
  static constexpr int kPromoteWarps = 8;
  static constexpr int kThreads = 128 + 32 * kPromoteWarps;
  static constexpr int kOutBuf = 4096;  // per promotion warp
  // Scales of a k-block: of the CTA's 128 rows, and of the tile's 256 columns (BVEC).  They are copied with the
  // k-block's operands and counted with them, so that partial sums that are there imply scales that are there.  A slot
  // is rewritten 16 k-blocks later.  The producer is at most kStages blocks ahead of the UMMAs, and those at most 2
  // ahead of the promotion, so by then every warp has left the slot's k-block; no barrier says so.
  static constexpr int kScaleSlots = 16;
  static constexpr int kSlotFloats = 128 + (BVEC ? 256 : 0);
  static constexpr int kSmem = 1024 + kStages * kStage + kPromoteWarps * kOutBuf + kScaleSlots * kSlotFloats * 4 + 512;
  static_assert(kStages + 4 < kScaleSlots, "see kScaleSlots");
  static constexpr int kStageBytes = kStage + kSlotFloats * 4;  // copied by a CTA for a k-block
  static_assert(kSmem <= 232448, "shared memory per block");
  // registers of the two warpgroups' kinds; together at most what the block is launched with (168 a thread)
  static constexpr int kIssueRegs = 40, kPromoteRegs = 232;
  static_assert(128 * kIssueRegs + 32 * kPromoteWarps * kPromoteRegs <= 168 * kThreads, "setmaxnreg split");
};

// Debug builds: is the scale of row `row` and 128-column block `block` of an 8-bit output inside its buffer?
__device__ __forceinline__ bool scale_ok(const GemmBlockParams& p, int block, int row) {
  return TPMLP_IN_BOUNDS(block, p.n_pad / kBlock, kBoundsBlockScales) && TPMLP_IN_BOUNDS(row, p.m_pad, kBoundsBlockScales);
}

// Where a warp's promotion leaves its 32 x 128 sums: float2 i of a thread.
//   rows (BVEC = false, tcgen05.ld 32x32b): row = lane, columns 2 i, 2 i + 1;
//   fragments (BVEC = true, 16x256b): i = 16 q + 8 h + 2 g + j, row 16 h + 8 j + lane / 4, columns 32 q + 8 g + 2 (lane % 4).
// The second form keeps only 32 columns a thread, so the columns' scales are 16 8-byte reads of shared memory a
// k-block and warp; with a row per thread they are 32 16-byte reads, every lane taking all of them, 1000 cycles of the
// SM's shared-memory bandwidth a k-block.

// Stage columns 32 q .. 32 q + 31 of the warp's rows as a box in `buf` (swizzled as the tensor maps say) and store it.
template <bool BVEC, bool F32>
__device__ __forceinline__ void store_box(const CUtensorMap* map, uint8_t* buf, const float2 (&acc)[64], int q,
                                          uint32_t lane, int col0, int row0, bool in) {
  if constexpr (BVEC) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 v = acc[16 * q + 8 * h + 2 * g + j];
          const uint32_t row = 16 * h + 8 * j + (lane >> 2);
          if constexpr (F32)
            *reinterpret_cast<float2*>(buf + row * 128 + (((2 * g + ((lane & 3) >> 1)) ^ (row & 7)) << 4) + 8 * (lane & 1)) = v;
          else
            *reinterpret_cast<uint32_t*>(buf + row * 64 + ((g ^ ((row >> 1) & 3)) << 4) + 4 * (lane & 3)) = pack_bf16x2(v.x, v.y);
        }
  } else if constexpr (F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 lo = acc[16 * q + 2 * j], hi = acc[16 * q + 2 * j + 1];
      *reinterpret_cast<float4*>(buf + lane * 128 + ((j ^ (lane & 7)) << 4)) = make_float4(lo.x, lo.y, hi.x, hi.y);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2* v = acc + 16 * q + 4 * j;
      *reinterpret_cast<uint4*>(buf + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
          make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y),
                     pack_bf16x2(v[3].x, v[3].y));
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (in) tma_store_2d(map, buf, col0 + 32 * q, row0);
    bulk_commit_group();  // an empty group where nothing is stored: the waits count groups
  }
}

// A warp's wait: short tries first, which cover the gaps of the pipeline's steady state, then the bounded wait.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtx& w, uint32_t site) {
#pragma unroll 1
  for (int i = 0; i < 8; ++i)
    if (__all_sync(0xffffffffu, mbar_try_wait_short(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_bounded(bar, parity, w, site));
}

template <int OUT, bool BVEC>
__global__ void __launch_bounds__(BlockPairShape<BVEC>::kThreads, 1) k_gemm_block_pair(const __grid_constant__ GemmBlockParams p) {
  using S = BlockPairShape<BVEC>;
  constexpr bool kFrag = BVEC;  // layout of the sums, see store_box
  constexpr int STAGES = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + STAGES * S::kATile;
  uint8_t* out_bufs = sB + STAGES * S::kBTile;
  float* scale_ring = reinterpret_cast<float*>(out_bufs + S::kPromoteWarps * S::kOutBuf);
  uint64_t* full = reinterpret_cast<uint64_t*>(scale_ring + S::kScaleSlots * S::kSlotFloats);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull + a, 1);
      mbar_init(tempty + a, 2 * S::kPromoteWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.tmA);
    tma_prefetch_desc(&p.tmB);
    tma_prefetch_desc(OUT == kOutGelu8 ? &p.tmH : &p.tmC);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();  // the peer's barriers are initialised before any remote arrive or copy
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  const WaitCtx wc{abort_flag, p.err, p.timeout_ns};
  const int num_tiles = p.m_blocks * p.n_blocks;
  const int cluster_id = blockIdx.x >> 1;
  const int num_clusters = gridDim.x >> 1;
  // Tile t: groups of kGroupM row blocks, column by column.  The quotient by a whole group comes from the host's factor
  // (a division of unknown operands is over a hundred cycles, on every warp's way into a tile).
  auto tile_at = [&](int t, int& mb, int& nb) {
    const int g = static_cast<int>((__umulhi(static_cast<uint32_t>(t), p.group_factor) + static_cast<uint32_t>(t)) >> p.group_shift);
    const int first = g * kGroupM, rest = t - first * p.n_blocks, gm = p.m_blocks - first;
    if (gm >= kGroupM) {
      mb = first + rest % kGroupM;
      nb = rest / kGroupM;
    } else {
      mb = first + rest % gm;
      nb = rest / gm;
    }
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kIssueRegs));
    if (warp == 0) {
      if (lane == 0) {
        // ------------------------------------------------------------------ producer (both CTAs)
        const uint64_t pol_a = policy_evict_normal(), pol_b = policy_evict_last();
        int stage = 0;
        uint32_t phase = 0, issued = 0, issued_parity = 0, blk = 0;
        bool ok = true;
        for (int t = cluster_id; ok && t < num_tiles; t += num_clusters) {
          int mb, nb;
          tile_at(t, mb, nb);
          const int m0 = mb * 256 + static_cast<int>(rank) * 128, n0 = nb * 256 + static_cast<int>(rank) * 128;
          for (int kb = 0; kb < p.k_blocks; ++kb, ++blk) {
            if (!wait_bounded(empty + stage, phase ^ 1u, wc, kSiteBlockProducer)) {
              ok = false;
              break;
            }
            if (leader) mbar_arrive_expect_tx(full + stage, 2 * S::kStageBytes);
            const uint32_t bar = mapa_shared(smem_u32(full + stage), 0);
            tma_load_2d_pair(sA + stage * S::kATile, &p.tmA, bar, kb * 128, m0, pol_a);
            tma_load_2d_pair(sB + stage * S::kBTile, &p.tmB, bar, kb * 128, n0, pol_b);
            float* slot = scale_ring + (blk & (S::kScaleSlots - 1)) * S::kSlotFloats;
            tma_load_2d_pair(slot, &p.tmSA, bar, m0, kb, pol_a);
            if (BVEC) tma_load_2d_pair(slot + 128, &p.tmSB, bar, nb * 256, kb, pol_a);
            issued |= 1u << stage;
            issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        // copies in flight land before shared memory is released (the odd CTA is held at the closing cluster barrier)
        if (leader)
          for (int s = 0; s < STAGES; ++s)
            if (issued & (1u << s)) wait_drain(full + s, (issued_parity >> s) & 1u, p.timeout_ns);
      }
    } else if (warp == 1) {
      if (leader) {
        // ------------------------------------------------------------------ MMA issuer (even CTA)
        // The whole warp walks the loop and one elected lane issues: descriptors are then warp-uniform, and an issue
        // costs a few cycles where a loop of one lane alone took about 75 for each (measured, clock64).
        const uint32_t idesc = idesc_f8_f32(256, 256, static_cast<uint32_t>(p.g.a_fmt), static_cast<uint32_t>(p.g.b_fmt),
                                            false, false);
        const bool elected = elect_one();
        int stage = 0;
        uint32_t phase = 0, blk = 0;
        bool ok = true;
        for (int t = cluster_id; ok && t < num_tiles; t += num_clusters) {
          for (int kb = 0; kb < p.k_blocks; ++kb, ++blk) {
            const uint32_t acc = blk & 1u;
            if (!warp_wait(full + stage, phase, wc, kSiteBlockMmaFull) ||
                !warp_wait(tempty + acc, ((blk >> 1) & 1u) ^ 1u, wc, kSiteBlockMmaEmpty)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            const uint32_t a_base = smem_u32(sA + stage * S::kATile), b_base = smem_u32(sB + stage * S::kBTile);
            if (elected) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_f8_pair(tmem_base + acc * 256, sdesc_sw128(a_base + k * 32, 16, 1024),
                             sdesc_sw128(b_base + k * 32, 16, 1024), idesc, k != 0 ? 1u : 0u);
              umma_commit_pair_multicast(tfull + acc, 0x3);
              umma_commit_pair_multicast(empty + stage, 0x3);
            }
            __syncwarp();
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        if (elected) {
          umma_commit_pair(drain);
          wait_drain(drain, 0, p.timeout_ns);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kPromoteRegs));
    // -------------------------------------------------------------------- promotion and epilogue (both CTAs)
    const int quad = warp & 3, half = (warp - 4) >> 2;
    uint8_t* buf = out_bufs + (warp - 4) * S::kOutBuf;
    const uint32_t tempty0 = mapa_shared(smem_u32(tempty), 0), tempty1 = mapa_shared(smem_u32(tempty + 1), 0);
    const uint32_t trow = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(half * 128);
    uint32_t blk = 0;
    bool ok = true;
    for (int t = cluster_id; ok && t < num_tiles; t += num_clusters) {
      int mb, nb;
      tile_at(t, mb, nb);
      const int row0 = mb * 256 + static_cast<int>(rank) * 128 + quad * 32;
      const int row = row0 + static_cast<int>(lane);
      const int col0 = nb * 256 + half * 128;
      // Weight scales (one per 128 columns and k-block): lane l holds that of block 32 j + l.
      const float* sb = p.g.b_scales + (BVEC || col0 >= p.n_pad ? 0 : static_cast<long long>(col0 >> 7) * p.k_blocks);
      float sb_cur = 0.f, sb_next = 0.f;
      if (!BVEC) {
        if (static_cast<int>(lane) < p.k_blocks) sb_cur = __ldg(sb + lane);
        if (32 + static_cast<int>(lane) < p.k_blocks) sb_next = __ldg(sb + 32 + lane);
      }
      float2 acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.f, 0.f);
      for (int kb = 0; kb < p.k_blocks; ++kb, ++blk) {
        const uint32_t ab = blk & 1u;
        const float* slot = scale_ring + (blk & (S::kScaleSlots - 1)) * S::kSlotFloats;
        ok = warp_wait(tfull + ab, (blk >> 1) & 1u, wc, kSiteBlockPromote);
        if (!ok) break;
        tc_fence_after_sync();
        const uint32_t tcol = trow + ab * 256;
        auto release = [&] {  // every load has returned: the buffer is free before the last sums, not after them
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) {
            if (leader) mbar_arrive(tempty + ab);
            else mbar_arrive_remote_relaxed(ab ? tempty1 : tempty0);
          }
        };
        if constexpr (kFrag) {
          // 4096 x 16384 x 8192: 570 us, without the products 366, without the loads 509.  Both of the latter hand the buffer
          // back where it is handed back now, so they do not tell the products' time from a buffer's stay with this warp;
          // the FMA pipe is busy 42% of the time.  A packed instruction takes longer the more registers it reads: rows
          // first, one scale for four products in a row, then columns, one scale for four sums (columns first: 593; a
          // row's two steps after each other: 593; scalar: 691).
          uint32_t r[4][16];
          auto load = [&](int u) {  // rows 0 to 15 and 16 to 31 of columns 32 u to 32 u + 31
#pragma unroll
            for (int h = 0; h < 2; ++h)
              tmem_load_16x32_async(tcol + (static_cast<uint32_t>(h * 16) << 16) + u * 32, r[2 * (u & 1) + h]);
          };
          load(0);
          float2 rs[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float f = slot[quad * 32 + 8 * i + (lane >> 2)];
            rs[i] = make_float2(f, f);
          }
          const float* cs = slot + 128 + half * 128 + 2 * (lane & 3);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float2 c2[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) c2[g] = *reinterpret_cast<const float2*>(cs + u * 32 + 8 * g);
            tmem_wait_ld(r[2 * (u & 1)]);
            tmem_wait_ld(r[2 * (u & 1) + 1]);
            if (u == 3) release();
            else load(u + 1);
            float2 q[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                const uint32_t* v = r[2 * (u & 1) + (i >> 1)] + 4 * g + 2 * (i & 1);
                q[i][g] = make_float2(__uint_as_float(v[0]), __uint_as_float(v[1]));
              }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int g = 0; g < 4; ++g) q[i][g] = __fmul2_rn(q[i][g], rs[i]);
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float2& a = acc[16 * u + 8 * (i >> 1) + 2 * g + (i & 1)];
                a = __ffma2_rn(q[i][g], c2[g], a);
              }
          }
        } else {
          uint32_t r[3][16];
#pragma unroll
          for (int c = 0; c < 3; ++c) tmem_load_16cols_async(tcol + c * 16, r[c]);
          const float f = slot[quad * 32 + lane] * __shfl_sync(0xffffffffu, sb_cur, kb & 31);
          const float2 rs = make_float2(f, f);
          if ((kb & 31) == 31) {
            sb_cur = sb_next;
            const int next = kb + 33 + static_cast<int>(lane);
            sb_next = next < p.k_blocks ? __ldg(sb + next) : 0.f;
          }
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t(&v)[16] = r[c % 3];
            tmem_wait_ld(v);
            if (c == 5) {
              tmem_wait_ld(r[0]);
              tmem_wait_ld(r[1]);
              release();
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              acc[c * 8 + i] = __ffma2_rn(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), rs, acc[c * 8 + i]);
            if (c < 5) tmem_load_16cols_async(tcol + (c + 3) * 16, v);
          }
        }
      }
      if (!ok) break;
      // ------------------------------------------------------------------ epilogue of the tile
      const bool in_m = row0 < p.g.M;
      if (p.g.bias != nullptr) {
        const __nv_bfloat16* bias = static_cast<const __nv_bfloat16*>(p.g.bias) + col0;
        if constexpr (kFrag) {
#pragma unroll
          for (int g = 0; g < 16; ++g) {
            const int c = 8 * g + 2 * static_cast<int>(lane & 3);
            const float2 b = col0 + c < p.g.N && TPMLP_IN_BOUNDS(col0 + c + 1, p.g.N, kBoundsBlockBias) ? unpack_bf16x2(__ldg(reinterpret_cast<const uint32_t*>(bias + c)))
                                              : make_float2(0.f, 0.f);
#pragma unroll
            for (int hj = 0; hj < 4; ++hj) {
              float2& a = acc[16 * (g >> 2) + 8 * (hj >> 1) + 2 * (g & 3) + (hj & 1)];
              a = __fadd2_rn(a, b);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint4 u = col0 + 8 * j < p.g.N && TPMLP_IN_BOUNDS(col0 + 8 * j + 7, p.g.N, kBoundsBlockBias) ? __ldg(reinterpret_cast<const uint4*>(bias) + j) : make_uint4(0, 0, 0, 0);
            acc[4 * j] = __fadd2_rn(acc[4 * j], unpack_bf16x2(u.x));
            acc[4 * j + 1] = __fadd2_rn(acc[4 * j + 1], unpack_bf16x2(u.y));
            acc[4 * j + 2] = __fadd2_rn(acc[4 * j + 2], unpack_bf16x2(u.z));
            acc[4 * j + 3] = __fadd2_rn(acc[4 * j + 3], unpack_bf16x2(u.w));
          }
        }
      }
      if (OUT != kOutGelu8 || p.g.pre != nullptr) {
        constexpr bool kF32 = OUT == kOutFp32;  // a 4 KB box, or 2 KB boxes in the halves of the buffer
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          // what was stored from this part of the buffer has left it
          if (lane == 0) {
            if (kF32 || q == 0) bulk_wait_read_all();
            else if (q >= 2) bulk_wait_read_1();
          }
          __syncwarp();
          store_box<kFrag, kF32>(&p.tmC, buf + (kF32 ? 0 : (q & 1) * 2048), acc, q, lane, col0, row0,
                                in_m && col0 + 32 * q < p.g.N);
        }
      }
      if constexpr (OUT == kOutGelu8) {
        // GeLU and the thread's own 1 x 128 block (columns at or past N hold zeros, GeLU(0) = 0)
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          acc[i] = gelu2(acc[i]);
          amax = fmaxf(amax, fmaxf(fabsf(acc[i].x), fabsf(acc[i].y)));
        }
        const BlockScale b = block_scale(amax, 448.f);
        if (row < p.g.M && col0 < p.g.N && scale_ok(p, col0 >> 7, row))
          p.g.h_scales[(col0 >> 7) * p.m_pad + row] = b.scale;
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2* h = acc + 8 * j;
          *reinterpret_cast<uint4*>(buf + lane * 128 + ((j ^ (lane & 7)) << 4)) =
              make_uint4(e4m3x4(h[0].x, h[0].y, h[1].x, h[1].y, b.inv), e4m3x4(h[2].x, h[2].y, h[3].x, h[3].y, b.inv),
                         e4m3x4(h[4].x, h[4].y, h[5].x, h[5].y, b.inv), e4m3x4(h[6].x, h[6].y, h[7].x, h[7].y, b.inv));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && in_m && col0 < p.g.N) {
          tma_store_2d(&p.tmH, buf, col0, row0);
          bulk_commit_group();
        }
      }
    }
    if (lane == 0) bulk_wait_all();  // box stores complete before the block's shared memory is released
  }

  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

}  // namespace tpmlp
