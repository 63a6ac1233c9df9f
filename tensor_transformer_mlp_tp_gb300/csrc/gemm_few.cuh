// The bf16 product for few rows (decoded tokens): every weight is read once, so the time is that of streaming the weights.
// W [K x N] as it is stored (math layout).  The operands change sides: a CTA takes 128 columns of W as the UMMA's M
// (MN-major) and up to BT rows of X as its N, so that a k-block of 64 is four 128 x BT x 16 UMMAs and X costs next to
// nothing.  MATS = 2: the same columns of both projections of the gated block, act(G) * U formed at the end.  The
// k-blocks are split over a cluster of CTAs, whose fp32 sums are joined through distributed shared memory in rank order: no
// workspace, no atomics, the same bits every time.
//
// Measured, d = 4096, F = 16384, both products of the gated block (403 MB of weights): 60.3 us for one token (6.6 TB/s, 0.99 of
// the measured copy rate), 61.1 for 8, 65.3 for 32, 68.6 for 64, 77.5 for 128.  Two CTAs an SM up to 32 rows: while one joins
// or starts, the other keeps copies in flight.
//
// Warp 0 copies (TMA ring), warp 1 issues, warps 2..5 bring the sums from TMEM to shared memory; then every warp finishes
// rows, four consecutive columns a lane.
#pragma once

#include "gated.cuh"

namespace tpmlp {

constexpr int kFewCols = 128;  // columns of W a CTA
constexpr int kFewRanks = 8;   // CTAs of a cluster at most

struct GemmFewParams {
  CUtensorMap tmX, tmW[2];  // X: boxes of 64 x box_rows; W: boxes of 64 columns x 64 rows
  int M, N, k_blocks, ranks, box_rows;
  int act;
  int early_weights;        // W is not written by the kernel before: its first copies need not wait for that one's end
  const void* bias[2];      // [N] bf16 or nullptr
  void* out;                // [M x N] bf16
  void* pre[2];             // MATS = 2: both factors before the activation, or nullptr
  unsigned int* err;
  unsigned long long timeout_ns;
};

template <int BT, int MATS>
struct GemmFewShape {
  static_assert(BT == 16 || BT == 32 || BT == 64 || BT == 128, "BT");
  static constexpr int kWTile = MATS * kFewCols * kBK * 2, kXTile = BT * kBK * 2, kStage = kWTile + kXTile;
  static constexpr int kCtas = BT <= 32 ? 2 : 1;  // an SM
  static constexpr int kStages = (kCtas == 2 ? 111000 : 210000) / kStage;
  static constexpr int kTmemCols = MATS * BT < 32 ? 32 : MATS * BT;
  static constexpr int kThreads = 192;
  static constexpr int kSmem = 1024 + kStages * kStage + 256;
  static_assert(kStages >= 3 && kStages <= 12, "ring");
  static_assert(kStages * kStage >= MATS * BT * kFewCols * 4, "the sums are joined in the ring's memory");
  static_assert(kCtas * (kSmem + 1024) <= 233472, "shared memory");
};

// grid: (cluster size x column tiles)
template <int BT, int MATS>
__global__ void __launch_bounds__(GemmFewShape<BT, MATS>::kThreads, GemmFewShape<BT, MATS>::kCtas)
    k_gemm_few(const __grid_constant__ GemmFewParams p) {
  using S = GemmFewShape<BT, MATS>;
  constexpr int STAGES = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * S::kStage);
  uint64_t* empty = full + STAGES;
  uint64_t* done = empty + STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31u;
  const int rank = static_cast<int>(cluster_ctarank()), ranks = p.ranks;
  const int n0 = static_cast<int>(blockIdx.x) / ranks * kFewCols;
  const int kb0 = static_cast<int>(static_cast<long long>(p.k_blocks) * rank / ranks);
  const int kbs = static_cast<int>(static_cast<long long>(p.k_blocks) * (rank + 1) / ranks) - kb0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.tmX);
    for (int i = 0; i < MATS; ++i) tma_prefetch_desc(&p.tmW[i]);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  const WaitCtx wc{abort_flag, p.err, p.timeout_ns};

  const uint64_t pol = policy_evict_normal();
  const uint32_t stage_bytes = static_cast<uint32_t>(S::kWTile + p.box_rows * kBK * 2);
  auto load_weights = [&](int b) {
    uint8_t* dst = smem + b % STAGES * S::kStage;
#pragma unroll
    for (int i = 0; i < MATS; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        tma_load_2d(dst + (2 * i + j) * 64 * kBK * 2, &p.tmW[i], full + b % STAGES, n0 + 64 * j, (kb0 + b) * kBK, pol);
  };
  int ahead = 0;  // stages whose weights are on their way
  if (p.early_weights && warp == 0 && lane == 0)
    for (; ahead < STAGES && ahead < kbs; ++ahead) {
      mbar_arrive_expect_tx(full + ahead, stage_bytes);
      load_weights(ahead);
    }
  griddep_wait();
  griddep_launch_dependents();

  if (warp == 0) {
    if (lane == 0) {
      uint32_t issued = 0, issued_parity = 0;
      for (int b = 0; b < kbs; ++b) {
        const int stage = b % STAGES;
        const uint32_t phase = static_cast<uint32_t>(b / STAGES) & 1u;
        if (b >= ahead) {
          if (!wait_bounded(empty + stage, phase ^ 1u, wc, kSiteFewProducer)) break;
          mbar_arrive_expect_tx(full + stage, stage_bytes);
          load_weights(b);
        }
        tma_load_2d(smem + stage * S::kStage + S::kWTile, &p.tmX, full + stage, (kb0 + b) * kBK, 0, pol);
        issued |= 1u << stage;
        issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
      }
      for (int s = 0; s < STAGES; ++s)  // copies in flight land before their memory is used again
        if (issued & (1u << s)) wait_drain(full + s, (issued_parity >> s) & 1u, p.timeout_ns);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(kFewCols, BT, true, false);
      for (int b = 0; b < kbs; ++b) {
        const int stage = b % STAGES;
        if (!wait_bounded(full + stage, static_cast<uint32_t>(b / STAGES) & 1u, wc, kSiteFewMma)) break;
        tc_fence_after_sync();
        const uint32_t w_base = smem_u32(smem + stage * S::kStage), x_base = w_base + S::kWTile;
#pragma unroll
        for (int i = 0; i < MATS; ++i)
#pragma unroll
          for (int k = 0; k < kBK / kUmmaK; ++k)
            umma_bf16(tmem_base + i * BT, sdesc_sw128(w_base + i * (kFewCols * kBK * 2) + k * 2048, 64 * kBK * 2, 1024),
                      sdesc_sw128(x_base + k * 32, 16, 1024), idesc, (b | k) != 0 ? 1u : 0u);
        umma_commit(empty + stage);
      }
      umma_commit(done);
      wait_drain(done, 0, p.timeout_ns);
    }
  }
  // Every copy has landed and, once `done` completes, every UMMA has read it: the ring's memory holds the CTA's sums
  // [MATS][BT][128] from here on.
  float* red = reinterpret_cast<float*>(smem);
  if (warp >= 2) {
    int ok = 1;
    if (lane == 0) ok = wait_bounded(done, 0, wc, kSiteFewEpilogue) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    tc_fence_after_sync();
    const int quad = warp & 3;
    if (ok) {
      const uint32_t trow = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
      for (int c = 0; c < MATS * BT; c += 16) {
        if (c % BT >= p.M) continue;
        uint32_t r[16];
        tmem_load_16cols_async(trow + c, r);
        tmem_wait_ld(r);
#pragma unroll
        for (int j = 0; j < 16; ++j) red[(c + j) * kFewCols + quad * 32 + lane] = __uint_as_float(r[j]);
      }
    }
    tc_fence_before_sync();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, S::kTmemCols);
  }
  cluster_sync_all();  // every CTA's sums are written (a cluster of one: a block barrier)
  const int col = n0 + static_cast<int>(lane) * 4;
  const bool col_in = col < p.N;
  const uint32_t red_addr = smem_u32(red);
  for (int row = rank + ranks * warp; row < p.M; row += ranks * (S::kThreads / 32)) {
    float v[MATS][4];
#pragma unroll
    for (int i = 0; i < MATS; ++i) {
      float4 q[kFewRanks];
#pragma unroll
      for (int r = 0; r < kFewRanks; ++r)
        q[r] = r < ranks ? ld_cluster_f4(mapa_shared(red_addr + ((i * BT + row) * kFewCols + lane * 4) * 4, static_cast<uint32_t>(r)))
                         : make_float4(0.f, 0.f, 0.f, 0.f);
      v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.f;
#pragma unroll
      for (int r = 0; r < kFewRanks; ++r) {  // in rank order
        v[i][0] += q[r].x; v[i][1] += q[r].y; v[i][2] += q[r].z; v[i][3] += q[r].w;
      }
      if (p.bias[i] != nullptr && col_in) {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.bias[i]) + col));
        const float2 lo = unpack_bf16x2(u.x), hi = unpack_bf16x2(u.y);
        v[i][0] += lo.x; v[i][1] += lo.y; v[i][2] += hi.x; v[i][3] += hi.y;
      }
    }
    const long long at = static_cast<long long>(row) * p.N + col;
    if (!col_in || !TPMLP_IN_BOUNDS(at + 3, static_cast<long long>(p.M) * p.N, kBoundsGemmFew)) continue;
    if constexpr (MATS == 2) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (p.pre[i] != nullptr)
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.pre[i]) + at) =
              make_uint2(pack_bf16x2(v[i][0], v[i][1]), pack_bf16x2(v[i][2], v[i][3]));
      const float2 a = __fmul2_rn(act2(p.act, make_float2(v[0][0], v[0][1])), make_float2(v[1][0], v[1][1]));
      const float2 b = __fmul2_rn(act2(p.act, make_float2(v[0][2], v[0][3])), make_float2(v[1][2], v[1][3]));
      v[0][0] = a.x; v[0][1] = a.y; v[0][2] = b.x; v[0][3] = b.y;
    }
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) =
        make_uint2(pack_bf16x2(v[0][0], v[0][1]), pack_bf16x2(v[0][2], v[0][3]));
  }
  cluster_sync_all();  // the cluster has read this CTA's sums
}

}  // namespace tpmlp
