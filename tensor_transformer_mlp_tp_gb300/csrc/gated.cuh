// Epilogues of the gated feed-forward block: H = act(G) * U of two products that lie side by side in TMEM, and its
// derivatives  dU = dH act(G),  dG = dH U act'(G).
// SiLU(x) = x s(x) with s(x) = 1 / (1 + exp(-x)), SiLU'(x) = s(x) (1 + x (1 - s(x))); the exact GeLU x Phi(x) as in
// ptx.cuh.  All of it in fp32 on the hardware's 2^x and 1/x; an output is rounded once.  H, dG and dU are rounded to bf16
// between the products, whose operands are bf16: Y and the gradients are then off by about 1.4 roundings of their type instead
// of one (2.3e-3 instead of 1.7e-3 of the norm).
#pragma once

#include "gemm_tc.cuh"

namespace tpmlp {

constexpr float kLog2e = 1.4426950408889634f;

// s(x) of two values: exp(-x) = 2^(-x log2 e); past its range 1 / (1 + inf) = 0.
__device__ __forceinline__ float2 sigmoid2(float2 x) {
  const float2 m = __fmul2_rn(make_float2(-kLog2e, -kLog2e), x);
  return make_float2(rcp_approx(1.f + ex2_approx(m.x)), rcp_approx(1.f + ex2_approx(m.y)));
}

__device__ __forceinline__ float2 act2(int act, float2 x) {
  return act == kActSilu ? __fmul2_rn(x, sigmoid2(x)) : gelu2(x);
}

// act(x) and act'(x) of two values.
__device__ __forceinline__ void act_slope2(int act, float2 x, float2& a, float2& slope) {
  if (act == kActSilu) {
    const float2 s = sigmoid2(x);
    a = __fmul2_rn(x, s);
    // s + x s (1 - s)
    slope = __ffma2_rn(a, __ffma2_rn(make_float2(-1.f, -1.f), s, make_float2(1.f, 1.f)), s);
  } else {
    const NormalCdfPdf2 n = normal_cdf_pdf2(x);
    a = __fmul2_rn(x, n.cdf);
    slope = __ffma2_rn(x, n.pdf, n.cdf);
  }
}

__device__ __forceinline__ void add_bias_32(const void* bias, int col0, int N, float (&v)[32]) {
  if (bias == nullptr) return;
  float b[32];
  load_row32(static_cast<const __nv_bfloat16*>(bias), col0, N, b);
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] += b[i];
}

// 32 columns of output `which` (0, 1, 2), through a box store where p.tma_out has its bit.
__device__ __forceinline__ void put_row32(const GemmParams& p, int which, const CUtensorMap* map, void* out, long long ld,
                                          const float (&v)[32], int row, int col0, uint32_t lane, uint8_t* sbuf) {
  if (p.tma_out >> which & 1) {
    box_store_bf16_32(map, sbuf, v, lane, col0, row - static_cast<int>(lane), p.M, p.N);
  } else if (row < p.M) {
    store_row32(static_cast<__nv_bfloat16*>(out) + static_cast<long long>(row) * ld, col0, p.N, v);
  }
}

// g, u: 32 columns of one row of both products.
__device__ __forceinline__ void gated_epilogue_32(const GemmParams& p, float (&g)[32], float (&u)[32], int row, int col0,
                                                  uint32_t lane, uint8_t* sbuf) {
  add_bias_32(p.bias, col0, p.N, g);
  add_bias_32(p.bias_u, col0, p.N, u);
  if (p.out1 != nullptr) put_row32(p, 1, &p.tmC1, p.out1, p.ld1, g, row, col0, lane, sbuf);
  if (p.out2 != nullptr) put_row32(p, 2, &p.tmC2, p.out2, p.ld1, u, row, col0, lane, sbuf);
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float2 h = __fmul2_rn(act2(p.act, make_float2(g[i], g[i + 1])), make_float2(u[i], u[i + 1]));
    g[i] = h.x;
    g[i + 1] = h.y;
  }
  put_row32(p, 0, &p.tmC0, p.out0, p.ld0, g, row, col0, lane, sbuf);
}

// Sums of 32 columns over a warp's rows into its partial row (four a 128-row block; see epilogue_32).
__device__ __forceinline__ void colsum_32(const GemmParams& p, float* colsum, float (&v)[32], int col0, int mb, int quad,
                                          uint32_t lane) {
  const float s = warp_column_sums(v, lane);
  const int col = col0 + static_cast<int>(lane);
  if (col < p.N && mb * kBM < p.M && TPMLP_IN_BOUNDS(mb * 4 + quad, 4 * ((p.M + kBM - 1) / kBM), kBoundsGemmColsum))
    colsum[(mb * 4 + quad) * p.ld_colsum + col] = s;
}

// d: 32 columns of dH = dY B^T; raw: G and U there (zeros outside the matrix).
__device__ __forceinline__ void dgated_epilogue_32(const GemmParams& p, float (&d)[32], const uint4 (&g_raw)[4],
                                                   const uint4 (&u_raw)[4], int row, int col0, int mb, int quad,
                                                   uint32_t lane, uint8_t* sbuf) {
  float g[32], u[32];
  unpack_row32(g_raw, g);
  unpack_row32(u_raw, u);
  const bool row_ok = row < p.M;
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    float2 a, slope;
    act_slope2(p.act, make_float2(g[i], g[i + 1]), a, slope);
    const float2 uu = make_float2(u[i], u[i + 1]);
    const float2 dd = row_ok ? make_float2(d[i], d[i + 1]) : make_float2(0.f, 0.f);
    const float2 h = __fmul2_rn(a, uu), dg = __fmul2_rn(__fmul2_rn(dd, uu), slope), du = __fmul2_rn(dd, a);
    g[i] = dg.x; g[i + 1] = dg.y;
    u[i] = du.x; u[i + 1] = du.y;
    d[i] = h.x; d[i + 1] = h.y;
  }
  put_row32(p, 0, &p.tmC0, p.out0, p.ld0, g, row, col0, lane, sbuf);
  put_row32(p, 1, &p.tmC1, p.out1, p.ld1, u, row, col0, lane, sbuf);
  if (p.out2 != nullptr) put_row32(p, 2, &p.tmC2, p.out2, p.ld1, d, row, col0, lane, sbuf);
  if (p.colsum != nullptr) colsum_32(p, p.colsum, g, col0, mb, quad, lane);
  if (p.colsum_u != nullptr) colsum_32(p, p.colsum_u, u, col0, mb, quad, lane);
}

}  // namespace tpmlp
