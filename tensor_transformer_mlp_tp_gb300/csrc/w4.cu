// Products with 4-bit weights and group scales, their quantiser and its inverse.
#include <cuda_bf16.h>

#include <climits>

#include "debug_bounds.cuh"
#include "gated.cuh"
#include "w4.cuh"

namespace tpmlp {
namespace {

constexpr float kW4Tiny = 7.8886090522101181e-31f;  // 2^-100, the least range a scale is made from
constexpr float kW4Big = 3.3895313892515355e38f;    // bf16's largest number, the largest

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

constexpr int kWarps = 8;

// Eight tokens (blockIdx.y) and 16 columns (blockIdx.x) a block; its warps share K and join their sums in shared memory.
template <bool GATED>
__global__ void __launch_bounds__(32 * kWarps) k_gemm_w4(const __grid_constant__ W4Launch p) {
  constexpr int MATS = GATED ? 2 : 1;
  __shared__ float red[kWarps][MATS][16][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kW4Cols, m = blockIdx.y * 8 + g;
  const int k_tiles = (p.K + kW4Rows - 1) / kW4Rows, groups = (p.K + p.group - 1) / p.group;
  const int kt0 = static_cast<int>(static_cast<long long>(k_tiles) * warp / kWarps);
  const int kt1 = static_cast<int>(static_cast<long long>(k_tiles) * (warp + 1) / kWarps);
  const uint32_t* x = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.x) + static_cast<long long>(m < p.M ? m : 0) * p.K);
  float sum[MATS][4] = {};
  for (int kt = kt0; kt < kt1; ++kt) {
    uint32_t b[4][2];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = kt * kW4Rows + 16 * j + 8 * h + 2 * t;
        b[j][h] = m < p.M && k < p.K ? __ldg(x + k / 2) : 0u;
      }
#pragma unroll
    for (int i = 0; i < MATS; ++i) {
      const W4Matrix& w = p.w[i];
      const uint4 q4 = __ldg(w.q + (static_cast<long long>(blockIdx.x) * k_tiles + kt) * 32 + lane);
      const uint32_t q[4] = {q4.x, q4.y, q4.z, q4.w};
      const int steps = p.group == 32 ? 2 : 4;  // of 16 rows, with one scale
      for (int j0 = 0; j0 < 4; j0 += steps) {
        const int grp = min((kt * kW4Rows + 16 * j0) / p.group, groups - 1);
        const long long at = static_cast<long long>(grp) * p.N + n0 + g;
        const bool in0 = n0 + g < p.N, in1 = n0 + g + 8 < p.N;
        const __nv_bfloat16* sc = static_cast<const __nv_bfloat16*>(w.scales) + at;
        const float s0 = in0 ? __bfloat162float(sc[0]) : 0.f, s1 = in1 ? __bfloat162float(sc[8]) : 0.f;
        const uint32_t z0 = w.zeros != nullptr && in0 ? w4_base(w.zeros[at]) : kW4Base8;
        const uint32_t z1 = w.zeros != nullptr && in1 ? w4_base(w.zeros[at + 8]) : kW4Base8;
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        for (int j = j0; j < j0 + steps; ++j) {
          const uint32_t a[4] = {w4_minus(w4_pair<0>(q[j]), z0), w4_minus(w4_pair<1>(q[j]), z1),
                                 w4_minus(w4_pair<2>(q[j]), z0), w4_minus(w4_pair<3>(q[j]), z1)};
          mma_16816(c, a, b[j]);
        }
        sum[i][0] = fmaf(c[0], s0, sum[i][0]);
        sum[i][1] = fmaf(c[1], s0, sum[i][1]);
        sum[i][2] = fmaf(c[2], s1, sum[i][2]);
        sum[i][3] = fmaf(c[3], s1, sum[i][3]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MATS; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[warp][i][g + 8 * (r >> 1)][2 * t + (r & 1)] = sum[i][r];
  __syncthreads();
  if (threadIdx.x < 128) {
    const int c = threadIdx.x & 15, row = blockIdx.y * 8 + (threadIdx.x >> 4), col = n0 + c;
    if (row < p.M && col < p.N && TPMLP_IN_BOUNDS(static_cast<long long>(row) * p.N + col, static_cast<long long>(p.M) * p.N, kBoundsW4Out)) {
      float v[MATS] = {};
#pragma unroll
      for (int i = 0; i < MATS; ++i) {
        for (int w = 0; w < kWarps; ++w) v[i] += red[w][i][c][threadIdx.x >> 4];
        if (p.w[i].bias != nullptr) v[i] += __bfloat162float(static_cast<const __nv_bfloat16*>(p.w[i].bias)[col]);
      }
      if constexpr (GATED) v[0] = act2(p.act, make_float2(v[0], v[0])).x * v[1];
      static_cast<__nv_bfloat16*>(p.y)[static_cast<long long>(row) * p.N + col] = __float2bfloat16_rn(v[0]);
    }
  }
}

// One warp a group of a column tile: lane l < 16 takes column l.
__global__ void __launch_bounds__(128) k_quantize_w4_scales(const __grid_constant__ W4Pack p) {
  const int col = blockIdx.x * blockDim.x + threadIdx.x, grp = blockIdx.y;
  if (col >= p.N) return;
  float lo = 0.f, hi = 0.f;
  for (int k = grp * p.group; k < min(p.K, (grp + 1) * p.group); ++k) {
    const float v = __bfloat162float(static_cast<const __nv_bfloat16*>(p.w)[static_cast<long long>(k) * p.N + col]);
    lo = fminf(lo, v);
    hi = fmaxf(hi, v);
  }
  const float span = fminf(fmaxf(p.zeros != nullptr ? hi - lo : fmaxf(hi, -lo), kW4Tiny), kW4Big);
  const __nv_bfloat16 s = __float2bfloat16_rn(span / (p.zeros != nullptr ? 15.f : 7.f));
  const long long at = static_cast<long long>(grp) * p.N + col;
  static_cast<__nv_bfloat16*>(p.scales)[at] = s;
  if (p.zeros != nullptr) p.zeros[at] = static_cast<uint8_t>(fminf(fmaxf(rintf(-lo / __bfloat162float(s)), 0.f), 15.f));
}

// One thread a word of a tile.
__global__ void __launch_bounds__(128) k_quantize_w4_codes(const __grid_constant__ W4Pack p) {
  const int word = threadIdx.x, l = word >> 2, j = word & 3, g = l >> 2, t = l & 3;
  uint32_t w = 0;
  for (int b = 0; b < 8; ++b) {
    const int i = b & 3, h = b >> 2;
    const int n = blockIdx.x * kW4Cols + 8 * (i & 1) + g, k = blockIdx.y * kW4Rows + 16 * j + 8 * (i >> 1) + 2 * t + h;
    uint32_t q = 8;
    if (n < p.N && k < p.K) {
      const long long at = static_cast<long long>(k / p.group) * p.N + n;
      float v = __bfloat162float(static_cast<const __nv_bfloat16*>(p.w)[static_cast<long long>(k) * p.N + n]);
      if (isnan(v)) v = 0.f;
      const float s = __bfloat162float(static_cast<const __nv_bfloat16*>(p.scales)[at]);
      const float z = p.zeros != nullptr ? static_cast<float>(p.zeros[at]) : 8.f;
      q = static_cast<uint32_t>(fminf(fmaxf(rintf(fminf(fmaxf(v / s, -16.f), 16.f)) + z, 0.f), 15.f));
    }
    w |= q << (4 * i + 16 * h);
  }
  reinterpret_cast<uint32_t*>(p.q)[(static_cast<long long>(blockIdx.x) * gridDim.y + blockIdx.y) * 128 + word] = w;
}

__global__ void __launch_bounds__(128) k_dequantize_w4(const __grid_constant__ W4Pack p) {
  const int word = threadIdx.x, l = word >> 2, j = word & 3, g = l >> 2, t = l & 3;
  const uint32_t w = reinterpret_cast<const uint32_t*>(p.q)[(static_cast<long long>(blockIdx.x) * gridDim.y + blockIdx.y) * 128 + word];
  for (int b = 0; b < 8; ++b) {
    const int i = b & 3, h = b >> 2;
    const int n = blockIdx.x * kW4Cols + 8 * (i & 1) + g, k = blockIdx.y * kW4Rows + 16 * j + 8 * (i >> 1) + 2 * t + h;
    if (n < p.N && k < p.K) {
      const long long at = static_cast<long long>(k / p.group) * p.N + n;
      const float s = __bfloat162float(static_cast<const __nv_bfloat16*>(p.scales)[at]);
      const int z = p.zeros != nullptr ? p.zeros[at] : 8;
      static_cast<__nv_bfloat16*>(p.w)[static_cast<long long>(k) * p.N + n] =
          __float2bfloat16_rn(s * static_cast<float>(static_cast<int>(w >> (4 * i + 16 * h) & 15u) - z));
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

cudaError_t launch_gemm_w4(const W4Launch& g, const DeviceCtx&, cudaStream_t s) {
  const dim3 grid((g.N + kW4Cols - 1) / kW4Cols, (g.M + 7) / 8);
  if (g.gated) k_gemm_w4<true><<<grid, 32 * kWarps, 0, s>>>(g);
  else k_gemm_w4<false><<<grid, 32 * kWarps, 0, s>>>(g);
  return cudaGetLastError();
}

cudaError_t launch_quantize_w4(const W4Pack& p, cudaStream_t s) {
  const dim3 tiles((p.N + kW4Cols - 1) / kW4Cols, (p.K + kW4Rows - 1) / kW4Rows);
  k_quantize_w4_scales<<<dim3((p.N + 127) / 128, (p.K + p.group - 1) / p.group), 128, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  k_quantize_w4_codes<<<tiles, 128, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_dequantize_w4(const W4Pack& p, cudaStream_t s) {
  const dim3 tiles((p.N + kW4Cols - 1) / kW4Cols, (p.K + kW4Rows - 1) / kW4Rows);
  k_dequantize_w4<<<tiles, 128, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace tpmlp
