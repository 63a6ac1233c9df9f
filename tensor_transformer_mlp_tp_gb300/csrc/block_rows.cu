// Row kernels of the block-scaled FP8 operators: the residual RMS norm with an 8-bit output, its backward, and
// the block quantiser.  All three are bound by memory: a few operations per byte.
#include <cuda_bf16.h>

#include "block_fp8.cuh"

namespace tpmlp {
namespace {

__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the block in a fixed order; every thread gets it.
__device__ __forceinline__ float block_add(float v, float* red) {
  v = warp_add(v);
  const int warp = threadIdx.x >> 5, n = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  __syncthreads();
  float t = 0.f;
  for (int w = 0; w < n; ++w) t += red[w];
  __syncthreads();
  return t;
}

template <typename T>
__device__ __forceinline__ T* chunk_at(T* const* chunks, int rows_per_chunk, int row, long long elems_per_row) {
  const int j = row / rows_per_chunk;
  return chunks[j] + static_cast<long long>(row - j * rows_per_chunk) * elems_per_row;
}

// s = bf16(x + r), y = s rsqrt(mean(s^2) + eps) w.  One block per row; thread t holds the 16-byte vectors
// t + k blockDim (k < V) in registers, so the row is read once and the 16 vectors of a 1 x 128 block sit on
// the 16 lanes of a half warp.  The statistics are of the stored (rounded) sum, the value the backward reads;
// y is rounded once, to bf16 or to E4M3.
template <int V>
__global__ void __launch_bounds__(V == 4 ? 1024 : 512) k_rmsnorm_add(const RmsBlockParams p) {
  __shared__ float red[32];
  const int row = blockIdx.x, nv = p.d / 8;
  const int j = row / p.rows_per_chunk;
  const long long off = static_cast<long long>(row - j * p.rows_per_chunk) * nv;
  const uint4* x4 = static_cast<const uint4*>(p.x.p[j]) + off;
  const bool has_r = p.r.p[0] != nullptr;
  float f[V][8];
  float q = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int v = threadIdx.x + k * blockDim.x;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[k][e] = 0.f;
    if (v < nv) {
      unpack_vec8(x4[v], f[k]);
      if (has_r) {
        float r[8];
        unpack_vec8((static_cast<const uint4*>(p.r.p[j]) + off)[v], r);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[k][e] += r[e];
        const uint4 s = pack_vec8(f[k]);
        if (p.s.p[0] != nullptr) (static_cast<uint4*>(p.s.p[j]) + off)[v] = s;
        unpack_vec8(s, f[k]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) q += f[k][e] * f[k][e];
    }
  }
  const float rstd = rsqrtf(block_add(q, red) / static_cast<float>(p.d) + p.eps);
  const long long row_off = static_cast<long long>(row) * nv;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int v = threadIdx.x + k * blockDim.x;
    const bool in = v < nv;
    float w[8], y[8];
    unpack_vec8(in ? __ldg(static_cast<const uint4*>(p.weight) + v) : make_uint4(0, 0, 0, 0), w);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = f[k][e] * rstd * w[e];
    if (p.xg != nullptr && in) (static_cast<uint4*>(p.xg) + row_off)[v] = pack_vec8(y);
    if (p.xq != nullptr) {
      const BlockScale b = block_scale(half_warp_max(abs_max8(y)), 448.f);
      if (in) (reinterpret_cast<uint2*>(p.xq) + row_off)[v] = fp8x8<0>(y, b.inv);
      if (in && (v & 15) == 0) p.scales[(v >> 4) * p.rows_pad + row] = b.scale;
    }
  }
}

// With xhat = s rstd and g = dy w:  dx = rstd (g - xhat mean(g xhat)) + ds,  dweight = sum over rows of dy xhat.
// Blocks walk rows blockIdx, blockIdx + gridDim, ... and keep their dweight sums in registers (fp32); the
// blocks' partial rows are summed in a fixed order by a second kernel.
template <int V>
__global__ void __launch_bounds__(V == 4 ? 1024 : 512) k_rmsnorm_add_bwd(const RmsBlockParams p) {
  __shared__ float red[32];
  const int nv = p.d / 8;
  const bool has_r = p.r.p[0] != nullptr;
  float dw[V][8];
#pragma unroll
  for (int k = 0; k < V; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[k][e] = 0.f;
  for (int row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int j = row / p.rows_per_chunk;
    const long long off = static_cast<long long>(row - j * p.rows_per_chunk) * nv;
    const uint4* x4 = static_cast<const uint4*>(p.x.p[j]) + off;
    const uint4* y4 = static_cast<const uint4*>(p.dy) + static_cast<long long>(row) * nv;
    float x[V][8], dy[V][8], sq = 0.f, sgx = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int v = threadIdx.x + k * blockDim.x;
      const bool in = v < nv;
      float w[8];
      unpack_vec8(in ? x4[v] : make_uint4(0, 0, 0, 0), x[k]);
      unpack_vec8(in ? y4[v] : make_uint4(0, 0, 0, 0), dy[k]);
      unpack_vec8(in ? __ldg(static_cast<const uint4*>(p.weight) + v) : make_uint4(0, 0, 0, 0), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sq += x[k][e] * x[k][e];
        sgx += dy[k][e] * w[e] * x[k][e];
      }
    }
    const float rstd = rsqrtf(block_add(sq, red) / static_cast<float>(p.d) + p.eps);
    const float c = block_add(sgx, red) * rstd * rstd * rstd / static_cast<float>(p.d);  // rstd mean(g xhat) rstd
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int v = threadIdx.x + k * blockDim.x;
      if (v >= nv) continue;
      float w[8], o[8];
      unpack_vec8(__ldg(static_cast<const uint4*>(p.weight) + v), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dw[k][e] += dy[k][e] * (x[k][e] * rstd);
        o[e] = rstd * (dy[k][e] * w[e]) - x[k][e] * c;
      }
      if (has_r) {
        float r[8];
        unpack_vec8((static_cast<const uint4*>(p.r.p[j]) + off)[v], r);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += r[e];
      }
      (static_cast<uint4*>(p.s.p[j]) + off)[v] = pack_vec8(o);
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int v = threadIdx.x + k * blockDim.x;
    if (v >= nv) continue;
    float4* out = reinterpret_cast<float4*>(p.partial + static_cast<long long>(blockIdx.x) * p.d + v * 8);
    out[0] = make_float4(dw[k][0], dw[k][1], dw[k][2], dw[k][3]);
    out[1] = make_float4(dw[k][4], dw[k][5], dw[k][6], dw[k][7]);
  }
}

constexpr int kBwdMaxBlocks = 592;  // dweight partial rows

struct RowLaunch {
  int threads, v;
};
RowLaunch row_launch(int d) {
  const int nv = d / 8;
  const int v = nv <= 512 ? 1 : nv <= 1024 ? 2 : 4;
  return {(nv + v * 32 - 1) / (v * 32) * 32, v};
}

// ----------------------------------------------------------------------------- quantiser

// One 128 x 128 tile per block of 256 threads, through shared memory: thread t reads 16-byte vectors t % 16 of
// rows t / 16 + 16 i.  A row's (or the tile's) amax comes from shuffles, a column's from shared memory.
constexpr int kQPitch = 130;  // bf16 elements: rows start 65 words apart, so a column walk is conflict-free
template <int FMT, bool TILE>
__global__ void __launch_bounds__(256) k_quantize_block(const QuantBlockParams p) {
  __shared__ __nv_bfloat16 tile[kBlock * kQPitch];
  __shared__ float red[8];
  const int r0 = blockIdx.y * kBlock, c0 = blockIdx.x * kBlock;
  const int t = threadIdx.x, vc = t & 15, vr = t >> 4;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.src);
  float m = 0.f;
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + vr + 16 * i, c = c0 + vc * 8;
    const uint4 u = r < p.rows && c < p.cols ? *reinterpret_cast<const uint4*>(src + r * p.ld + c) : make_uint4(0, 0, 0, 0);
    uint32_t* row = reinterpret_cast<uint32_t*>(tile + (vr + 16 * i) * kQPitch + vc * 8);
    row[0] = u.x;
    row[1] = u.y;
    row[2] = u.z;
    row[3] = u.w;
    float f[8];
    unpack_vec8(u, f);
    m = fmaxf(m, abs_max8(f));
  }
  BlockScale b{};
  if constexpr (TILE) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((t & 31) == 0) red[t >> 5] = m;
    __syncthreads();
    for (int w = 0; w < 8; ++w) m = fmaxf(m, red[w]);
    b = block_scale(m, fp8_max(FMT));
    if (t == 0) {
      if (p.scales != nullptr) p.scales[static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x] = b.scale;
      if (p.scales_t != nullptr) p.scales_t[static_cast<long long>(blockIdx.x) * gridDim.y + blockIdx.y] = b.scale;
    }
  }
  __syncthreads();
  if (p.q != nullptr) {
    const long long rows_pad = static_cast<long long>(gridDim.y) * kBlock;
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + vr + 16 * i, c = c0 + vc * 8;
      const uint32_t* row = reinterpret_cast<const uint32_t*>(tile + (vr + 16 * i) * kQPitch + vc * 8);
      float f[8];
      unpack_vec8(make_uint4(row[0], row[1], row[2], row[3]), f);
      if constexpr (!TILE) b = block_scale(half_warp_max(abs_max8(f)), fp8_max(FMT));
      if (r < p.rows && c < p.cols)
        *reinterpret_cast<uint2*>(p.q + static_cast<long long>(r) * p.cols + c) = fp8x8<FMT>(f, b.inv);
      if (!TILE && vc == 0 && r < p.rows) p.scales[blockIdx.x * rows_pad + r] = b.scale;
    }
  }
  if (p.qt != nullptr) {
    const long long cols_pad = static_cast<long long>(gridDim.x) * kBlock;
    const long long pitch = (p.rows + 15) / 16 * 16;
    for (int i = 0; i < 8; ++i) {  // destination row (source column) vr + 16 i, source rows 8 vc .. + 7
      const int c = c0 + vr + 16 * i, r = r0 + vc * 8;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = __bfloat162float(tile[(vc * 8 + e) * kQPitch + vr + 16 * i]);
      if constexpr (!TILE) b = block_scale(half_warp_max(abs_max8(f)), fp8_max(FMT));
      if (c < p.cols && r < pitch) *reinterpret_cast<uint2*>(p.qt + c * pitch + r) = fp8x8<FMT>(f, b.inv);
      if (!TILE && vc == 0 && c < p.cols) p.scales_t[blockIdx.y * cols_pad + c] = b.scale;
    }
  }
}

}  // namespace

cudaError_t launch_rmsnorm_add(const RmsBlockParams& p, const DeviceCtx&, cudaStream_t s) {
  const RowLaunch l = row_launch(p.d);
  if (l.v == 1) k_rmsnorm_add<1><<<p.rows, l.threads, 0, s>>>(p);
  else if (l.v == 2) k_rmsnorm_add<2><<<p.rows, l.threads, 0, s>>>(p);
  else k_rmsnorm_add<4><<<p.rows, l.threads, 0, s>>>(p);
  return cudaGetLastError();
}

size_t rmsnorm_add_bwd_scratch_floats(int rows, int d) {
  return static_cast<size_t>(rows < kBwdMaxBlocks ? rows : kBwdMaxBlocks) * d;
}

cudaError_t launch_rmsnorm_add_bwd(const RmsBlockParams& p, float* dweight, const DeviceCtx&, cudaStream_t s) {
  const RowLaunch l = row_launch(p.d);
  const int blocks = p.rows < kBwdMaxBlocks ? p.rows : kBwdMaxBlocks;
  if (l.v == 1) k_rmsnorm_add_bwd<1><<<blocks, l.threads, 0, s>>>(p);
  else if (l.v == 2) k_rmsnorm_add_bwd<2><<<blocks, l.threads, 0, s>>>(p);
  else k_rmsnorm_add_bwd<4><<<blocks, l.threads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_column_sum(p.partial, blocks, p.d, dweight, false, s);
}

cudaError_t launch_quantize_block(const QuantBlockParams& p, cudaStream_t s) {
  const dim3 grid((p.cols + kBlock - 1) / kBlock, (p.rows + kBlock - 1) / kBlock);
  if (p.fmt == 0 && p.block_rows == 1) k_quantize_block<0, false><<<grid, 256, 0, s>>>(p);
  else if (p.fmt == 0) k_quantize_block<0, true><<<grid, 256, 0, s>>>(p);
  else if (p.block_rows == 1) k_quantize_block<1, false><<<grid, 256, 0, s>>>(p);
  else k_quantize_block<1, true><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace tpmlp
