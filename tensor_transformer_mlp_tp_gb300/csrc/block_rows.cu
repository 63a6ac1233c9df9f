// Row kernels of the block-scaled FP8 operators: the residual RMS norm with an 8-bit output, its backward, and
// the block quantiser.  All three are bound by memory: a few operations per byte.
#include <cuda_bf16.h>

#include "block_fp8.cuh"
#include "bwd_ring.h"
#include "debug_bounds.cuh"

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

// Debug builds: are the chunk of row `row`, and vectors v of that row, inside their tensors?
__device__ __forceinline__ bool chunk_ok(const RmsBlockParams& p, int row, int chunk, uint32_t site) {
  return TPMLP_IN_BOUNDS(row, p.rows, site) && TPMLP_IN_BOUNDS(chunk, p.n_chunks, site) &&
         TPMLP_IN_BOUNDS(row - chunk * p.rows_per_chunk, p.rows_per_chunk, site);
}
__device__ __forceinline__ bool row_ok(const RmsBlockParams& p, int row, int v, uint32_t site) {
  return TPMLP_IN_BOUNDS(row, p.rows, site) && TPMLP_IN_BOUNDS(v, p.d / 8, site);
}

// s = bf16(x + r), y = s rsqrt(mean(s^2) + eps) w.  A team of TW warps per row; thread t of the team holds the 16-byte
// vectors t + 32 TW k (k < V) in registers, so the row is read once, all its loads in flight together, and the 16 vectors
// of a 1 x 128 block sit on the 16 lanes of a half warp.  The statistics are of the stored (rounded) sum, the value the
// backward reads; y is rounded once, to bf16 or to E4M3.  Measured: 8192 x 4096 over 8 chunks 38 us (6.2 TB/s, 0.93 of the
// copy rate; 52 us with one vector a thread), 1037 x 1024 2.8 us, one row of 4096 2.4 us.
template <int V>
__global__ void __launch_bounds__(V == 4 ? 1024 : 512) k_rmsnorm_add(const RmsBlockParams p, int tw) {
  __shared__ float red[32];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, team = warp / tw, nv = p.d / 8;
  const int step = 32 * tw, j0 = threadIdx.x - team * step;
  const int row = blockIdx.x * (static_cast<int>(blockDim.x >> 5) / tw) + team;
  const bool valid = row < p.rows;
  int j = valid ? row / p.rows_per_chunk : 0;
  long long off = valid ? static_cast<long long>(row - j * p.rows_per_chunk) * nv : 0;
  if (valid && !chunk_ok(p, row, j, kBoundsInChunk)) off = j = 0;
  const uint4* x4 = static_cast<const uint4*>(p.x.p[j]) + off;
  const uint4* r4 = static_cast<const uint4*>(p.r.p[j]) + off;
  const bool has_r = p.r.p[0] != nullptr;
  uint4 x[V], r[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int v = j0 + k * step;
    x[k] = valid && v < nv ? x4[v] : make_uint4(0, 0, 0, 0);
  }
  if (has_r) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int v = j0 + k * step;
      r[k] = valid && v < nv ? r4[v] : make_uint4(0, 0, 0, 0);
    }
  }
  float q = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    float f[8];
    unpack_vec8(x[k], f);
    if (has_r) {
      float g[8];
      unpack_vec8(r[k], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] += g[e];
      x[k] = pack_vec8(f);
      const int v = j0 + k * step;
      if (p.s.p[0] != nullptr && valid && v < nv && row_ok(p, row, v, kBoundsOutChunk))
        (static_cast<uint4*>(p.s.p[j]) + off)[v] = x[k];
      unpack_vec8(x[k], f);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) q += f[e] * f[e];
  }
  q = warp_add(q);
  if (tw > 1) {
    if ((threadIdx.x & 31) == 0) red[warp] = q;
    __syncthreads();
    q = 0.f;
    for (int w = 0; w < tw; ++w) q += red[team * tw + w];
  }
  const float rstd = rsqrtf(q / static_cast<float>(p.d) + p.eps);
  const long long row_off = static_cast<long long>(valid ? row : 0) * nv;
  float y[V][8], amax = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int v = j0 + k * step;
    float f[8], w[8];
    unpack_vec8(x[k], f);
    unpack_vec8(v < nv ? __ldg(static_cast<const uint4*>(p.weight) + v) : make_uint4(0, 0, 0, 0), w);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[k][e] = f[e] * rstd * w[e];
    if (p.xg != nullptr && valid && v < nv && row_ok(p, row, v, kBoundsRowStore))
      (static_cast<uint4*>(p.xg) + row_off)[v] = pack_vec8(y[k]);
    if (p.xq != nullptr) {
      const float a = half_warp_max(abs_max8(y[k]));
      if ((threadIdx.x & (V - 1)) == k) amax = a;
    }
  }
  if (p.xq == nullptr) return;
  // the divisions of the thread's V blocks are shared out: lane k of each half warp makes those of block k
  const BlockScale b = block_scale(amax, 448.f);
  const int kl = threadIdx.x & 15, block = (j0 + kl * step) >> 4;
  if (kl < V && valid && block * 16 < nv && TPMLP_IN_BOUNDS(row, p.rows_pad, kBoundsBlockScales) &&
      TPMLP_IN_BOUNDS(block, (p.d + kBlock - 1) / kBlock, kBoundsBlockScales))
    p.scales[block * p.rows_pad + row] = b.scale;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int v = j0 + k * step;
    const float inv = __shfl_sync(0xffffffffu, b.inv, k, 16);
    if (valid && v < nv && row_ok(p, row, v, kBoundsBlockCodes))
      (reinterpret_cast<uint2*>(p.xq) + row_off)[v] = fp8x8<0>(y[k], inv);
  }
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// With xhat = s rstd and g = dy w:  dx = rstd (g - xhat mean(g xhat)) + ds,  dweight = sum over rows of dy xhat.
//
// One persistent block an SM.  Warp 0 keeps the next groups of rows of s, dy and ds coming into a ring in shared memory
// (bulk copies of about 8 KB, so a group has several rows where rows are short; up to 190 KB in flight an SM), teams of
// TW of the 16 consumer warps take a row each: thread j of a team has the vectors j + 32 TW k (k < VT), takes them from
// the ring once (VT = 2, rows up to 8192) or once for the two sums and once for the output (VT = 4), and keeps the
// weights and its dweight sums in registers.  Row i of the block belongs to team i % teams, so the order of every sum is
// fixed; which rings are safe with that: bwd_ring_ok.  Measured: 8192 x 4096 46.4 us with the final sum's 2.3 (5.8 TB/s,
// 0.86 of the copy rate; 58 us with VT = 4, 83 us with rows in registers and no ring), 65536 x 128 37 us (148 us with a
// row a copy), 320 x 1024 5.5 us.
template <int VT>
__global__ void __launch_bounds__(32 * (kBwdConsumers + 1), 1)
    k_rmsnorm_add_bwd(const RmsBlockParams p, int tw, int group, int slots, unsigned int* err,
                      unsigned long long timeout_ns) {
  constexpr bool kKeep = VT == 2;  // s and dy stay in registers between the two passes
  extern __shared__ __align__(128) uint8_t bwd_smem[];
  __shared__ float2 red[2][kBwdConsumers];
  __shared__ int vote[2][kBwdConsumers];
  __shared__ __align__(8) uint64_t full[kBwdMaxSlots], empty[kBwdMaxSlots];
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool has_r = p.r.p[0] != nullptr;
  const uint32_t row_bytes = static_cast<uint32_t>(p.d) * 2u, part_bytes = row_bytes * static_cast<uint32_t>(group);
  const uint32_t slot_bytes = part_bytes * 3u;  // [s | dy | ds] of a group
  if (threadIdx.x == 0) {
    for (int s = 0; s < slots; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, tw * group);
    }
    abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const WaitCtx wc{&abort_flag, err, timeout_ns};
  const int grid = static_cast<int>(gridDim.x), first = static_cast<int>(blockIdx.x);
  const int groups = (p.rows + group - 1) / group, n_groups = (groups - first + grid - 1) / grid;
  const int cw = warp - 1, team = cw / tw, teams = kBwdConsumers / tw;
  const int nv = p.d / 8, step = 32 * tw, j = (cw - team * tw) * 32 + lane;
  float2 dw[VT][4];
#pragma unroll
  for (int k = 0; k < VT; ++k)
#pragma unroll
    for (int w = 0; w < 4; ++w) dw[k][w] = make_float2(0.f, 0.f);
  if (warp == 0) {
    if (lane == 0) {
      uint32_t phase = 0;
      int slot = 0, issued = 0;
      for (int i = 0; i < n_groups; ++i) {
        if (!wait_bounded(empty + slot, phase ^ 1u, wc, kSiteRmsProducer)) break;
        int r0 = (first + i * grid) * group;
        const int n = min(group, p.rows - r0);
        if (!TPMLP_IN_BOUNDS(r0, p.rows, kBoundsRowLoad) || !TPMLP_IN_BOUNDS(r0 + n - 1, p.rows, kBoundsRowLoad)) r0 = 0;
        uint8_t* dst = bwd_smem + static_cast<long long>(slot) * slot_bytes;
        mbar_arrive_expect_tx(full + slot, static_cast<uint32_t>(n) * row_bytes * (has_r ? 3u : 2u));
        bulk_load(dst + part_bytes, static_cast<const uint8_t*>(p.dy) + static_cast<long long>(r0) * row_bytes,
                  static_cast<uint32_t>(n) * row_bytes, full + slot);
        for (int r = 0; r < n;) {  // the group's rows of one chunk after the other
          int c = (r0 + r) / p.rows_per_chunk, in = r0 + r - c * p.rows_per_chunk;
          if (!chunk_ok(p, r0 + r, c, kBoundsInChunk)) c = in = 0;
          const int m = min(n - r, p.rows_per_chunk - in);
          const long long off = static_cast<long long>(in) * row_bytes;
          const uint32_t bytes = static_cast<uint32_t>(m) * row_bytes, at = static_cast<uint32_t>(r) * row_bytes;
          bulk_load(dst + at, static_cast<const uint8_t*>(p.x.p[c]) + off, bytes, full + slot);
          if (has_r) bulk_load(dst + 2 * part_bytes + at, static_cast<const uint8_t*>(p.r.p[c]) + off, bytes, full + slot);
          r += m;
        }
        ++issued;
        if (++slot == slots) {
          slot = 0;
          phase ^= 1u;
        }
      }
      // copies in flight land before their memory is used again
      for (int i = issued > slots ? issued - slots : 0; i < issued; ++i)
        wait_drain(full + i % slots, static_cast<uint32_t>(i / slots) & 1u, timeout_ns);
    }
  } else {
    uint4 w4[VT];
#pragma unroll
    for (int k = 0; k < VT; ++k)
      w4[k] = j + k * step < nv ? __ldg(static_cast<const uint4*>(p.weight) + j + k * step) : make_uint4(0, 0, 0, 0);
    const float inv_d = 1.f / static_cast<float>(p.d);
    // the team's next row: row `in` of the block's group gi, in slot `slot` (phase: how often the ring went round)
    int gi = team / group, in = team - gi * group, slot = gi % slots;
    uint32_t phase = static_cast<uint32_t>(gi / slots) & 1u;
    const int dgi = teams / group, din = teams - dgi * group;
    for (int par = 0;; par ^= 1) {
      const int row = (first + gi * grid) * group + in;
      if (gi >= n_groups || row >= p.rows) break;
      // every warp waits (bounded) on its own; the outcomes are voted on, so a team leaves the loop together
      const bool ok = __all_sync(0xffffffffu, wait_bounded(full + slot, phase, wc, kSiteRmsConsumer));
      const uint4* xs = reinterpret_cast<const uint4*>(bwd_smem + static_cast<long long>(slot) * slot_bytes) + in * nv;
      const uint4* ys = xs + group * nv;
      const uint4* rs = ys + group * nv;
      uint4 x4[kKeep ? VT : 1], y4[kKeep ? VT : 1];
      float2 sq = make_float2(0.f, 0.f), sg = sq;
      if (ok) {
#pragma unroll
        for (int k = 0; k < VT; ++k) {
          const int v = j + k * step;
          if (v >= nv) continue;
          const uint4 x = xs[v], y = ys[v];
          if (kKeep) {
            x4[kKeep ? k : 0] = x;
            y4[kKeep ? k : 0] = y;
          }
          const uint32_t xa[4] = {x.x, x.y, x.z, x.w}, ya[4] = {y.x, y.y, y.z, y.w};
          const uint32_t wa[4] = {w4[k].x, w4[k].y, w4[k].z, w4[k].w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float2 xf = unpack_bf16x2(xa[w]);
            sq = __ffma2_rn(xf, xf, sq);
            sg = __ffma2_rn(__fmul2_rn(unpack_bf16x2(ya[w]), unpack_bf16x2(wa[w])), xf, sg);
          }
        }
      }
      float2 t = make_float2(warp_add(sq.x + sq.y), warp_add(sg.x + sg.y));
      bool team_ok = ok;
      if (tw > 1) {
        if (lane == 0) {
          red[par][cw] = t;
          vote[par][cw] = ok ? 1 : 0;
        }
        bar_sync(1 + team, step);
        t = make_float2(0.f, 0.f);
        for (int w = 0; w < tw; ++w) {
          t.x += red[par][team * tw + w].x;
          t.y += red[par][team * tw + w].y;
          team_ok = team_ok && vote[par][team * tw + w] != 0;
        }
      }
      if (!team_ok) break;
      const float rstd = rsqrtf(t.x * inv_d + p.eps);
      const float c = t.y * rstd * rstd * rstd * inv_d;  // rstd mean(g xhat) rstd
      const float2 r2 = make_float2(rstd, rstd), nc2 = make_float2(-c, -c);
      const int ch = row / p.rows_per_chunk;
      const bool out_ok = chunk_ok(p, row, ch, kBoundsOutChunk);
      uint4* out = static_cast<uint4*>(p.s.p[ch]) + static_cast<long long>(row - ch * p.rows_per_chunk) * nv;
#pragma unroll
      for (int k = 0; k < VT; ++k) {
        const int v = j + k * step;
        if (v >= nv) continue;
        const uint4 x = kKeep ? x4[kKeep ? k : 0] : xs[v], y = kKeep ? y4[kKeep ? k : 0] : ys[v];
        const uint4 r = has_r ? rs[v] : make_uint4(0, 0, 0, 0);
        const uint32_t xa[4] = {x.x, x.y, x.z, x.w}, ya[4] = {y.x, y.y, y.z, y.w}, ra[4] = {r.x, r.y, r.z, r.w};
        const uint32_t wa[4] = {w4[k].x, w4[k].y, w4[k].z, w4[k].w};
        uint32_t o[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 xf = unpack_bf16x2(xa[w]), yr = __fmul2_rn(unpack_bf16x2(ya[w]), r2);
          dw[k][w] = __ffma2_rn(yr, xf, dw[k][w]);
          const float2 dx = __fadd2_rn(__ffma2_rn(xf, nc2, __fmul2_rn(yr, unpack_bf16x2(wa[w]))), unpack_bf16x2(ra[w]));
          o[w] = pack_bf16x2(dx.x, dx.y);
        }
        if (out_ok && row_ok(p, row, v, kBoundsOutChunk)) out[v] = make_uint4(o[0], o[1], o[2], o[3]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + slot);
      int ahead = dgi;
      if ((in += din) >= group) {
        in -= group;
        ++ahead;
      }
      gi += ahead;
      for (slot += ahead; slot >= slots; slot -= slots) phase ^= 1u;
    }
  }
  __syncthreads();  // the producer has drained its copies: the ring's memory is free for the teams' sums [teams][d]
  float* acc = reinterpret_cast<float*>(bwd_smem);
  if (warp > 0) {
#pragma unroll
    for (int k = 0; k < VT; ++k) {
      const int v = j + k * step;
      if (v >= nv) continue;
      float4* a = reinterpret_cast<float4*>(acc + static_cast<long long>(team) * p.d + v * 8);
      a[0] = make_float4(dw[k][0].x, dw[k][0].y, dw[k][1].x, dw[k][1].y);
      a[1] = make_float4(dw[k][2].x, dw[k][2].y, dw[k][3].x, dw[k][3].y);
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < p.d; c += blockDim.x) {
    float t = 0.f;
    for (int tm = 0; tm < teams; ++tm) t += acc[static_cast<long long>(tm) * p.d + c];
    if (TPMLP_IN_BOUNDS(first, min(p.rows, kBwdMaxBlocks), kBoundsPartial))
      p.partial[static_cast<long long>(first) * p.d + c] = t;
  }
}

// dweight[c] = the sum of the blocks' partial rows, in a fixed order: 32 columns a block, the rows over its 32 warps, so
// that all of a warp's loads are in flight together.
__global__ void __launch_bounds__(1024) k_dweight_sum(const float* partial, int rows, int d, float* dweight) {
  __shared__ float red[32][33];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float a[(kBwdMaxBlocks + 31) / 32];
#pragma unroll
  for (int u = 0; u < (kBwdMaxBlocks + 31) / 32; ++u) {
    const int r = warp + 32 * u;
    a[u] = c < d && r < rows ? partial[static_cast<long long>(r) * d + c] : 0.f;
  }
  float t = 0.f;
#pragma unroll
  for (int u = 0; u < (kBwdMaxBlocks + 31) / 32; ++u) t += a[u];
  red[warp][lane] = t;
  __syncthreads();
  if (warp == 0 && c < d) {
    t = 0.f;
#pragma unroll
    for (int w = 0; w < 32; ++w) t += red[w][lane];
    if (TPMLP_IN_BOUNDS(c, d, kBoundsPartial)) dweight[c] = t;
  }
}

// Rows wider than the ring kernel's, in registers: one block per row at a time, blocks walk the rows.  A thread's 96 sums
// and values in fp32 are more than a block of 1024 threads has registers for, so most of them live in local memory, which
// bounds it: 2048 x 32768 about 340 us (its bytes alone are 80), 2048 x 16392 about 180 (40).
template <int V>
__global__ void __launch_bounds__(1024) k_rmsnorm_add_bwd_wide(const RmsBlockParams p) {
  __shared__ float red[32];
  griddep_launch_dependents();
  const int nv = p.d / 8;
  const bool has_r = p.r.p[0] != nullptr;
  float dw[V][8];
#pragma unroll
  for (int k = 0; k < V; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[k][e] = 0.f;
  for (int row = blockIdx.x; row < p.rows; row += gridDim.x) {
    int j = row / p.rows_per_chunk;
    long long off = static_cast<long long>(row - j * p.rows_per_chunk) * nv;
    if (!chunk_ok(p, row, j, kBoundsInChunk)) off = j = 0;
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
      if (row_ok(p, row, v, kBoundsOutChunk)) (static_cast<uint4*>(p.s.p[j]) + off)[v] = pack_vec8(o);
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int v = threadIdx.x + k * blockDim.x;
    if (v >= nv || !TPMLP_IN_BOUNDS(blockIdx.x, min(p.rows, kBwdMaxBlocks), kBoundsPartial)) continue;
    float4* out = reinterpret_cast<float4*>(p.partial + static_cast<long long>(blockIdx.x) * p.d + v * 8);
    out[0] = make_float4(dw[k][0], dw[k][1], dw[k][2], dw[k][3]);
    out[1] = make_float4(dw[k][4], dw[k][5], dw[k][6], dw[k][7]);
  }
}

// ----------------------------------------------------------------------------- quantiser

// One 128 x 128 tile per block of 256 threads.  Thread t holds the 16-byte vectors t % 16 of rows t / 16 + 16 i (i < 8)
// in registers, all eight loads in flight at once; src is read once for both outputs.
//   q:  the 16 vectors of a row are on the 16 lanes of a half warp: amax by shuffles, codes stored from registers.
//   qT: column amaxes over a thread's rows, its half warps (shuffle) and the eight warps (shared memory); the codes
//       cross a 16 KB byte tile and leave as 16 consecutive bytes of a destination row, eight lanes a 128-byte line.
// In the byte tile, word w of row r sits at word w ^ 4 (r / 16): a warp's reads (four words of rows 16 g + i, g < 8) and
// its 8-byte writes are then free of bank conflicts.
template <int FMT, bool TILE>
__global__ void __launch_bounds__(256) k_quantize_block(const QuantBlockParams p) {
  __shared__ __align__(16) uint32_t tile[kBlock * kBlock / 4];
  __shared__ float red[8][kBlock];  // column amaxes of the warps; row 0: the columns' factors.  TILE: red[0][warp]
  griddep_wait();
  griddep_launch_dependents();
  const int r0 = blockIdx.y * kBlock, c0 = blockIdx.x * kBlock;
  const int t = threadIdx.x, vc = t & 15, vr = t >> 4, warp = t >> 5;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.src);
  const int c = c0 + vc * 8;
  uint4 u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + vr + 16 * i;
    u[i] = r < p.rows && c < p.cols && TPMLP_IN_BOUNDS(r * p.ld + c + 7, (p.rows - 1) * p.ld + p.cols, kBoundsBlockSource)
               ? __ldg(reinterpret_cast<const uint4*>(src + r * p.ld + c)) : make_uint4(0, 0, 0, 0);
  }
  constexpr float kF = fp8_max(FMT);
  BlockScale b{};
  if constexpr (TILE) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f[8];
      unpack_vec8(u[i], f);
      m = fmaxf(m, abs_max8(f));
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((t & 31) == 0) red[0][warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = fmaxf(m, red[0][w]);
    b = block_scale(m, kF);
    if (t == 0) {
      if (p.scales != nullptr && TPMLP_IN_BOUNDS(c0, p.cols, kBoundsBlockScales) &&
          TPMLP_IN_BOUNDS(r0, p.rows, kBoundsBlockScales))
        p.scales[static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x] = b.scale;
      if (p.scales_t != nullptr && TPMLP_IN_BOUNDS(c0, p.cols, kBoundsBlockScales) &&
          TPMLP_IN_BOUNDS(r0, p.rows, kBoundsBlockScales))
        p.scales_t[static_cast<long long>(blockIdx.x) * gridDim.y + blockIdx.y] = b.scale;
    }
  } else if (p.qt != nullptr) {
    float m[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f[8];
      unpack_vec8(u[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) m[e] = fmaxf(m[e], fabsf(f[e]));
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) m[e] = fmaxf(m[e], __shfl_xor_sync(0xffffffffu, m[e], 16));
    if ((t & 16) == 0) {
      reinterpret_cast<float4*>(red[warp] + vc * 8)[0] = make_float4(m[0], m[1], m[2], m[3]);
      reinterpret_cast<float4*>(red[warp] + vc * 8)[1] = make_float4(m[4], m[5], m[6], m[7]);
    }
    __syncthreads();
    if (t < kBlock) {
      float a = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) a = fmaxf(a, red[w][t]);
      const BlockScale col = block_scale(a, kF);
      red[0][t] = col.inv;
      if (c0 + t < p.cols && TPMLP_IN_BOUNDS(blockIdx.y, (p.rows + kBlock - 1) / kBlock, kBoundsBlockScales) &&
          TPMLP_IN_BOUNDS(c0 + t, gridDim.x * kBlock, kBoundsBlockScales))
        p.scales_t[blockIdx.y * (static_cast<long long>(gridDim.x) * kBlock) + c0 + t] = col.scale;
    }
    __syncthreads();
  }
  float inv[8];
  if (p.qt != nullptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) inv[e] = TILE ? b.inv : red[0][vc * 8 + e];
  }
  const long long rows_pad = static_cast<long long>(gridDim.y) * kBlock;
  auto code_ok = [&](int r, int c) {  // debug builds
    return TPMLP_IN_BOUNDS(static_cast<long long>(r) * p.cols + c + 7, static_cast<long long>(p.rows) * p.cols,
                           kBoundsBlockCodes);
  };
  float row_inv = 0.f;  // lane vc < 8 of a half warp: of row vr + 16 vc
  if (!TILE && p.q != nullptr) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f[8];
      unpack_vec8(u[i], f);
      const float a = half_warp_max(abs_max8(f));
      if ((vc & 7) == i) m = a;
    }
    const BlockScale row = block_scale(m, kF);
    row_inv = row.inv;
    const int r = r0 + vr + 16 * (vc & 7);
    if (vc < 8 && r < p.rows && TPMLP_IN_BOUNDS(blockIdx.x, (p.cols + kBlock - 1) / kBlock, kBoundsBlockScales) &&
        TPMLP_IN_BOUNDS(r, rows_pad, kBoundsBlockScales))
      p.scales[blockIdx.x * rows_pad + r] = row.scale;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + vr + 16 * i;
    float f[8];
    unpack_vec8(u[i], f);
    if constexpr (TILE) {
      const uint2 codes = fp8x8<FMT>(f, b.inv);
      if (p.q != nullptr && r < p.rows && c < p.cols && code_ok(r, c))
        *reinterpret_cast<uint2*>(p.q + static_cast<long long>(r) * p.cols + c) = codes;
      if (p.qt != nullptr) *reinterpret_cast<uint2*>(tile + (vr + 16 * i) * 32 + ((2 * vc) ^ (4 * i))) = codes;
    } else {
      if (p.q != nullptr) {
        const float row = __shfl_sync(0xffffffffu, row_inv, i, 16);
        if (r < p.rows && c < p.cols && code_ok(r, c))
          *reinterpret_cast<uint2*>(p.q + static_cast<long long>(r) * p.cols + c) = fp8x8<FMT>(f, row);
      }
      if (p.qt != nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= inv[e];
        *reinterpret_cast<uint2*>(tile + (vr + 16 * i) * 32 + ((2 * vc) ^ (4 * i))) = fp8x8<FMT>(f, 1.f);
      }
    }
  }
  if (p.qt == nullptr) return;
  __syncthreads();
  // lane: rows 16 g .. + 15 (g = lane % 8) of the four columns of word w
  const int g = t & 7, w = (t >> 3) & 31;
  const long long pitch = (p.rows + 15) / 16 * 16;
  uint32_t out[4][4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {  // a 4 x 4 byte transpose: words of rows 16 g + 4 k .. + 3
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = tile[(16 * g + 4 * k + i) * 32 + (w ^ (4 * g))];
    const uint32_t lo01 = __byte_perm(x[0], x[1], 0x5140), hi01 = __byte_perm(x[0], x[1], 0x7362);
    const uint32_t lo23 = __byte_perm(x[2], x[3], 0x5140), hi23 = __byte_perm(x[2], x[3], 0x7362);
    out[0][k] = __byte_perm(lo01, lo23, 0x5410);
    out[1][k] = __byte_perm(lo01, lo23, 0x7632);
    out[2][k] = __byte_perm(hi01, hi23, 0x5410);
    out[3][k] = __byte_perm(hi01, hi23, 0x7632);
  }
  const int r = r0 + 16 * g;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int oc = c0 + 4 * w + e;
    if (oc < p.cols && r < pitch && TPMLP_IN_BOUNDS(oc * pitch + r + 15, p.cols * pitch, kBoundsBlockCodes))
      *reinterpret_cast<uint4*>(p.qt + oc * pitch + r) = make_uint4(out[e][0], out[e][1], out[e][2], out[e][3]);
  }
}

}  // namespace

namespace {

// Launch with programmatic stream serialisation: the kernel may be set up while the previous one ends (each waits for
// that one, griddep_wait, before its first global access).
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

}  // namespace

cudaError_t launch_rmsnorm_add(const RmsBlockParams& p, const DeviceCtx& ctx, cudaStream_t s) {
  // More vectors than two fillings of the SMs' threads: four a thread, so that the registers hold as many rows' loads as
  // they can.  Below that one a thread, the shortest path from load to store.
  const int nv = p.d / 8;
  const int v = nv > 1024 || static_cast<long long>(p.rows) * nv > 4096ll * ctx.sm_count ? 4 : nv > 512 ? 2 : 1;
  int tw = 1;
  while (32 * tw * v < nv) tw *= 2;
  const int warps = tw < 4 ? 4 : tw, rows = warps / tw;
  const int grid = (p.rows + rows - 1) / rows;
  auto kern = v == 1 ? k_rmsnorm_add<1> : v == 2 ? k_rmsnorm_add<2> : k_rmsnorm_add<4>;
  return launch_overlapped(kern, dim3(grid), dim3(32 * warps), 0, s, p, tw);
}

size_t rmsnorm_add_bwd_scratch_floats(int rows, int d) {
  return static_cast<size_t>(rows < kBwdMaxBlocks ? rows : kBwdMaxBlocks) * d;
}

cudaError_t launch_rmsnorm_add_bwd(const RmsBlockParams& p, float* dweight, const DeviceCtx& ctx, cudaStream_t s) {
  const int sms = ctx.sm_count < kBwdMaxBlocks ? ctx.sm_count : kBwdMaxBlocks, blocks = p.rows < sms ? p.rows : sms;
  cudaError_t e;
  if (p.d <= kBwdMaxD) {
    const BwdRing r = bwd_ring(p.rows, p.d, ctx.sm_count);
    // Asked here and not at the kernel's entry: a return or an empty loop for such blocks there makes the compiler's code
    // for the others slower (8192 x 4096: 46.4 -> 47.4 to 48.3 us).
    if (!bwd_ring_ok(r.most, r.group, r.slots, r.teams)) return cudaErrorInvalidConfiguration;
    static std::atomic<unsigned long long> set[2][64] = {};
    auto kern = r.vt == 2 ? k_rmsnorm_add_bwd<2> : k_rmsnorm_add_bwd<4>;
    e = raise_smem_once(kern, kBwdSmem, ctx, set[r.vt == 2 ? 0 : 1]);
    if (e != cudaSuccess) return e;
    e = launch_overlapped(kern, dim3(r.blocks), dim3(32 * (kBwdConsumers + 1)), r.smem, s, p, r.team_warps, r.group,
                          r.slots, ctx.err, ctx.timeout_ns);
  } else {
    k_rmsnorm_add_bwd_wide<4><<<blocks, (p.d / 8 + 127) / 128 * 32, 0, s>>>(p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  return launch_overlapped(k_dweight_sum, dim3((p.d + 31) / 32), dim3(1024), 0, s, static_cast<const float*>(p.partial),
                           blocks, p.d, dweight);
}

cudaError_t block_rows_bounds_status(unsigned int* count, unsigned int* site) {
#ifdef TPMLP_DEBUG_BOUNDS
  return bounds_read_and_clear(count, site);
#else
  *count = *site = 0;
  return cudaSuccess;
#endif
}

cudaError_t launch_quantize_block(const QuantBlockParams& p, cudaStream_t s) {
  const dim3 grid((p.cols + kBlock - 1) / kBlock, (p.rows + kBlock - 1) / kBlock);
  auto kern = p.block_rows == 1 ? (p.fmt == 0 ? k_quantize_block<0, false> : k_quantize_block<1, false>)
                                : (p.fmt == 0 ? k_quantize_block<0, true> : k_quantize_block<1, true>);
  return launch_overlapped(kern, grid, dim3(256), 0, s, p);
}

}  // namespace tpmlp
