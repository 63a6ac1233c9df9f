// Block-scaled FP8 operators: parameters and launchers (internal).
//
// An 8-bit operand Q [R x K] (row-major bytes, E4M3 or E5M2) stands for Q * scale with one fp32 scale for each
// block of 128 along K, either per row or per tile of 128 rows:
//   block_rows = 1:   scales[kb * R_pad + r], kb = k / 128, R_pad = 128 ceil(R / 128) (k-block major, so the
//                     scales of consecutive rows are consecutive; the entries of rows >= R are never read into
//                     a result),
//   block_rows = 128: scales[(r / 128) * KB + kb], KB = ceil(K / 128).
// scale = max(amax, 2^-100) / F with F the format's largest finite value (448, 57344) and amax the block's
// largest magnitude (a NaN does not count, an infinity counts as the largest finite float); a code is
// FP8(x * (F / max(amax, 2^-100))), saturating, round to nearest even: NaN stays NaN.
#pragma once

#include <cuda_runtime.h>

#include "launch.h"

namespace tpmlp {

constexpr int kBlock = 128;
constexpr int kBlockMaxD = 32768;  // widest row of the residual RMS norm (1024 threads x 4 vectors of 8)

inline long long pad128(long long n) { return (n + kBlock - 1) / kBlock * kBlock; }

struct RmsBlockParams {
  ConstChunkPtrs x;       // N chunks [rows_per_chunk x d]
  ConstChunkPtrs r;       // residual chunks, or p[0] == nullptr
  ChunkPtrs s;            // sum chunks (forward; p[0] == nullptr: not kept) or dX chunks (backward)
  const void* weight;     // [d] bf16
  const void* dy;         // backward: dXg [rows x d] bf16
  void* xg;               // forward: [rows x d] bf16 or nullptr
  uint8_t* xq;            // forward: [rows x d] E4M3 or nullptr
  float* scales;          // forward: [ceil(d / 128) x rows_pad]
  float* partial;         // backward: dweight partial sums [blocks x d]
  int rows, d, n_chunks, rows_per_chunk;
  long long rows_pad;
  float eps;
};

cudaError_t launch_rmsnorm_add(const RmsBlockParams& p, const DeviceCtx& ctx, cudaStream_t s);
// dX and the dweight partials, then their fixed-order sum into dweight [d] fp32.
cudaError_t launch_rmsnorm_add_bwd(const RmsBlockParams& p, float* dweight, const DeviceCtx& ctx, cudaStream_t s);
size_t rmsnorm_add_bwd_scratch_floats(int rows, int d);

struct QuantBlockParams {
  const void* src;        // [rows x cols] bf16, ld elements between rows
  long long ld;
  int rows, cols;
  int block_rows;         // 1 or 128
  int fmt;                // 0 = E4M3, 1 = E5M2
  uint8_t* q;             // [rows x cols] or nullptr
  float* scales;
  uint8_t* qt;            // [cols x rows_pitch] or nullptr, rows_pitch = 16 ceil(rows / 16), padding zeroed
  float* scales_t;
};
cudaError_t launch_quantize_block(const QuantBlockParams& p, cudaStream_t s);

// C [M x N] = sum over blocks kb of sA sB (A8 B8^T restricted to block kb) + bias.  Exactly one of
//   c:  C in bf16 or fp32 with ldc elements between rows,
//   hq: GeLU(C) as E4M3 [M x N] with 1 x 128 blocks (h_scales [ceil(N / 128) x M_pad]), pre: C in bf16 or nullptr.
struct GemmBlockLaunch {
  const uint8_t* a;
  const uint8_t* b;
  const float* a_scales;  // per row
  const float* b_scales;
  int b_block_rows;       // 1 or 128
  int a_fmt, b_fmt;
  int M, N, K;
  const void* bias;       // [N] bf16 or nullptr
  void* c;
  int c_fp32;
  long long ldc;
  uint8_t* hq;
  float* h_scales;
  void* pre;
};
cudaError_t launch_gemm_block(const GemmBlockLaunch& g, const DeviceCtx& ctx, cudaStream_t s);

}  // namespace tpmlp
