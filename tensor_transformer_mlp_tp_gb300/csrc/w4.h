// Launch parameters of the 4-bit weights (host side).
//
// A matrix W [K x N] stands for (q - z) s: codes q in 0..15, a bf16 scale s and a zero point z (8 without zero points) for
// each group of 32, 64 or 128 rows of a column.  The codes' layout is that of the m16n8k16 products' A operand with the
// columns of W as its rows, a tile of 16 columns x 64 rows in 512 bytes: lane 4 g + t of a warp holds 16 bytes, word j of
// them the 16 rows 16 j .. of the tile, its bits 4 i + 16 h the code of column 8 (i % 2) + g, row 8 (i / 2) + 2 t + h.
// A warp's 16-byte loads then read the tile as it lies, and a shift and a mask make a register of two codes.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.h"
#include "few_plan_w4.h"

namespace tpmlp {

struct W4Matrix {
  const uint4* q;          // [n_tiles][k_tiles][32]
  const void* scales;      // [groups x N] bf16
  const uint8_t* zeros;    // [groups x N] or nullptr
  const void* bias;        // [N] bf16 or nullptr
};

// Y [M x N] bf16 = X [M x K] W (+ bias), or act(X W0 + b0) * (X W1 + b1) with `gated`.
struct W4Launch {
  const void* x;
  W4Matrix w[2];
  bool gated;
  int act;
  void* y;
  int M, N, K, group;
};

struct W4Pack {
  void* w;                 // [K x N] bf16, read by the quantiser and written by its inverse
  uint4* q;
  void* scales;
  uint8_t* zeros;
  int K, N, group;
};

cudaError_t launch_gemm_w4(const W4Launch& g, const DeviceCtx& ctx, cudaStream_t s);
cudaError_t launch_quantize_w4(const W4Pack& p, cudaStream_t s);
cudaError_t launch_dequantize_w4(const W4Pack& p, cudaStream_t s);

}  // namespace tpmlp
