// Device helpers of the 4-bit weights.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "w4.h"

namespace tpmlp {

// Codes i of a word (its bits 4 i and 16 + 4 i) as two bf16 of 128 + q: an integer below 256 is exact in bf16, and 128 + q
// is 0x4300 | q.
template <int I>
__device__ __forceinline__ uint32_t w4_pair(uint32_t word) {
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x000F000F, 0x43004300, 0xEA;" : "=r"(r) : "r"(I == 0 ? word : word >> (4 * I)));
  return r;
}

// (128 + q) - (128 + z), exact.
__device__ __forceinline__ uint32_t w4_minus(uint32_t pair, uint32_t base) {
  const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&pair), *reinterpret_cast<const __nv_bfloat162*>(&base));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 128 + z in both halves.
__device__ __forceinline__ uint32_t w4_base(uint32_t z) { return 0x43004300u + z * 0x00010001u; }

constexpr uint32_t kW4Base8 = 0x43084308u;  // z = 8, without zero points

}  // namespace tpmlp
