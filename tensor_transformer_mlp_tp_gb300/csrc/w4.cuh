// Device helpers of the 4-bit weights.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "w4.h"

namespace tpmlp {

// A word of codes as the four registers of an m16n8k16 product's A operand: bits 4 i and 16 + 4 i are register i.  In fp16,
// 1024 + q is 0x6400 | q and 1024 + 16 q is 0x6400 | q << 4, so that codes at odd places need no shift of their own: they
// come out sixteen times as large, which is their columns' scale's to undo.  base0 = 1024 + z, base1 = 1024 + 16 z twice;
// the differences are exact.
__device__ __forceinline__ uint32_t w4_minus(uint32_t pair, uint32_t base) {
  const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&pair), *reinterpret_cast<const __half2*>(&base));
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <uint32_t MASK>
__device__ __forceinline__ uint32_t w4_pair(uint32_t word) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, 0x64006400, 0xEA;" : "=r"(r) : "r"(word), "n"(MASK));
  return r;
}

__device__ __forceinline__ void w4_unpack(uint32_t word, uint32_t base0, uint32_t base1, uint32_t (&a)[4]) {
  const uint32_t high = word >> 8;
  a[0] = w4_minus(w4_pair<0x000F000Fu>(word), base0);
  a[1] = w4_minus(w4_pair<0x00F000F0u>(word), base1);
  a[2] = w4_minus(w4_pair<0x000F000Fu>(high), base0);
  a[3] = w4_minus(w4_pair<0x00F000F0u>(high), base1);
}

// The same as bf16, with a shift for every code, times a power of two that ONE, a bf16 number of no fraction, gives: ONE's seven
// fraction bits count ONE / 128, so that ONE | q is ONE + q ONE / 128.  base0 and base1 are w4_base<ONE> of columns g and g + 8.
constexpr uint32_t kW4One = 0x4300u;      // 128: q - z
constexpr uint32_t kW4OneLow = 0x3D80u;   // 2^-4: (q - z) 2^-11

template <uint32_t ONE, int I>
__device__ __forceinline__ uint32_t w4_bf16(uint32_t word, uint32_t base) {
  uint32_t pair;
  asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(pair) : "r"(I == 0 ? word : word >> (4 * I)), "n"(ONE * 0x00010001u));
  const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&pair), *reinterpret_cast<const __nv_bfloat162*>(&base));
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <uint32_t ONE>
__device__ __forceinline__ void w4_unpack_bf16(uint32_t word, uint32_t base0, uint32_t base1, uint32_t* a) {
  a[0] = w4_bf16<ONE, 0>(word, base0);
  a[1] = w4_bf16<ONE, 1>(word, base1);
  a[2] = w4_bf16<ONE, 2>(word, base0);
  a[3] = w4_bf16<ONE, 3>(word, base1);
}

template <uint32_t ONE>
__device__ __forceinline__ uint32_t w4_base(uint32_t z) { return (ONE + z) * 0x00010001u; }

__device__ __forceinline__ uint32_t w4_base0(uint32_t z) { return 0x64006400u + z * 0x00010001u; }
__device__ __forceinline__ uint32_t w4_base1(uint32_t z) { return 0x64006400u + z * 0x00100010u; }

}  // namespace tpmlp
