// Device helpers of the block-scaled FP8 operators.
#pragma once

#include <cfloat>

#include "block_fp8.h"
#include "fp8.cuh"
#include "ptx.cuh"

namespace tpmlp {

// The scale of a block with largest magnitude `amax` and the factor its values are multiplied by before the
// cast.  The floor of 2^-100 keeps both finite and normal for a block of zeros; infinities count as FLT_MAX.
struct BlockScale {
  float scale, inv;
};
__device__ __forceinline__ BlockScale block_scale(float amax, float fmax) {
  const float a = fminf(fmaxf(amax, 0x1p-100f), FLT_MAX);
  return {__fdiv_rn(a, fmax), __fdiv_rn(fmax, a)};
}

__host__ __device__ constexpr float fp8_max(int fmt) { return fmt == 0 ? 448.f : 57344.f; }

__device__ __forceinline__ void unpack_vec8(const uint4& u, float (&f)[8]) {
  const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y), c = unpack_bf16x2(u.z), d = unpack_bf16x2(u.w);
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y; f[4] = c.x; f[5] = c.y; f[6] = d.x; f[7] = d.y;
}

__device__ __forceinline__ uint4 pack_vec8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ float abs_max8(const float (&f)[8]) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
  return m;
}

// Largest value over the 16 lanes of a half warp (a 1 x 128 block is 16 vectors of 8 on consecutive lanes).
__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

}  // namespace tpmlp
