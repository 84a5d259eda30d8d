// Device helpers of the 4-bit kernels: one block's scale and codes.
#pragma once

#include "mx4.hpp"

namespace vggt3 {
namespace mx4 {

constexpr uint32_t kInfBits = 0x7f800000u;

// Scale byte of a block from the largest |x| of it, as fp32 bits (compared as
// integers, so that Inf and NaN, which lie above every finite value, win):
// 2^(floor(log2 max) - 2) puts the largest value in [4, 8), at least 2^-127;
// a block that holds an Inf or a NaN is NaN as a whole (255).
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return amax_bits >= kInfBits ? 255u : (e > 2u ? e - 2u : 0u);
}

// The scale as fp32 (2^-127 is subnormal there). Not for 255.
__device__ __forceinline__ float scale_value(uint32_t s) { return __uint_as_float(s == 0u ? 0x00400000u : s << 23); }

// Eight values -> eight codes, rounded to nearest with ties to the even code,
// saturating at 6 (the converter divides by the scale).
__device__ __forceinline__ uint32_t encode8(const float* v, float scale) {
  uint32_t o = 0;
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[0], v[1], scale, 0);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[2], v[3], scale, 1);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[4], v[5], scale, 2);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[6], v[7], scale, 3);
  return o;
}

// Byte offset of the scale of (row, block) in the tiles of a matrix of nb = kp/128.
__device__ __forceinline__ int64_t scale_at(int64_t row, int block, int nb) {
  return ((row >> 6) * nb + (block >> 2)) * 256 + (((block & 3) * 16 + (int)(row & 15)) << 2) + ((row >> 4) & 3);
}

}  // namespace mx4
}  // namespace vggt3
