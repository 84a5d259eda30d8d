// Device helpers of the 4-bit kernels: one block's scale and codes.
#pragma once

#include "bf16_ops.hpp"
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

// The 32 values of a row [k] from column k0 on, 0 past k. VEC: 16-byte loads
// (rows start at 16-byte boundaries, k is a whole number of them).
template <bool BF16, bool VEC>
__device__ __forceinline__ void load_block(const void* X, int64_t row, int k0, int k, float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = 0.0f;
  if constexpr (VEC) {
    constexpr int E = BF16 ? 8 : 4;
    const char* p = (const char*)X + (row * (int64_t)k + k0) * (BF16 ? 2 : 4);
#pragma unroll
    for (int c = 0; c < 32 / E; ++c) {
      if (k0 + c * E >= k) continue;
      const u32x4 q = ld16(p + 16 * c);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (BF16) {
          v[c * E + 2 * j] = bf16_lo(q[j]);
          v[c * E + 2 * j + 1] = bf16_hi(q[j]);
        } else {
          v[c * E + j] = __uint_as_float(q[j]);
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int64_t i = row * (int64_t)k + k0 + j;
      if (k0 + j < k) v[j] = BF16 ? bf16_bits_to_f32(((const uint16_t*)X)[i]) : ((const float*)X)[i];
    }
  }
}

// A block's scale byte and its 32 codes.
__device__ __forceinline__ uint32_t quantize_block(const float (&v)[32], u32x4& codes) {
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const uint32_t a = __float_as_uint(v[j]) & 0x7fffffffu;
    amax = a > amax ? a : amax;
  }
  const uint32_t s = scale_byte(amax);
  codes = u32x4{0u, 0u, 0u, 0u};
  if (s != 255u) {
    const float f = scale_value(s);
#pragma unroll
    for (int c = 0; c < 4; ++c) codes[c] = encode8(v + 8 * c, f);
  }
  return s;
}

// Byte offset of the scale of (row, block) in the tiles of a matrix of nb = kp/128.
__device__ __forceinline__ int64_t scale_at(int64_t row, int block, int nb) {
  return ((row >> 6) * nb + (block >> 2)) * 256 + (((block & 3) * 16 + (int)(row & 15)) << 2) + ((row >> 4) & 3);
}

}  // namespace mx4
}  // namespace vggt3
