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

template <bool BF16>
__device__ __forceinline__ float load1(const void* X, int64_t i) {
  if (BF16) return bf16_bits_to_f32(((const uint16_t*)X)[i]);
  return ((const float*)X)[i];
}

// The 8 values of a row [k] from column k0 on, 0 past k. VEC: 16-byte loads (rows
// start at 16-byte boundaries, k is a whole number of them).
template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(const void* X, int64_t row, int k0, int k, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  if constexpr (VEC && BF16) {
    if (k0 >= k) return;
    const u32x4 q = ld16((const uint16_t*)X + row * k + k0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_lo(q[j]);
      v[2 * j + 1] = bf16_hi(q[j]);
    }
  } else if constexpr (VEC) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (k0 + 4 * h >= k) continue;
      const f32x4 q = *(const f32x4*)((const float*)X + row * k + k0 + 4 * h);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * h + j] = q[j];
    }
  } else if (k0 + 8 <= k) {
    if constexpr (BF16) {
      const u32x4 q = ld16_any((const uint16_t*)X + row * k + k0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = bf16_lo(q[j]);
        v[2 * j + 1] = bf16_hi(q[j]);
      }
    } else {
      const float* p = (const float*)X + row * k + k0;
      const f32x4 a = *(const f32x4_any*)p, b = *(const f32x4_any*)(p + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = a[j];
        v[4 + j] = b[j];
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (k0 + j < k) v[j] = load1<BF16>(X, row * (int64_t)k + k0 + j);
  }
}

// Largest of 4 neighbouring lanes, by DPP.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xb1, 0xf, 0xf, false);  // lane ^ 1
  v = o > v ? o : v;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4e, 0xf, 0xf, false);  // lane ^ 2
  return o > v ? o : v;
}

// A quarter of a block, its other 24 values in the 3 neighbours of a group of 4
// lanes: the block's scale byte and the lane's codes.
__device__ __forceinline__ uint32_t quantize8(const float (&v)[8], uint32_t& s) {
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t a = __float_as_uint(v[j]) & 0x7fffffffu;
    amax = a > amax ? a : amax;
  }
  s = scale_byte(quad_max(amax));
  return s == 255u ? 0u : encode8(v, scale_value(s));
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
