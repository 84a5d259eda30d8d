// Quantisation to microscaled 4-bit and back.
//
// For each row and block of 32 columns: e = max(floor(log2 max|x|) - 2, -127),
// code = x / 2^e rounded to {0, .5, 1, 1.5, 2, 3, 4, 6} (nearest, ties to the
// even code, saturating). The scale is a power of two and the division exact,
// so each value is rounded once.
#include "bf16_ops.hpp"
#include "mx4_ops.hpp"

namespace vggt3 {
namespace mx4 {
namespace {

constexpr int NTHR = 256;

template <bool BF16>
__device__ __forceinline__ float load1(const void* X, int64_t i) {
  if (BF16) return bf16_bits_to_f32(((const uint16_t*)X)[i]);
  return ((const float*)X)[i];
}

// One workgroup per 64 rows x 128 columns, one thread per (row, block): the
// maximum needs no exchange between lanes, and the 256 scale bytes of the
// workgroup are one whole scale tile, put together in LDS. VEC: rows start at
// 16-byte boundaries and k is a multiple of a 16-byte load.
template <bool BF16, bool TRANS, bool VEC>
__global__ __launch_bounds__(NTHR) void quantize_kernel(const void* X, uint8_t* codes, uint8_t* scales, int64_t rows,
                                                        int k, int nb) {
  __shared__ uint32_t sc[64];
  const int t = threadIdx.x;
  const int64_t R = blockIdx.x / nb;
  const int B = (int)(blockIdx.x % nb);
  // Row-major: 4 neighbouring threads share a row (256 or 512 consecutive
  // bytes); transposed: a wave takes 64 neighbouring rows of one block.
  const int rr = TRANS ? (t & 63) : (t >> 2), g = TRANS ? (t >> 6) : (t & 3);
  const int64_t row = R * 64 + rr;
  const int k0 = B * 128 + g * 32;
  const bool live = row < rows;
  float v[32];
  if constexpr (TRANS) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = live && k0 + j < k ? load1<BF16>(X, (int64_t)(k0 + j) * rows + row) : 0.0f;
  } else {
    load_block<BF16, VEC>(X, live ? row : 0, k0, live ? k : 0, v);
  }
  u32x4 o;
  const uint32_t s = quantize_block(v, o);
  if (live) st16(codes + row * (int64_t)(nb * 64) + B * 64 + g * 16, o);
  ((uint8_t*)sc)[(g * 16 + (rr & 15)) * 4 + (rr >> 4)] = (uint8_t)s;
  __syncthreads();
  if (t < 64) ((uint32_t*)scales)[(R * nb + B) * 64 + t] = sc[t];
}

// One thread per 8 columns of a row.
template <bool BF16, bool VEC>
__global__ __launch_bounds__(NTHR) void dequantize_kernel(const uint8_t* codes, const uint8_t* scales, void* X,
                                                          int64_t rows, int k, int nb) {
  const int groups = (k + 7) / 8;
  const int64_t i = (int64_t)blockIdx.x * NTHR + threadIdx.x;
  if (i >= rows * groups) return;
  const int64_t row = i / groups;
  const int c = (int)(i % groups);
  const uint32_t q = ((const uint32_t*)(codes + row * (int64_t)(nb * 64)))[c];
  const uint32_t s = scales[scale_at(row, c >> 2, nb)];
  const float f = s == 255u ? __uint_as_float(0x7fc00000u) : scale_value(s);
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t code = (q >> (4 * j)) & 15u, m = code & 7u;
    // {0, .5, 1, 1.5, 2, 3, 4, 6}: .5 m below 2, else (1 + .5 (m & 1)) 2^(m / 2 - 1)
    const float a = m < 4u ? 0.5f * (float)m : (float)(2u + (m & 1u)) * (m < 6u ? 1.0f : 2.0f);
    v[j] = (code & 8u ? -a : a) * f;
  }
  if (VEC) {
    if (BF16) {
      st16((uint16_t*)X + row * k + 8 * c, as_u32x4(pack8(v)));
    } else {
      float* p = (float*)X + row * k + 8 * c;
      *(f32x4*)p = f32x4{v[0], v[1], v[2], v[3]};
      *(f32x4*)(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (8 * c + j >= k) continue;
      if (BF16)
        ((uint16_t*)X)[row * k + 8 * c + j] = f32_to_bf16_bits(v[j]);
      else
        ((float*)X)[row * k + 8 * c + j] = v[j];
    }
  }
}

}  // namespace

hipError_t launch_quantize(const void* X, bool transposed, bool bf16, uint8_t* codes, uint8_t* scales, int64_t rows,
                           int k, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const int nb = (int)(padded_k(k) / kPad);
  const dim3 grid((unsigned)(row_tiles(rows) * nb)), block(NTHR);
  const bool vec = k % (bf16 ? 8 : 4) == 0;
#define GO(B, T, V) quantize_kernel<B, T, V><<<grid, block, 0, stream>>>(X, codes, scales, rows, k, nb)
  if (bf16) {
    if (transposed) GO(true, true, false);
    else if (vec) GO(true, false, true);
    else GO(true, false, false);
  } else {
    if (transposed) GO(false, true, false);
    else if (vec) GO(false, false, true);
    else GO(false, false, false);
  }
#undef GO
  return hipGetLastError();
}

hipError_t launch_dequantize(const uint8_t* codes, const uint8_t* scales, void* X, bool bf16, int64_t rows, int k,
                             hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const int nb = (int)(padded_k(k) / kPad);
  const dim3 grid((unsigned)((rows * ((k + 7) / 8) + NTHR - 1) / NTHR)), block(NTHR);
  const bool vec = k % 8 == 0;
#define GO(B, V) dequantize_kernel<B, V><<<grid, block, 0, stream>>>(codes, scales, X, rows, k, nb)
  if (bf16) {
    if (vec) GO(true, true);
    else GO(true, false);
  } else {
    if (vec) GO(false, true);
    else GO(false, false);
  }
#undef GO
  return hipGetLastError();
}

}  // namespace mx4
}  // namespace vggt3
