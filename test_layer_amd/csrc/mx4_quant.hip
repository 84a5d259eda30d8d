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

// Both directions are bound by memory; a workgroup takes 64 rows x 128 columns, one
// scale tile. Row-major: thread t has 8 columns (16 neighbouring threads a row: 256
// or 512 consecutive bytes) of the rows t / 16 + 16 i, i = 0..3, so that the 4 scale
// bytes of one block column that it is part of are one dword of the tile, and a
// block is 4 neighbouring lanes. (One thread per block of 32 needs no exchange
// between lanes, but its loads step 64 bytes from lane to lane: 137,400 x 1024 bf16
// took 90 us that way.)
template <bool BF16, bool VEC>
__global__ __launch_bounds__(NTHR) void quantize_kernel(const void* X, uint8_t* codes, uint8_t* scales, int64_t rows,
                                                        int k, int nb) {
  const int t = threadIdx.x, piece = t & 15, r = t >> 4;
  const int64_t R = blockIdx.x / (uint32_t)nb;
  const int B = (int)(blockIdx.x % (uint32_t)nb);
  const int k0 = B * 128 + piece * 8;
  float v[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = R * 64 + 16 * i + r;
    load8<BF16, VEC>(X, row, k0, row < rows ? k : 0, v[i]);
  }
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t s;
    const uint32_t q = quantize8(v[i], s);
    word |= s << (8 * i);
    const int64_t row = R * 64 + 16 * i + r;
    if (row < rows) ((uint32_t*)(codes + row * (int64_t)(nb * 64) + B * 64))[piece] = q;
  }
  if ((piece & 3) == 0) ((uint32_t*)scales)[(R * nb + B) * 64 + 16 * (piece >> 2) + r] = word;
}

// X [k][rows]: a wave takes 64 neighbouring rows of one block, a thread one block.
template <bool BF16>
__global__ __launch_bounds__(NTHR) void quantize_transposed_kernel(const void* X, uint8_t* codes, uint8_t* scales,
                                                                   int64_t rows, int k, int nb) {
  __shared__ uint32_t sc[64];
  const int t = threadIdx.x, rr = t & 63, g = t >> 6;
  const int64_t R = blockIdx.x / (uint32_t)nb;
  const int B = (int)(blockIdx.x % (uint32_t)nb);
  const int64_t row = R * 64 + rr;
  const int k0 = B * 128 + g * 32;
  const bool live = row < rows;
  float v[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = live && k0 + j < k ? load1<BF16>(X, (int64_t)(k0 + j) * rows + row) : 0.0f;
  u32x4 o;
  const uint32_t s = quantize_block(v, o);
  if (live) st16(codes + row * (int64_t)(nb * 64) + B * 64 + g * 16, o);
  ((uint8_t*)sc)[(g * 16 + (rr & 15)) * 4 + (rr >> 4)] = (uint8_t)s;
  __syncthreads();
  if (t < 64) ((uint32_t*)scales)[(R * nb + B) * 64 + t] = sc[t];
}

// Thread t has V columns, 16 bytes of X (8 of bf16, 4 of fp32), of the rows
// t / (128 / V) + (2 V) i: stores of a wave lie side by side (with 8 columns of fp32
// a thread they step 32 bytes: 178 us instead of
// 125 for 137,400 x 1024, or 104 streamed).
template <bool BF16, bool VEC, bool STREAM>
__global__ __launch_bounds__(NTHR) void dequantize_kernel(const uint8_t* codes, const uint8_t* scales, void* X,
                                                          int64_t rows, int k, int nb) {
  constexpr int V = BF16 ? 8 : 4, LANES = 128 / V, PASS = NTHR / LANES, N = 64 / PASS;
  constexpr int WORDS = PASS < 16 ? 16 / PASS : 1;  // scale dwords: the rows of a pass modulo 16
  const int t = threadIdx.x, piece = t % LANES, r = t / LANES;
  const int64_t R = blockIdx.x / (uint32_t)nb;
  const int B = (int)(blockIdx.x % (uint32_t)nb);
  const int k0 = B * 128 + piece * V;
  if (k0 >= k) return;
  uint32_t word[WORDS], q[N];
#pragma unroll
  for (int w = 0; w < WORDS; ++w)
    word[w] = ((const uint32_t*)scales)[(R * nb + B) * 64 + 16 * (piece * V / 32) + r + PASS * w];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t row = R * 64 + PASS * i + r;
    const uint8_t* p = codes + row * (int64_t)(nb * 64) + B * 64 + piece * V / 2;
    q[i] = row < rows ? (V == 8 ? *(const uint32_t*)p : *(const uint16_t*)p) : 0u;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t row = R * 64 + PASS * i + r;
    if (row >= rows) continue;
    const uint32_t s = word[i % WORDS] >> (8 * (i / WORDS)) & 255u;
    const float f = scale_value(s);
    float v[8];
#define PAIR(j)                                                                   \
  {                                                                               \
    const auto p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], f, j);          \
    v[2 * j] = s == 255u ? __uint_as_float(0x7fc00000u) : p[0];                   \
    v[2 * j + 1] = s == 255u ? __uint_as_float(0x7fc00000u) : p[1];               \
  }
    PAIR(0) PAIR(1)
    if constexpr (V == 8) {
      PAIR(2) PAIR(3)
    }
#undef PAIR
    if constexpr (VEC) {
      if constexpr (BF16)
        st16<STREAM>((uint16_t*)X + row * k + k0, as_u32x4(pack8(v)));
      else
        st16<STREAM>((float*)X + row * k + k0, __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}));
    } else if (k0 + V <= k) {
      if constexpr (BF16)
        st16_any((uint16_t*)X + row * k + k0, as_u32x4(pack8(v)));
      else
        st16_any((float*)X + row * k + k0, __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}));
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (k0 + j >= k) continue;
        if constexpr (BF16)
          ((uint16_t*)X)[row * k + k0 + j] = f32_to_bf16_bits(v[j]);
        else
          ((float*)X)[row * k + k0 + j] = v[j];
      }
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
#define GO(KERNEL) KERNEL<<<grid, block, 0, stream>>>(X, codes, scales, rows, k, nb)
  if (transposed) {
    if (bf16) GO(quantize_transposed_kernel<true>);
    else GO(quantize_transposed_kernel<false>);
  } else if (bf16) {
    if (vec) GO((quantize_kernel<true, true>));
    else GO((quantize_kernel<true, false>));
  } else {
    if (vec) GO((quantize_kernel<false, true>));
    else GO((quantize_kernel<false, false>));
  }
#undef GO
  return hipGetLastError();
}

hipError_t launch_dequantize(const uint8_t* codes, const uint8_t* scales, void* X, bool bf16, int64_t rows, int k,
                             hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const int nb = (int)(padded_k(k) / kPad);
  const dim3 grid((unsigned)(row_tiles(rows) * nb)), block(NTHR);
  const bool vec = k % (bf16 ? 8 : 4) == 0;
  const bool past = vec && streams(rows * k * (bf16 ? 2 : 4));
#define GO(B, V, S) dequantize_kernel<B, V, S><<<grid, block, 0, stream>>>(codes, scales, X, rows, k, nb)
  if (bf16) {
    if (past) GO(true, true, true);
    else if (vec) GO(true, true, false);
    else GO(true, false, false);
  } else {
    if (past) GO(false, true, true);
    else if (vec) GO(false, true, false);
    else GO(false, false, false);
  }
#undef GO
  return hipGetLastError();
}

}  // namespace mx4
}  // namespace vggt3
