// Microscaled 4-bit matrices (MX, element type e2m1, block 32, e8m0 scales):
// the stored form and the launchers of its kernels.
//
// A matrix [rows][k] is two arrays, with kp = k rounded up to 128:
//   codes   [rows][kp/2] bytes, two values each, the even column in the low
//           nibble. Bit 3 is the sign, bits 0-2 index {0, .5, 1, 1.5, 2, 3, 4, 6}.
//   scales  one byte s per row and 32 columns, standing for 2^(s - 127) (255:
//           the block is NaN), as tiles [ceil(rows/64)][kp/128][64][4]: the byte
//           of row 64 R + 16 i + r and block 4 B + g is [R][B][16 g + r][i].
// Columns k .. kp-1 hold code 0 and, in whole blocks, scale 0, so they add 0 to
// a product; tile rows past `rows` hold scale 0.
//
// A 16x16x128 scaled MFMA takes from lane 16 g + r the 32 values of row r,
// columns 32 g .. 32 g + 31 (16 bytes) and, out of a 32-bit register, the scale
// byte that a 2-bit immediate selects. So one scale tile (256 bytes, one dword
// a lane, one coalesced load) serves 64 rows x 128 columns, with i as the
// immediate, and no scale passes through LDS or is shuffled.
#pragma once

#include "common.hpp"

namespace vggt3 {
namespace mx4 {

constexpr int kBlock = 32;    // values a scale covers
constexpr int kPad = 128;     // k is padded to the depth of one MFMA
constexpr int kTileRows = 64;  // rows of a scale tile

constexpr int64_t padded_k(int64_t k) { return (k + kPad - 1) / kPad * kPad; }
constexpr int64_t row_tiles(int64_t rows) { return (rows + kTileRows - 1) / kTileRows; }
constexpr int64_t code_bytes(int64_t rows, int64_t k) { return rows * (padded_k(k) / 2); }
constexpr int64_t scale_bytes(int64_t rows, int64_t k) { return row_tiles(rows) * kTileRows * (padded_k(k) / kBlock); }

struct Matrix {  // [rows][kp], read only
  const uint8_t* codes;
  const uint8_t* scales;
};

// X [rows][k] (or, transposed, [k][rows]) -> codes, scales.
hipError_t launch_quantize(const void* X, bool transposed, bool bf16, uint8_t* codes, uint8_t* scales, int64_t rows,
                           int k, hipStream_t stream);
// codes, scales -> X [rows][k].
hipError_t launch_dequantize(const uint8_t* codes, const uint8_t* scales, void* X, bool bf16, int64_t rows, int k,
                             hipStream_t stream);

// C[i][j] = sum_k A[i][k] W[j][k], fp32 accumulation, C [m][n] bf16 or fp32.
hipError_t launch_gemm(const Matrix& A, const Matrix& W, void* C, bool bf16, int64_t m, int n, int k,
                       hipStream_t stream);
// H = quantised(silu(A Wg^T) * (A Wu^T)), n hidden units (a multiple of 128).
hipError_t launch_gemm_swiglu(const Matrix& A, const Matrix& Wg, const Matrix& Wu, uint8_t* h_codes,
                              uint8_t* h_scales, int64_t m, int n, int k, hipStream_t stream);
// The same for a few tokens A [m][k], quantised inside the product; only where
// takes_tokens says so.
bool takes_tokens(int64_t m, int k);
hipError_t launch_gemm_tokens(const void* A, bool a_bf16, const Matrix& W, void* C, bool bf16, int64_t m, int n, int k,
                              hipStream_t stream);
hipError_t launch_gemm_swiglu_tokens(const void* A, const Matrix& Wg, const Matrix& Wu, uint8_t* h_codes,
                                     uint8_t* h_scales, int64_t m, int n, int k, hipStream_t stream);

}  // namespace mx4
}  // namespace vggt3
