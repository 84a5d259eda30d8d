// What the columns of a chunk's products share (forward and backward): rows in
// LDS, decays, and the 32 x 32 matrices as operands. See delta_scan.hip for the
// formulas.
#pragma once

#include <cstddef>

#include "delta.hpp"
#include "delta_ops.hpp"

namespace vggt3 {
namespace delta {

constexpr double kLog2eD = 1.4426950408889634074;

// Parts of an operand that holds fp32 values whole, and its 16-byte pieces.
template <class T>
constexpr int kWhole = sizeof(T) == 2 ? 3 : 1;
template <class T>
constexpr int kOperand = 64 * (sizeof(T) == 2 ? 3 : 2);
// Rows of D values in LDS, 16 bytes apart in the banks.
template <class T, int D>
constexpr int kPitch = D + 16 / (int)sizeof(T);

// Rows 0 .. len - 1 of src, `ld` apart, to LDS, zeros behind them, by COUNT threads.
template <class T, int D, int COUNT>
__device__ __forceinline__ void stage(T* dst, const T* src, int64_t ld, int len, int thread) {
  constexpr int kPiece = 16 / sizeof(T), kPieces = D / kPiece;
#pragma unroll
  for (int x = 0; x < kChunk * kPieces / COUNT; ++x) {
    const int at = x * COUNT + thread, row = at / kPieces, col = at % kPieces * kPiece;
    u32x4 w = {0, 0, 0, 0};
    if (row < len) w = ld16(src + row * ld + col);
    st16(dst + row * kPitch<T, D> + col, w);
  }
}

// Lane t % 32's token: the chunk's decay up to it, as a power of 2 in 64 bits, so that
// a difference of two is right whatever lies before them; and beta. (Below 2^-2000 a
// decay is 0 in either form.)
struct Gates {
  double G, end;  // end: of the whole chunk
  float beta;
};
__device__ __forceinline__ Gates gates(const Args& a, int64_t first, int len, int h, int lane) {
  const int t = lane % 32;
  Gates x{0.0, 0.0, 0.0f};
  if (t < len) {
    if (a.g) {
      const float g = a.g[(first + t) * a.hv + h];
      x.G = (g < -2000.0f ? -2000.0f : g) * kLog2eD;
    }
    x.beta = a.beta[(first + t) * a.hv + h];
  }
  if (a.g) {
#pragma unroll
    for (int off = 1; off < kChunk; off *= 2) {
      const double up = __shfl_up(x.G, off, 32);
      if (t >= off) x.G += up;
    }
    x.end = __shfl(x.G, 31, 32);
  }
  return x;
}
__device__ __forceinline__ float exp2d(double x) { return __builtin_amdgcn_exp2f((float)x); }

// The gates that a chunk's columns use, by token.
struct Rows {
  float decay[kChunk];  // from the chunk's start
  float rest[kChunk];   // to its end
  float beta[kChunk];
  float total;
};
__device__ __forceinline__ void put_rows(Rows& m, const Gates& x, int lane) {
  if (lane >= kChunk) return;
  m.decay[lane] = exp2d(x.G);
  m.rest[lane] = exp2d(x.end - x.G);
  m.beta[lane] = x.beta;
  if (lane == 31) m.total = exp2d(x.G);
}
__device__ __forceinline__ f32x4 rows4(const float* v, int it, int q) {
  return *reinterpret_cast<const f32x4*>(v + 16 * it + 4 * q);
}

// The three tiles of a lower triangle [32][32]: 00, 10 (below) and 11.
struct Tri {
  f32x4 t00, t10, t11;
};

// D_ij x_ij for j < i (strict) or j <= i, 0 elsewhere, times beta_j if `beta`, times f.
// FORWARD: lane (c, q) holds rows i = 4q + r of columns j = c; otherwise columns
// 4q + r of rows i = c.
template <bool FORWARD>
__device__ __forceinline__ void decay_tri(Tri& m, const Gates& x, bool strict, bool beta, float f, int lane) {
  const int c = lane % 16, q = lane / 16;
  const double Gc0 = __shfl(x.G, c, 32), Gc1 = __shfl(x.G, 16 + c, 32);
  const float bc0 = __shfl(x.beta, c, 32), bc1 = __shfl(x.beta, 16 + c, 32);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int e = 4 * q + r;
    const double Ge0 = __shfl(x.G, e, 32), Ge1 = __shfl(x.G, 16 + e, 32);
    float d00, d10, d11, b0 = 1.0f, b1 = 1.0f;
    bool in;
    if (FORWARD) {
      d00 = exp2d(Ge0 - Gc0);
      d10 = exp2d(Ge1 - Gc0);
      d11 = exp2d(Ge1 - Gc1);
      in = strict ? c < e : c <= e;
      if (beta) {
        b0 = bc0;
        b1 = bc1;
      }
    } else {
      d00 = exp2d(Gc0 - Ge0);
      d10 = exp2d(Gc1 - Ge0);
      d11 = exp2d(Gc1 - Ge1);
      in = strict ? e < c : e <= c;
      if (beta) {
        b0 = __shfl(x.beta, e, 32);
        b1 = __shfl(x.beta, 16 + e, 32);
      }
    }
    m.t00[r] = in ? m.t00[r] * d00 * b0 * f : 0.0f;
    m.t10[r] = m.t10[r] * d10 * b0 * f;
    m.t11[r] = in ? m.t11[r] * d11 * b1 * f : 0.0f;
  }
}

// Tiles of X Y^T, X and Y [kChunk][pitch] in LDS, where lane (c, q) gets rows 4q + r
// of X and column c of Y: 00, 10 (rows of X 16-31, columns 0-15 of Y) and 11.
template <int NX, int NY, class T, int D, class LX, class LY>
__device__ __forceinline__ Tri products(LX x, LY y, int q) {
  Tri m{zero4(), zero4(), zero4()};
#pragma unroll
  for (int s = 0; s < D / 32; ++s) {
    Frag<T> x0, x1, y0, y1;
    x(x0, 0, 32 * s + 8 * q);
    x(x1, 16, 32 * s + 8 * q);
    y(y0, 0, 32 * s + 8 * q);
    y(y1, 16, 32 * s + 8 * q);
    m.t00 = mm<NX, NY>(x0, y0, m.t00);
    m.t10 = mm<NX, NY>(x1, y0, m.t10);
    m.t11 = mm<NX, NY>(x1, y1, m.t11);
  }
  return m;
}

// A triangle as a left operand: L from tiles that hold its rows i by lane (columns
// 4q + r), and L^T from tiles that hold its columns j by lane.
template <class T, int P>
__device__ __forceinline__ void put_lower(u32x4* at, const Tri& m, int lane) {
  Frag<T> f;
  make<P>(f, m.t00, zero4());
  put<P>(at, f, lane);
  make<P>(f, m.t10, m.t11);
  put<P>(at + kOperand<T>, f, lane);
}
template <class T, int P>
__device__ __forceinline__ void put_upper(u32x4* at, const Tri& m, int lane) {
  Frag<T> f;
  make<P>(f, m.t00, m.t10);
  put<P>(at, f, lane);
  make<P>(f, zero4(), m.t11);
  put<P>(at + kOperand<T>, f, lane);
}

// Tiles by row -> the same tiles by column (and back): a product with the unit
// matrix, exact.
__device__ __forceinline__ f32x4 turned(const f32x4& x, int lane) {
  f32x4 one;
#pragma unroll
  for (int r = 0; r < 4; ++r) one[r] = 4 * (lane / 16) + r == lane % 16 ? 1.0f : 0.0f;
  return mm16(x, one, zero4());
}

// A chunk's shared matrices in memory, as operands: tiles 00, 10, 11 of T and B by row,
// and for the gradient of their transposes (tiles by column). B of the forward alone is
// in two bf16 parts (bf16).
struct Matrices {
  f32x4 t[3][64];
  f32x4 b[3][64];
  Rows rows;
  float pad[kChunk - 1];
  f32x4 tt[3][64];  // the gradient's only
  f32x4 bt[3][64];
};
__host__ __device__ constexpr size_t matrices_bytes(bool keep) {
  return keep ? sizeof(Matrices) : offsetof(Matrices, tt);
}
__device__ __forceinline__ Matrices* matrices_of(void* base, int64_t at, bool keep) {
  return reinterpret_cast<Matrices*>(static_cast<char*>(base) + at * matrices_bytes(keep));
}
__device__ __forceinline__ void put_tri(f32x4 (*to)[64], const Tri& m, int lane) {
  to[0][lane] = m.t00;
  to[1][lane] = m.t10;
  to[2][lane] = m.t11;
}
// A tile in two bf16 parts, and two of them as an operand.
template <class T>
__device__ __forceinline__ u32x4 tile_parts(const f32x4& x) {
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(u32x4, x);
  } else {
    const uint32_t a = pack_bf16x2(x[0], x[1]), b = pack_bf16x2(x[2], x[3]);
    return u32x4{a, b, pack_bf16x2(x[0] - bf16_lo(a), x[1] - bf16_hi(a)), pack_bf16x2(x[2] - bf16_lo(b), x[3] - bf16_hi(b))};
  }
}
template <class T>
__device__ __forceinline__ void put_tri_parts(f32x4 (*to)[64], const Tri& m, int lane) {
  to[0][lane] = __builtin_bit_cast(f32x4, tile_parts<T>(m.t00));
  to[1][lane] = __builtin_bit_cast(f32x4, tile_parts<T>(m.t10));
  to[2][lane] = __builtin_bit_cast(f32x4, tile_parts<T>(m.t11));
}
__device__ __forceinline__ void parts_frag(Frag<uint16_t>& f, const u32x4& x, const u32x4& y) {
  f.part[0] = as_bf16x8(u32x4{x[0], x[1], y[0], y[1]});
  f.part[1] = as_bf16x8(u32x4{x[2], x[3], y[2], y[3]});
}
__device__ __forceinline__ void parts_frag(Frag<float>& f, const u32x4& x, const u32x4& y) {
  f.a = __builtin_bit_cast(f32x4, x);
  f.b = __builtin_bit_cast(f32x4, y);
}

// The tile of 16 * NCT columns that a lane has NCT of, to and from rows in memory.
template <int DK, int NCT>
__device__ __forceinline__ void load_state(f32x4 (*S)[NCT], const float* from, int64_t ld, int q) {
#pragma unroll
  for (int t = 0; t < DK / 16; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float w[NCT];
#pragma unroll
      for (int x = 0; x < NCT; ++x) w[x] = 0.0f;
      if (from) load_n<NCT>(w, from + channel(t, 4 * q + r) * ld);
#pragma unroll
      for (int x = 0; x < NCT; ++x) S[t][x][r] = w[x];
    }
}
template <int DK, int NCT>
__device__ __forceinline__ void store_state(const f32x4 (*S)[NCT], float* to, int64_t ld, int q) {
#pragma unroll
  for (int t = 0; t < DK / 16; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float w[NCT];
#pragma unroll
      for (int x = 0; x < NCT; ++x) w[x] = S[t][x][r];
      store_n<NCT>(to + channel(t, 4 * q + r) * ld, w);
    }
}
template <int DK, int NCT>
__device__ __forceinline__ void unit_state(f32x4 (*S)[NCT], int col, int q) {
#pragma unroll
  for (int t = 0; t < DK / 16; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int x = 0; x < NCT; ++x) S[t][x][r] = channel(t, 4 * q + r) == col + x ? 1.0f : 0.0f;
}
// Rows of a chunk's values, 0 behind its end.
template <int NCT, class T>
__device__ __forceinline__ void load_rows(f32x4 (*V)[NCT], const T* from, int64_t ld, int len, int q) {
#pragma unroll
  for (int it = 0; it < 2; ++it)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * it + 4 * q + r;
      float w[NCT];
#pragma unroll
      for (int x = 0; x < NCT; ++x) w[x] = 0.0f;
      if (row < len) load_n<NCT>(w, from + row * ld);
#pragma unroll
      for (int x = 0; x < NCT; ++x) V[it][x][r] = w[x];
    }
}
template <int NCT, class T>
__device__ __forceinline__ void store_rows(T* to, const f32x4 (*V)[NCT], int64_t ld, int len, int q) {
#pragma unroll
  for (int it = 0; it < 2; ++it)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * it + 4 * q + r;
      float w[NCT];
#pragma unroll
      for (int x = 0; x < NCT; ++x) w[x] = V[it][x][r];
      if (row < len) store_n<NCT>(to + row * ld, w);
    }
}

__device__ __forceinline__ Tri turned(const Tri& m, int lane) {
  return Tri{turned(m.t00, lane), turned(m.t10, lane), turned(m.t11, lane)};
}

}  // namespace delta
}  // namespace vggt3
