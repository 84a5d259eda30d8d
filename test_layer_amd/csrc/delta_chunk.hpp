// What the columns of a chunk's products share (forward and backward): rows in
// LDS, decays, and the 32 x 32 matrices as operands. See delta_scan.hip for the
// formulas.
#pragma once

#include <cstddef>

#include "delta.hpp"
#include "delta_ops.hpp"

namespace vggt3 {
namespace delta {

// Parts of an operand that holds fp32 values whole.
template <class T>
constexpr int kWhole = sizeof(T) == 2 ? 3 : 1;
// Rows of D values in LDS, 16 bytes apart in the banks.
template <class T, int D>
constexpr int kPitch = D + 16 / (int)sizeof(T);

// The gates that a chunk's columns use, by token. Its decay up to a token is
// 2^(high + low): high a multiple of 2^-6, so that sums and differences of it are
// exact (at most 32 * 2885 in size), low what that leaves, at most 2^-7 a token. So
// the decay between two tokens is right whatever lies before them, and by a power of 2
// each, since their sum's rounding would show in it: 11 u at e^-20 (u = 2^-24), 44 u at
// e^-80. (Below e^-2000 a token's decay is 0 in either form.)
struct Rows {
  float decay[kChunk];  // from the chunk's start
  float rest[kChunk];   // to its end
  float beta[kChunk];
  float high[kChunk];
  float low[kChunk];
  float total, pad[3];
};

template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float shifted(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, ROWS, 0xf, false));
}
// Sums over the lanes before and with each, in every 32.
__device__ __forceinline__ float running_sum(float x) {
  x += shifted<0x111>(x);  // one lane down, within 16; then 2, 4, 8
  x += shifted<0x112>(x);
  x += shifted<0x114>(x);
  x += shifted<0x118>(x);
  x += shifted<0x142, 0xa>(x);  // the first 16's sum to the second's lanes
  return x;
}

__device__ __forceinline__ float power(float high, float low) {
  return __builtin_amdgcn_exp2f(high) * __builtin_amdgcn_exp2f(low);
}

__device__ __forceinline__ void put_rows(Rows& m, const Args& a, int64_t first, int len, int h, int lane) {
#pragma clang fp contract(off)  // (g log2 e - high would have the product's rest, which low has by itself)
  const int t = lane % 32;
  float high = 0.0f, low = 0.0f, beta = 0.0f;
  if (t < len) {
    if (a.g) {
      float g = a.g[(first + t) * a.hv + h];
      g = g < -2000.0f ? -2000.0f : g;
      constexpr float kLog2e = 1.44269502162933349609f, kMore = 1.92596299112661746887e-08f;  // their sum: log2 e
      const float x = g * kLog2e;
      high = __builtin_rintf(x * 64.0f) * 0.015625f;
      low = __builtin_fmaf(g, kMore, __builtin_fmaf(g, kLog2e, -x)) + (x - high);  // (x - high is exact)
    }
    beta = a.beta[(first + t) * a.hv + h];
  }
  if (a.g) {
    high = running_sum(high);
    low = running_sum(low);
  }
  const float end = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, high), 31)),
              more = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, low), 31));
  if (lane >= kChunk) return;
  m.decay[lane] = power(high, low);
  m.rest[lane] = power(end - high, more - low);
  m.beta[lane] = beta;
  m.high[lane] = high;
  m.low[lane] = low;
  if (lane == 0) m.total = power(end, more);
}
__device__ __forceinline__ f32x4 rows4(const float* v, int it, int q) {
  return *reinterpret_cast<const f32x4*>(v + 16 * it + 4 * q);
}

// The three tiles of a lower triangle [32][32]: 00, 10 (below) and 11.
struct Tri {
  f32x4 t00, t10, t11;
};

__device__ __forceinline__ Tri operator*(const Tri& x, const Tri& y) {
  return Tri{x.t00 * y.t00, x.t10 * y.t10, x.t11 * y.t11};
}

// The decays D_ij from token j to token i. FORWARD: lane (c, q) has rows i = 4q + r of
// columns j = c; otherwise columns j = 4q + r of rows i = c. (Above the diagonal:
// anything.)
template <bool FORWARD>
__device__ __forceinline__ Tri decays(const Rows& m, int lane) {
  const int c = lane % 16, q = lane / 16;
  const float hc[2] = {m.high[c], m.high[16 + c]}, lc[2] = {m.low[c], m.low[16 + c]};
  const f32x4 he[2] = {rows4(m.high, 0, q), rows4(m.high, 1, q)}, le[2] = {rows4(m.low, 0, q), rows4(m.low, 1, q)};
  Tri d;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const auto decay = [&](int i, int j) {
      const float hi = FORWARD ? he[i][r] : hc[i], li = FORWARD ? le[i][r] : lc[i];
      const float hj = FORWARD ? hc[j] : he[j][r], lj = FORWARD ? lc[j] : le[j][r];
      return power(hi - hj, li - lj);
    };
    d.t00[r] = decay(0, 0);
    d.t10[r] = decay(1, 0);
    d.t11[r] = decay(1, 1);
  }
  return d;
}
// What lies on and above (strict: or on) the diagonal to 0.
template <bool FORWARD, bool STRICT>
__device__ __forceinline__ Tri lower(const Tri& m, int lane) {
  const int c = lane % 16, q = lane / 16;
  Tri o = m;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = FORWARD ? 4 * q + r : c, j = FORWARD ? c : 4 * q + r;
    const bool in = STRICT ? j < i : j <= i;
    o.t00[r] = in ? m.t00[r] : 0.0f;
    o.t11[r] = in ? m.t11[r] : 0.0f;
  }
  return o;
}

// A triangle L as a left operand of its rows (tiles with columns 4q + r of rows c), and
// L^T as one (tiles with rows 4q + r of columns c).
template <int P, class T>
__device__ __forceinline__ void lower_rows(Frag<T> (&f)[2], const Tri& m) {
  make<P>(f[0], m.t00, zero4());
  make<P>(f[1], m.t10, m.t11);
}
template <int P, class T>
__device__ __forceinline__ void upper_rows(Frag<T> (&f)[2], const Tri& m) {
  make<P>(f[0], m.t00, m.t10);
  make<P>(f[1], zero4(), m.t11);
}

// Tiles by row -> the same tiles by column (and back): a product with the unit
// matrix, exact.
__device__ __forceinline__ f32x4 turned(const f32x4& x, int lane) {
  f32x4 one;
#pragma unroll
  for (int r = 0; r < 4; ++r) one[r] = 4 * (lane / 16) + r == lane % 16 ? 1.0f : 0.0f;
  return mm16(x, one, zero4());
}

// A chunk's shared matrices in memory, tile by tile as lanes hold them: T = (I + N)^-1
// and B by row, and for the gradient X = (I + beta N')^-1 and B with tiles by column
// (the operands X^T and B^T).
struct Matrices {
  f32x4 t[3][64];
  f32x4 b[3][64];
  Rows rows;
  f32x4 x[3][64];  // the gradient's only
  f32x4 bt[3][64];
};
__host__ __device__ constexpr size_t matrices_bytes(bool keep) {
  return keep ? sizeof(Matrices) : offsetof(Matrices, x);
}
__device__ __forceinline__ Matrices* matrices_of(void* base, int64_t at, bool keep) {
  return reinterpret_cast<Matrices*>(static_cast<char*>(base) + at * matrices_bytes(keep));
}
__device__ __forceinline__ Tri get_tri(const f32x4 (*from)[64], int lane) {
  return Tri{from[0][lane], from[1][lane], from[2][lane]};
}
__device__ __forceinline__ void put_tri(f32x4 (*to)[64], const Tri& m, int lane) {
  to[0][lane] = m.t00;
  to[1][lane] = m.t10;
  to[2][lane] = m.t11;
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
__device__ __forceinline__ Tri turned(const Tri& m, int lane) {
  return Tri{turned(m.t00, lane), turned(m.t10, lane), turned(m.t11, lane)};
}

}  // namespace delta
}  // namespace vggt3
