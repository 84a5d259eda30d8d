// Products of microscaled 4-bit matrices on the scaled MFMA of gfx950.
//
//   C[i][j] = sum_b 2^(sa[i][b] + sw[j][b]) sum_{k in block b} a[i][k] w[j][k]
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes 4-bit operands and their scales and
// adds 128 products a lane group in fp32. The weight rows are its first operand and
// the token rows its second, so a lane ends with 4 neighbouring columns of one
// row of C.
#include <utility>

#include "bf16_ops.hpp"
#include "kernels.hpp"
#include "mx4_ops.hpp"

namespace vggt3 {
namespace mx4 {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lu8;
typedef __attribute__((address_space(3))) i32x4 li32x4;
typedef __attribute__((address_space(3))) void lvoid;

template <int... I, class F>
__device__ __forceinline__ void unrolled(std::integer_sequence<int, I...>, F&& f) {
  (f(std::integral_constant<int, I>{}), ...);
}

// 16x16x128 product of 4-bit operands (format 4 of the instruction's five).
//   A: lane l holds row l%16, columns 32 (l/16) ..+31; B likewise
//   C: lane l, register r holds C[row = 4 (l/16) + r][col = l%16]
template <int IA, int IB>
__device__ __forceinline__ f32x4 mfma4(const i32x4& a, const i32x4& b, const f32x4& c, uint32_t sa, uint32_t sb) {
  const i32x8 a8 = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8 b8 = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, IA, (int)sa, IB, (int)sb);
}

struct Args {
  Matrix A, W, W2;  // token rows, weight rows (W2: the up matrix of the SwiGLU)
  const void* tokens;  // A as tokens [m][k] (direct_kernel)
  int64_t m;
  int n, k, nb;  // nb = kp / 128
  void* out;     // C, or the codes of H
  uint8_t* h_scales;
};

enum Epi { EPI_BF16, EPI_F32, EPI_SWIGLU };

// Four neighbouring columns of one row of C.
template <int EPI>
__device__ __forceinline__ void store_tile(const Args& g, const f32x4& v, int64_t row, int64_t col) {
  if (row >= g.m) return;
  if constexpr (EPI == EPI_BF16) {
    uint16_t* o = (uint16_t*)g.out + row * g.n + col;
    if (g.n % 4 == 0 && col < g.n) {
      st8(o, u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])});
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (col + r < g.n) o[r] = f32_to_bf16_bits(v[r]);
    }
  } else {
    float* o = (float*)g.out + row * g.n + col;
    if (g.n % 4 == 0 && col < g.n) {
      *(f32x4*)o = v;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (col + r < g.n) o[r] = v[r];
    }
  }
}

// One block of H: a lane's 8 of 32 gate and up sums of one row (units 4 (l/16)
// ..+3 and 16 more), the other 24 in the lanes 16, 32 and 48 further.
// Quantised from fp32; the lane's codes are two 16-bit halves, 8 bytes apart.
__device__ __forceinline__ uint32_t swiglu_codes(const f32x4 (&gate)[2], const f32x4 (&up)[2], uint32_t& s) {
  float h[8];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float v = gate[i][r] * sigmoid_fast(gate[i][r]) * up[i][r];
      h[4 * i + r] = v;
      const uint32_t a = __float_as_uint(v) & 0x7fffffffu;
      amax = a > amax ? a : amax;
    }
#pragma unroll
  for (int off = 16; off <= 32; off <<= 1) {
    const uint32_t o = __shfl_xor(amax, off, 64);
    amax = o > amax ? o : amax;
  }
  s = scale_byte(amax);
  return s == 255u ? 0u : encode8(h, scale_value(s));
}

// LDS tiles: [rows][128 bytes] (256 columns), 16-byte piece c of a row kept at
// position c ^ ((row / 2) % 8): the 16 lanes of an operand read (16 rows, one
// piece) then touch every bank equally often.
constexpr int BKB = 128;
__device__ __forceinline__ int swz(int row) { return (row >> 1) & 7; }

__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// BN x BM tile of C^T per workgroup of WN x WM waves, each TN x TM tiles of
// 16x16; k stages of 256 columns (two MFMA steps) in a double-buffered LDS,
// filled by direct global-to-LDS loads. The scales go straight to registers.
template <int TN, int TM, int WN, int WM, int EPI>
__global__ __launch_bounds__(64 * WN * WM) void gemm_kernel(Args g) {
  constexpr int NW = WN * WM, NTHR = 64 * NW;
  constexpr int BN = 16 * TN * WN, BM = 16 * TM * WM;
  static_assert(TN % 4 == 0 && TM % 4 == 0, "a wave's rows are whole scale tiles");
  constexpr int SN = TN / 4, SM = TM / 4;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * (BN + BM) * BKB];
  lu8* const lds = (lu8*)smem;

  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int wn = wid % WN, wm = wid / WN;
  const int64_t tiles_n = (g.n + (EPI == EPI_SWIGLU ? BN / 2 : BN) - 1) / (EPI == EPI_SWIGLU ? BN / 2 : BN);
  const int64_t b = xcd_remap(blockIdx.x, gridDim.x);
  const int64_t n0 = (b % tiles_n) * (EPI == EPI_SWIGLU ? BN / 2 : BN), m0 = (b / tiles_n) * BM;

  const int nst = (g.nb + 1) / 2;
  const int64_t ld = (int64_t)g.nb * 64;

  // Rows past the end read the last one: they give values of C that are not stored.
  auto dma = [&](lu8* tile, const uint8_t* src, int64_t r0, int64_t rows, int R, int st) {
    const uint8_t* base = src + r0 * ld + (int64_t)st * BKB;
    const int rmax = (int)(rows - r0 - 1);
    const bool half = 2 * st + 1 >= g.nb;  // the last stage of an odd nb: 64 bytes a row
    for (int i = 0; i < R * 8 / NTHR; ++i) {
      const int p = (NW * i + wid) * 64 + lane;
      const int row = p >> 3;
      int c = (p & 7) ^ swz(row);
      if (half) c &= 3;
      __builtin_amdgcn_global_load_lds(base + (int64_t)(row < rmax ? row : rmax) * ld + 16 * c,
                                       (lvoid*)(tile + (NW * i + wid) * 1024), 16, 0, 0);
    }
  };
  // SwiGLU: tile rows are [32 gate units | the same 32 up units] in turn.
  auto dma_gu = [&](lu8* tile, int st) {
    const bool half = 2 * st + 1 >= g.nb;
    for (int i = 0; i < BN * 8 / NTHR; ++i) {
      const int p = (NW * i + wid) * 64 + lane;
      const int row = p >> 3;
      int c = (p & 7) ^ swz(row);
      if (half) c &= 3;
      const uint8_t* src = (row & 32) ? g.W2.codes : g.W.codes;
      const int64_t unit = n0 + (row >> 6) * 32 + (row & 31);
      __builtin_amdgcn_global_load_lds(src + unit * ld + (int64_t)st * BKB + 16 * c,
                                       (lvoid*)(tile + (NW * i + wid) * 1024), 16, 0, 0);
    }
  };
  const int64_t nrt = row_tiles(g.n), mrt = row_tiles(g.m);
  auto scale_word = [&](const uint8_t* s, int64_t rt, int blk) {
    return ((const uint32_t*)s)[(rt * g.nb + (blk < g.nb ? blk : g.nb - 1)) * 64 + lane];
  };
  auto load_scales = [&](uint32_t (&sn)[2][SN], uint32_t (&sm)[2][SM], int st) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (EPI == EPI_SWIGLU) {
        const int64_t unit = n0 + 32 * wn;
        const int sh = (unit & 32) ? 16 : 0;  // the lower or upper 32 rows of a scale tile
        const uint32_t a = scale_word(g.W.scales, unit >> 6, 2 * st + u) >> sh;
        const uint32_t c = scale_word(g.W2.scales, unit >> 6, 2 * st + u) >> sh;
        sn[u][0] = (a & 0xffffu) | (c << 16);
      } else {
#pragma unroll
        for (int i = 0; i < SN; ++i) {
          const int64_t rt = (n0 >> 6) + wn * SN + i;
          sn[u][i] = scale_word(g.W.scales, rt < nrt ? rt : nrt - 1, 2 * st + u);
        }
      }
#pragma unroll
      for (int i = 0; i < SM; ++i) {
        const int64_t rt = (m0 >> 6) + wm * SM + i;
        sm[u][i] = scale_word(g.A.scales, rt < mrt ? rt : mrt - 1, 2 * st + u);
      }
    }
  };

  f32x4 acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  uint32_t sn[2][2][SN], sm[2][2][SM];
  auto issue = [&](int st, int s) {
    lu8* const P = lds + s * (BN + BM) * BKB;
    if (EPI == EPI_SWIGLU)
      dma_gu(P, st);
    else
      dma(P, g.W.codes, n0, g.n, BN, st);
    dma(P + BN * BKB, g.A.codes, m0, g.m, BM, st);
  };
  const int i16 = lane & 15, g4 = lane >> 4;
  auto compute = [&](int st, int s, const uint32_t (&ssn)[2][SN], const uint32_t (&ssm)[2][SM]) {
    const lu8* const P = lds + s * (BN + BM) * BKB;
    const lu8* const Q = P + BN * BKB;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (u == 1 && 2 * st + 1 >= g.nb) break;
      const int off = i16 * BKB + 16 * ((4 * u + g4) ^ swz(i16));
      i32x4 p[TN], q[TM];
#pragma unroll
      for (int i = 0; i < TN; ++i) p[i] = *(const li32x4*)(P + (wn * TN + i) * 16 * BKB + off);
#pragma unroll
      for (int j = 0; j < TM; ++j) q[j] = *(const li32x4*)(Q + (wm * TM + j) * 16 * BKB + off);
      unrolled(std::make_integer_sequence<int, TM>{}, [&](auto J) {
        constexpr int j = decltype(J)::value;
        unrolled(std::make_integer_sequence<int, TN>{}, [&](auto I) {
          constexpr int i = decltype(I)::value;
          acc[i][j] = mfma4<i & 3, j & 3>(p[i], q[j], acc[i][j], ssn[u][i >> 2], ssm[u][j >> 2]);
        });
      });
    }
  };

  issue(0, 0);
  load_scales(sn[0], sm[0], 0);
  wait_loads();
  __syncthreads();
  for (int st = 0; st < nst; st += 2) {
    if (st + 1 < nst) {
      issue(st + 1, 1);
      load_scales(sn[1], sm[1], st + 1);
    }
    compute(st, 0, sn[0], sm[0]);
    wait_loads();
    __syncthreads();
    if (st + 1 >= nst) break;
    if (st + 2 < nst) {
      issue(st + 2, 0);
      load_scales(sn[0], sm[0], st + 2);
    }
    compute(st + 1, 1, sn[1], sm[1]);
    wait_loads();
    __syncthreads();
  }

  if constexpr (EPI == EPI_SWIGLU) {
    // Each wave holds gate (tiles 0, 1) and up (tiles 2, 3) of the same 32
    // units: one block of H per row. Codes and scales are gathered in LDS.
    constexpr int HB = BN / 4;  // bytes of codes per row of this tile
    lu8* const hc = lds;                 // [BM][HB]
    lu8* const hs = lds + BM * HB;       // [BM / 64][64][4], the scale tiles
    static_assert(EPI != EPI_SWIGLU || (TN == 4 && WN == 4), "a tile is 128 units: one scale tile wide");
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int row = (wm * TM + j) * 16 + i16;
      const f32x4 c0[2] = {acc[0][j], acc[1][j]}, c1[2] = {acc[2][j], acc[3][j]};
      uint32_t s;
      const uint32_t q = swiglu_codes(c0, c1, s);
      if (m0 + row >= g.m) s = 0;
      lu8* const d = hc + row * HB + wn * 16 + 2 * g4;
      *(__attribute__((address_space(3))) uint16_t*)d = (uint16_t)q;
      *(__attribute__((address_space(3))) uint16_t*)(d + 8) = (uint16_t)(q >> 16);
      if (g4 == 0) hs[(row >> 6) * 256 + (wn * 16 + i16) * 4 + ((row >> 4) & 3)] = (uint8_t)s;
    }
    __syncthreads();
    const int hnb = g.n / 128;  // scale tiles across H
    for (int p = threadIdx.x; p < BM * HB / 16; p += NTHR) {
      const int row = p / (HB / 16), c = p % (HB / 16);
      if (m0 + row < g.m)
        *(i32x4*)((uint8_t*)g.out + (m0 + row) * (int64_t)(hnb * 64) + n0 / 2 + 16 * c) =
            *(const li32x4*)(hc + row * HB + 16 * c);
    }
    for (int p = threadIdx.x; p < BM; p += NTHR) {
      const int64_t rt = (m0 >> 6) + (p >> 6);
      if (rt < mrt)
        ((uint32_t*)g.h_scales)[(rt * hnb + n0 / 128) * 64 + (p & 63)] =
            *(__attribute__((address_space(3))) uint32_t*)(hs + p * 4);
    }
    return;
  }

#pragma unroll
  for (int j = 0; j < TM; ++j)
#pragma unroll
    for (int i = 0; i < TN; ++i)
      store_tile<EPI>(g, acc[i][j], m0 + (wm * TM + j) * 16 + i16, n0 + (wn * TN + i) * 16 + 4 * g4);
}

// Products with few tiles: a tile of 16 TN x 16 TM per workgroup, its KW waves
// splitting k between them, operands straight from global memory to registers
// (nothing is shared between the waves), the waves' sums joined in LDS in wave
// order. TOK: A comes as tokens (at most 16 rows), which every workgroup
// quantises for itself into LDS: one launch instead of two.
enum Tok { TOK_NONE, TOK_BF16, TOK_F32 };

template <int TN, int TM, int KW, int EPI, int TOK>
__global__ __launch_bounds__(64 * KW) void direct_kernel(Args g) {
  static_assert(4 % TN == 0 && 4 % TM == 0, "a tile's rows lie in one scale tile");
  static_assert(EPI != EPI_SWIGLU || TN == 4, "two gate tiles, two up tiles");
  static_assert(TOK == TOK_NONE || TM == 1, "tokens: one row tile");
  constexpr int NT = TN * TM;
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  __shared__ __attribute__((aligned(16))) float red[KW > 1 ? KW * NT * 256 : 4];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int i16 = lane & 15, g4 = lane >> 4;
  constexpr int BN = EPI == EPI_SWIGLU ? 32 : 16 * TN;
  const int tiles_n = (g.n + BN - 1) / BN;
  const int64_t b = xcd_remap(blockIdx.x, gridDim.x);
  const int64_t n0 = (b % tiles_n) * BN, m0 = b / tiles_n * (16 * TM);
  const int64_t ld = (int64_t)g.nb * 64;

  // Quantised tokens in LDS: rows of nb * 64 + 16 bytes (the 16 spread the rows
  // over the banks), then the scale bytes, rows of nb * 4.
  const int qld = g.nb * 64 + 16;  // (tokens only)
  uint8_t* const qs = dyn + (TOK == TOK_NONE ? 0 : (int)g.m * qld);
  if constexpr (TOK != TOK_NONE) {
    const int kb = g.nb * 4;
    for (int i = threadIdx.x; i < (int)g.m * kb; i += 64 * KW) {
      const int row = i / kb, blk = i % kb;
      float v[32];
      if (g.k % (TOK == TOK_BF16 ? 8 : 4) == 0)
        load_block<TOK == TOK_BF16, true>(g.tokens, row, blk * 32, g.k, v);
      else
        load_block<TOK == TOK_BF16, false>(g.tokens, row, blk * 32, g.k, v);
      u32x4 o;
      const uint32_t s = quantize_block(v, o);
      st16(dyn + row * qld + blk * 16, o);
      qs[row * kb + blk] = (uint8_t)s;
    }
    __syncthreads();
  }

  const uint8_t* wrow[TN];
#pragma unroll
  for (int i = 0; i < TN; ++i) {
    if (EPI == EPI_SWIGLU) {
      wrow[i] = (i < 2 ? g.W.codes : g.W2.codes) + (n0 + 16 * (i & 1) + i16) * ld + 16 * g4;
    } else {
      const int64_t row = n0 + 16 * i + i16;
      wrow[i] = g.W.codes + (row < g.n ? row : g.n - 1) * ld + 16 * g4;
    }
  }
  const uint8_t* arow[TM];
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int64_t row = m0 + 16 * j + i16;
    arow[j] = TOK == TOK_NONE ? g.A.codes + (row < g.m ? row : g.m - 1) * ld + 16 * g4
                              : dyn + (row < g.m ? row : g.m - 1) * qld + 16 * g4;
  }
  const uint32_t* const ws = (const uint32_t*)g.W.scales + (n0 >> 6) * g.nb * 64 + lane;
  const uint32_t* const ws2 = (const uint32_t*)g.W2.scales + (n0 >> 6) * g.nb * 64 + lane;
  const uint32_t* const as = (const uint32_t*)g.A.scales + (m0 >> 6) * g.nb * 64 + lane;
  const int wsh = 8 * (int)((n0 >> 4) & 3), ash = 8 * (int)((m0 >> 4) & 3);

  struct Frag {
    i32x4 p[TN], q[TM];
    uint32_t sp, sq;
  };
  auto load = [&](Frag& f, int blk) {
#pragma unroll
    for (int i = 0; i < TN; ++i) f.p[i] = *(const i32x4*)(wrow[i] + blk * 64);
#pragma unroll
    for (int j = 0; j < TM; ++j) f.q[j] = *(const i32x4*)(arow[j] + blk * 64);
    f.sp = ws[blk * 64] >> wsh;
    if constexpr (EPI == EPI_SWIGLU) f.sp = (f.sp & 0xffffu) | (ws2[blk * 64] >> wsh << 16);
    if constexpr (TOK == TOK_NONE)
      f.sq = as[blk * 64] >> ash;
    else
      f.sq = qs[(i16 < g.m ? i16 : g.m - 1) * (g.nb * 4) + blk * 4 + g4];
  };
  f32x4 acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto mma = [&](const Frag& f) {
    unrolled(std::make_integer_sequence<int, TM>{}, [&](auto J) {
      constexpr int j = decltype(J)::value;
      unrolled(std::make_integer_sequence<int, TN>{}, [&](auto I) {
        constexpr int i = decltype(I)::value;
        acc[i][j] = mfma4<i, j>(f.p[i], f.q[j], acc[i][j], f.sp, f.sq);
      });
    });
  };
  const int b0 = g.nb * wid / KW, b1 = g.nb * (wid + 1) / KW;
  if (b0 < b1) {
    Frag f0, f1;
    load(f0, b0);
    for (int blk = b0; blk < b1; blk += 2) {
      if (blk + 1 < b1) load(f1, blk + 1);
      mma(f0);
      if (blk + 1 >= b1) break;
      if (blk + 2 < b1) load(f0, blk + 2);
      mma(f1);
    }
  }
  if constexpr (KW > 1) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) *(f32x4*)(red + ((wid * NT + j * TN + i) * 64 + lane) * 4) = acc[i][j];
    __syncthreads();
  }
  auto joined = [&](int t) {  // tile t = j * TN + i, summed over the waves
    f32x4 v = *(const f32x4*)(red + (t * 64 + lane) * 4);
    for (int w = 1; w < KW; ++w) v += *(const f32x4*)(red + ((w * NT + t) * 64 + lane) * 4);
    return v;
  };

  if constexpr (EPI == EPI_SWIGLU) {
    const int hnb = g.n / 128;
    for (int j = wid; j < TM; j += KW) {
      f32x4 a[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = joined(j * 4 + i);
      const f32x4 c0[2] = {a[0], a[1]}, c1[2] = {a[2], a[3]};
      uint32_t s;
      const uint32_t q = swiglu_codes(c0, c1, s);
      const int64_t row = m0 + 16 * j + i16;
      if (row < g.m) {
        uint8_t* d = (uint8_t*)g.out + row * (int64_t)(hnb * 64) + n0 / 2 + 2 * g4;
        *(uint16_t*)d = (uint16_t)q;
        *(uint16_t*)(d + 8) = (uint16_t)(q >> 16);
      }
      if (g4 == 0) g.h_scales[scale_at(row, (int)(n0 >> 5), hnb)] = row < g.m ? (uint8_t)s : 0;
    }
  } else {
    for (int t = wid; t < NT; t += KW)
      store_tile<EPI>(g, joined(t), m0 + 16 * (t / TN) + i16, n0 + 16 * (t % TN) + 4 * g4);
  }
}

template <int TN, int TM, int WN, int WM, int EPI>
hipError_t go(const Args& g, hipStream_t stream) {
  constexpr int BN = 16 * TN * WN / (EPI == EPI_SWIGLU ? 2 : 1), BM = 16 * TM * WM;
  const int64_t tiles = ((g.n + BN - 1) / BN) * ((g.m + BM - 1) / BM);
  gemm_kernel<TN, TM, WN, WM, EPI><<<dim3((unsigned)tiles), dim3(64 * WN * WM), 0, stream>>>(g);
  return hipGetLastError();
}

template <int TN, int TM, int KW, int EPI, int TOK = TOK_NONE>
hipError_t go_direct(const Args& g, hipStream_t stream) {
  constexpr int BN = EPI == EPI_SWIGLU ? 32 : 16 * TN, BM = 16 * TM;
  const int64_t tiles = ((g.n + BN - 1) / BN) * ((g.m + BM - 1) / BM);
  const size_t lds = TOK == TOK_NONE ? 0 : (size_t)g.m * (g.nb * 68 + 16);  // at most 16384 values: 9 KB
  direct_kernel<TN, TM, KW, EPI, TOK><<<dim3((unsigned)tiles), dim3(64 * KW), lds, stream>>>(g);
  return hipGetLastError();
}

template <int EPI>
hipError_t product(const Args& g, hipStream_t stream) {
  const int64_t big = ((g.n + 127) / 128) * ((g.m + 127) / 128);
  if (g.m <= 16) return go_direct<1, 1, 8, EPI>(g, stream);
  if (g.m <= 64) return go_direct<1, 4, 4, EPI>(g, stream);
  if (big < 256) return go_direct<4, 4, 4, EPI>(g, stream);
  return go<4, 4, 2, 2, EPI>(g, stream);
}

}  // namespace

bool takes_tokens(int64_t m, int k) { return m >= 1 && m <= 16 && m * padded_k(k) <= 16384; }

hipError_t launch_gemm(const Matrix& A, const Matrix& W, void* C, bool bf16, int64_t m, int n, int k,
                       hipStream_t stream) {
  if (m == 0) return hipSuccess;
  Args g{};
  g.A = A; g.W = W; g.m = m; g.n = n; g.k = k; g.nb = (int)(padded_k(k) / kPad); g.out = C;
  return bf16 ? product<EPI_BF16>(g, stream) : product<EPI_F32>(g, stream);
}

hipError_t launch_gemm_tokens(const void* A, bool a_bf16, const Matrix& W, void* C, bool bf16, int64_t m, int n, int k,
                              hipStream_t stream) {
  Args g{};
  g.tokens = A; g.W = W; g.m = m; g.n = n; g.k = k; g.nb = (int)(padded_k(k) / kPad); g.out = C;
  if (a_bf16) return bf16 ? go_direct<1, 1, 8, EPI_BF16, TOK_BF16>(g, stream) : go_direct<1, 1, 8, EPI_F32, TOK_BF16>(g, stream);
  return bf16 ? go_direct<1, 1, 8, EPI_BF16, TOK_F32>(g, stream) : go_direct<1, 1, 8, EPI_F32, TOK_F32>(g, stream);
}

hipError_t launch_gemm_swiglu(const Matrix& A, const Matrix& Wg, const Matrix& Wu, uint8_t* h_codes,
                              uint8_t* h_scales, int64_t m, int n, int k, hipStream_t stream) {
  if (m == 0) return hipSuccess;
  Args g{};
  g.A = A; g.W = Wg; g.W2 = Wu; g.m = m; g.n = n; g.k = k; g.nb = (int)(padded_k(k) / kPad);
  g.out = h_codes; g.h_scales = h_scales;
  if (m <= 16) return go_direct<4, 1, 8, EPI_SWIGLU>(g, stream);
  if (m <= 256) return go_direct<4, 4, 4, EPI_SWIGLU>(g, stream);
  return go<4, 4, 4, 2, EPI_SWIGLU>(g, stream);
}

hipError_t launch_gemm_swiglu_tokens(const void* A, const Matrix& Wg, const Matrix& Wu, uint8_t* h_codes,
                                     uint8_t* h_scales, int64_t m, int n, int k, hipStream_t stream) {
  Args g{};
  g.tokens = A; g.W = Wg; g.W2 = Wu; g.m = m; g.n = n; g.k = k; g.nb = (int)(padded_k(k) / kPad);
  g.out = h_codes; g.h_scales = h_scales;
  return go_direct<4, 1, 8, EPI_SWIGLU, TOK_BF16>(g, stream);
}

}  // namespace mx4
}  // namespace vggt3
