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
  int64_t m;
  int n, nb, splits;  // nb = kp / 128
  void* out;          // C, fp32 partials, or the codes of H
  uint8_t* h_scales;
};

enum Epi { EPI_BF16, EPI_F32, EPI_PART, EPI_SWIGLU };

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
  const int64_t tiles_m = (g.m + BM - 1) / BM;
  const int64_t b = xcd_remap(blockIdx.x, gridDim.x);
  const int slice = (int)(b / (tiles_n * tiles_m));
  const int64_t t = b % (tiles_n * tiles_m);
  const int64_t n0 = (t % tiles_n) * (EPI == EPI_SWIGLU ? BN / 2 : BN), m0 = (t / tiles_n) * BM;

  const int nst = (g.nb + 1) / 2;
  const int st0 = (int)((int64_t)nst * slice / g.splits), st1 = (int)((int64_t)nst * (slice + 1) / g.splits);
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

  if (st0 < st1) {
    issue(st0, 0);
    load_scales(sn[0], sm[0], st0);
  }
  wait_loads();
  __syncthreads();
  for (int st = st0; st < st1; st += 2) {
    if (st + 1 < st1) {
      issue(st + 1, 1);
      load_scales(sn[1], sm[1], st + 1);
    }
    compute(st, 0, sn[0], sm[0]);
    wait_loads();
    __syncthreads();
    if (st + 1 >= st1) break;
    if (st + 2 < st1) {
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
      float h[8];
      uint32_t amax = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float gg = acc[i][j][r];
          const float v = gg * sigmoid_fast(gg) * acc[i + 2][j][r];
          h[4 * i + r] = v;
          const uint32_t a = __float_as_uint(v) & 0x7fffffffu;
          amax = a > amax ? a : amax;
        }
#pragma unroll
      for (int off = 16; off <= 32; off <<= 1) {
        const uint32_t o = __shfl_xor(amax, off, 64);
        amax = o > amax ? o : amax;
      }
      const int row = (wm * TM + j) * 16 + i16;
      uint32_t s = scale_byte(amax);
      const uint32_t q = s == 255u ? 0u : encode8(h, scale_value(s));
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

  const bool quad = g.n % 4 == 0;
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int64_t row = m0 + (wm * TM + j) * 16 + i16;
    if (row >= g.m) continue;
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      const int64_t col = n0 + (wn * TN + i) * 16 + 4 * g4;
      const f32x4 v = acc[i][j];
      if (EPI == EPI_BF16) {
        uint16_t* o = (uint16_t*)g.out + row * g.n + col;
        if (quad && col < g.n) {
          st8(o, u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])});
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (col + r < g.n) o[r] = f32_to_bf16_bits(v[r]);
        }
      } else {
        float* o = (float*)g.out + (EPI == EPI_PART ? (int64_t)slice * g.m * g.n : 0) + row * g.n + col;
        if (quad && col < g.n) {
          *(f32x4*)o = v;
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (col + r < g.n) o[r] = v[r];
        }
      }
    }
  }
}

// C = the sum over the k slices, in slice order.
template <bool BF16>
__global__ __launch_bounds__(256) void sum_slices_kernel(const float* part, int splits, int64_t count, void* out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= count) return;
  float v = part[i];
  for (int s = 1; s < splits; ++s) v += part[s * count + i];
  if (BF16)
    ((uint16_t*)out)[i] = f32_to_bf16_bits(v);
  else
    ((float*)out)[i] = v;
}

template <int TN, int TM, int WN, int WM, int EPI>
hipError_t go(const Args& g, hipStream_t stream) {
  constexpr int BN = 16 * TN * WN / (EPI == EPI_SWIGLU ? 2 : 1), BM = 16 * TM * WM;
  const int64_t tiles = ((g.n + BN - 1) / BN) * ((g.m + BM - 1) / BM);
  gemm_kernel<TN, TM, WN, WM, EPI><<<dim3((unsigned)(tiles * g.splits)), dim3(64 * WN * WM), 0, stream>>>(g);
  return hipGetLastError();
}

}  // namespace

int gemm_splits(int64_t m, int n, int kp) {
  (void)m; (void)n; (void)kp;
  return 1;
}

hipError_t launch_gemm(const Matrix& A, const Matrix& W, void* C, bool bf16, int64_t m, int n, int kp, float* part,
                       hipStream_t stream) {
  if (m == 0) return hipSuccess;
  Args g{};
  g.A = A; g.W = W; g.m = m; g.n = n; g.nb = kp / kPad; g.out = C;
  g.splits = gemm_splits(m, n, kp);
  if (g.splits == 1) return bf16 ? go<4, 4, 2, 2, EPI_BF16>(g, stream) : go<4, 4, 2, 2, EPI_F32>(g, stream);
  g.out = part;
  const hipError_t e = go<4, 4, 2, 2, EPI_PART>(g, stream);
  if (e != hipSuccess) return e;
  const int64_t count = m * n;
  const dim3 grid((unsigned)((count + 255) / 256));
  if (bf16) sum_slices_kernel<true><<<grid, 256, 0, stream>>>(part, g.splits, count, C);
  else sum_slices_kernel<false><<<grid, 256, 0, stream>>>(part, g.splits, count, C);
  return hipGetLastError();
}

hipError_t launch_gemm_swiglu(const Matrix& A, const Matrix& Wg, const Matrix& Wu, uint8_t* h_codes,
                              uint8_t* h_scales, int64_t m, int n, int kp, hipStream_t stream) {
  if (m == 0) return hipSuccess;
  Args g{};
  g.A = A; g.W = Wg; g.W2 = Wu; g.m = m; g.n = n; g.nb = kp / kPad; g.splits = 1;
  g.out = h_codes; g.h_scales = h_scales;
  return go<4, 4, 4, 2, EPI_SWIGLU>(g, stream);
}

}  // namespace mx4
}  // namespace vggt3
