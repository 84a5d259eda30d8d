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
typedef __attribute__((address_space(3))) uint32_t lu32;
typedef __attribute__((address_space(3))) uint16_t lu16;
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

enum Epi { EPI_BF16, EPI_BF16_STREAM, EPI_F32, EPI_SWIGLU };
constexpr bool to_bf16(int epi) { return epi == EPI_BF16 || epi == EPI_BF16_STREAM; }

// Four neighbouring columns of one row of C.
template <int EPI>
__device__ __forceinline__ void store_tile(const Args& g, const f32x4& v, int64_t row, int64_t col) {
  if (row >= g.m) return;
  if constexpr (to_bf16(EPI)) {
    uint16_t* o = (uint16_t*)g.out + row * g.n + col;
    if (col + 4 <= g.n) {
      *(u32x2_any*)o = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (col + r < g.n) o[r] = f32_to_bf16_bits(v[r]);
    }
  } else {
    float* o = (float*)g.out + row * g.n + col;
    if (col + 4 <= g.n) {
      *(f32x4_any*)o = v;
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
// (The sigmoid goes to the gate first: gate * up may pass fp32 where silu(gate) * up
// does not, and Inf * 0 would make the block NaN.)
__device__ __forceinline__ uint32_t swiglu_codes(const f32x4 (&gate)[2], const f32x4 (&up)[2], uint32_t& s) {
  float h[8], top = 0.0f;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      h[4 * i + r] = gate[i][r] * sigmoid_fast(gate[i][r]) * up[i][r];
      top = __builtin_elementwise_maximum(top, __builtin_fabsf(h[4 * i + r]));  // a NaN stays
    }
#pragma unroll
  for (int off = 16; off <= 32; off <<= 1) top = __builtin_elementwise_maximum(top, __shfl_xor(top, off, 64));
  const uint32_t amax = __float_as_uint(top);
  s = scale_byte(amax);
  return s == 255u ? 0u : encode8(h, scale_value(s));
}

// ------------------------------------------------------------ tiled products
// A workgroup of WN x WM waves works through BN x BM tiles of C^T, TN x TM tiles of
// 16x16 a wave, in steps of 128 columns (one MFMA deep). LDS holds a ring of RING
// steps, each [BN + BM rows][64 bytes] of codes and the scale tiles of those rows,
// filled by direct global-to-LDS loads RING steps ahead. The steps of all the
// workgroup's tiles are one stream: while a tile's last steps are worked on and its
// results stored, the next tile's first steps are under way. (At k = 1024 a tile
// has 8 steps, 3.6 us of MFMAs; as a workgroup of its own it would spend more than
// that on its first loads and its stores.)
//
// A 16-byte piece c of row r is kept at position c ^ ((r / 4) % 4): the 16 lanes
// of an operand read (16 rows, one piece) then touch every bank once.
constexpr int STEP = 64;  // bytes of a row and step
__device__ __forceinline__ int swz(int row) { return (row >> 2) & 3; }

// Wait until at most N of this wave's global loads, or none of its LDS reads, are
// under way. (Builtins: the compiler then knows, and adds no waits of its own.)
template <int N>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4 << 14) | 0x0f70);
}
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xc07f); }

// A choice between values (of variables, ?: would choose between their places, and
// so keep them in memory).
template <class T>
__device__ __forceinline__ T pick(bool c, T a, T b) {
  return c ? a : b;
}
// Lambdas that stay calls would keep what they refer to in memory.
#define INLINE __attribute__((always_inline))

// 16 or 4 bytes a lane from memory to LDS, the lanes of a wave side by side from dst
// on. (As buffer loads: a scalar base and offset, a 32-bit lane offset. Their
// global_load form also counts as a possible LDS access of the wave's own, which
// makes the compiler wait for every LDS read in front of each use of one.)
__device__ __forceinline__ void to_lds16(const uint8_t* p, uint32_t lane_off, uint32_t off, lu8* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(__builtin_amdgcn_make_buffer_rsrc((void*)p, 0, 0x7fffffff, 0x00027000),
                                           (lvoid*)dst, 16, lane_off, off, 0, 0);
}
__device__ __forceinline__ void to_lds4(const uint8_t* p, uint32_t lane_off, uint32_t off, lu8* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(__builtin_amdgcn_make_buffer_rsrc((void*)p, 0, 0x7fffffff, 0x00027000),
                                           (lvoid*)dst, 4, lane_off, off, 0, 0);
}
__device__ __forceinline__ void swap_rows(uint32_t& a, uint32_t& b) {
  // odd 16-lane rows of a <-> even rows of b
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
  // upper 32 lanes of a <-> lower 32 lanes of b
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

template <int TN, int TM, int WN, int WM, int RING, int EPI>
__global__ __launch_bounds__(64 * WN * WM) __attribute__((amdgpu_waves_per_eu(2))) void gemm_kernel(Args g) {
  constexpr int NW = WN * WM;
  constexpr int BN = 16 * TN * WN, BM = 16 * TM * WM;
  static_assert(TN % 4 == 0 && TM % 4 == 0, "a wave's rows are whole scale tiles");
  constexpr int SN = TN / 4, SM = TM / 4;
  constexpr int CODES = (BN + BM) * STEP, STAGE = CODES + (BN + BM) * 4;
  constexpr int DN = BN / 16 / NW, DM = BM / 16 / NW, DS = ((BN + BM) / 64 + NW - 1) / NW;  // loads a wave and step
  static_assert(DN * NW * 16 == BN && DM * NW * 16 == BM, "whole loads");
  constexpr int LOADS = DN + DM + DS;
  // Stores (at least) a wave makes of a tile that lies inside C.
  constexpr int STORES = EPI == EPI_SWIGLU ? 2 * SN : to_bf16(EPI) ? TN * TM / 2 : TN * TM;
  static_assert(RING >= 2 && (RING - 2) * LOADS + STORES < 64, "vmcnt");
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  lu8* const lds = (lu8*)smem;

  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wid % WN, wm = wid / WN;
  constexpr int CN = EPI == EPI_SWIGLU ? BN / 2 : BN;  // columns (hidden units) a tile
  const uint32_t tiles_n = (g.n + CN - 1) / CN, tiles_m = (uint32_t)((g.m + BM - 1) / BM);
  const int steps = g.nb;
  const int64_t ld = (int64_t)g.nb * 64;

  // This workgroup's tiles: the XCD it runs on (number % 8) has a contiguous range,
  // which its workgroups go through side by side.
  uint32_t tile, tile_end, stride;
  {
    const uint32_t x = blockIdx.x % kNumXcd, q = gridDim.x / kNumXcd, r = gridDim.x % kNumXcd;
    const uint32_t before = x * q + (x < r ? x : r);
    const uint64_t tiles = (uint64_t)tiles_n * tiles_m;
    stride = q + (x < r ? 1 : 0);
    tile = __builtin_amdgcn_readfirstlane((uint32_t)(tiles * before / gridDim.x) + blockIdx.x / kNumXcd);
    tile_end = __builtin_amdgcn_readfirstlane((uint32_t)(tiles * (before + stride) / gridDim.x));
  }
  if (tile >= tile_end) return;
  // Tiles in groups of GM row tiles x all column tiles, row-fastest, so that those
  // side by side share rows of both operands.
  auto place = [&](uint32_t t, int64_t& n0, int64_t& m0) INLINE {
    constexpr uint32_t GM = 4;
    const uint32_t first = t / (GM * tiles_n) * GM, in = t % (GM * tiles_n);
    const uint32_t rows = tiles_m - first < GM ? tiles_m - first : GM;
    // (the divisions go through vector registers)
    m0 = (int64_t)__builtin_amdgcn_readfirstlane(first + in % rows) * BM;
    n0 = (int64_t)__builtin_amdgcn_readfirstlane(in / rows) * CN;
  };

  // The stream of loads: the tile and step it has come to, where that tile's rows
  // are, and this lane's places in them. Rows and scale tiles past the end read the
  // last ones: they give values of C that are not stored.
  const uint8_t *wp, *up, *ap, *wsp, *usp, *asp;
  int wtiles, atiles;
  uint32_t off_n[DN], off_m[DM];
  const uint32_t tile_bytes = (uint32_t)g.nb * 256;
  auto aim = [&](uint32_t t) INLINE {
    int64_t n0, m0;
    place(t, n0, m0);
    wp = g.W.codes + n0 * ld;
    up = EPI == EPI_SWIGLU ? g.W2.codes + n0 * ld : wp;
    ap = g.A.codes + m0 * ld;
    wsp = g.W.scales + (n0 >> 6) * tile_bytes;
    usp = EPI == EPI_SWIGLU ? g.W2.scales + (n0 >> 6) * tile_bytes : wsp;
    asp = g.A.scales + (m0 >> 6) * tile_bytes;
    const int64_t wt = row_tiles(g.n) - (n0 >> 6), at = row_tiles(g.m) - (m0 >> 6);
    wtiles = wt < 64 ? (int)wt : 64;
    atiles = at < 64 ? (int)at : 64;
    const int nmost = (int)(g.n - n0 < BN ? g.n - n0 : BN) - 1, mmost = (int)(g.m - m0 < BM ? g.m - m0 : BM) - 1;
    const int row = lane >> 2;
    const uint32_t piece = 16 * ((lane & 3) ^ swz(row));
#pragma unroll
    for (int i = 0; i < DN; ++i) {
      const int r = (NW * i + wid) * 16 + row;
      // SwiGLU: rows are [32 gate units | the same 32 up units] in turn
      const int from = EPI == EPI_SWIGLU ? (r >> 6) * 32 + (r & 31) : r < nmost ? r : nmost;
      off_n[i] = (uint32_t)from * (uint32_t)ld + piece;
    }
#pragma unroll
    for (int i = 0; i < DM; ++i) {
      const int r = (NW * i + wid) * 16 + row;
      off_m[i] = (uint32_t)(r < mmost ? r : mmost) * (uint32_t)ld + piece;
    }
  };
  auto issue = [&](int step, lu8* stage) INLINE {
#pragma unroll
    for (int i = 0; i < DN; ++i) {
      // a load covers 16 rows, so it lies in one of gate and up
      to_lds16(EPI == EPI_SWIGLU ? pick((NW * i + wid) & 2, up, wp) : +wp, off_n[i], step * STEP, stage + (NW * i + wid) * 1024);
    }
#pragma unroll
    for (int i = 0; i < DM; ++i) to_lds16(ap, off_m[i], step * STEP, stage + BN * STEP + (NW * i + wid) * 1024);
#pragma unroll
    for (int i = 0; i < DS; ++i) {
      // the scale tiles of W (of gate, then of up), then of A; where there are fewer
      // than loads, several waves load the last one
      const int want = NW * i + wid, slot = want < (BN + BM) / 64 ? want : (BN + BM) / 64 - 1;
      const bool of_a = slot >= BN / 64, of_up = EPI == EPI_SWIGLU && slot >= BN / 128;
      const int t = of_a ? slot - BN / 64 : of_up ? slot - BN / 128 : slot;
      const int most = pick(of_a, atiles, wtiles) - 1;
      const uint8_t* p = pick(of_a, asp, pick(of_up, usp, wsp));
      to_lds4(p, lane * 4, (uint32_t)(t < most ? t : most) * tile_bytes + step * 256, stage + CODES + slot * 256);
    }
  };
  // The step after the one just issued. Behind the last one it stays where it is:
  // the loads beyond the end are copies that nothing uses, so that every round is
  // the same.
  uint32_t at = tile;
  int at_step = 0;
  auto load_on = [&]() INLINE {
    if (at_step + 1 < steps) {
      ++at_step;
    } else if (stride < tile_end - at) {
      at_step = 0;
      at += stride;
      aim(at);
    }
  };

  const int i16 = lane & 15, g4 = lane >> 4;
  const int foff = i16 * STEP + 16 * (g4 ^ swz(i16));
  struct Cols {               // one step's token rows, and all scales
    i32x4 q[TM];
    uint32_t sp[SN], sq[SM];
    uint32_t su[EPI == EPI_SWIGLU ? SN : 1];  // (sp: gate's scales, su: up's)
  };
  auto fetch_row = [&](int i, const lu8* stage) INLINE {
    return *(const li32x4*)(stage + (wn * TN + i) * 16 * STEP + foff);
  };
  auto fetch_cols = [&](Cols& f, const lu8* stage) INLINE {
    const lu8* const Q = stage + BN * STEP + wm * TM * 16 * STEP + foff;
    const lu8* const S = stage + CODES + lane * 4;
#pragma unroll
    for (int i = 0; i < SN; ++i) {
      if (EPI == EPI_SWIGLU) {
        const int t = (wn * SN + i) >> 1;
        f.sp[i] = *(const lu32*)(S + t * 256);
        f.su[i] = *(const lu32*)(S + (BN / 128 + t) * 256);
      } else {
        f.sp[i] = *(const lu32*)(S + (wn * SN + i) * 256);
      }
    }
#pragma unroll
    for (int j = 0; j < SM; ++j) f.sq[j] = *(const lu32*)(S + (BN / 64 + wm * SM + j) * 256);
#pragma unroll
    for (int j = 0; j < TM; ++j) f.q[j] = *(const li32x4*)(Q + j * 16 * STEP);
  };
  f32x4 acc[TN][TM];
  auto clear = [&]() INLINE {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  };
  // The MFMAs of weight row tile i (p) with all token rows.
  auto mma = [&](auto I, const i32x4& p, const Cols& c) INLINE {
    constexpr int i = decltype(I)::value;
    // SwiGLU: the wave's 32 of a tile's 64 gate units, and the same up units
    const int sh = 16 * ((wn * SN + i / 4) & 1);
    const uint32_t sp =
        EPI == EPI_SWIGLU ? (c.sp[i / 4] >> sh & 0xffffu) | (c.su[EPI == EPI_SWIGLU ? i / 4 : 0] >> sh << 16) : c.sp[i / 4];
    unrolled(std::make_integer_sequence<int, TM>{}, [&](auto J) INLINE {
      constexpr int j = decltype(J)::value;
      acc[i][j] = mfma4<i & 3, j & 3>(p, c.q[j], acc[i][j], sp, c.sq[j >> 2]);
    });
  };

  aim(tile);
  issue(0, lds);
  for (int i = 1; i < RING; ++i) {
    load_on();
    issue(at_step, lds + i * STAGE);
  }
  wait_loads<0>();
  __builtin_amdgcn_s_barrier();
  i32x4 rows[TN];
  Cols cols, next;
  fetch_cols(cols, lds);
#pragma unroll
  for (int i = 0; i < TN; ++i) rows[i] = fetch_row(i, lds);
  clear();
  int ring = 0;  // place of the present step
  for (;; tile += stride) {
    // Work on the present step, in registers, and read the next one, each part as
    // the registers of its predecessor fall free. The next step's loads are waited
    // for; those of RING - 2 later steps may be under way and, in the first RING - 1
    // rounds, whose loads were issued ahead of them (or are done), the stores of the
    // tile before. The reads of this step are waited for too, so behind the barrier
    // every wave has them and their place takes the step RING ahead (68,700 rows
    // through a frozen read: 531 us; 543 with the reads' wait behind the barrier and
    // the loads one step less ahead). The scheduling fences keep the reads ahead of the
    // MFMAs that hide them. The questions come first: between the reads and the MFMAs
    // on one side and the end of the round on the other there is no branch for them to
    // cross.
    for (int s = 0; s < steps; ++s) {
      load_on();
      if (s < RING - 1)
        wait_loads<(RING - 2) * LOADS + STORES>();
      else
        wait_loads<(RING - 2) * LOADS>();
      // (The compiler takes the loads to LDS for LDS accesses of this wave's and would
      // wait for all reads at the first use of one; with this wait there is none.)
      wait_lds();
      __builtin_amdgcn_s_barrier();
      issue(at_step, lds + ring * STAGE);
      ring = ring + 1 == RING ? 0 : ring + 1;
      const lu8* const stage = lds + ring * STAGE;
      fetch_cols(next, stage);
      __builtin_amdgcn_sched_barrier(0);
      unrolled(std::make_integer_sequence<int, TN>{}, [&](auto I) INLINE {
        constexpr int i = decltype(I)::value;
        mma(I, rows[i], cols);
        __builtin_amdgcn_sched_barrier(0);
        rows[i] = fetch_row(i, stage);
        __builtin_amdgcn_sched_barrier(0);
      });
      cols = next;
    }

    int64_t n0, m0;
    place(tile, n0, m0);
    const bool inside = m0 + BM <= g.m && n0 + CN <= g.n;
    if constexpr (EPI == EPI_SWIGLU) {
      // Each wave holds gate (tiles 0, 1 of four) and up (tiles 2, 3) of the same 32
      // units: one block of H per row, whose 16 bytes of codes lie in 4 lanes, 4 each.
      // A transposition over 4 row tiles and the 4 16-lane rows brings a block
      // together: lane 16 j + r gets that of row 16 j + r, to store in one piece.
      static_assert(EPI != EPI_SWIGLU || (TM == 4 && BN == 256), "64 rows a wave, 128 units a tile");
      const int hnb = g.n / 128;  // scale tiles across H
      const int64_t row0 = m0 + wm * 64;
#pragma unroll
      for (int q = 0; q < SN; ++q) {
        const int blk = wn * SN + q;  // of the tile's four
        uint32_t d[4], word = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4 gate[2] = {acc[4 * q][j], acc[4 * q + 1][j]}, upv[2] = {acc[4 * q + 2][j], acc[4 * q + 3][j]};
          uint32_t sc;
          d[j] = swiglu_codes(gate, upv, sc);
          if (row0 + 16 * j + i16 < g.m) word |= sc << (8 * j);
        }
        swap_halves(d[0], d[2]);
        swap_halves(d[1], d[3]);
        swap_rows(d[0], d[1]);
        swap_rows(d[2], d[3]);
        const u32x4 codes = {(d[0] & 0xffffu) | d[1] << 16, (d[2] & 0xffffu) | d[3] << 16,
                             d[0] >> 16 | (d[1] & 0xffff0000u), d[2] >> 16 | (d[3] & 0xffff0000u)};
        const int64_t row = row0 + lane;
        if (row < g.m) st16((uint8_t*)g.out + row * (int64_t)(hnb * 64) + n0 / 2 + 16 * blk, codes);
        if (g4 == 0 && row0 < g.m)
          ((uint32_t*)g.h_scales)[((row0 >> 6) * hnb + n0 / 128) * 64 + 16 * blk + i16] = word;
      }
    } else {
      const int64_t row0 = m0 + wm * TM * 16 + i16, col0 = n0 + wn * TN * 16;
      if (!inside) {
#pragma unroll
        for (int j = 0; j < TM; ++j)
#pragma unroll
          for (int i = 0; i < TN; ++i) store_tile<EPI>(g, acc[i][j], row0 + 16 * j, col0 + 16 * i + 4 * g4);
      } else if constexpr (to_bf16(EPI)) {
        // Lanes of odd 16-lane rows trade one column tile for its neighbour's, so
        // that each lane has 8 neighbouring columns: 16-byte stores, 64 bytes a row,
        // streamed when C is large (68,700 x 1024 x 4096: 222 us, 232 with ordinary
        // stores; in fp32, whose stores are 64 bytes a row too, 388 against 342).
        uint16_t* const o = (uint16_t*)g.out + row0 * g.n + col0 + 16 * (g4 & 1) + 4 * (g4 & 2);
#pragma unroll
        for (int j = 0; j < TM; ++j)
#pragma unroll
          for (int i = 0; i < TN; i += 2) {
            const f32x4 a = acc[i][j], b = acc[i + 1][j];
            uint32_t a0 = pack_bf16x2(a[0], a[1]), a1 = pack_bf16x2(a[2], a[3]);
            uint32_t b0 = pack_bf16x2(b[0], b[1]), b1 = pack_bf16x2(b[2], b[3]);
            swap_rows(a0, b0);
            swap_rows(a1, b1);
            uint16_t* const at = o + (int64_t)(16 * j) * g.n + 16 * i;
            if constexpr (EPI == EPI_BF16_STREAM)
              st16<true>(at, u32x4{a0, a1, b0, b1});
            else
              st16_any(at, u32x4{a0, a1, b0, b1});
          }
      } else {
        float* const o = (float*)g.out + row0 * g.n + col0 + 4 * g4;
#pragma unroll
        for (int j = 0; j < TM; ++j)
#pragma unroll
          for (int i = 0; i < TN; ++i) *(f32x4_any*)(o + (int64_t)(16 * j) * g.n + 16 * i) = acc[i][j];
      }
    }
    if (stride >= tile_end - tile) break;
    clear();
    // A tile over the edge makes fewer stores than the waits above allow for.
    if (!inside) wait_loads<0>();
  }
  wait_loads<0>();  // the copies beyond the end still go to this workgroup's LDS
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
    const int kb = g.nb * 4, pieces = g.nb * 16;  // blocks and pieces of 8 a row
    for (int i = threadIdx.x; i < (int)g.m * pieces; i += 64 * KW) {
      const int row = i / pieces, piece = i % pieces;
      float v[8];
      if (g.k % (TOK == TOK_BF16 ? 8 : 4) == 0)
        load8<TOK == TOK_BF16, true>(g.tokens, row, piece * 8, g.k, v);
      else
        load8<TOK == TOK_BF16, false>(g.tokens, row, piece * 8, g.k, v);
      uint32_t s;
      *(uint32_t*)(dyn + row * qld + piece * 4) = quantize8(v, s);
      if ((piece & 3) == 0) qs[row * kb + piece / 4] = (uint8_t)s;
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

template <int TN, int TM, int WN, int WM, int RING, int EPI>
hipError_t go(const Args& g, hipStream_t stream) {
  constexpr int BN = 16 * TN * WN, BM = 16 * TM * WM, CN = EPI == EPI_SWIGLU ? BN / 2 : BN;
  constexpr size_t lds = (size_t)RING * (BN + BM) * (STEP + 4);
  static_assert(lds <= 160 * 1024, "LDS of one workgroup");
  // as many workgroups as 256 compute units hold at once
  const int64_t most = 256 * (160 * 1024 / lds < 8 / (WN * WM) ? 160 * 1024 / lds : 8 / (WN * WM));
  const int64_t tiles = ((g.n + CN - 1) / CN) * ((g.m + BM - 1) / BM);
  gemm_kernel<TN, TM, WN, WM, RING, EPI>
      <<<dim3((unsigned)(tiles < most ? tiles : most)), dim3(64 * WN * WM), lds, stream>>>(g);
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

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Which kernel (measured at n x k = 4096 x 1024 and 1024 x 4096, us):
//  up to 16 rows    16 x 16 tiles, 8 waves splitting k;
//  up to 64 rows    16 columns x 64 rows (64 rows: 3.8, 6.8; 64 x 64 tiles: 5.7, 10.7);
//  64 x 64 tiles    while the 256 compute units hold them all (200 rows: 6.0, 10.8;
//                   128 x 128: 6.5, 14.0; at 300 rows, 4096 columns: 10.3 and 6.6);
//  128 x 128, 2 workgroups a unit, or 256 x 256, one: by the rounds that either
//                   needs. A round of 256 x 256 takes as long as two at k = 1024 (the
//                   stores' time; it hides them from the third round on) and one and
//                   a half at 4096 (1374 rows: 10.4, 14.5 and 13.6, 28.5; 2748: 13.8
//                   and 15.7; 10,992: 45.1, 38.9 and 45.4, 35.4; 68,700: 259, 202 and
//                   219, 170).
template <int EPI>
hipError_t product(const Args& g, hipStream_t stream) {
  if (g.m <= 16) return go_direct<1, 1, 8, EPI>(g, stream);
  if (g.m <= 64) return go_direct<1, 4, 4, EPI>(g, stream);
  auto tiles = [&](int edge) { return ceil_div(g.n, edge) * ceil_div(g.m, edge); };
  if (tiles(64) <= 256) return go_direct<4, 4, 4, EPI>(g, stream);
  const int64_t small = ceil_div(tiles(128), 512), large = ceil_div(tiles(256), 256);
  const bool use_large = g.nb >= 16 ? 3 * large <= 2 * small : large >= 3 && 2 * large <= small;
  if (!use_large) return go<4, 4, 2, 2, 4, EPI>(g, stream);
  if (EPI == EPI_BF16 && g.n % 8 == 0 && streams(g.m * g.n * 2)) return go<8, 4, 2, 4, 4, EPI_BF16_STREAM>(g, stream);
  return go<8, 4, 2, 4, 4, EPI>(g, stream);
}

}  // namespace

// Up to 16,384 values: every workgroup quantises them all (m x n x k of 1 x 4096 x 1024
// in fp32: 3.0 us, 4.7 in two launches; 4 x 1024 x 4096: 5.0 and 6.0; 16 x 4096 x 1024:
// 4.5 and 5.1; 8 x 1024 x 4096, twice as many values: 6.8 and 6.4).
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
  // as above (8192 x 1024: 256 rows 11.4 us in 64 x 64 tiles, 12.3 in 256 x 256; 300 rows
  // 15.7 and 13.3)
  if (m <= 16) return go_direct<4, 1, 8, EPI_SWIGLU>(g, stream);
  if (ceil_div(2 * (int64_t)n, 64) * ceil_div(m, 64) <= 512) return go_direct<4, 4, 4, EPI_SWIGLU>(g, stream);
  return go<8, 4, 2, 4, 4, EPI_SWIGLU>(g, stream);
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
