// Block join: the tail of one block and the head of the next in one pass.
//
//   h = post(f),  r = x + s * g * h  (stored),  y = pre(r)
//
// with post and pre each an RMS norm, a layer norm or nothing, s a residual
// scale per channel and g a gate per token (or group of tokens) and channel.
// y is the norm of the stored (rounded) r: the stream that later blocks and the
// gradient see.
//
// A row belongs to one unit of T threads (a wave up to 1024 channels, a
// workgroup beyond) and stays in its registers, E values a thread, so each
// tensor is read and written once; means and variances are two-pass, in fp32.
// A unit takes a contiguous range of rows, asks for its next row before it works
// on the present one, and keeps a gate row that several tokens share in
// registers. The channel parameters lie in LDS (they would take 80 registers a
// thread, and with them half of the waves that hide the loads).
#include "bf16_ops.hpp"
#include "join.hpp"
#include "mx4_ops.hpp"

#include <type_traits>

namespace vggt3 {
namespace join {
namespace {

// A workgroup is one unit, but for units of at most a wave, which never wait for
// each other.
constexpr int block_threads(int T) { return T <= 64 ? 256 : T; }

// How a unit's T threads share a row: 16-byte pieces in turn where the channel
// count is a multiple of a piece, single values otherwise. FULL: the pieces fill
// the unit (512, 1024, 2048, ... channels), so no load or store asks whether its
// column exists (the questions took a third of the instructions).
// (Pieces of odd rows, loaded at the alignment of their elements, are slower than
// single values: 65,952 x 999 bf16 took 223 us instead of 150.)
enum Mode { SCALAR, PIECES, FULL };

template <bool BF16, Mode MODE, int T, int E>
struct Row {
  static constexpr bool VEC = MODE != SCALAR;
  static constexpr int VL = VEC ? (BF16 ? 8 : 4) : 1;
  static constexpr int NC = E / VL;
  static constexpr uint32_t SZ = BF16 ? 2 : 4;
  static constexpr int U = block_threads(T) / T;  // units per workgroup
  static_assert(E % VL == 0, "whole pieces");

  __device__ static __forceinline__ int col(int c, int tid) { return (c * T + tid) * VL; }
  __device__ static __forceinline__ bool inside(int k, int C) { return MODE == FULL || k < C; }

  // A row as loaded, and as values (0 past C).
  struct Raw {
    std::conditional_t<VEC, u32x4, uint32_t> q[NC];
  };
  __device__ static __forceinline__ void load(const void* base, int64_t row, int C, int tid, Raw& raw) {
    const char* p = (const char*)base + row * C * SZ;  // the same in a whole wave: a scalar base
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const uint32_t k = col(c, tid);
      if constexpr (VEC) {
        raw.q[c] = inside(k, C) ? ld16(p + k * SZ) : u32x4{0u, 0u, 0u, 0u};
      } else {
        raw.q[c] = (int)k >= C ? 0u : BF16 ? *(const uint16_t*)(p + k * SZ) : *(const uint32_t*)(p + k * SZ);
      }
    }
  }
  __device__ static __forceinline__ void values(const Raw& raw, float (&v)[E]) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if constexpr (VEC) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (BF16) {
            v[c * VL + 2 * j] = bf16_lo(raw.q[c][j]);
            v[c * VL + 2 * j + 1] = bf16_hi(raw.q[c][j]);
          } else {
            v[c * VL + j] = __uint_as_float(raw.q[c][j]);
          }
        }
      } else {
        v[c] = BF16 ? bf16_bits_to_f32(raw.q[c]) : __uint_as_float(raw.q[c]);
      }
    }
  }

  __device__ static __forceinline__ void store(void* base, int64_t row, int C, int tid, const float (&v)[E]) {
    char* p = (char*)base + row * C * SZ;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const uint32_t k = col(c, tid);
      if (!inside(k, C)) continue;
      if constexpr (VEC) {
        u32x4 q;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (BF16)
            q[j] = pack_bf16x2(v[c * VL + 2 * j], v[c * VL + 2 * j + 1]);
          else
            q[j] = __float_as_uint(v[c * VL + j]);
        }
        st16(p + k * SZ, q);
      } else if constexpr (BF16) {
        *(uint16_t*)(p + k * SZ) = f32_to_bf16_bits(v[c]);
      } else {
        *(float*)(p + k * SZ) = v[c];
      }
    }
  }

  // fp32 channel parameters in LDS: element 4 i + j of thread tid's values at
  // [i][tid][j], so that a wave reads 16 bytes a lane in sequence. Each thread
  // takes its own columns, the units of a workgroup in turn.
  struct Quads {
    f32x4 v[(E / 4 + U - 1) / U];
  };
  // `absent` where there is no vector, 0 past C.
  __device__ static __forceinline__ void fetch_param(Quads& q, const float* p, float absent, int C, int tid, int uid) {
#pragma unroll
    for (int n = 0; n < (E / 4 + U - 1) / U; ++n) {
      const int i = uid + n * U;
#pragma unroll
      for (int j = 0; j < 4; ++j) q.v[n][j] = 0.0f;
      if (i >= E / 4) continue;
      if constexpr (VEC) {
        const int k = col(4 * i / VL, tid) + 4 * i % VL;
        if (inside(k, C)) q.v[n] = p ? *(const f32x4*)(p + k) : f32x4{absent, absent, absent, absent};
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = col(4 * i + j, tid);
          if (k < C) q.v[n][j] = p ? p[k] : absent;
        }
      }
    }
  }
  __device__ static __forceinline__ void stage_param(float* lds, const Quads& q, int tid, int uid) {
#pragma unroll
    for (int n = 0; n < (E / 4 + U - 1) / U; ++n)
      if (uid + n * U < E / 4) *(f32x4*)(lds + ((uid + n * U) * T + tid) * 4) = q.v[n];
  }
  __device__ static __forceinline__ f32x4 param(const float* lds, int i, int tid) {
    return *(const f32x4*)(lds + (i * T + tid) * 4);
  }

  __device__ static __forceinline__ void store_f32(float* p, int C, int tid, const float (&v)[E]) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      if constexpr (VEC) {
        const int k = col(4 * i / VL, tid) + 4 * i % VL;
        if (inside(k, C)) *(f32x4*)(p + k) = f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = col(4 * i + j, tid);
          if (k < C) p[k] = v[4 * i + j];
        }
      }
    }
  }
};

// Round to the token type and back.
template <bool BF16>
__device__ __forceinline__ float rounded(float v) {
  return BF16 ? bf16_bits_to_f32(f32_to_bf16_bits(v)) : v;
}

// Largest of N = 4, 8, 16 or 32 neighbouring lanes, the same in each.
template <int N>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  static_assert(N == 4 || N == 8 || N == 16 || N == 32, "parts of a DPP row, one, or two");
#define VGGT3_DPP(ctrl)                                                                      \
  {                                                                                          \
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xf, 0xf, false); \
    v = o > v ? o : v;                                                                       \
  }
  VGGT3_DPP(0xb1)                         // quad_perm 1,0,3,2
  VGGT3_DPP(0x4e)                         // quad_perm 2,3,0,1
  if constexpr (N >= 8) VGGT3_DPP(0x141)  // row_half_mirror
  if constexpr (N >= 16) VGGT3_DPP(0x140)  // row_mirror
  if constexpr (N == 32) {
    const uint32_t o = __shfl_xor(v, 16, 64);
    v = o > v ? o : v;
  }
#undef VGGT3_DPP
  return v;
}

#define VGGT3_DPP(v, ctrl, rows) \
  __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, rows, 0xf, false))
// Sum over T = 16, 32 or 64 neighbouring lanes, the same in each, by DPP (no LDS
// round trips, but for one with 32).
template <int T>
__device__ __forceinline__ float lanes_total(float v) {
  static_assert(T == 16 || T == 32 || T == 64, "a DPP row, two, or a wave");
  if constexpr (T <= 32) {
    v += VGGT3_DPP(v, 0xb1, 0xf);   // quad_perm 1,0,3,2
    v += VGGT3_DPP(v, 0x4e, 0xf);   // quad_perm 2,3,0,1
    v += VGGT3_DPP(v, 0x141, 0xf);  // row_half_mirror
    v += VGGT3_DPP(v, 0x140, 0xf);  // row_mirror
    if constexpr (T == 32) v += __shfl_xor(v, 16, 64);
    return v;
  } else {
    v += VGGT3_DPP(v, 0x111, 0xf);  // row_shr 1, 2, 4, 8: lane 15 of a row has its sum
    v += VGGT3_DPP(v, 0x112, 0xf);
    v += VGGT3_DPP(v, 0x114, 0xf);
    v += VGGT3_DPP(v, 0x118, 0xf);
    v += VGGT3_DPP(v, 0x142, 0xa);  // row_bcast:15 into rows 1, 3
    v += VGGT3_DPP(v, 0x143, 0xc);  // row_bcast:31 into rows 2, 3
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
  }
}
#undef VGGT3_DPP

// A workgroup barrier for LDS only. (__syncthreads also waits for the rows asked
// for and the stores under way, which is what asking ahead is to avoid.)
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Sums of N values over a unit, given to every thread of it. Across waves
// through LDS, in wave order.
template <int T, int N>
__device__ __forceinline__ void unit_sum(float (&v)[N], float* red, int tid) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lanes_total<(T < 64 ? T : 64)>(v[i]);
  if constexpr (T > 64) {
    constexpr int W = T / 64;
    lds_barrier();
    if ((tid & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[i * W + (tid >> 6)] = v[i];
    lds_barrier();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = red[i * W];
#pragma unroll
      for (int w = 1; w < W; ++w) s += red[i * W + w];
      v[i] = s;
    }
  }
}

// A unit's number within its workgroup, in a scalar register where a wave has one unit.
template <int T>
__device__ __forceinline__ int unit_of_thread() {
  const int u = threadIdx.x / T;
  return T >= 64 ? __builtin_amdgcn_readfirstlane(u) : u;
}

// Centre v for a layer norm and return 1/sqrt(mean square + eps); past C, v stays 0.
template <class R, int T, int E>
__device__ __forceinline__ float center(float (&v)[E], int kind, int C, float inv_c, float eps, float* red, int tid) {
  if (kind == kLayer) {
    float m[1] = {0.0f};
#pragma unroll
    for (int e = 0; e < E; ++e) m[0] += v[e];
    unit_sum<T>(m, red, tid);
    const float mean = m[0] * inv_c;
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = R::inside(R::col(e / R::VL, tid) + e % R::VL, C) ? v[e] - mean : 0.0f;
  }
  float q[1] = {0.0f};
#pragma unroll
  for (int e = 0; e < E; ++e) q[0] += v[e] * v[e];
  unit_sum<T>(q, red, tid);
  return rsqrtf(q[0] * inv_c + eps);
}

// One row of y in 4 bits (values already rounded to the token type): a block of 32
// columns lies in 32 / VL neighbouring threads, or in G column chunks of a unit of
// 16 threads with single values.
template <class R, int T, int E>
__device__ __forceinline__ void store_mx4(const float (&y)[E], int64_t row, int C, uint8_t* codes, uint8_t* scales,
                                          int tid) {
  constexpr int G = 32 / R::VL > T ? 32 / R::VL / T : 1;
  const int nb = (C + 127) / 128;
  // past C the value is 0 whatever the row holds (a NaN row has NaN there too)
  auto value = [&](int c, int j) { return R::inside(R::col(c, tid) + j, C) ? y[c * R::VL + j] : 0.0f; };
#pragma unroll
  for (int c0 = 0; c0 < R::NC; c0 += G) {
    if (R::VL == 1 && R::col(c0, 0) >= nb * 128) continue;
    uint32_t amax = 0;
#pragma unroll
    for (int c = c0; c < c0 + G; ++c)
#pragma unroll
      for (int j = 0; j < R::VL; ++j) {
        const uint32_t a = __float_as_uint(value(c, j)) & 0x7fffffffu;
        amax = a > amax ? a : amax;
      }
    const uint32_t s = mx4::scale_byte(lanes_max<32 / R::VL / G>(amax));
#pragma unroll
    for (int c = c0; c < c0 + G; ++c) {
      const int k = R::col(c, tid);
      uint32_t q = 0;
      if constexpr (R::VL == 1) {  // two lanes' values a byte
        const float v = value(c, 0);
        const float o = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xb1, 0xf, 0xf, false));
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v, o, mx4::scale_value(s), 0);
        if (s == 255u) q = 0;
      } else {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < R::VL ? value(c, j < R::VL ? j : 0) : 0.0f;
        q = s == 255u ? 0u : mx4::encode8(v, mx4::scale_value(s));
      }
      if (k >= nb * 128) continue;
      uint8_t* p = codes + row * (int64_t)(nb * 64) + k / 2;
      if constexpr (R::VL == 8)
        *(uint32_t*)p = q;
      else if constexpr (R::VL == 4)
        *(uint16_t*)p = (uint16_t)q;
      else if ((tid & 1) == 0)
        *p = (uint8_t)q;
      if ((k & 31) == 0) scales[mx4::scale_at(row, k >> 5, nb)] = (uint8_t)s;
    }
  }
}

// The rows of a gate along a unit's range: which group a row is in, counted
// along rather than divided, and the next group's row asked for ahead.
template <class R>
struct GateRows {
  int64_t group;
  int64_t left;  // rows of the group from here on
  typename R::Raw next;

  __device__ __forceinline__ void start(const Args& a, int64_t t0, int tid) {
    group = (uint32_t)t0 / (uint32_t)a.per;
    left = (group + 1) * a.per - t0;
    R::load(a.gate, group, a.C, tid, next);
  }
};

template <bool BF16, Mode MODE, int T, int E>
__global__ __launch_bounds__(block_threads(T)) void join_kernel(Args a) {
  typedef Row<BF16, MODE, T, E> R;
  constexpr int U = R::U;
  enum { PW, PB, W, B };  // post_w and post_b come with the residual scale multiplied in
  __shared__ float red[T > 64 ? T / 64 : 1];
  extern __shared__ __attribute__((aligned(16))) float params[];  // [NP][T * E]
  int tid = threadIdx.x % T;
  const int64_t unit = (int64_t)blockIdx.x * U + unit_of_thread<T>();
  const int C = a.C;
  const float inv_c = 1.0f / (float)C;
  // rows of the last scale tile past n hold scale 0
  const int64_t rows = a.y_codes ? mx4::row_tiles(a.n) * mx4::kTileRows : a.n;
  const int64_t t0 = unit * a.rows_per_unit;
  const int64_t t1 = t0 + a.rows_per_unit < rows ? t0 + a.rows_per_unit : rows;
  const int64_t end = t1 < a.n ? t1 : a.n;
  typename R::Raw nx, nf;
  GateRows<R> gate;
  if (t0 < end) {
    R::load(a.x, t0, C, tid, nx);
    if (a.f) R::load(a.f, t0, C, tid, nf);
    if (a.gate) gate.start(a, t0, tid);
  }
  {
    const int uid = threadIdx.x / T;
    typename R::Quads pw, pb, sc, w, b;
    R::fetch_param(pw, a.post_w, 1.0f, C, tid, uid);
    R::fetch_param(pb, a.post_b, 0.0f, C, tid, uid);
    R::fetch_param(sc, a.scale, 1.0f, C, tid, uid);
    R::fetch_param(w, a.pre_w, 1.0f, C, tid, uid);
    R::fetch_param(b, a.pre_b, 0.0f, C, tid, uid);
#pragma unroll
    for (size_t i = 0; i < sizeof(pw.v) / sizeof(f32x4); ++i) {
      pw.v[i] *= sc.v[i];
      if (a.post_b) pb.v[i] *= sc.v[i];  // no bias stays 0 where the scale is Inf
    }
    R::stage_param(params + PW * T * E, pw, tid, uid);
    R::stage_param(params + PB * T * E, pb, tid, uid);
    R::stage_param(params + W * T * E, w, tid, uid);
    R::stage_param(params + B * T * E, b, tid, uid);
  }
  __syncthreads();
  float g[E];
  bool fresh = true;
  for (int64_t row = t0; row < end; ++row) {
    // an opaque copy of the thread index, so that the parameters are read from
    // LDS in every round instead of being held in registers
    asm volatile("" : "+v"(tid));
    float x[E];
    R::values(nx, x);
    if (a.f) {
      float f[E];
      R::values(nf, f);
      if (a.gate) {
        if (fresh) R::values(gate.next, g);
        fresh = --gate.left == 0;
        if (fresh && row + 1 < end) {
          gate.left = a.per;
          R::load(a.gate, ++gate.group, C, tid, gate.next);
        }
      }
      if (row + 1 < end) {
        R::load(a.x, row + 1, C, tid, nx);
        R::load(a.f, row + 1, C, tid, nf);
      }
      const float rstd = a.post != kNone ? center<R, T>(f, a.post, C, inv_c, a.eps, red, tid) : 1.0f;
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        const f32x4 w = R::param(params + PW * T * E, i, tid), b = R::param(params + PB * T * E, i, tid);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = 4 * i + j;
          const float h = f[e] * rstd * w[j] + b[j];
          x[e] = rounded<BF16>(x[e] + (a.gate ? h * g[e] : h));
        }
      }
      R::store(a.r, row, C, tid, x);
    } else if (row + 1 < end) {
      R::load(a.x, row + 1, C, tid, nx);
    }
    if (a.pre == kNone) continue;
    const float rstd = center<R, T>(x, a.pre, C, inv_c, a.eps, red, tid);
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      const f32x4 w = R::param(params + W * T * E, i, tid), b = R::param(params + B * T * E, i, tid);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[4 * i + j] = x[4 * i + j] * rstd * w[j] + b[j];
    }
    if (a.y) {
      R::store(a.y, row, C, tid, x);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = rounded<BF16>(x[e]);
      store_mx4<R, T>(x, row, C, a.y_codes, a.y_scales, tid);
    }
  }
  const int nb = (C + 127) / 128;
  for (int64_t row = t0 > a.n ? t0 : a.n; row < t1; ++row)
    for (int blk = tid; blk < nb * 4; blk += T) a.y_scales[mx4::scale_at(row, blk, nb)] = 0;
}

// Gradient. With r-hat, f-hat the centred rows over their deviation:
//   dr' = dr + pre^T(dy),  norm^T(d) = rstd (d w - mean(d w v-hat) v-hat [- mean(d w)])
//   dx = dr',  dh = dr' s g,  df = post^T(dh)
//   dg = s dr' h (summed over a gate's tokens),  dpre_w = sum dy r-hat,  dpre_b = sum dy
// and, as s, post_w and post_b are the same for all tokens, from two sums
//   A = sum dr' g f-hat,  B = sum dr' g:
//   dscale = post_w A + post_b B,  dpost_w = s A,  dpost_b = s B.
// The norms are formed again from r and f: their rows are read in any case.
// Sums over tokens stay in registers over a unit's rows, are added up in unit
// order within a workgroup, and by launch_grad's second kernel in workgroup
// order: no atomics, the same bits each time.
// PREF: the next row is asked for while the present one is worked on (not for
// the widest rows, whose registers do not reach for both).
template <bool BF16, Mode MODE, int T, int E, bool PREF>
__global__ __launch_bounds__(block_threads(T)) void join_grad_kernel(Args a) {
  typedef Row<BF16, MODE, T, E> R;
  constexpr int U = R::U;
  enum { PW, PB, S, W };
  __shared__ float red[T > 64 ? 2 * T / 64 : 1];
  extern __shared__ __attribute__((aligned(16))) float params[];  // [NP][T * E]
  int tid = threadIdx.x % T;
  const int uid = unit_of_thread<T>();
  const int64_t unit = (int64_t)blockIdx.x * U + uid;
  const int C = a.C;
  const float inv_c = 1.0f / (float)C;
  const int64_t t0 = unit * a.rows_per_unit < a.n ? unit * a.rows_per_unit : a.n;
  const int64_t t1 = t0 + a.rows_per_unit < a.n ? t0 + a.rows_per_unit : a.n;
  typename R::Raw nd, nr, ndy, nf;
  GateRows<R> gate;
  auto ask = [&](int64_t row) {
    if (a.dr) R::load(a.dr, row, C, tid, nd);
    if (a.pre != kNone) {
      R::load(a.x, row, C, tid, nr);
      R::load(a.dy, row, C, tid, ndy);
    }
    if (PREF && a.f) R::load(a.f, row, C, tid, nf);
  };
  if (t0 < t1) {
    if (PREF) ask(t0);
    if (a.gate) gate.start(a, t0, tid);
  }
  {
    const int u = threadIdx.x / T;
    typename R::Quads pw, pb, sc, w;
    R::fetch_param(pw, a.post_w, 1.0f, C, tid, u);
    R::fetch_param(pb, a.post_b, 0.0f, C, tid, u);
    R::fetch_param(sc, a.scale, 1.0f, C, tid, u);
    R::fetch_param(w, a.pre_w, 1.0f, C, tid, u);
    R::stage_param(params + PW * T * E, pw, tid, u);
    R::stage_param(params + PB * T * E, pb, tid, u);
    R::stage_param(params + S * T * E, sc, tid, u);
    R::stage_param(params + W * T * E, w, tid, u);
  }
  __syncthreads();
  float acc[kVecs][E], g[E], dg[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    g[e] = dg[e] = 0.0f;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) acc[v][e] = 0.0f;
  }
  // A gate group within this unit's rows is complete here; the others (at most
  // the first and the last) leave their part to the second kernel.
  auto flush_gate = [&](int64_t group) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      const f32x4 s = R::param(params + S * T * E, i, tid);
#pragma unroll
      for (int j = 0; j < 4; ++j) dg[4 * i + j] *= s[j];
    }
    const int64_t q0 = group * a.per, q1 = q0 + a.per < a.n ? q0 + a.per : a.n;
    if (q0 >= t0 && q1 <= t1)
      R::store(a.dgate, group, C, tid, dg);
    else
      R::store_f32(a.edge + (2 * unit + (q0 <= t0 ? 0 : 1)) * C, C, tid, dg);
  };
  bool fresh = true;
  for (int64_t row = t0; row < t1; ++row) {
    asm volatile("" : "+v"(tid));  // as in join_kernel
    if (!PREF) ask(row);
    float d[E], f[E], r[E], dy[E];
    if (a.dr) {
      R::values(nd, d);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] = 0.0f;
    }
    if (a.pre != kNone) {
      R::values(nr, r);
      R::values(ndy, dy);
    }
    if (PREF && a.f) R::values(nf, f);
    const int64_t group = gate.group;
    bool last = false;  // the last row of the group here
    if (a.gate) {
      if (fresh) {
        R::values(gate.next, g);
#pragma unroll
        for (int e = 0; e < E; ++e) dg[e] = 0.0f;
      }
      fresh = --gate.left == 0;
      last = fresh || row + 1 == t1;
      if (fresh && row + 1 < t1) {
        gate.left = a.per;
        R::load(a.gate, ++gate.group, C, tid, gate.next);
      }
    }
    if (PREF && row + 1 < t1) ask(row + 1);
    if (a.pre != kNone) {
      const float rstd = center<R, T>(r, a.pre, C, inv_c, a.eps, red, tid);
      float m[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        const f32x4 w = R::param(params + W * T * E, i, tid);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = 4 * i + j;
          r[e] *= rstd;
          acc[kSumPreW][e] += dy[e] * r[e];
          acc[kSumPreB][e] += dy[e];
          dy[e] *= w[j];
          m[0] += dy[e] * r[e];
          m[1] += dy[e];
        }
      }
      unit_sum<T>(m, red, tid);
      const float m0 = m[0] * inv_c, m1 = a.pre == kLayer ? m[1] * inv_c : 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] += rstd * (dy[e] - r[e] * m0 - m1);
    }
    if (a.dx) R::store(a.dx, row, C, tid, d);
    if (!a.f) continue;
    if (!PREF) {
      R::load(a.f, row, C, tid, nf);
      R::values(nf, f);
    }
    float rstd = 1.0f;
    if (a.post != kNone) {
      rstd = center<R, T>(f, a.post, C, inv_c, a.eps, red, tid);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] *= rstd;
    }
    float m[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      const f32x4 pw = R::param(params + PW * T * E, i, tid), pb = R::param(params + PB * T * E, i, tid);
      const f32x4 s = R::param(params + S * T * E, i, tid);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = 4 * i + j;
        if (a.gate) {
          dg[e] += d[e] * (f[e] * pw[j] + pb[j]);
          d[e] *= g[e];
        }
        acc[kA][e] += d[e] * f[e];
        acc[kB][e] += d[e];
        d[e] *= s[j];
        if (a.post != kNone) {
          d[e] *= pw[j];
          m[0] += d[e] * f[e];
          m[1] += d[e];
        }
      }
    }
    if (last && a.dgate) flush_gate(group);
    if (a.post != kNone) {
      unit_sum<T>(m, red, tid);
      const float m0 = m[0] * inv_c, m1 = a.post == kLayer ? m[1] * inv_c : 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] = rstd * (d[e] - f[e] * m0 - m1);
    }
    if (a.df) R::store(a.df, row, C, tid, d);
  }
  // per-workgroup sums
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    if constexpr (U > 1) {
      float* const stage = params;  // U vectors, in place of the parameters
      __syncthreads();
#pragma unroll
      for (int e = 0; e < E; ++e) stage[uid * T * E + e * T + tid] = acc[v][e];
      __syncthreads();
      if (uid == 0) {
#pragma unroll
        for (int e = 0; e < E; ++e)
          for (int u = 1; u < U; ++u) acc[v][e] += stage[u * T * E + e * T + tid];
      }
    }
    if (uid == 0) R::store_f32(a.part + ((int64_t)blockIdx.x * kVecs + v) * C, C, tid, acc[v]);
  }
}

struct Outs {
  float* v[kOuts];
};

// Joins the sums that the runs of a workgroup have taken in turn, by a tree. Called
// by all threads; the total is run 0's.
template <int N, int RUNS, int COLS>
__device__ __forceinline__ void sum_runs(float (&s)[N], float (&red)[N][RUNS][COLS], int run, int col) {
#pragma unroll
  for (int i = 0; i < N; ++i) red[i][run][col] = s[i];
  for (int h = RUNS / 2; h >= 1; h >>= 1) {
    __syncthreads();
    if (run < h)
#pragma unroll
      for (int i = 0; i < N; ++i) red[i][run][col] += red[i][run + h][col];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = red[i][0][col];
}

// The sums over tokens from the workgroups' parts, in a fixed order, and the
// channel vectors from them. 16 columns a workgroup: narrow, so that there are
// workgroups enough to hide the reads.
constexpr int kSumCols = 16, kSumRuns = 64;
__global__ __launch_bounds__(1024) void sum_parts_kernel(Args a, int64_t blocks, Outs out) {
  const int col = threadIdx.x % kSumCols, c = blockIdx.x * kSumCols + col, run = threadIdx.x / kSumCols;
  const int v0 = blockIdx.y * 2;  // A and B, or the two of the norm before the next block
  __shared__ float red[2][kSumRuns][kSumCols];
  float s[2] = {0.0f, 0.0f};
  if (c < a.C)
#pragma unroll 4
    for (int64_t b = run; b < blocks; b += kSumRuns) {
      const float* p = a.part + (b * kVecs + v0) * a.C + c;
      s[0] += p[0];
      s[1] += p[a.C];
    }
  sum_runs(s, red, run, col);
  if (run != 0 || c >= a.C) return;
  const float s0 = s[0], s1 = s[1];
  if (v0 == kA) {
    const float sc = a.scale ? a.scale[c] : 1.0f;
    if (out.v[kDScale])
      out.v[kDScale][c] = (a.post_w ? a.post_w[c] * s0 : s0) + (a.post_b ? a.post_b[c] * s1 : 0.0f);
    if (out.v[kDPostW]) out.v[kDPostW][c] = sc * s0;
    if (out.v[kDPostB]) out.v[kDPostB][c] = sc * s1;
  } else {
    if (out.v[kDPreW]) out.v[kDPreW][c] = s0;
    if (out.v[kDPreB]) out.v[kDPreB][c] = s1;
  }
}

// Gate groups that several units share, each by the unit that it starts in.
template <bool BF16, bool BY_UNIT>
__global__ __launch_bounds__(BY_UNIT ? 256 : 1024) void sum_edges_kernel(Args a) {
  // One workgroup per group, its units shared out to 16 runs, or (BY_UNIT), where a
  // group has fewer units than that, one per unit for its last group. (1024 bf16
  // channels, the whole gradient in us, by group and by unit: 65,952 tokens in groups
  // of 2: 1004, 231; of 30: 289, 214; of 100, 2.3 units: 224, 201; of 1374, 32 units:
  // 202, 206. 1374 tokens in groups of 5: 36, 27; of 30, 10 units: 27, 27; of 100: 26, 29;
  // of 1374: 28, 71.)
  int64_t group = blockIdx.x;
  if (BY_UNIT) {
    const int64_t t1 = (group + 1) * a.rows_per_unit;
    group = ((t1 < a.n ? t1 : a.n) - 1) / a.per;
  }
  const int64_t q0 = group * a.per, q1 = q0 + a.per < a.n ? q0 + a.per : a.n;
  const int64_t u0 = q0 / a.rows_per_unit, u1 = (q1 - 1) / a.rows_per_unit, t0 = u0 * a.rows_per_unit;
  if (u0 == u1 || (BY_UNIT && u0 != blockIdx.x)) return;  // written whole, or another unit's
  constexpr int COLS = BY_UNIT ? 256 : 64, RUNS = BY_UNIT ? 1 : 16;
  const int col = threadIdx.x % COLS, c = blockIdx.y * COLS + col, run = threadIdx.x / COLS;
  __shared__ float red[1][RUNS][COLS];
  float s[1] = {0.0f};
  if (c < a.C)
#pragma unroll 4
    for (int64_t u = u0 + run; u <= u1; u += RUNS) {
      const int slot = u == u0 && q0 > t0 ? 1 : 0;
      s[0] += a.edge[(2 * u + slot) * a.C + c];
    }
  if constexpr (RUNS > 1) sum_runs(s, red, run, col);
  if (run != 0 || c >= a.C) return;
  if (BF16)
    ((uint16_t*)a.dgate)[group * a.C + c] = f32_to_bf16_bits(s[0]);
  else
    ((float*)a.dgate)[group * a.C + c] = s[0];
}

// (The powers of two from 128 on are the unit sizes T * E below.)
Mode row_mode(int C, bool bf16) {
  return C >= 128 && (C & (C - 1)) == 0 ? FULL : C % (bf16 ? 8 : 4) == 0 ? PIECES : SCALAR;
}

// Threads per row for C channels: forward, gradient. Rows of up to 256 channels
// share a wave: a unit's reductions take as long for few channels as for many (a
// wave a row against this, 65,952 bf16 rows: forward 34 and 14 us at 128 channels, 38
// and 25 at 256; gradient 74 and 37, 75 and 54). The gradient has 8 values a thread for
// the registers of its sums (1024 channels as 16 values x 64 threads: 293 us, 245 as
// 8 x 128).
int unit_threads(int C) {
  return C <= 256 ? 16 : C <= 1024 ? 64 : C <= 2048 ? 128 : C <= 4096 ? 256 : 512;
}
int grad_threads(int C) { return C <= 128 ? 16 : C <= 256 ? 32 : C <= 512 ? 64 : C <= 1024 ? 128 : C <= 2048 ? 256 : 512; }

}  // namespace

// PICK(bf16, mode) for the row's type and channel count.
#define VGGT3_JOIN_TYPES(PICK)                           \
  do {                                                   \
    const Mode mode = row_mode(a.C, bf16);               \
    if (bf16) {                                          \
      if (mode == FULL) PICK(true, FULL);                \
      else if (mode == PIECES) PICK(true, PIECES);       \
      else PICK(true, SCALAR);                           \
    } else {                                             \
      if (mode == FULL) PICK(false, FULL);               \
      else if (mode == PIECES) PICK(false, PIECES);      \
      else PICK(false, SCALAR);                          \
    }                                                    \
  } while (0)
// LDS: four parameter vectors, and in their place in the end one vector a unit.
constexpr size_t lds_bytes(int T, int E) {
  return (size_t)(block_threads(T) / T > 4 ? block_threads(T) / T : 4) * T * E * sizeof(float);
}
static_assert(lds_bytes(512, 16) + 2 * 8 * sizeof(float) <= 160 * 1024, "LDS of one workgroup");
#define VGGT3_JOIN_FORWARD(B, V)                                                                                 \
  do {                                                                                                           \
    if (a.C <= 128) VGGT3_JOIN_GO((join_kernel<B, V, 16, 8>), 16, 8);                                            \
    else if (a.C <= 256) VGGT3_JOIN_GO((join_kernel<B, V, 16, 16>), 16, 16);                                     \
    else if (a.C <= 512) VGGT3_JOIN_GO((join_kernel<B, V, 64, 8>), 64, 8);                                       \
    else if (a.C <= 1024) VGGT3_JOIN_GO((join_kernel<B, V, 64, 16>), 64, 16);                                    \
    else if (a.C <= 2048) VGGT3_JOIN_GO((join_kernel<B, V, 128, 16>), 128, 16);                                  \
    else if (a.C <= 4096) VGGT3_JOIN_GO((join_kernel<B, V, 256, 16>), 256, 16);                                  \
    else VGGT3_JOIN_GO((join_kernel<B, V, 512, 16>), 512, 16);                                                   \
  } while (0)
#define VGGT3_JOIN_GRAD(B, V)                                                                                    \
  do {                                                                                                           \
    if (a.C <= 128) VGGT3_JOIN_GO((join_grad_kernel<B, V, 16, 8, true>), 16, 8);                                 \
    else if (a.C <= 256) VGGT3_JOIN_GO((join_grad_kernel<B, V, 32, 8, true>), 32, 8);                            \
    else if (a.C <= 512) VGGT3_JOIN_GO((join_grad_kernel<B, V, 64, 8, true>), 64, 8);                            \
    else if (a.C <= 1024) VGGT3_JOIN_GO((join_grad_kernel<B, V, 128, 8, true>), 128, 8);           \
    else if (a.C <= 2048) VGGT3_JOIN_GO((join_grad_kernel<B, V, 256, 8, true>), 256, 8);                         \
    else if (a.C <= 4096) VGGT3_JOIN_GO((join_grad_kernel<B, V, 512, 8, true>), 512, 8);                         \
    else VGGT3_JOIN_GO((join_grad_kernel<B, (V == SCALAR ? SCALAR : PIECES), 512, 16, false>), 512, 16);         \
  } while (0)
#define VGGT3_JOIN_GO(KERNEL, T, E) \
  hipLaunchKernelGGL(KERNEL, dim3((unsigned)blocks), dim3(block_threads(T)), lds_bytes(T, E), stream, a)

hipError_t launch_forward(const Args& args, bool bf16, hipStream_t stream) {
  Args a = args;
  if (a.n == 0) return hipSuccess;
  const int T = unit_threads(a.C), U = block_threads(T) / T;
  const int64_t rows = a.y_codes ? mx4::row_tiles(a.n) * mx4::kTileRows : a.n;
  const int64_t most = 8192 * 64 / T;  // units
  a.rows_per_unit = (rows + most - 1) / most;
  const int64_t units = (rows + a.rows_per_unit - 1) / a.rows_per_unit;
  const int64_t blocks = (units + U - 1) / U;
  VGGT3_JOIN_TYPES(VGGT3_JOIN_FORWARD);
  return hipGetLastError();
}

GradPlan grad_plan(int64_t n, int C, bool bf16) {
  const int T = grad_threads(C), U = block_threads(T) / T;
  // As many units as 256 compute units hold at once: 12 waves each of the
  // kernels of up to 168 registers, 8 of the others.
  const int64_t waves = bf16 && row_mode(C, bf16) != SCALAR && T >= 64 && T <= 256 ? 12 : 8;
  const int64_t most = 256 * waves * 64 / T;
  // Few rows: up to 3 a unit, for a unit's start costs as much as a row or two and
  // its sums as many bytes as one (1374 x 1024: 19.8, 19.7, 20.4, 22.3 us for 1, 2, 3, 4
  // rows a unit in fp32, and 41, 32, 28, 28 in bf16 with one gate for all).
  const int64_t least = (n + 255) / 256 < 3 ? (n + 255) / 256 : 3;
  GradPlan p;
  p.rows_per_unit = (n + most - 1) / most;
  if (p.rows_per_unit < least) p.rows_per_unit = least;
  p.units = (n + p.rows_per_unit - 1) / p.rows_per_unit;
  p.blocks = (p.units + U - 1) / U;
  return p;
}

hipError_t launch_grad(const Args& args, const GradPlan& p, float* const* out, bool bf16, hipStream_t stream) {
  Args a = args;
  a.rows_per_unit = p.rows_per_unit;
  const int64_t blocks = p.blocks;
  hipError_t e = hipSuccess;
  if (a.n > 0) {
    VGGT3_JOIN_TYPES(VGGT3_JOIN_GRAD);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.n == 0) a.scale = a.post_w = a.post_b = nullptr;  // zeros, whatever the vectors hold
  Outs o;
  bool any = false;
  for (int v = 0; v < kOuts; ++v) any |= (o.v[v] = out[v]) != nullptr;
  if (any) sum_parts_kernel<<<dim3((a.C + kSumCols - 1) / kSumCols, kVecs / 2), dim3(1024), 0, stream>>>(a, blocks, o);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.n > 0 && a.dgate && a.per > 1) {
    const int64_t groups = (a.n + a.per - 1) / a.per;
    const bool by_unit = 16 * groups > p.units;
    const dim3 grid((unsigned)(by_unit ? p.units : groups), (a.C + (by_unit ? 255 : 63)) / (by_unit ? 256 : 64));
    if (by_unit) {
      if (bf16) sum_edges_kernel<true, true><<<grid, dim3(256), 0, stream>>>(a);
      else sum_edges_kernel<false, true><<<grid, dim3(256), 0, stream>>>(a);
    } else {
      if (bf16) sum_edges_kernel<true, false><<<grid, dim3(1024), 0, stream>>>(a);
      else sum_edges_kernel<false, false><<<grid, dim3(1024), 0, stream>>>(a);
    }
    e = hipGetLastError();
  }
  return e;
}

}  // namespace join
}  // namespace vggt3
