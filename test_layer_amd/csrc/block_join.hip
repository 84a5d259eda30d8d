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
// A unit takes a contiguous range of rows and keeps the channel parameters (and
// a gate row that several tokens share) in registers across it.
#include "bf16_ops.hpp"
#include "join.hpp"
#include "mx4_ops.hpp"

namespace vggt3 {
namespace join {
namespace {

// How a unit's T threads share a row: 16-byte pieces in turn where the channel
// count is a multiple of a piece (VEC), single values otherwise.
template <bool BF16, bool VEC, int T, int E>
struct Row {
  static constexpr int VL = VEC ? (BF16 ? 8 : 4) : 1;
  static constexpr int NC = E / VL;
  static_assert(E % VL == 0, "whole pieces");

  __device__ static __forceinline__ int col(int c, int tid) { return (c * T + tid) * VL; }

  __device__ static __forceinline__ void load(const void* base, int64_t row, int C, int tid, float (&v)[E]) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int k = col(c, tid);
      if (k < C) {
        if constexpr (VEC) {
          const u32x4 q = ld16((const char*)base + (row * C + k) * (BF16 ? 2 : 4));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (BF16) {
              v[c * VL + 2 * j] = bf16_lo(q[j]);
              v[c * VL + 2 * j + 1] = bf16_hi(q[j]);
            } else {
              v[c * VL + j] = __uint_as_float(q[j]);
            }
          }
        } else {
          v[c] = BF16 ? bf16_bits_to_f32(((const uint16_t*)base)[row * C + k]) : ((const float*)base)[row * C + k];
        }
      } else {
#pragma unroll
        for (int j = 0; j < VL; ++j) v[c * VL + j] = 0.0f;
      }
    }
  }

  __device__ static __forceinline__ void store(void* base, int64_t row, int C, int tid, const float (&v)[E]) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int k = col(c, tid);
      if (k >= C) continue;
      if constexpr (VEC) {
        u32x4 q;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (BF16)
            q[j] = pack_bf16x2(v[c * VL + 2 * j], v[c * VL + 2 * j + 1]);
          else
            q[j] = __float_as_uint(v[c * VL + j]);
        }
        st16((char*)base + (row * C + k) * (BF16 ? 2 : 4), q);
      } else if constexpr (BF16) {
        ((uint16_t*)base)[row * C + k] = f32_to_bf16_bits(v[c]);
      } else {
        ((float*)base)[row * C + k] = v[c];
      }
    }
  }

  // fp32 channel parameters; `absent` where there is no vector, 0 past C.
  __device__ static __forceinline__ void load_param(const float* p, float absent, int C, int tid, float (&v)[E]) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < VL; ++j) {
        const int k = col(c, tid) + j;
        v[c * VL + j] = k < C ? (p ? p[k] : absent) : 0.0f;
      }
  }

  __device__ static __forceinline__ void store_f32(float* p, int C, int tid, const float (&v)[E]) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < VL; ++j) {
        const int k = col(c, tid) + j;
        if (k < C) p[k] = v[c * VL + j];
      }
  }
};

// Round to the token type and back.
template <bool BF16>
__device__ __forceinline__ float rounded(float v) {
  return BF16 ? bf16_bits_to_f32(f32_to_bf16_bits(v)) : v;
}

// Sums of N values over a unit, given to every thread of it. One wave: a
// butterfly. More: then across waves through LDS, in wave order.
template <int T, int N>
__device__ __forceinline__ void unit_sum(float (&v)[N], float* red, int tid) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], off, 64);
  if constexpr (T > 64) {
    constexpr int W = T / 64;
    __syncthreads();
    if ((tid & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[i * W + (tid >> 6)] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = red[i * W];
      for (int w = 1; w < W; ++w) s += red[i * W + w];
      v[i] = s;
    }
  }
}

constexpr int block_threads(int T) { return T < 256 ? 256 : T; }

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
    for (int e = 0; e < E; ++e) v[e] = R::col(e / R::VL, tid) + e % R::VL < C ? v[e] - mean : 0.0f;
  }
  float q[1] = {0.0f};
#pragma unroll
  for (int e = 0; e < E; ++e) q[0] += v[e] * v[e];
  unit_sum<T>(q, red, tid);
  return rsqrtf(q[0] * inv_c + eps);
}

// One row of y in 4 bits (values already rounded to the token type): blocks of
// 32 columns lie in 32 / VL neighbouring threads.
template <class R, int T, int E>
__device__ __forceinline__ void store_mx4(const float (&y)[E], int64_t row, int C, uint8_t* codes, uint8_t* scales,
                                          int tid) {
  const int nb = (C + 127) / 128;
  // past C the value is 0 whatever the row holds (a NaN row has NaN there too)
  auto value = [&](int c, int j) { return R::col(c, tid) + j < C ? y[c * R::VL + j] : 0.0f; };
#pragma unroll
  for (int c = 0; c < R::NC; ++c) {
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < R::VL; ++j) {
      const uint32_t a = __float_as_uint(value(c, j)) & 0x7fffffffu;
      amax = a > amax ? a : amax;
    }
#pragma unroll
    for (int off = 1; off < 32 / R::VL; off <<= 1) {
      const uint32_t o = __shfl_xor(amax, off, 64);
      amax = o > amax ? o : amax;
    }
    const uint32_t s = mx4::scale_byte(amax);
    const int k = R::col(c, tid);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < R::VL ? value(c, j < R::VL ? j : 0) : 0.0f;
    uint32_t q = s == 255u ? 0u : mx4::encode8(v, mx4::scale_value(s));
    if constexpr (R::VL == 1) q |= (uint32_t)__shfl_xor((int)q, 1, 64) << 4;
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

template <bool BF16, bool VEC, int T, int E>
__global__ __launch_bounds__(block_threads(T)) void join_kernel(Args a) {
  typedef Row<BF16, VEC, T, E> R;
  constexpr int U = block_threads(T) / T;  // units per workgroup
  __shared__ float red[T > 64 ? T / 64 : 1];
  const int tid = threadIdx.x % T;
  const int64_t unit = (int64_t)blockIdx.x * U + threadIdx.x / T;
  const int C = a.C;
  const float inv_c = 1.0f / (float)C;
  // rows of the last scale tile past n hold scale 0
  const int64_t rows = a.y_codes ? mx4::row_tiles(a.n) * mx4::kTileRows : a.n;
  const int64_t t0 = unit * a.rows_per_unit;
  const int64_t t1 = t0 + a.rows_per_unit < rows ? t0 + a.rows_per_unit : rows;
  float pw[E], pb[E], s[E], w[E], b[E], g[E];
  R::load_param(a.post_w, 1.0f, C, tid, pw);
  R::load_param(a.post_b, 0.0f, C, tid, pb);
  R::load_param(a.scale, 1.0f, C, tid, s);
  R::load_param(a.pre_w, 1.0f, C, tid, w);
  R::load_param(a.pre_b, 0.0f, C, tid, b);
  int64_t group = -1;
  for (int64_t row = t0; row < t1; ++row) {
    if (row >= a.n) {
      const int nb = (C + 127) / 128;
      for (int blk = tid; blk < nb * 4; blk += T) a.y_scales[mx4::scale_at(row, blk, nb)] = 0;
      continue;
    }
    float x[E];
    R::load(a.x, row, C, tid, x);
    if (a.f) {
      float f[E];
      R::load(a.f, row, C, tid, f);
      if (a.gate && (int64_t)((uint32_t)row / (uint32_t)a.per) != group) {
        group = (uint32_t)row / (uint32_t)a.per;
        R::load(a.gate, group, C, tid, g);
      }
      if (a.post != kNone) {
        const float rstd = center<R, T>(f, a.post, C, inv_c, a.eps, red, tid);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = f[e] * rstd * pw[e] + pb[e];
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float h = a.gate ? f[e] * g[e] : f[e];
        x[e] = rounded<BF16>(x[e] + h * s[e]);
      }
      R::store(a.r, row, C, tid, x);
    }
    if (a.pre == kNone) continue;
    const float rstd = center<R, T>(x, a.pre, C, inv_c, a.eps, red, tid);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = x[e] * rstd * w[e] + b[e];
    if (a.y) {
      R::store(a.y, row, C, tid, x);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = rounded<BF16>(x[e]);
      store_mx4<R, T>(x, row, C, a.y_codes, a.y_scales, tid);
    }
  }
}

// Gradient. With r-hat, f-hat the centred rows over their deviation:
//   dr' = dr + pre^T(dy),  norm^T(d) = rstd (d w - mean(d w v-hat) v-hat [- mean(d w)])
//   dx = dr',  dh = dr' s g,  df = post^T(dh)
//   ds = sum dr' g h,  dg = dr' s h (summed over a gate's tokens),
//   dw = sum d v-hat,  db = sum d
// The norms are formed again from r and f: their rows are read in any case.
// Sums over tokens stay in registers over a unit's rows, are added up in unit
// order within a workgroup, and by launch_grad's second kernel in workgroup
// order: no atomics, the same bits each time.
template <bool BF16, bool VEC, int T, int E>
__global__ __launch_bounds__(block_threads(T)) void join_grad_kernel(Args a) {
  typedef Row<BF16, VEC, T, E> R;
  constexpr int U = block_threads(T) / T;
  __shared__ float red[T > 64 ? 2 * T / 64 : 1];
  __shared__ float stage[U > 1 ? U * T * E : 1];
  const int tid = threadIdx.x % T, uid = threadIdx.x / T;
  const int64_t unit = (int64_t)blockIdx.x * U + uid;
  const int C = a.C;
  const float inv_c = 1.0f / (float)C;
  const int64_t t0 = unit * a.rows_per_unit < a.n ? unit * a.rows_per_unit : a.n;
  const int64_t t1 = t0 + a.rows_per_unit < a.n ? t0 + a.rows_per_unit : a.n;
  float pw[E], pb[E], s[E], w[E], g[E];
  R::load_param(a.post_w, 1.0f, C, tid, pw);
  R::load_param(a.post_b, 0.0f, C, tid, pb);
  R::load_param(a.scale, 1.0f, C, tid, s);
  R::load_param(a.pre_w, 1.0f, C, tid, w);
  float acc[kVecs][E], dg[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    dg[e] = 0.0f;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) acc[v][e] = 0.0f;
  }
  int64_t group = -1;
  // A gate group within this unit's rows is complete here; the others (at most
  // the first and the last) leave their part to the second kernel.
  auto flush_gate = [&]() {
    const int64_t q0 = group * a.per, q1 = q0 + a.per < a.n ? q0 + a.per : a.n;
    if (q0 >= t0 && q1 <= t1)
      R::store(a.dgate, group, C, tid, dg);
    else
      R::store_f32(a.edge + (2 * unit + (t0 / a.per == group ? 0 : 1)) * C, C, tid, dg);
  };
  for (int64_t row = t0; row < t1; ++row) {
    float d[E];
    if (a.dr) {
      R::load(a.dr, row, C, tid, d);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] = 0.0f;
    }
    if (a.pre != kNone) {
      float r[E], dy[E];
      R::load(a.x, row, C, tid, r);
      R::load(a.dy, row, C, tid, dy);
      const float rstd = center<R, T>(r, a.pre, C, inv_c, a.eps, red, tid);
      float m[2] = {0.0f, 0.0f};
#pragma unroll
      for (int e = 0; e < E; ++e) {
        r[e] *= rstd;
        acc[kDPreW][e] += dy[e] * r[e];
        acc[kDPreB][e] += dy[e];
        dy[e] *= w[e];
        m[0] += dy[e] * r[e];
        m[1] += dy[e];
      }
      unit_sum<T>(m, red, tid);
      const float m0 = m[0] * inv_c, m1 = a.pre == kLayer ? m[1] * inv_c : 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] += rstd * (dy[e] - r[e] * m0 - m1);
    }
    if (a.dx) R::store(a.dx, row, C, tid, d);
    if (!a.f) continue;
    float f[E];
    R::load(a.f, row, C, tid, f);
    float rstd = 1.0f;
    if (a.post != kNone) {
      rstd = center<R, T>(f, a.post, C, inv_c, a.eps, red, tid);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] *= rstd;
    }
    if (a.gate) {
      if ((int64_t)((uint32_t)row / (uint32_t)a.per) != group) {
        if (group >= 0 && a.dgate) flush_gate();
        group = (uint32_t)row / (uint32_t)a.per;
        R::load(a.gate, group, C, tid, g);
#pragma unroll
        for (int e = 0; e < E; ++e) dg[e] = 0.0f;
      }
    }
    float m[2] = {0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float h = f[e] * pw[e] + pb[e];
      if (a.gate) {
        dg[e] += d[e] * s[e] * h;
        d[e] *= g[e];
      }
      acc[kDScale][e] += d[e] * h;
      d[e] *= s[e];
      acc[kDPostW][e] += d[e] * f[e];
      acc[kDPostB][e] += d[e];
      if (a.post != kNone) {
        d[e] *= pw[e];
        m[0] += d[e] * f[e];
        m[1] += d[e];
      }
    }
    if (a.post != kNone) {
      unit_sum<T>(m, red, tid);
      const float m0 = m[0] * inv_c, m1 = a.post == kLayer ? m[1] * inv_c : 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] = rstd * (d[e] - f[e] * m0 - m1);
    }
    if (a.df) R::store(a.df, row, C, tid, d);
  }
  if (group >= 0 && a.dgate) flush_gate();
  // per-workgroup sums
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    if constexpr (U > 1) {
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
  float* v[kVecs];
};

// out[v][c] = sum of the workgroups' parts, in a fixed order: 16 interleaved
// runs, then a tree over them.
__global__ __launch_bounds__(1024) void sum_parts_kernel(const float* part, int64_t blocks, int C, Outs out) {
  const int v = blockIdx.y, c = blockIdx.x * 64 + (threadIdx.x & 63), run = threadIdx.x >> 6;
  float* o = out.v[v];
  if (!o) return;
  __shared__ float red[16][64];
  float s = 0.0f;
  if (c < C)
    for (int64_t b = run; b < blocks; b += 16) s += part[(b * kVecs + v) * C + c];
  red[run][threadIdx.x & 63] = s;
  for (int h = 8; h >= 1; h >>= 1) {
    __syncthreads();
    if (run < h) red[run][threadIdx.x & 63] += red[run + h][threadIdx.x & 63];
  }
  if (run == 0 && c < C) o[c] = red[0][threadIdx.x];
}

// Gate groups that several units share: their parts in unit order.
template <bool BF16>
__global__ __launch_bounds__(256) void sum_edges_kernel(Args a) {
  const int64_t group = blockIdx.x;
  const int64_t q0 = group * a.per, q1 = q0 + a.per < a.n ? q0 + a.per : a.n;
  const int64_t u0 = q0 / a.rows_per_unit, u1 = (q1 - 1) / a.rows_per_unit;
  if (u0 == u1) return;  // written by its unit
  for (int c = blockIdx.y * 256 + threadIdx.x; c < a.C; c += gridDim.y * 256) {
    float s = 0.0f;
    for (int64_t u = u0; u <= u1; ++u) {
      const int slot = u * a.rows_per_unit / a.per == group ? 0 : 1;
      s += a.edge[(2 * u + slot) * a.C + c];
    }
    if (BF16)
      ((uint16_t*)a.dgate)[group * a.C + c] = f32_to_bf16_bits(s);
    else
      ((float*)a.dgate)[group * a.C + c] = s;
  }
}

// Threads per row for C channels, and whether rows are whole 16-byte pieces.
int unit_threads(int C) { return C <= 1024 ? 64 : C <= 4096 ? 256 : 512; }
bool vec_rows(int C, bool bf16) { return C % (bf16 ? 8 : 4) == 0; }

}  // namespace

#define VGGT3_JOIN_DISPATCH(KERNEL)                                                                        \
  do {                                                                                                     \
    const bool vec = vec_rows(a.C, bf16);                                                                  \
    const dim3 grid((unsigned)blocks);                                                                     \
    if (bf16) {                                                                                            \
      if (vec) VGGT3_JOIN_T(KERNEL, true, true);                                                           \
      else VGGT3_JOIN_T(KERNEL, true, false);                                                              \
    } else {                                                                                               \
      if (vec) VGGT3_JOIN_T(KERNEL, false, true);                                                          \
      else VGGT3_JOIN_T(KERNEL, false, false);                                                             \
    }                                                                                                      \
  } while (0)
#define VGGT3_JOIN_T(KERNEL, B, V)                                                                         \
  do {                                                                                                     \
    if (a.C <= 512) KERNEL<B, V, 64, 8><<<grid, dim3(256), 0, stream>>>(a);                                \
    else if (a.C <= 1024) KERNEL<B, V, 64, 16><<<grid, dim3(256), 0, stream>>>(a);                         \
    else if (a.C <= 4096) KERNEL<B, V, 256, 16><<<grid, dim3(256), 0, stream>>>(a);                        \
    else KERNEL<B, V, 512, 16><<<grid, dim3(512), 0, stream>>>(a);                                         \
  } while (0)

hipError_t launch_forward(const Args& args, bool bf16, hipStream_t stream) {
  Args a = args;
  if (a.n == 0) return hipSuccess;
  const int T = unit_threads(a.C), U = block_threads(T) / T;
  const int64_t rows = a.y_codes ? mx4::row_tiles(a.n) * mx4::kTileRows : a.n;
  const int64_t most = 8192 / (T / 64);  // units
  a.rows_per_unit = (rows + most - 1) / most;
  const int64_t units = (rows + a.rows_per_unit - 1) / a.rows_per_unit;
  const int64_t blocks = (units + U - 1) / U;
  VGGT3_JOIN_DISPATCH(join_kernel);
  return hipGetLastError();
}

GradPlan grad_plan(int64_t n, int C, bool) {
  const int T = unit_threads(C), U = block_threads(T) / T;
  const int64_t most = 2048 / (T / 64);
  GradPlan p;
  p.rows_per_unit = (n + most - 1) / most;
  if (p.rows_per_unit < 4) p.rows_per_unit = 4;
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
    VGGT3_JOIN_DISPATCH(join_grad_kernel);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  Outs o;
  bool any = false;
  for (int v = 0; v < kVecs; ++v) any |= (o.v[v] = out[v]) != nullptr;
  if (any) sum_parts_kernel<<<dim3((a.C + 63) / 64, kVecs), dim3(1024), 0, stream>>>(a.part, blocks, a.C, o);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.n > 0 && a.dgate && a.per > 1) {
    const dim3 grid((unsigned)((a.n + a.per - 1) / a.per), (a.C + 255) / 256);
    if (bf16) sum_edges_kernel<true><<<grid, dim3(256), 0, stream>>>(a);
    else sum_edges_kernel<false><<<grid, dim3(256), 0, stream>>>(a);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace join
}  // namespace vggt3
