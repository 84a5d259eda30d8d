// The gradient of the gated delta rule, chunk by chunk, from the state S before each
// chunk and the gradient dS of the state after it (delta_scan.hip). With the forward's
// y, u, o and the reverse scan's du, x = X^T du, dR = beta . x,
//
//   dV = dR,    dbeta_i = x_i . y_i
//   F = scale D . (dO u^T) (lower),    E = D . (dR u^T) (strictly lower)
//   dQ = scale G . (dO S^T) + F K
//   dK = F^T Q + G_end / G . (u dS^T) - G . (dR S^T) - E K - E^T K
//   dg_t = sum over i >= t of (o_i . dO_i - v_i . dR_i) + <dS, the state after>
//
// The last line: G enters o_i as its query's factor, and each token's error as its
// read key's factor minus its write key's, whose sum is -v_i . dR_i; a whole chunk
// back from its end, what the later chunks say is in <dS, state>. (One such sum over
// the whole sequence would lose the small terms; over 32 tokens it does not.)
//
// Four waves to a chunk and head: each has a quarter of the value channels (u, x, o and
// the row sums, in fp32 values whole), then two forms each of F and E, then a quarter
// of the key channels (dQ, dK, from operands in two bf16 parts). u and dR change from
// columns by lane to rows by lane through LDS.
#include <type_traits>

#include "delta_chunk.hpp"

namespace vggt3 {
namespace delta {
namespace {

constexpr int kWaves = 4;

template <class T, int DK, int DV>
struct GradShared {
  static constexpr int kParts = sizeof(T) == 2 ? 2 : 1;  // of u and dR
  static constexpr int kTwo = 128;                       // an operand of two parts, or of fp32 values
  T k[kChunk][kPitch<T, DK>];
  T q[kChunk][kPitch<T, DK>];
  T u[kParts][kChunk][kPitch<T, DV>];
  T dr[kParts][kChunk][kPitch<T, DV>];
  u32x4 op[4][2][kTwo];  // F, F^T, -E, -E^T, 16 rows each
  float along[kWaves][kChunk], step[kWaves][kChunk], all[kWaves];
};

// A tile pair's values as rows of LDS, split into parts.
template <int PITCH>
__device__ __forceinline__ void put_tile(uint16_t* to, const f32x4& v0, const f32x4& v1, int part, int col, int q) {
  f32x4 v[2] = {v0, v1};
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint16_t b = f32_to_bf16_bits(v[it][r]);
        to[p * part + (16 * it + 4 * q + r) * PITCH + col] = b;
        v[it][r] -= bf16_bits_to_f32(b);
      }
}
template <int PITCH>
__device__ __forceinline__ void put_tile(float* to, const f32x4& v0, const f32x4& v1, int, int col, int q) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    to[(4 * q + r) * PITCH + col] = v0[r];
    to[(16 + 4 * q + r) * PITCH + col] = v1[r];
  }
}
template <int PITCH>
__device__ __forceinline__ void row_parts(Frag<uint16_t>& f, const uint16_t* from, int part, int row, int col) {
  f.part[0] = ld_op(from + row * PITCH + col);
  f.part[1] = ld_op(from + part + row * PITCH + col);
}
template <int PITCH>
__device__ __forceinline__ void row_parts(Frag<float>& f, const float* from, int, int row, int col) {
  row8(f, from + row * PITCH + col);
}

// Sum over a row's 16 lanes, in all of them.
template <int CTRL>
__device__ __forceinline__ float row_add(float x) {
  return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float row_sum(float x) {
  return row_add<0x140>(row_add<0x141>(row_add<0x4E>(row_add<0xB1>(x))));
}

template <class T, int DK, int DV>
__global__ __launch_bounds__(64 * kWaves, DK + DV == 128 ? 3 : 1) void grad_kernel(const Args a) {
  using Sh = GradShared<T, DK, DV>;
  constexpr int kP = kWhole<T>, kV = DV / 64, kK = DK / 64, kPV = kPitch<T, DV>, kPK = kPitch<T, DK>, kB = (int)sizeof(T);
  __shared__ Sh m;
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int c = lane % 16, q = lane / 16;
  const int h = blockIdx.x % a.hv;
  const int64_t slot = blockIdx.x / a.hv;
  const Piece p = find_piece(a.cu, a.nseq, a.n, kChunk, slot, lane);
  if (p.seg < 0 || p.len == 0) return;
  const int kh = h / (a.hv / a.hk), len = p.len;
  const int64_t ldk = (int64_t)a.hk * DK, ldv = (int64_t)a.hv * DV;
  const Window kw = window<DK>(static_cast<const T*>(a.k) + p.first * ldk + kh * DK, ldk, len);
  const Window qw = window<DK>(static_cast<const T*>(a.q) + p.first * ldk + kh * DK, ldk, len);
  const Window vw = window<DV>(static_cast<const T*>(a.v) + p.first * ldv + h * DV, ldv, len);
  const Window ow = window<DV>(static_cast<const T*>(a.dout) + p.first * ldv + h * DV, ldv, len);
  const float* S0 = a.states + (slot * a.hv + h) * DK * DV;
  const float* S1 = a.dstates + (slot * a.hv + h) * DK * DV;
  const Matrices& mat = *matrices_of(a.mats, slot * a.hv + h, true);
  const int orow = (int)((c * ldv + 8 * q) * kB), onext = (int)(16 * ldv * kB);  // dO by rows

  {  // K and Q to LDS
    constexpr int kPieces = DK / 8, kEach = kChunk * kPieces / (64 * kWaves);
    Raw<T> kr[kEach], qr[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int at = i * 64 * kWaves + threadIdx.x, off = (int)((at / kPieces * ldk + at % kPieces * 8) * kB);
      load_raw(kr[i], kw, off);
      load_raw(qr[i], qw, off);
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int at = i * 64 * kWaves + threadIdx.x;
      put_raw(&m.k[at / kPieces][at % kPieces * 8], kr[i]);
      put_raw(&m.q[at / kPieces][at % kPieces * 8], qr[i]);
    }
  }

  // this wave's value channels
  {
    const int col = wave * 16 * kV + kV * c;
    const int voff = (int)((4 * q * ldv + col) * kB), vrow = (int)(ldv * kB);
    RawN<T, kV> vr[2][4], dr[2][4];
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        load_rawn(vr[it][r], vw, voff + (16 * it + r) * vrow);
        load_rawn(dr[it][r], ow, voff + (16 * it + r) * vrow);
      }
    const Tri t = get_tri(mat.t, lane), b = get_tri(mat.b, lane), bt = get_tri(mat.bt, lane), xt = get_tri(mat.x, lane);
    f32x4 dec[2], rest[2], beta[2], along[2], step[2];
#pragma unroll
    for (int it = 0; it < 2; ++it) {
      dec[it] = rows4(mat.rows.decay, it, q);
      rest[it] = rows4(mat.rows.rest, it, q);
      beta[it] = rows4(mat.rows.beta, it, q);
      along[it] = step[it] = zero4();
    }
    f32x4 ks[2][kV], kd[2][kV], qs[2][kV];
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int x = 0; x < kV; ++x) ks[it][x] = kd[it][x] = qs[it][x] = zero4();
    float both = 0.0f;  // <dS, S>
    __syncthreads();
#pragma unroll
    for (int s = 0; s < DK / 32; ++s) {
      f32x4 st[2][kV], ds[2][kV];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float w0[kV], w1[kV];
          const int at = channel(2 * s + i, 4 * q + r) * DV + col;
          load_n<kV>(w0, S0 + at);
          load_n<kV>(w1, S1 + at);
#pragma unroll
          for (int x = 0; x < kV; ++x) {
            st[i][x][r] = w0[x];
            ds[i][x][r] = w1[x];
            both += w0[x] * w1[x];
          }
        }
      Frag<T> k0, k1, q0, q1;
      row8(k0, &m.k[c][32 * s + 8 * q]);
      row8(k1, &m.k[16 + c][32 * s + 8 * q]);
      row8(q0, &m.q[c][32 * s + 8 * q]);
      row8(q1, &m.q[16 + c][32 * s + 8 * q]);
#pragma unroll
      for (int x = 0; x < kV; ++x) {
        Frag<T> f;
        make<kP>(f, st[0][x], st[1][x]);
        ks[0][x] = mm<1, kP>(k0, f, ks[0][x]);
        ks[1][x] = mm<1, kP>(k1, f, ks[1][x]);
        qs[0][x] = mm<1, kP>(q0, f, qs[0][x]);
        qs[1][x] = mm<1, kP>(q1, f, qs[1][x]);
        make<kP>(f, ds[0][x], ds[1][x]);
        kd[0][x] = mm<1, kP>(k0, f, kd[0][x]);
        kd[1][x] = mm<1, kP>(k1, f, kd[1][x]);
      }
    }
    both *= mat.rows.total;
    Frag<T> o[2];
    f32x4 dR[2][kV];
#pragma unroll
    for (int x = 0; x < kV; ++x) {
      f32x4 V[2], dO[2];
#pragma unroll
      for (int it = 0; it < 2; ++it)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          V[it][r] = value_of(vr[it][r], x);
          dO[it][r] = value_of(dr[it][r], x);
        }
      Frag<T> f;
      make<kP>(f, V[0] - dec[0] * ks[0][x], V[1] - dec[1] * ks[1][x]);
      lower_rows<kP>(o, t);
      const f32x4 y0 = mm<kP, kP>(o[0], f, zero4()), y1 = mm<kP, kP>(o[1], f, zero4());
      const f32x4 u0 = y0 * beta[0], u1 = y1 * beta[1];
      put_tile<kPV>(&m.u[0][0][0], u0, u1, kChunk * kPV, col + x, q);
      make<kP>(f, u0, u1);
      lower_rows<kP>(o, b);
      along[0] += dO[0] * mm<kP, kP>(o[0], f, qs[0][x] * (dec[0] * a.scale));
      along[1] += dO[1] * mm<kP, kP>(o[1], f, qs[1][x] * (dec[1] * a.scale));
      make<1>(f, dO[0], dO[1]);
      upper_rows<kP>(o, bt);
      const f32x4 e0 = kd[0][x] * rest[0], e1 = kd[1][x] * rest[1];
      const f32x4 du0 = mm<kP, 1>(o[0], f, e0), du1 = mm<kP, 1>(o[1], f, e1);
      make<kP>(f, du0, du1);
      upper_rows<kP>(o, xt);
      const f32x4 x0 = mm<kP, kP>(o[0], f, zero4()), x1 = mm<kP, kP>(o[1], f, zero4());
      dR[0][x] = x0 * beta[0];
      dR[1][x] = x1 * beta[1];
      put_tile<kPV>(&m.dr[0][0][0], dR[0][x], dR[1][x], kChunk * kPV, col + x, q);
      along[0] -= V[0] * dR[0][x];
      along[1] -= V[1] * dR[1][x];
      step[0] += y0 * x0;
      step[1] += y1 * x1;
#pragma unroll
      for (int r = 0; r < 4; ++r) both += e0[r] * u0[r] + e1[r] * u1[r];
    }
    if (a.dv_out) {
      const Window dw = window<DV>(static_cast<const T*>(a.dv_out) + p.first * ldv + h * DV, ldv, len);
#pragma unroll
      for (int it = 0; it < 2; ++it)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float w[kV];
#pragma unroll
          for (int x = 0; x < kV; ++x) w[x] = dR[it][x][r];
          store_rawn<T, kV>(dw, voff + (16 * it + r) * vrow, w);
        }
    }
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float s0 = row_sum(along[it][r]), s1 = row_sum(step[it][r]);
        if (c == 0) {
          m.along[wave][16 * it + 4 * q + r] = s0;
          m.step[wave][16 * it + 4 * q + r] = s1;
        }
      }
    both = wave_sum(both);
    if (lane == 0) m.all[wave] = both;
  }
  __syncthreads();

  // F and E, rows by lane and columns by lane: waves 0 and 1 dO u^T, waves 2 and 3 dR u^T
  {
    Tri w{zero4(), zero4(), zero4()};
    const bool by_row = wave % 2 == 0, of_e = wave >= 2;
#pragma unroll
    for (int s = 0; s < DV / 32; ++s) {
      Frag<T> l0, l1, u0, u1;
      const int col = 32 * s + 8 * q;
      row_parts<kPV>(u0, &m.u[0][0][0], kChunk * kPV, c, col);
      row_parts<kPV>(u1, &m.u[0][0][0], kChunk * kPV, 16 + c, col);
      if (of_e) {
        row_parts<kPV>(l0, &m.dr[0][0][0], kChunk * kPV, c, col);
        row_parts<kPV>(l1, &m.dr[0][0][0], kChunk * kPV, 16 + c, col);
        if (by_row) {
          w.t00 = mm<2, 2>(u0, l0, w.t00);
          w.t10 = mm<2, 2>(u0, l1, w.t10);
          w.t11 = mm<2, 2>(u1, l1, w.t11);
        } else {
          w.t00 = mm<2, 2>(l0, u0, w.t00);
          w.t10 = mm<2, 2>(l1, u0, w.t10);
          w.t11 = mm<2, 2>(l1, u1, w.t11);
        }
      } else {
        Raw<T> r0, r1;
        load_raw(r0, ow, orow + 32 * s * kB);
        load_raw(r1, ow, orow + onext + 32 * s * kB);
        as_frag(l0, r0);
        as_frag(l1, r1);
        if (by_row) {
          w.t00 = mm<2, 1>(u0, l0, w.t00);
          w.t10 = mm<2, 1>(u0, l1, w.t10);
          w.t11 = mm<2, 1>(u1, l1, w.t11);
        } else {
          w.t00 = mm<1, 2>(l0, u0, w.t00);
          w.t10 = mm<1, 2>(l1, u0, w.t10);
          w.t11 = mm<1, 2>(l1, u1, w.t11);
        }
      }
    }
    const float f = of_e ? -1.0f : a.scale;
    Frag<T> o[2];
    if (by_row) {
      w = w * decays<false>(mat.rows, lane);
      w = of_e ? lower<false, true>(w, lane) : lower<false, false>(w, lane);
    } else {
      w = w * decays<true>(mat.rows, lane);
      w = of_e ? lower<true, true>(w, lane) : lower<true, false>(w, lane);
    }
    w.t00 *= f;
    w.t10 *= f;
    w.t11 *= f;
    if (by_row)
      lower_rows<2>(o, w);
    else
      upper_rows<2>(o, w);
    put<2>(m.op[wave][0], o[0], lane);
    put<2>(m.op[wave][1], o[1], lane);
  }
  if (wave == 3 && lane < kChunk) {
    double x = 0.0;
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      x += m.along[w][lane];
      s += m.step[w][lane];
    }
#pragma unroll
    for (int off = 1; off < kChunk; off *= 2) {
      const double down = __shfl_down(x, off, 32);
      if (lane + off < kChunk) x += down;
    }
    const double all = (double)m.all[0] + m.all[1] + m.all[2] + m.all[3];
    if (lane < len) {
      if (a.dg) a.dg[(p.first + lane) * a.hv + h] = (float)(x + all);
      if (a.dbeta) a.dbeta[(p.first + lane) * a.hv + h] = s;
    }
  }
  __syncthreads();

  // this wave's key channels: lane c has channels kK wave 16 + kK c and the next
  if (a.dq == nullptr && a.dk_out == nullptr) return;
  f32x4 dq[2][kK], dk[2][kK];
#pragma unroll
  for (int x = 0; x < kK; ++x) {
    f32x4 ds[2], rs[2];
#pragma unroll
    for (int it = 0; it < 2; ++it) dq[it][x] = ds[it] = rs[it] = zero4();
    const int row = (16 * kK * wave + kK * c + x) * DV;
#pragma unroll
    for (int s = 0; s < DV / 32; ++s) {
      const int col = 32 * s + 8 * q;
      Frag<T> s0, s1, l;
      make<2>(s0, *reinterpret_cast<const f32x4*>(S0 + row + col), *reinterpret_cast<const f32x4*>(S0 + row + col + 4));
      make<2>(s1, *reinterpret_cast<const f32x4*>(S1 + row + col), *reinterpret_cast<const f32x4*>(S1 + row + col + 4));
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        Raw<T> r;
        load_raw(r, ow, orow + it * onext + 32 * s * kB);
        as_frag(l, r);
        dq[it][x] = mm<1, 2>(l, s0, dq[it][x]);
        row_parts<kPV>(l, &m.dr[0][0][0], kChunk * kPV, 16 * it + c, col);
        rs[it] = mm<2, 2>(l, s0, rs[it]);
        row_parts<kPV>(l, &m.u[0][0][0], kChunk * kPV, 16 * it + c, col);
        ds[it] = mm<2, 2>(l, s1, ds[it]);
      }
    }
    Frag<T> kc, qc;
    token_columns<kK, kPK>(kc, &m.k[0][0], 16 * kK * wave, x, lane);
    token_columns<kK, kPK>(qc, &m.q[0][0], 16 * kK * wave, x, lane);
#pragma unroll
    for (int it = 0; it < 2; ++it) {
      const f32x4 dec = rows4(mat.rows.decay, it, q), rest = rows4(mat.rows.rest, it, q);
      Frag<T> l;
      get<2>(l, m.op[0][it], lane);
      dq[it][x] = mm<2, 1>(l, kc, dq[it][x] * (dec * a.scale));
      f32x4 d = ds[it] * rest - rs[it] * dec;
      get<2>(l, m.op[1][it], lane);
      d = mm<2, 1>(l, qc, d);
      get<2>(l, m.op[2][it], lane);
      d = mm<2, 1>(l, kc, d);
      get<2>(l, m.op[3][it], lane);
      dk[it][x] = mm<2, 1>(l, kc, d);
    }
  }
  const int ch = 16 * kK * wave + kK * c;
  const auto store = [&](auto* to, int64_t ld, const f32x4(*v)[kK]) {
    using U = std::remove_pointer_t<decltype(to)>;
    const Window w = window<DK>(to, ld, len);
    const int off = (int)((4 * q * ld + ch) * (int)sizeof(U)), next = (int)(ld * (int)sizeof(U));
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float o[kK];
#pragma unroll
        for (int x = 0; x < kK; ++x) o[x] = v[it][x][r];
        store_rawn<U, kK>(w, off + (16 * it + r) * next, o);
      }
  };
  if (a.dq_part) {
    store(a.dq_part + (p.first * a.hv + h) * DK, (int64_t)a.hv * DK, dq);
    store(a.dk_part + (p.first * a.hv + h) * DK, (int64_t)a.hv * DK, dk);
  } else {
    if (a.dq) store(static_cast<T*>(a.dq) + p.first * ldk + kh * DK, ldk, dq);
    if (a.dk_out) store(static_cast<T*>(a.dk_out) + p.first * ldk + kh * DK, ldk, dk);
  }
}

// dq, dk of key heads that several value heads share, in the heads' order. Rows of
// no sequence are left as they are.
template <class T>
__global__ __launch_bounds__(256) void group_kernel(const Args a) {
  const uint32_t row = blockIdx.x;
  bool inside = a.cu == nullptr;
  for (int b = threadIdx.x; !inside && b < a.nseq; b += 256)
    inside = row >= bound(a.cu, b, a.n) && row < bound(a.cu, b + 1, a.n);
  if (!__syncthreads_or(inside)) return;
  const int group = a.hv / a.hk, width = a.hk * a.dk;
  const float* from = blockIdx.y ? a.dk_part : a.dq_part;
  T* to = static_cast<T*>(blockIdx.y ? a.dk_out : a.dq);
  if (from == nullptr || to == nullptr) return;
  for (int i = 4 * threadIdx.x; i < width; i += 1024) {
    const int kh = i / a.dk, ch = i % a.dk;
    f32x4 s = zero4();
    for (int g = 0; g < group; ++g)
      s += *reinterpret_cast<const f32x4*>(from + ((int64_t)row * a.hv + kh * group + g) * a.dk + ch);
    const float w[4] = {s[0], s[1], s[2], s[3]};
    store_n<4>(to + (int64_t)row * width + i, w);
  }
}

template <class T, int DK, int DV>
hipError_t run(const Args& a, hipStream_t s) {
  grad_kernel<T, DK, DV><<<(unsigned)(chunk_slots(a.n, a.nseq) * a.hv), 64 * kWaves, 0, s>>>(a);
  return hipGetLastError();
}
template <class T>
hipError_t grad_of(const Args& a, hipStream_t s) {
  hipError_t e = a.dk == 64 ? (a.dv == 64 ? run<T, 64, 64>(a, s) : run<T, 64, 128>(a, s))
                            : (a.dv == 64 ? run<T, 128, 64>(a, s) : run<T, 128, 128>(a, s));
  if (e != hipSuccess || a.dq_part == nullptr || (a.dq == nullptr && a.dk_out == nullptr)) return e;
  group_kernel<T><<<dim3((unsigned)a.n, 2), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grad(const Args& a, bool bf16, hipStream_t stream) {
  if (a.n == 0) return hipSuccess;
  return bf16 ? grad_of<uint16_t>(a, stream) : grad_of<float>(a, stream);
}

}  // namespace delta
}  // namespace vggt3
