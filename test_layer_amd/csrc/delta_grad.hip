// The gradient of the gated delta rule, chunk by chunk, from the state S before each
// chunk and the gradient dS of the state after it (delta_scan.hip). With the forward's
// y, u and the reverse scan's du, x = X^T du, dR = beta . x,
//
//   dV = dR,    dbeta_i = x_i . y_i
//   F = scale D . (dO u^T) (lower),    E = D . (dR u^T) (strictly lower)
//   dQ = scale G . (dO S^T) + F K
//   dK = F^T Q + G_end / G . (u dS^T) - G . (dR S^T) - E K - E^T K
//   dg_t = sum over i >= t of A_i + over j < t of C_j + over i >= t > j of W_ij + G_end <dS, S>
//   A_i = G_i (scale q_i S . dO_i - k_i S . dR_i),  C_j = G_end / G_j  k_j dS . u_j
//   W = B . (dO u^T) - E . (K K^T) (strictly lower)
//
// The last lines: token t's decay is a factor of what crosses it, from the state or a
// token j < t to a token i >= t or the state behind. Every term has it as a factor, so
// dg is right however small the decay makes it. (o_i . dO_i - v_i . dR_i summed over i >= t
// is the same value by terms without that factor, which must cancel: nothing of dg is left
// where e^g is 2^-24.)
//
// A wave has 64 value channels of a chunk and head, 4 neighbours a lane (u, x and the
// row sums), then F and E, then its share of the key channels (dQ, dK). In bf16 all
// fp32 operands are whole, in three parts (in two: 48 views' chunks 803 us for 928, but
// more last bits of dQ and dK differ than an order of sums explains). u and dR change
// from columns by lane to rows by lane through LDS; the triangles stay in registers.
//
// 48 views (65,952 tokens), 16 heads of 64 x 64 in bf16: 888 to 928 us. The wave fills a
// SIMD's registers, so nothing runs while it waits: 39% of its cycles are instructions (33%
// vector), 13% wait to issue behind a product, 48% wait for memory and LDS. S and dS are read
// once by columns and once by rows, and of the second reading half comes from memory again
// (3.2 GB fetched, 2.0 needed; 0.47 written). With operands in two parts, 785 us: turning both
// in LDS instead saves that but took 1070 (its writes and conflicts, and 45 registers spilled),
// asking for the next chunk's lines ahead 950 (the L2 has no room for them), four waves of 16
// columns, which convert each triangle four times over, 1300.
#include <type_traits>

#include "delta_chunk.hpp"

namespace vggt3 {
namespace delta {
namespace {

template <class T, int DK, int DV>
struct GradShared {
  static constexpr int kParts = kWhole<T>;  // of u and dR
  T k[kChunk][kPitch<T, DK>];
  T q[kChunk][kPitch<T, DK>];
  T u[kParts][kChunk][kPitch<T, DV>];
  T dr[kParts][kChunk][kPitch<T, DV>];
  float in[DV / 64][kChunk], out[DV / 64][kChunk], step[DV / 64][kChunk], all[DV / 64];  // A, C, dbeta and <dS, S>
};

// 4 neighbouring values of a row to LDS, split into three parts (bf16).
__device__ __forceinline__ void put_four(uint16_t* to, int part, const float* v) {
  float x[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    const uint32_t a = pack_bf16x2(x[0], x[1]), b = pack_bf16x2(x[2], x[3]);
    st8(to + p * part, u32x2{a, b});
    x[0] = less_lo(x[0], a);
    x[1] = less_hi(x[1], a);
    x[2] = less_lo(x[2], b);
    x[3] = less_hi(x[3], b);
  }
}
__device__ __forceinline__ void put_four(float* to, int, const float* v) {
  *reinterpret_cast<f32x4*>(to) = f32x4{v[0], v[1], v[2], v[3]};
}
template <int PITCH>
__device__ __forceinline__ void row_parts(Frag<uint16_t>& f, const uint16_t* from, int part, int row, int col) {
#pragma unroll
  for (int p = 0; p < 3; ++p) f.part[p] = ld_op(from + p * part + row * PITCH + col);
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

// The sums of a strict triangle's values over i >= t > j, in lanes t < 32: over its columns
// by a product with a triangle of ones, then over its rows.
__device__ __forceinline__ float crossing(const Tri& w, int lane) {
  const int c = lane % 16, q = lane / 16;
  f32x4 before, one;  // j < t, and all j
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    before[r] = 4 * q + r < c ? 1.0f : 0.0f;
    one[r] = 1.0f;
  }
  const f32x4 m00 = mm16(w.t00, before, zero4()), m10 = mm16(w.t10, before, zero4());
  const f32x4 m11 = mm16(w.t11, before, mm16(w.t10, one, zero4()));
  float x = 0.0f, y = 0.0f;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const bool from = 4 * q + r >= c;
    x += (from ? m00[r] : 0.0f) + m10[r];
    y += from ? m11[r] : 0.0f;
  }
#pragma unroll
  for (int off = 16; off < 64; off *= 2) {
    x += __shfl_xor(x, off, 64);
    y += __shfl_xor(y, off, 64);
  }
  return q == 0 ? x : y;
}

// A value that the compiler takes as a new one: what was made of it before is made
// again, instead of being held in registers until then.
__device__ __forceinline__ void anew(uint32_t& x) { asm volatile("" : "+v"(x)); }
__device__ __forceinline__ void anew(f32x4& x) { asm volatile("" : "+v"(x)); }

// Between the waves of a workgroup, or a wave's own LDS accesses.
template <int W>
__device__ __forceinline__ void meet() {
  if constexpr (W == 1)
    wave_lds_order();
  else
    __syncthreads();
}

template <class T, int DK, int DV>
__global__ __launch_bounds__(DV, 1) void grad_kernel(const Args a) {
  using Sh = GradShared<T, DK, DV>;
  constexpr int kW = DV / 64, kP = kWhole<T>, kPV = kPitch<T, DV>, kPK = kPitch<T, DK>, kB = (int)sizeof(T);
  constexpr int kPart = kChunk * kPV, kS = DK / 32;
  __shared__ Sh m;
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int c = lane % 16, q = lane / 16;
  const int h = blockIdx.x % a.hv;
  const int64_t slot = blockIdx.x / a.hv;
  const Piece p = find_piece(a, kChunk, slot, lane);
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
  const int krow = (int)((c * ldk + 8 * q) * kB), knext = (int)(16 * ldk * kB);
  const int orow = (int)((c * ldv + 8 * q) * kB), onext = (int)(16 * ldv * kB);
  const int col = wave * 64 + 4 * c;
  const int voff = (int)((4 * q * ldv + col) * kB), vrow = (int)(ldv * kB);

  Raw<T> kr[2][kS], qr[2][kS];
#pragma unroll
  for (int it = 0; it < 2; ++it)
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      load_raw(kr[it][s], kw, krow + it * knext + 32 * s * kB);
      load_raw(qr[it][s], qw, krow + it * knext + 32 * s * kB);
    }
  f32x4 dec[2], rest[2], beta[2];
#pragma unroll
  for (int it = 0; it < 2; ++it) {
    dec[it] = rows4(mat.rows.decay, it, q);
    rest[it] = rows4(mat.rows.rest, it, q);
    beta[it] = rows4(mat.rows.beta, it, q);
  }
#pragma unroll
  for (int it = 0; it < 2; ++it)
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      if (s % kW != wave) continue;
      put_raw(&m.k[16 * it + c][32 * s + 8 * q], kr[it][s]);
      put_raw(&m.q[16 * it + c][32 * s + 8 * q], qr[it][s]);
    }
  // 128 key channels of them by rows would take 64 registers: they come from LDS again
  constexpr bool kAgain = DK > 64;
  if constexpr (kAgain) meet<kW>();
  const auto rows_of = [&](Frag<T>& f0, Frag<T>& f1, const Raw<T>(*r)[kS], const T* from, int s) {
    if constexpr (!kAgain) {
      as_frag(f0, r[0][s]);
      as_frag(f1, r[1][s]);
    } else {
      row8(f0, from + c * kPK + 32 * s + 8 * q);
      row8(f1, from + (16 + c) * kPK + 32 * s + 8 * q);
    }
  };

  // this wave's value channels: u, then x and dR
  RawN<T, 4> vr[2][4], dr[2][4];
  f32x4 y[2][4], dR[2][4], ks[2][4];  // ks: G . (K S)
  f32x4 in[2] = {zero4(), zero4()}, out[2] = {zero4(), zero4()}, step[2] = {zero4(), zero4()};
  {
    f32x4 qs[2][4];
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int x = 0; x < 4; ++x) ks[it][x] = qs[it][x] = zero4();
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      f32x4 st[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const f32x4 w = *reinterpret_cast<const f32x4*>(S0 + channel(2 * s + i, 4 * q + r) * DV + col);
#pragma unroll
          for (int x = 0; x < 4; ++x) st[i][x][r] = w[x];
        }
      Frag<T> k0, k1, q0, q1;
      rows_of(k0, k1, kr, &m.k[0][0], s);
      rows_of(q0, q1, qr, &m.q[0][0], s);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        Frag<T> f;
        make<kP>(f, st[0][x], st[1][x]);
        ks[0][x] = mm<1, kP>(k0, f, ks[0][x]);
        ks[1][x] = mm<1, kP>(k1, f, ks[1][x]);
        qs[0][x] = mm<1, kP>(q0, f, qs[0][x]);
        qs[1][x] = mm<1, kP>(q1, f, qs[1][x]);
      }
    }
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        load_rawn(vr[it][r], vw, voff + (16 * it + r) * vrow);
        load_rawn(dr[it][r], ow, voff + (16 * it + r) * vrow);
      }
    Frag<T> tf[2];
    lower_rows<kP>(tf, get_tri(mat.t, lane));
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      f32x4 V[2], dO[2];
#pragma unroll
      for (int it = 0; it < 2; ++it)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          V[it][r] = value_of(vr[it][r], x);
          dO[it][r] = value_of(dr[it][r], x);
        }
      Frag<T> f;
      ks[0][x] *= dec[0];
      ks[1][x] *= dec[1];
      make<kP>(f, V[0] - ks[0][x], V[1] - ks[1][x]);
      y[0][x] = mm<kP, kP>(tf[0], f, zero4());
      y[1][x] = mm<kP, kP>(tf[1], f, zero4());
      in[0] += dO[0] * (qs[0][x] * (dec[0] * a.scale));
      in[1] += dO[1] * (qs[1][x] * (dec[1] * a.scale));
    }
  }
#pragma unroll
  for (int it = 0; it < 2; ++it) {
    anew(beta[it]);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < (int)sizeof(T); ++i) anew(dr[it][r].r[i]);
  }
  {
    f32x4 kd[2][4];
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int x = 0; x < 4; ++x) kd[it][x] = zero4();
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      f32x4 ds[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const f32x4 w = *reinterpret_cast<const f32x4*>(S1 + channel(2 * s + i, 4 * q + r) * DV + col);
#pragma unroll
          for (int x = 0; x < 4; ++x) ds[i][x][r] = w[x];
        }
      Frag<T> k0, k1;
      rows_of(k0, k1, kr, &m.k[0][0], s);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        Frag<T> f;
        make<kP>(f, ds[0][x], ds[1][x]);
        kd[0][x] = mm<1, kP>(k0, f, kd[0][x]);
        kd[1][x] = mm<1, kP>(k1, f, kd[1][x]);
      }
    }
    Frag<T> btf[2], xf[2];
    upper_rows<kP>(btf, get_tri(mat.bt, lane));
    upper_rows<kP>(xf, get_tri(mat.x, lane));
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      f32x4 dO[2];
#pragma unroll
      for (int it = 0; it < 2; ++it)
#pragma unroll
        for (int r = 0; r < 4; ++r) dO[it][r] = value_of(dr[it][r], x);
      Frag<T> f;
      make<1>(f, dO[0], dO[1]);
      const f32x4 e0 = kd[0][x] * rest[0], e1 = kd[1][x] * rest[1];
      out[0] += e0 * (y[0][x] * beta[0]);
      out[1] += e1 * (y[1][x] * beta[1]);
      const f32x4 du0 = mm<kP, 1>(btf[0], f, e0), du1 = mm<kP, 1>(btf[1], f, e1);
      make<kP>(f, du0, du1);
      const f32x4 x0 = mm<kP, kP>(xf[0], f, zero4()), x1 = mm<kP, kP>(xf[1], f, zero4());
      step[0] += y[0][x] * x0;
      step[1] += y[1][x] * x1;
      dR[0][x] = x0 * beta[0];
      dR[1][x] = x1 * beta[1];
      in[0] -= ks[0][x] * dR[0][x];
      in[1] -= ks[1][x] * dR[1][x];
    }
  }
  anew(beta[0]);
  anew(beta[1]);
  {
    const Window dw = window<DV>(static_cast<const T*>(a.dv_out) + p.first * ldv + h * DV, ldv, a.dv_out ? len : 0);
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float w[4] = {y[it][0][r] * beta[it][r], y[it][1][r] * beta[it][r], y[it][2][r] * beta[it][r],
                            y[it][3][r] * beta[it][r]};
        const float z[4] = {dR[it][0][r], dR[it][1][r], dR[it][2][r], dR[it][3][r]};
        put_four(&m.u[0][16 * it + 4 * q + r][col], kPart, w);
        put_four(&m.dr[0][16 * it + 4 * q + r][col], kPart, z);
        store_rawn<T, 4>(dw, voff + (16 * it + r) * vrow, z);
      }
  }
#pragma unroll
  for (int it = 0; it < 2; ++it)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float s0 = row_sum(in[it][r]), s1 = row_sum(out[it][r]), s2 = row_sum(step[it][r]);
      if (c == 0) {
        m.in[wave][16 * it + 4 * q + r] = s0;
        m.out[wave][16 * it + 4 * q + r] = s1;
        m.step[wave][16 * it + 4 * q + r] = s2;
      }
    }
  meet<kW>();

  // F = dO u^T and E = dR u^T, with rows by lane (as F, -E) and columns by lane (F^T, -E^T)
  Frag<T> ff[2], ft[2], ef[2], et[2];
  float between = 0.0f;  // lane t < 32: W's sum over i >= t > j
  const auto triangles = [&]() {
    Tri f{zero4(), zero4(), zero4()}, g = f, e = f, d = f;
#pragma unroll
    for (int s = 0; s < DV / 32; ++s) {
      Frag<T> r0, r1, u0, u1, o0, o1;
      const int at = 32 * s + 8 * q;
      row_parts<kPV>(u0, &m.u[0][0][0], kPart, c, at);
      row_parts<kPV>(u1, &m.u[0][0][0], kPart, 16 + c, at);
      row_parts<kPV>(r0, &m.dr[0][0][0], kPart, c, at);
      row_parts<kPV>(r1, &m.dr[0][0][0], kPart, 16 + c, at);
      Raw<T> w0, w1;
      load_raw(w0, ow, orow + 32 * s * kB);
      load_raw(w1, ow, orow + onext + 32 * s * kB);
      as_frag(o0, w0);
      as_frag(o1, w1);
      f.t00 = mm<kP, 1>(u0, o0, f.t00);
      f.t10 = mm<kP, 1>(u0, o1, f.t10);
      f.t11 = mm<kP, 1>(u1, o1, f.t11);
      g.t00 = mm<1, kP>(o0, u0, g.t00);
      g.t10 = mm<1, kP>(o1, u0, g.t10);
      g.t11 = mm<1, kP>(o1, u1, g.t11);
      e.t00 = mm<kP, kP>(u0, r0, e.t00);
      e.t10 = mm<kP, kP>(u0, r1, e.t10);
      e.t11 = mm<kP, kP>(u1, r1, e.t11);
      d.t00 = mm<kP, kP>(r0, u0, d.t00);
      d.t10 = mm<kP, kP>(r1, u0, d.t10);
      d.t11 = mm<kP, kP>(r1, u1, d.t11);
    }
    Tri w = decays<false>(mat.rows, lane);
    e = lower<false, true>(e * w, lane);
    {
      Tri kk{zero4(), zero4(), zero4()};
#pragma unroll
      for (int s = 0; s < kS; ++s) {
        Frag<T> k0, k1;
        row8(k0, &m.k[c][32 * s + 8 * q]);
        row8(k1, &m.k[16 + c][32 * s + 8 * q]);
        kk.t00 = mm<1, 1>(k0, k0, kk.t00);
        kk.t10 = mm<1, 1>(k0, k1, kk.t10);
        kk.t11 = mm<1, 1>(k1, k1, kk.t11);
      }
      kk = e * kk;
      const Tri o = lower<false, true>(f * get_tri(mat.b, lane), lane);
      between = crossing(Tri{o.t00 - kk.t00, o.t10 - kk.t10, o.t11 - kk.t11}, lane);
    }
    const f32x4 one = {1.0f, 1.0f, 1.0f, 1.0f}, sc = one * a.scale;
    f = lower<false, false>(f * w, lane);
    lower_rows<kP>(ff, f * Tri{sc, sc, sc});
    lower_rows<kP>(ef, e * Tri{-one, -one, -one});
    w = decays<true>(mat.rows, lane);
    d = lower<true, true>(d * w, lane);
    g = lower<true, false>(g * w, lane);
    upper_rows<kP>(ft, g * Tri{sc, sc, sc});
    upper_rows<kP>(et, d * Tri{-one, -one, -one});
  };

  // this wave's key channels, kN neighbours a lane at a time
  constexpr int kEach = DK / kW, kN = kEach / 16 < 4 ? kEach / 16 : 4;
  float apart = 0.0f;  // <dS, S before the chunk>, by rows
  f32x4 dq[2][kN], dk[2][kN];
  // what S and dS have of them
  const auto by_states = [&](int base) {
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int x = 0; x < kN; ++x) dq[it][x] = dk[it][x] = zero4();
    const int row = (base + kN * c) * DV + 8 * q;
    const auto eight = [&](f32x4* w, const float* from, int x, int s) {
      const float* at = from + row + x * DV + 32 * s;
      w[0] = *reinterpret_cast<const f32x4*>(at);
      w[1] = *reinterpret_cast<const f32x4*>(at + 4);
    };
#pragma unroll
    for (int s = 0; s < DV / 32; ++s) {
      Frag<T> o[2], r[2];
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        Raw<T> w;
        load_raw(w, ow, orow + it * onext + 32 * s * kB);
        as_frag(o[it], w);
        row_parts<kPV>(r[it], &m.dr[0][0][0], kPart, 16 * it + c, 32 * s + 8 * q);
      }
#pragma unroll
      for (int x = 0; x < kN; ++x) {
        f32x4 w[2];
        eight(w, S0, x, s);
        Frag<T> f;
        make<kP>(f, w[0], w[1]);
#pragma unroll
        for (int it = 0; it < 2; ++it) {
          dq[it][x] = mm<1, kP>(o[it], f, dq[it][x]);
          dk[it][x] = mm<kP, kP>(r[it], f, dk[it][x]);
        }
      }
    }
    f32x4 us[2][kN];
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int x = 0; x < kN; ++x) us[it][x] = zero4();
#pragma unroll
    for (int s = 0; s < DV / 32; ++s) {
      Frag<T> u[2];
#pragma unroll
      for (int it = 0; it < 2; ++it) row_parts<kPV>(u[it], &m.u[0][0][0], kPart, 16 * it + c, 32 * s + 8 * q);
#pragma unroll
      for (int x = 0; x < kN; ++x) {
        f32x4 w[2], z[2];
        eight(w, S1, x, s);
        eight(z, S0, x, s);
#pragma unroll
        for (int r = 0; r < 4; ++r) apart += w[0][r] * z[0][r] + w[1][r] * z[1][r];
        Frag<T> f;
        make<kP>(f, w[0], w[1]);
#pragma unroll
        for (int it = 0; it < 2; ++it) us[it][x] = mm<kP, kP>(u[it], f, us[it][x]);
      }
    }
#pragma unroll
    for (int x = 0; x < kN; ++x)
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        dq[it][x] *= dec[it] * a.scale;
        dk[it][x] = us[it][x] * rest[it] - dk[it][x] * dec[it];
      }
  };
  // what the chunk's own keys and queries have
  const auto by_tokens = [&](int base) {
#pragma unroll
    for (int x = 0; x < kN; ++x) {
      Frag<T> kc, qc;
      token_columns<kN, kPK>(kc, &m.k[0][0], base, x, lane);
      token_columns<kN, kPK>(qc, &m.q[0][0], base, x, lane);
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        dq[it][x] = mm<kP, 1>(ff[it], kc, dq[it][x]);
        dk[it][x] = mm<kP, 1>(ft[it], qc, dk[it][x]);
        dk[it][x] = mm<kP, 1>(ef[it], kc, dk[it][x]);
        dk[it][x] = mm<kP, 1>(et[it], kc, dk[it][x]);
      }
    }
    const auto store = [&](auto* to, int64_t ld, const f32x4(*v)[kN]) {
      using U = std::remove_pointer_t<decltype(to)>;
      const Window w = window<DK>(to, ld, len);
      const int off = (int)((4 * q * ld + base + kN * c) * (int)sizeof(U)), next = (int)(ld * (int)sizeof(U));
#pragma unroll
      for (int it = 0; it < 2; ++it)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float z[kN];
#pragma unroll
          for (int x = 0; x < kN; ++x) z[x] = v[it][x][r];
          store_rawn<U, kN>(w, off + (16 * it + r) * next, z);
        }
    };
    if (a.dq_part) {
      store(a.dq_part + (p.first * a.hv + h) * DK, (int64_t)a.hv * DK, dq);
      store(a.dk_part + (p.first * a.hv + h) * DK, (int64_t)a.hv * DK, dk);
    } else {
      if (a.dq) store(static_cast<T*>(a.dq) + p.first * ldk + kh * DK, ldk, dq);
      if (a.dk_out) store(static_cast<T*>(a.dk_out) + p.first * ldk + kh * DK, ldk, dk);
    }
  };
  triangles();
#pragma unroll 1
  for (int base = wave * kEach; base < (wave + 1) * kEach; base += 16 * kN) {
    by_states(base);
    by_tokens(base);
  }
  apart = wave_sum(apart * mat.rows.total);
  if (lane == 0) m.all[wave] = apart;
  meet<kW>();
  if (wave == 0 && lane < kChunk) {
    float x = 0.0f, y = 0.0f, s = 0.0f, all = 0.0f;
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      x += m.in[w][lane];
      y += m.out[w][lane];
      s += m.step[w][lane];
      all += m.all[w];
    }
    // A from each token on, C before it
#pragma unroll
    for (int off = 1; off < kChunk; off *= 2) {
      const float down = __shfl_down(x, off, 32), up = __shfl_up(y, off, 32);
      if (lane + off < kChunk) x += down;
      if (lane >= off) y += up;
    }
    y = __shfl_up(y, 1, 32);
    if (lane == 0) y = 0.0f;
    if (lane < len) {
      if (a.dg) a.dg[(p.first + lane) * a.hv + h] = (x + y) + (between + all);
      if (a.dbeta) a.dbeta[(p.first + lane) * a.hv + h] = s;
    }
  }
}

// dq, dk of key heads that several value heads share, in the heads' order, a chunk's rows
// a workgroup. Rows of no sequence are of no chunk.
template <class T>
__global__ __launch_bounds__(256) void group_kernel(const Args a) {
  const Piece p = find_piece(a, kChunk, blockIdx.x, threadIdx.x % 64);
  const int group = a.hv / a.hk, width = a.hk * a.dk;
  const float* from = blockIdx.y ? a.dk_part : a.dq_part;
  T* to = static_cast<T*>(blockIdx.y ? a.dk_out : a.dq);
  if (p.seg < 0 || to == nullptr) return;
  for (int at = 4 * threadIdx.x; at < p.len * width; at += 1024) {
    const int64_t row = p.first + at / width;
    const int i = at % width, kh = i / a.dk, ch = i % a.dk;
    f32x4 s = zero4();
    for (int g = 0; g < group; ++g)
      s += *reinterpret_cast<const f32x4*>(from + (row * a.hv + kh * group + g) * a.dk + ch);
    const float w[4] = {s[0], s[1], s[2], s[3]};
    store_n<4>(to + row * width + i, w);
  }
}

template <class T, int DK, int DV>
hipError_t run(const Args& a, hipStream_t s) {
  grad_kernel<T, DK, DV><<<(unsigned)(chunk_slots(a.n, a.nseq) * a.hv), DV, 0, s>>>(a);
  return hipGetLastError();
}
template <class T>
hipError_t grad_of(const Args& a, hipStream_t s) {
  hipError_t e = a.dk == 64 ? (a.dv == 64 ? run<T, 64, 64>(a, s) : run<T, 64, 128>(a, s))
                            : (a.dv == 64 ? run<T, 128, 64>(a, s) : run<T, 128, 128>(a, s));
  if (e != hipSuccess || a.dq_part == nullptr || (a.dq == nullptr && a.dk_out == nullptr)) return e;
  group_kernel<T><<<dim3((unsigned)chunk_slots(a.n, a.nseq), 2), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grad(const Args& a, bool bf16, hipStream_t stream) {
  if (a.n == 0) return hipSuccess;
  return bf16 ? grad_of<uint16_t>(a, stream) : grad_of<float>(a, stream);
}

}  // namespace delta
}  // namespace vggt3
