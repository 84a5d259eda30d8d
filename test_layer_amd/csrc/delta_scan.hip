// The gated delta rule over whole sequences.
//
//   p_t = a_t S_{t-1}^T k_t,  u_t = beta_t (v_t - p_t),  S_t = a_t S_{t-1} + k_t u_t^T,  o_t = scale S_t^T q_t
//
// by chunks of 32 tokens. With G_i the chunk's decay up to token i, D_ij = G_i / G_j
// and S the state before the chunk,
//
//   N' = strict lower triangle of D . (K K^T),    T = (I + N' beta)^-1
//   y = T (V - G . (K S)),  u = beta . y
//   O = scale (G . (Q S) + (lower triangle of D . (Q K^T)) u)
//   S <- G_end S + K^T (G_end / G . u)
//
// A column of S, and of everything that u and O are made of, depends on no other
// column. So a wave keeps NCT tiles of 16 columns of S in registers over its whole
// piece of a sequence, and the products chain through its registers (delta_ops.hpp).
// T and the triangle of Q K^T, which all columns share and no state enters, are formed
// beforehand for all chunks at once (matrices_kernel) and read as operands. A wave
// works by itself: it asks for the next chunk's rows and operands while it computes,
// and passes K alone through LDS, for its transpose.
//
// Long sequences are cut into pieces that are worked on at once: a first pass finds
// what each piece makes of its first state (M S + R: the columns of M are those of
// a value-free run that starts from the unit matrix), join_kernel goes through the
// pieces, and the main pass starts each piece from its own first state. (A
// sequence's first piece starts from the sequence's first state in both passes.)
//
// 100 views (137,400 tokens) as one sequence, 16 heads of 64 x 64 in bf16: 179 to 202 us
// for the matrices (1.1 GB: memory), 453 to 541 for the summary, 52 for the join, 367 to
// 427 for the main pass. One wave a SIMD, whose registers 64 columns of S fill, so a wave's
// waiting is the SIMD's. Its cycles, by counters: 59% (main pass) and 65% (summary) vector
// instructions, most of which cut fp32 values into 3 bf16 parts before each product, 6 and 7%
// others, 24 and 20% waiting to issue behind a product that is not done, 11 and 8% waiting for
// memory and LDS. (48 views' states: 54, 6, 16 and 24%, on 768 waves for 1024 SIMDs.) Two
// waves a SIMD of 32 columns, interleaved products, or S held in parts were not faster.
#include "delta_chunk.hpp"

namespace vggt3 {
namespace delta {
namespace {

// One wave to a chunk and head: its shared matrices. KEEP: those of the gradient too.
template <class T, int DK, bool KEEP>
__global__ __launch_bounds__(256) void matrices_kernel(const Args a) {
  __shared__ float scratch[4][2 * 16 * 20];
  __shared__ Rows gates[4];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int c = lane % 16, q = lane / 16;
  const uint32_t id = blockIdx.x * 4 + wave, slot = id / a.hv;
  const int h = (int)(id % a.hv);
  const Piece p = find_piece(a, kChunk, slot, lane);
  if (p.seg < 0 || p.len == 0) return;
  const int64_t ld = (int64_t)a.hk * DK;
  const int64_t at = p.first * ld + h / (a.hv / a.hk) * DK;
  const Window kw = window<DK>(static_cast<const T*>(a.k) + at, ld, p.len);
  const Window qw = window<DK>(static_cast<const T*>(a.q) + at, ld, p.len);
  const int off = (int)((c * ld + 8 * q) * (int)sizeof(T)), next = (int)(16 * ld * (int)sizeof(T));
  Raw<T> kr[2][DK / 32], qr[2][DK / 32];
#pragma unroll
  for (int s = 0; s < DK / 32; ++s)
#pragma unroll
    for (int it = 0; it < 2; ++it) {
      load_raw(kr[it][s], kw, off + it * next + 32 * s * (int)sizeof(T));
      load_raw(qr[it][s], qw, off + it * next + 32 * s * (int)sizeof(T));
    }
  Rows& rows = gates[wave];
  put_rows(rows, a, p.first, p.len, h, lane);
  // keys as a tile's rows: N' and Q K^T with rows by lane
  Tri n{zero4(), zero4(), zero4()}, b = n;
#pragma unroll
  for (int s = 0; s < DK / 32; ++s) {
    Frag<T> k0, k1, q0, q1;
    as_frag(k0, kr[0][s]);
    as_frag(k1, kr[1][s]);
    as_frag(q0, qr[0][s]);
    as_frag(q1, qr[1][s]);
    n.t00 = mm<1, 1>(k0, k0, n.t00);
    n.t10 = mm<1, 1>(k0, k1, n.t10);
    n.t11 = mm<1, 1>(k1, k1, n.t11);
    b.t00 = mm<1, 1>(k0, q0, b.t00);
    b.t10 = mm<1, 1>(k0, q1, b.t10);
    b.t11 = mm<1, 1>(k1, q1, b.t11);
  }
  wave_lds_order();
  const Tri d = decays<false>(rows, lane);
  n = lower<false, true>(n * d, lane);
  b = lower<false, false>(b * d, lane);
  b.t00 *= a.scale;
  b.t10 *= a.scale;
  b.t11 *= a.scale;
  const f32x4 b0 = rows4(rows.beta, 0, q), b1 = rows4(rows.beta, 1, q);
  Tri t;
  unit_inverse(n.t00 * b0, n.t10 * b0, n.t11 * b1, t.t00, t.t10, t.t11, scratch[wave], lane);
  Matrices* m = matrices_of(a.mats, (int64_t)slot * a.hv + h, KEEP);
  put_tri(m->t, t, lane);
  put_tri(m->b, b, lane);
  if constexpr (KEEP) {
    put_tri(m->bt, turned(b, lane), lane);
    // X = (I + beta N')^-1 = I - beta (T N'): one inverse serves both sides' scaling
    n = turned(n, lane);
    f32x4 one;
#pragma unroll
    for (int r = 0; r < 4; ++r) one[r] = 4 * q + r == c ? 1.0f : 0.0f;
    Tri x;
    x.t00 = one - b0 * mm16(t.t00, n.t00, zero4());
    x.t10 = -b1 * mm16(t.t11, n.t10, mm16(t.t10, n.t00, zero4()));
    x.t11 = one - b1 * mm16(t.t11, n.t11, zero4());
    put_tri(m->x, x, lane);
  }
  const float* from = reinterpret_cast<const float*>(&rows);
  float* to = reinterpret_cast<float*>(&m->rows);
#pragma unroll
  for (int i = lane; i < (int)(sizeof(Rows) / 4); i += 64) to[i] = from[i];
}

// kStates: the state before every chunk, for the gradient (no outputs).
enum Mode { kForward, kSummary, kStates };

// What a wave has of a chunk before it computes.
template <class T, int DK, int NCT, Mode MODE>
struct Loaded {
  Raw<T> k[2][DK / 32], q[MODE == kForward ? 2 : 0][DK / 32];
  RawN<T, NCT> v[2][4];
  f32x4 t[3], b[3];
  f32x4 decay[2], rest[2], beta[2];
  float total;
};

template <class T, int DK, int DV, int NCT, Mode MODE>
__global__ __launch_bounds__(64 * (4 / NCT), DK * NCT <= 64 ? 2 : 1) void scan_kernel(const Args a) {
  constexpr int kTiles = DK / 16, kSteps = DK / 32, kP = kWhole<T>, kW = 4 / NCT, kB = (int)sizeof(T);
  // The next chunk's rows into the registers that this one's leave, half a chunk ahead, or
  // whole chunks in two sets by turns: the one is half the code and registers (48 views'
  // states 256 us, 261 by turns; 24 views in fp32 220 + 201, 224 + 206), the other further
  // ahead (a scene's two passes in bf16 538 + 388 us, 574 + 416 in one set).
  constexpr bool kOnce = sizeof(T) == 4 || MODE == kStates;
  __shared__ T ks_rows[kW][kChunk * kPitch<T, DK>];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int c = lane % 16, q = lane / 16;
  const int h = blockIdx.x % a.hv;
  const int64_t sid = blockIdx.x / a.hv;
  const Piece p = find_piece(a, a.per, sid, lane);
  if (p.seg < 0) return;
  if (MODE == kSummary && p.seg == p.segs - 1) return;  // nothing follows it
  // this lane's columns: NCT neighbours
  const int col0 = blockIdx.y * 64 + wave * 16 * NCT, col = col0 + NCT * c;
  const bool unit = MODE == kSummary && blockIdx.y * 64 >= DV;
  if (unit && p.seg == 0) return;  // its first state is known
  T* const kt_rows = ks_rows[wave];

  f32x4 S[kTiles][NCT];
  if (unit) {
    unit_state<DK, NCT>(S, col - DV, q);
  } else {
    const float* from = nullptr;
    if (MODE != kSummary && p.segs > 1)
      from = a.seg_n + (sid * a.hv + h) * DK * DV + col;
    else if (a.state && p.seg == 0)
      from = a.state + ((int64_t)p.b * a.hv + h) * DK * DV + col;
    load_state<DK, NCT>(S, from, DV, q);
  }

  const int64_t ldq = (int64_t)a.hk * DK, ldv = (int64_t)a.hv * DV;
  const int kh = h / (a.hv / a.hk);
  const int chunks = (p.len + kChunk - 1) / kChunk;
  const int64_t slot0 = p.slot;
  const int koff = (int)((c * ldq + 8 * q) * kB), knext = (int)(16 * ldq * kB);
  const int voff = (int)((4 * q * ldv + NCT * c) * kB), vrow = (int)(ldv * kB);

  typedef Loaded<T, DK, NCT, MODE> L;
  const auto load_keys = [&](L& x, int i) {
    const int64_t first = p.first + (int64_t)i * kChunk;
    const int len = min(kChunk, p.len - i * kChunk);
    const Window kw = window<DK>(static_cast<const T*>(a.k) + first * ldq + kh * DK, ldq, len);
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int s = 0; s < kSteps; ++s) load_raw(x.k[it][s], kw, koff + it * knext + 32 * s * kB);
    if constexpr (MODE == kForward) {
      const Window qw = window<DK>(static_cast<const T*>(a.q) + first * ldq + kh * DK, ldq, len);
#pragma unroll
      for (int it = 0; it < 2; ++it)
#pragma unroll
        for (int s = 0; s < kSteps; ++s) load_raw(x.q[it][s], qw, koff + it * knext + 32 * s * kB);
    }
  };
  const auto load_rest = [&](L& x, int i) {
    const int64_t first = p.first + (int64_t)i * kChunk;
    const int len = min(kChunk, p.len - i * kChunk);
    const Window vw = window<16 * NCT>(static_cast<const T*>(a.v) + first * ldv + h * DV + (unit ? 0 : col0), ldv,
                                       unit ? 0 : len);
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int r = 0; r < 4; ++r) load_rawn(x.v[it][r], vw, voff + (16 * it + r) * vrow);
    const Matrices* m = matrices_of(a.mats, (slot0 + i) * a.hv + h, a.keep);
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      x.t[j] = m->t[j][lane];
      if constexpr (MODE == kForward) x.b[j] = m->b[j][lane];
    }
#pragma unroll
    for (int it = 0; it < 2; ++it) {
      x.decay[it] = rows4(m->rows.decay, it, q);
      x.rest[it] = rows4(m->rows.rest, it, q);
      x.beta[it] = rows4(m->rows.beta, it, q);
    }
    x.total = m->rows.total;
  };
  const auto load = [&](L& x, int i) {
    load_keys(x, i);
    load_rest(x, i);
  };
  const auto compute = [&](L& x, int i) {
    const int next = min(i + 1, chunks - 1);
    if constexpr (MODE == kStates)
      store_state<DK, NCT>(S, a.states + ((slot0 + i) * a.hv + h) * DK * DV + col, DV, q);
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int s = 0; s < kSteps; ++s) put_raw(kt_rows + (16 * it + c) * kPitch<T, DK> + 32 * s + 8 * q, x.k[it][s]);
    f32x4 ks[2][NCT], o[2][NCT];
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int y = 0; y < NCT; ++y) ks[it][y] = o[it][y] = zero4();
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      Frag<T> k0, k1, q0, q1;
      as_frag(k0, x.k[0][s]);
      as_frag(k1, x.k[1][s]);
      if constexpr (MODE == kForward) {
        as_frag(q0, x.q[0][s]);
        as_frag(q1, x.q[1][s]);
      }
#pragma unroll
      for (int y = 0; y < NCT; ++y) {
        Frag<T> f;
        make<kP>(f, S[2 * s][y], S[2 * s + 1][y]);
        ks[0][y] = mm<1, kP>(k0, f, ks[0][y]);
        ks[1][y] = mm<1, kP>(k1, f, ks[1][y]);
        if constexpr (MODE == kForward) {
          o[0][y] = mm<1, kP>(q0, f, o[0][y]);
          o[1][y] = mm<1, kP>(q1, f, o[1][y]);
        }
      }
    }
    if constexpr (kOnce) load_keys(x, next);
    Frag<T> t0, t1, b0, b1;
    make<kP>(t0, x.t[0], zero4());
    make<kP>(t1, x.t[1], x.t[2]);
    if constexpr (MODE == kForward) {
      make<kP>(b0, x.b[0], zero4());
      make<kP>(b1, x.b[1], x.b[2]);
    }
    Frag<T> uf[NCT];
#pragma unroll
    for (int y = 0; y < NCT; ++y) {
      f32x4 R[2];
#pragma unroll
      for (int it = 0; it < 2; ++it)
#pragma unroll
        for (int r = 0; r < 4; ++r) R[it][r] = value_of(x.v[it][r], y) - x.decay[it][r] * ks[it][y][r];
      Frag<T> f;
      make<kP>(f, R[0], R[1]);
      const f32x4 u0 = mm<kP, kP>(t0, f, zero4()) * x.beta[0], u1 = mm<kP, kP>(t1, f, zero4()) * x.beta[1];
      if constexpr (MODE == kForward) {
        make<kP>(f, u0, u1);
        o[0][y] = mm<kP, kP>(b0, f, o[0][y] * (x.decay[0] * a.scale));
        o[1][y] = mm<kP, kP>(b1, f, o[1][y] * (x.decay[1] * a.scale));
      }
      make<kP>(uf[y], u0 * x.rest[0], u1 * x.rest[1]);
    }
    const float total = x.total;
    if constexpr (kOnce) load_rest(x, next);
    wave_lds_order();
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      Frag<T> kt;
      state_rows<kPitch<T, DK>>(kt, (const T*)kt_rows, t, lane);
#pragma unroll
      for (int y = 0; y < NCT; ++y) S[t][y] = mm<1, kP>(kt, uf[y], S[t][y] * total);
    }
    wave_lds_order();
    if constexpr (MODE == kForward) {
      const int64_t first = p.first + (int64_t)i * kChunk;
      const Window ow = window<16 * NCT>(static_cast<const T*>(a.o) + first * ldv + h * DV + col0, ldv,
                                         min(kChunk, p.len - i * kChunk));
#pragma unroll
      for (int it = 0; it < 2; ++it)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float w[NCT];
#pragma unroll
          for (int y = 0; y < NCT; ++y) w[y] = o[it][y][r];
          store_rawn<T, NCT>(ow, voff + (16 * it + r) * vrow, w);
        }
    }
  };
  if (kOnce && chunks > 0) {
    L x;
    load(x, 0);
    for (int i = 0; i < chunks; ++i) compute(x, i);
  } else if (chunks > 0) {
    L x, y;
    load(x, 0);
    for (int i = 0; i < chunks; i += 2) {
      load(y, min(i + 1, chunks - 1));
      compute(x, i);
      if (i + 1 >= chunks) break;
      load(x, min(i + 2, chunks - 1));
      compute(y, i + 1);
    }
  }

  if constexpr (MODE == kForward) {
    if (a.state_out && p.seg == p.segs - 1)
      store_state<DK, NCT>(S, a.state_out + ((int64_t)p.b * a.hv + h) * DK * DV + col, DV, q);
  } else if constexpr (MODE == kSummary) {
    if (unit)
      store_state<DK, NCT>(S, a.seg_m + (sid * a.hv + h) * DK * DK + col - DV, DK, q);
    else
      store_state<DK, NCT>(S, a.seg_n + (sid * a.hv + h) * DK * DV + col, DV, q);
  }
}

// The reverse of the scan, for the gradient. With dS the gradient of the state after a
// chunk,
//
//   du = B^T dO + G_end / G . (K dS),  dR = beta . X^T du  (the gradient of V),
//   dS <- G_end dS + Q^T (scale G . dO) - K^T (G . dR)
//
// with B = scale D . Q K^T (lower) and X = (I + beta N')^-1,
//
// by the same columns, with dS in the registers. kBack: dS after every chunk is
// stored; kBackSummary: what a piece makes of the dS behind it.
enum BackMode { kBack, kBackSummary };

template <class T, int DK, int NCT>
struct BackLoaded {
  Raw<T> k[2][DK / 32], q[2][DK / 32];
  RawN<T, NCT> d[2][4];
  f32x4 xt[3], bt[3];
  f32x4 decay[2], rest[2], beta[2];
  float total;
};

template <class T, int DK, int DV, int NCT, BackMode MODE>
__global__ __launch_bounds__(64 * (4 / NCT), DK * NCT <= 64 ? 2 : 1) void back_kernel(const Args a) {
  constexpr int kTiles = DK / 16, kSteps = DK / 32, kP = kWhole<T>, kW = 4 / NCT, kB = (int)sizeof(T);
  __shared__ T rows[kW][2][kChunk * kPitch<T, DK>];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int c = lane % 16, q = lane / 16;
  const int h = blockIdx.x % a.hv;
  const int64_t sid = blockIdx.x / a.hv;
  const Piece p = find_piece(a, a.per, sid, lane);
  if (p.seg < 0) return;
  if (MODE == kBackSummary && p.seg == 0) return;  // nothing lies before it
  const int col0 = blockIdx.y * 64 + wave * 16 * NCT, col = col0 + NCT * c;
  const bool unit = MODE == kBackSummary && blockIdx.y * 64 >= DV;
  if (unit && p.seg == p.segs - 1) return;  // the dS behind it is known
  T* const kt_rows = rows[wave][0];
  T* const qt_rows = rows[wave][1];

  f32x4 S[kTiles][NCT];
  if (unit) {
    unit_state<DK, NCT>(S, col - DV, q);
  } else {
    const float* from = nullptr;
    if (MODE == kBack && p.segs > 1)
      from = a.seg_n + (sid * a.hv + h) * DK * DV + col;
    else if (a.dlast && p.seg == p.segs - 1)
      from = a.dlast + ((int64_t)p.b * a.hv + h) * DK * DV + col;
    load_state<DK, NCT>(S, from, DV, q);
  }

  const int64_t ldq = (int64_t)a.hk * DK, ldv = (int64_t)a.hv * DV;
  const int kh = h / (a.hv / a.hk);
  const int chunks = (p.len + kChunk - 1) / kChunk;
  const int64_t slot0 = p.slot;
  const int koff = (int)((c * ldq + 8 * q) * kB), knext = (int)(16 * ldq * kB);
  const int voff = (int)((4 * q * ldv + NCT * c) * kB), vrow = (int)(ldv * kB);

  typedef BackLoaded<T, DK, NCT> L;
  const auto load_keys = [&](L& x, int i) {
    const int64_t first = p.first + (int64_t)i * kChunk;
    const int len = min(kChunk, p.len - i * kChunk);
    const Window kw = window<DK>(static_cast<const T*>(a.k) + first * ldq + kh * DK, ldq, len);
    const Window qw = window<DK>(static_cast<const T*>(a.q) + first * ldq + kh * DK, ldq, len);
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        load_raw(x.k[it][s], kw, koff + it * knext + 32 * s * kB);
        load_raw(x.q[it][s], qw, koff + it * knext + 32 * s * kB);
      }
  };
  const auto load_rest = [&](L& x, int i) {
    const int64_t first = p.first + (int64_t)i * kChunk;
    const int len = min(kChunk, p.len - i * kChunk);
    const Window dw = window<16 * NCT>(static_cast<const T*>(a.dout) + first * ldv + h * DV + (unit ? 0 : col0), ldv,
                                       unit ? 0 : len);
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int r = 0; r < 4; ++r) load_rawn(x.d[it][r], dw, voff + (16 * it + r) * vrow);
    const Matrices* m = matrices_of(a.mats, (slot0 + i) * a.hv + h, true);
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      x.xt[j] = m->x[j][lane];
      x.bt[j] = m->bt[j][lane];
    }
#pragma unroll
    for (int it = 0; it < 2; ++it) {
      x.decay[it] = rows4(m->rows.decay, it, q);
      x.rest[it] = rows4(m->rows.rest, it, q);
      x.beta[it] = rows4(m->rows.beta, it, q);
    }
    x.total = m->rows.total;
  };
  const auto compute = [&](L& x, int i) {
    const int next = max(i - 1, 0);
    if constexpr (MODE == kBack)
      store_state<DK, NCT>(S, a.dstates + ((slot0 + i) * a.hv + h) * DK * DV + col, DV, q);
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        put_raw(kt_rows + (16 * it + c) * kPitch<T, DK> + 32 * s + 8 * q, x.k[it][s]);
        put_raw(qt_rows + (16 * it + c) * kPitch<T, DK> + 32 * s + 8 * q, x.q[it][s]);
      }
    f32x4 kd[2][NCT];
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int y = 0; y < NCT; ++y) kd[it][y] = zero4();
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      Frag<T> k0, k1;
      as_frag(k0, x.k[0][s]);
      as_frag(k1, x.k[1][s]);
#pragma unroll
      for (int y = 0; y < NCT; ++y) {
        Frag<T> f;
        make<kP>(f, S[2 * s][y], S[2 * s + 1][y]);
        kd[0][y] = mm<1, kP>(k0, f, kd[0][y]);
        kd[1][y] = mm<1, kP>(k1, f, kd[1][y]);
      }
    }
    load_keys(x, next);
    Frag<T> t0, t1, b0, b1;
    make<kP>(t0, x.xt[0], x.xt[1]);
    make<kP>(t1, zero4(), x.xt[2]);
    make<kP>(b0, x.bt[0], x.bt[1]);
    make<kP>(b1, zero4(), x.bt[2]);
    Frag<T> df[NCT], rf[NCT];
#pragma unroll
    for (int y = 0; y < NCT; ++y) {
      f32x4 dO[2];
#pragma unroll
      for (int it = 0; it < 2; ++it)
#pragma unroll
        for (int r = 0; r < 4; ++r) dO[it][r] = value_of(x.d[it][r], y);
      Frag<T> f;
      make<1>(f, dO[0], dO[1]);
      const f32x4 du0 = mm<kP, 1>(b0, f, kd[0][y] * x.rest[0]), du1 = mm<kP, 1>(b1, f, kd[1][y] * x.rest[1]);
      make<kP>(f, du0, du1);
      const f32x4 dR0 = mm<kP, kP>(t0, f, zero4()) * x.beta[0], dR1 = mm<kP, kP>(t1, f, zero4()) * x.beta[1];
      make<kP>(df[y], dO[0] * (x.decay[0] * a.scale), dO[1] * (x.decay[1] * a.scale));
      make<kP>(rf[y], -dR0 * x.decay[0], -dR1 * x.decay[1]);
    }
    const float total = x.total;
    load_rest(x, next);
    wave_lds_order();
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      Frag<T> kt, qt;
      state_rows<kPitch<T, DK>>(kt, (const T*)kt_rows, t, lane);
      state_rows<kPitch<T, DK>>(qt, (const T*)qt_rows, t, lane);
#pragma unroll
      for (int y = 0; y < NCT; ++y) S[t][y] = mm<1, kP>(kt, rf[y], mm<1, kP>(qt, df[y], S[t][y] * total));
    }
    wave_lds_order();
  };
  // the next chunk's rows into the registers that this one's leave (one view in fp32 26 +
  // 18 us; by turns in two sets, with twice the code for the first to read, 33 + 31)
  if (chunks > 0) {
    L x;
    load_keys(x, chunks - 1);
    load_rest(x, chunks - 1);
    for (int i = chunks - 1; i >= 0; --i) compute(x, i);
  }

  if constexpr (MODE == kBack) {
    if (a.dfirst && p.seg == 0)
      store_state<DK, NCT>(S, a.dfirst + ((int64_t)p.b * a.hv + h) * DK * DV + col, DV, q);
  } else {
    if (unit)
      store_state<DK, NCT>(S, a.seg_m + (sid * a.hv + h) * DK * DK + col - DV, DK, q);
    else
      store_state<DK, NCT>(S, a.seg_n + (sid * a.hv + h) * DK * DV + col, DV, q);
  }
}

// First states of a sequence's pieces, in seg_n's place: S <- M S + R from piece to
// piece (BACK: from the last piece to the first). One step waits for the one before, so
// it is cut short: DK / 16 waves share 16 columns, a wave has 16 rows of the products
// (in fp32 for both types: they are few) and its rows of the next 2 pieces' M and R at
// hand, and the new S goes round through LDS. 64 pieces 53 us, 15 pieces 10.7 (4 at
// hand: 54 and 12), most of it the 16 products one after the other.
template <int DK, int DV, bool BACK>
__global__ __launch_bounds__(4 * DK) void join_kernel(const Args a) {
  constexpr int kSteps = DK / 32, kAhead = 2;
  __shared__ f32x4 rows[2][DK / 16][64];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int c = lane % 16, q = lane / 16;
  const int h = blockIdx.x % a.hv, b = blockIdx.x / a.hv;
  const int col = blockIdx.y * 16 + c;
  const Sequence seq = sequence(a, (uint32_t)a.per, b, lane);
  const int segs = (int)pieces_of(seq.begin, seq.end, (uint32_t)a.per);
  const int64_t sid = seq.piece;
  if (segs < 2 || sid + segs > a.pieces) return;
  const float* from = BACK ? a.dlast : a.state;
  const int64_t own = (int64_t)channel(wave, 4 * q) * DV + col;  // its 4 rows are neighbours
  const int64_t mine = (int64_t)channel(wave, c) * DK + 8 * q;
  const int64_t nstep = (int64_t)a.hv * DK * DV * (BACK ? -1 : 1), mstep = (int64_t)a.hv * DK * DK * (BACK ? -1 : 1);
  const int64_t first = sid + (BACK ? segs - 1 : 0);
  float* np = a.seg_n + (first * a.hv + h) * DK * DV + own;
  const float* mp = a.seg_m + (first * a.hv + h) * DK * DK + mine;
  f32x4 S = zero4(), R[kAhead];
  Frag<float> M[kAhead][kSteps];
  const auto load = [&](f32x4& R, Frag<float>* M, int i) {
    i = min(i, segs - 1);  // (behind the last piece: anything)
#pragma unroll
    for (int r = 0; r < 4; ++r) R[r] = np[i * nstep + r * DV];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) row8(M[s], mp + i * mstep + 32 * s);
  };
  const auto store = [&](int i) {
#pragma unroll
    for (int r = 0; r < 4; ++r) np[i * nstep + r * DV] = S[r];
  };
  const auto step = [&](const f32x4& R, const Frag<float>* M, int i) {
    rows[i & 1][wave][lane] = S;
    __syncthreads();
    S = R;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      Frag<float> f;
      make<1>(f, rows[i & 1][2 * s][lane], rows[i & 1][2 * s + 1][lane]);
      S = mm<1, 1>(M[s], f, S);
    }
  };
  if (from) {
#pragma unroll
    for (int r = 0; r < 4; ++r) S[r] = from[((int64_t)b * a.hv + h) * DK * DV + own + r * DV];
  }
  // the first piece was run from the given state
  f32x4 next;
#pragma unroll
  for (int r = 0; r < 4; ++r) next[r] = np[r * DV];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) load(R[j], M[j], 1 + j);
  store(0);
  S = next;
  int i = 1;
  for (; i + kAhead < segs; i += kAhead) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      store(i + j);
      step(R[j], M[j], i + j);
      load(R[j], M[j], i + j + kAhead);
    }
  }
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    if (i + j >= segs) break;
    store(i + j);
    if (i + j + 1 < segs) step(R[j], M[j], i + j);
  }
}

// The first pieces and chunks of many sequences: 4 sequences a thread, 4096 a turn.
// (Counts past the room there is, of sequences that share rows, stay at it.)
__global__ __launch_bounds__(1024) void cuts_kernel(const Args a) {
  __shared__ uint64_t sums[2][2][16];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const uint32_t n = (uint32_t)a.n, per = (uint32_t)a.per;
  const uint64_t room[2] = {(uint64_t)a.pieces, (uint64_t)chunk_slots(a.n, a.nseq)};
  uint64_t before[2] = {0, 0};
  for (int64_t base = 0, turn = 0; base < a.nseq; base += 4096, turn ^= 1) {
    const int64_t b = base + 4 * threadIdx.x;
    uint32_t v[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) v[i] = b + i <= a.nseq ? bound(a.cu, (uint32_t)(b + i), n) : 0;
    uint64_t count[2][4], all[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      all[j] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        count[j][i] = b + i < a.nseq ? pieces_of(v[i], v[i + 1], j == 0 ? per : (uint32_t)kChunk) : 0;
        all[j] += count[j][i];
      }
      uint64_t x = all[j];
#pragma unroll
      for (int off = 1; off < 64; off *= 2) {
        const uint64_t y = __shfl_up(x, off, 64);
        if (lane >= off) x += y;
      }
      if (lane == 63) sums[turn][j][wave] = x;
      all[j] = x - all[j];  // of the lanes before
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint64_t at = before[j] + all[j];
      for (int w = 0; w < 16; ++w) {
        if (w < wave) at += sums[turn][j][w];
        before[j] += sums[turn][j][w];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (b + i < a.nseq) a.cuts[j * (int64_t)a.nseq + b + i] = (uint32_t)(at < room[j] ? at : room[j]);
        at += count[j][i];
      }
    }
  }
}

template <class T, int DK, bool KEEP>
hipError_t run_matrices(const Args& a, hipStream_t stream) {
  const int64_t waves = chunk_slots(a.n, a.nseq) * a.hv;
  matrices_kernel<T, DK, KEEP><<<(unsigned)((waves + 3) / 4), 256, 0, stream>>>(a);
  return hipGetLastError();
}

template <class T, int DK, int DV, int NCT, Mode MODE>
hipError_t run_forward(const Args& a, const Plan& p, hipStream_t stream) {
  constexpr int kThreads = 64 * (4 / NCT);
  const unsigned x = (unsigned)(p.pieces * a.hv);
  if (a.cuts) {
    cuts_kernel<<<1, 1024, 0, stream>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (hipError_t e = run_matrices<T, DK, MODE == kStates>(a, stream)) return e;
  if (p.split) {
    scan_kernel<T, DK, DV, NCT, kSummary><<<dim3(x, (DV + DK) / 64), kThreads, 0, stream>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
    join_kernel<DK, DV, false><<<dim3((unsigned)(a.nseq * a.hv), DV / 16), 4 * DK, 0, stream>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
  }
  scan_kernel<T, DK, DV, NCT, MODE><<<dim3(x, DV / 64), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

template <class T, int DK, int DV, int NCT>
hipError_t run_back(const Args& a, const Plan& p, hipStream_t stream) {
  constexpr int kThreads = 64 * (4 / NCT);
  const unsigned x = (unsigned)(p.pieces * a.hv);
  if (p.split) {
    back_kernel<T, DK, DV, NCT, kBackSummary><<<dim3(x, (DV + DK) / 64), kThreads, 0, stream>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
    join_kernel<DK, DV, true><<<dim3((unsigned)(a.nseq * a.hv), DV / 16), 4 * DK, 0, stream>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
  }
  back_kernel<T, DK, DV, NCT, kBack><<<dim3(x, DV / 64), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

enum What { kOutputs, kKeepStates, kReverse };

template <class T, int DK, int DV, int NCT>
hipError_t run_wide(const Args& a, const Plan& p, What what, hipStream_t s) {
  if (what == kOutputs) return run_forward<T, DK, DV, NCT, kForward>(a, p, s);
  if (what == kKeepStates) return run_forward<T, DK, DV, NCT, kStates>(a, p, s);
  return run_back<T, DK, DV, NCT>(a, p, s);
}
template <class T, int DK, int DV>
hipError_t run(const Args& a, const Plan& p, What what, hipStream_t s) {
  return p.wide ? run_wide<T, DK, DV, DK == 64 ? 4 : 2>(a, p, what, s) : run_wide<T, DK, DV, 1>(a, p, what, s);
}
template <class T>
hipError_t run_of(const Args& a, const Plan& p, What what, hipStream_t s) {
  if (a.dk == 64) return a.dv == 64 ? run<T, 64, 64>(a, p, what, s) : run<T, 64, 128>(a, p, what, s);
  return a.dv == 64 ? run<T, 128, 64>(a, p, what, s) : run<T, 128, 128>(a, p, what, s);
}

}  // namespace

hipError_t launch_forward(const Args& a, const Plan& p, bool bf16, hipStream_t stream) {
  return bf16 ? run_of<uint16_t>(a, p, kOutputs, stream) : run_of<float>(a, p, kOutputs, stream);
}
hipError_t launch_states(const Args& a, const Plan& p, bool bf16, hipStream_t stream) {
  return bf16 ? run_of<uint16_t>(a, p, kKeepStates, stream) : run_of<float>(a, p, kKeepStates, stream);
}
hipError_t launch_back(const Args& a, const Plan& p, bool bf16, hipStream_t stream) {
  return bf16 ? run_of<uint16_t>(a, p, kReverse, stream) : run_of<float>(a, p, kReverse, stream);
}

size_t matrix_bytes(bool keep) { return matrices_bytes(keep); }

// Wide waves pay where they alone fill the GPU: against narrow ones a 100-view scene takes
// 1025 us (1467), 48 views' gradient 1520 (1762), 24 views in fp32 462 (549), and 12
// views with heads of 128, below the limit, 978 (698). Where narrow ones need no cut,
// they have to fill half of it (32 sequences of 1374 tokens, 16 heads: 302 us, their
// gradient 1100, narrow 313 and 1196; 24 of them 300 and 1053, narrow 276 and 993).
// Pieces are as long as fill the GPU with waves (one a SIMD where they are wide: 1025 us
// for the scene, with half as many 1166, with twice as many 1085; half as many narrow
// ones: 698 us with heads of 128, with one a SIMD 1095), at least 3 chunks (one view's
// gradient 141 us; of 2: 164, of 4: 149). Sequences are cut only where much longer than
// that, since a cut costs a pass over all pieces with d_k more columns (48 views of 48
// sequences uncut 1520 us, cut 1796; 24 views in 10 sequences cut 462, uncut 529).
Plan plan(int64_t n, int nseq, int64_t longest, int hv, int dk, int dv) {
  const int64_t chunks = (n + kChunk - 1) / kChunk, rows = (int64_t)hv * (dv / 64);
  Plan p;
  const auto cut = [&](bool wide) {
    const int64_t waves = wide ? 1024 : 512;
    int64_t each = (chunks * rows + waves - 1) / waves;
    if (each < 3) each = 3;
    p.wide = wide;
    p.split = longest > each * kChunk * 5 / 2;
    p.per = p.split ? each * kChunk : (n / kChunk + 1) * kChunk;
    p.pieces = n / p.per + nseq;
  };
  cut(false);
  if (chunks * rows >= 16384 && (p.split || nseq * rows >= 512)) cut(true);
  return p;
}

}  // namespace delta
}  // namespace vggt3
