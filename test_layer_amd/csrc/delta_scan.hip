// The gated delta rule over whole sequences.
//
//   p_t = a_t S_{t-1}^T k_t,  u_t = beta_t (v_t - p_t),  S_t = a_t S_{t-1} + k_t u_t^T,  o_t = scale S_t^T q_t
//
// by chunks of 32 tokens. With G_i the chunk's decay up to token i, D_ij = G_i / G_j
// and S the state before the chunk,
//
//   N = strict lower triangle of D . (K K^T) . beta_j,    T = (I + N)^-1
//   y = T (V - G . (K S)),  u = beta . y
//   O = scale (G . (Q S) + (lower triangle of D . (Q K^T)) u)
//   S <- G_end S + K^T (G_end / G . u)
//
// A column of S, and of everything that u and O are made of, depends on no other
// column. So a wave keeps NCT tiles of 16 columns of S in registers over its whole
// piece of a sequence, and the products chain through its registers (delta_ops.hpp);
// only K, T and the triangle of Q K^T, which all columns share, pass through LDS.
// A workgroup takes GC chunks at a time: each of GC waves prepares one chunk's
// shared matrices by itself, then all waves run through the chunks.
//
// Long sequences are cut into pieces that are worked on at once: a first pass finds
// what each piece makes of its first state (M S + R: the columns of M are those of
// a value-free run that starts from the unit matrix), join_kernel goes through the
// pieces, and the main pass starts each piece from its own first state. (A
// sequence's first piece starts from the sequence's first state in both passes.)
#include "delta_chunk.hpp"

namespace vggt3 {
namespace delta {
namespace {

// kStates: the state before every chunk, for the gradient (no outputs).
enum Mode { kForward, kSummary, kStates };

template <class T, int DK>
struct Shared {
  T k[kChunk][kPitch<T, DK>];
  u32x4 t[2 * kOperand<T>];  // T
  u32x4 b[2 * kOperand<T>];  // the triangle of Q K^T
  Rows rows;
};

// One wave prepares a chunk: rows first .. first + len - 1, len in 1 .. 32 (rows
// behind them count as zeros).
template <class T, int DK, bool QK>
__device__ __forceinline__ void prepare(Shared<T, DK>& sh, const Args& a, int64_t first, int len, int h, int lane) {
  const int kh = h / (a.hv / a.hk), c = lane % 16, q = lane / 16;
  const int64_t ld = (int64_t)a.hk * DK;
  stage<T, DK, 64>(&sh.k[0][0], static_cast<const T*>(a.k) + first * ld + kh * DK, ld, len, lane);
  const Gates gt = gates(a, first, len, h, lane);
  put_rows(sh.rows, gt, lane);
  wave_lds_order();
  // keys as a tile's rows: results by row of N and of Q K^T
  const auto key = [&](Frag<T>& f, int row, int col) { row8(f, &sh.k[row + c][col]); };
  const T* qp = static_cast<const T*>(a.q) + first * ld + kh * DK;
  const auto query = [&](Frag<T>& f, int row, int col) {
    clear(f);
    if (row + c < len) row8(f, qp + (row + c) * ld + col);
  };
  Tri n{zero4(), zero4(), zero4()}, w = n;
#pragma unroll
  for (int s = 0; s < DK / 32; ++s) {
    Frag<T> k0, k1, q0, q1;
    key(k0, 0, 32 * s + 8 * q);
    key(k1, 16, 32 * s + 8 * q);
    n.t00 = mm<1, 1>(k0, k0, n.t00);
    n.t10 = mm<1, 1>(k0, k1, n.t10);
    n.t11 = mm<1, 1>(k1, k1, n.t11);
    if constexpr (QK) {
      query(q0, 0, 32 * s + 8 * q);
      query(q1, 16, 32 * s + 8 * q);
      w.t00 = mm<1, 1>(k0, q0, w.t00);
      w.t10 = mm<1, 1>(k0, q1, w.t10);
      w.t11 = mm<1, 1>(k1, q1, w.t11);
    }
  }
  decay_tri<false>(n, gt, true, true, 1.0f, lane);
  Tri t;
  unit_inverse(n.t00, n.t10, n.t11, t.t00, t.t10, t.t11, reinterpret_cast<float*>(sh.t), lane);
  put_lower<T, kWhole<T>>(sh.t, t, lane);
  if constexpr (QK) {
    decay_tri<false>(w, gt, false, false, a.scale, lane);
    put_lower<T, 2>(sh.b, w, lane);
  }
}

template <class T, int DK, int DV, int NCT, int W, int GC, Mode MODE>
__global__ __launch_bounds__(64 * W, 1) void scan_kernel(const Args a) {
  constexpr int kTiles = DK / 16, kSteps = DK / 32, kP = kWhole<T>;
  __shared__ Shared<T, DK> sh[GC];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int c = lane % 16, q = lane / 16;
  const int h = blockIdx.x % a.hv;
  const int64_t sid = blockIdx.x / a.hv;
  const Piece p = find_piece(a.cu, a.nseq, a.n, a.per, sid, lane);
  if (p.seg < 0) return;
  if (MODE == kSummary && p.seg == p.segs - 1) return;  // nothing follows it
  // this lane's columns: NCT neighbours
  const int col = (blockIdx.y * W + wave) * 16 * NCT + NCT * c;
  const bool unit = MODE == kSummary && col >= DV;
  if (unit && p.seg == 0) return;  // its first state is known (whole workgroups: DV is a multiple of their columns)

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
  for (int c0 = 0; c0 < chunks; c0 += GC) {
    if (wave < GC && c0 + wave < chunks) {
      const int at = (c0 + wave) * kChunk;
      prepare<T, DK, MODE == kForward>(sh[wave], a, p.first + at, min(kChunk, p.len - at), h, lane);
    }
    __syncthreads();
    for (int i = 0; i < GC && c0 + i < chunks; ++i) {
      const Shared<T, DK>& m = sh[i];
      const int64_t first = p.first + (int64_t)(c0 + i) * kChunk;
      const int len = min(kChunk, p.len - (c0 + i) * kChunk);
      if constexpr (MODE == kStates) {
        const int64_t slot = p.begin / kChunk + p.b + (p.first - p.begin) / kChunk + c0 + i;
        store_state<DK, NCT>(S, a.states + (slot * a.hv + h) * DK * DV + col, DV, q);
      }
      f32x4 V[2][NCT];
      load_rows<NCT>(V, static_cast<const T*>(a.v) + first * ldv + h * DV + col, ldv, unit ? 0 : len, q);
      Frag<T> qf[2][kSteps];
      if constexpr (MODE == kForward) {
#pragma unroll
        for (int it = 0; it < 2; ++it)
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {
            clear(qf[it][s]);
            if (16 * it + c < len)
              row8(qf[it][s], static_cast<const T*>(a.q) + (first + 16 * it + c) * ldq + kh * DK + 32 * s + 8 * q);
          }
      }
      f32x4 ks[2][NCT], o[2][NCT];
#pragma unroll
      for (int it = 0; it < 2; ++it)
#pragma unroll
        for (int x = 0; x < NCT; ++x) ks[it][x] = o[it][x] = zero4();
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        Frag<T> k0, k1;
        row8(k0, &m.k[c][32 * s + 8 * q]);
        row8(k1, &m.k[16 + c][32 * s + 8 * q]);
#pragma unroll
        for (int x = 0; x < NCT; ++x) {
          Frag<T> f;
          make<kP>(f, S[2 * s][x], S[2 * s + 1][x]);
          ks[0][x] = mm<1, kP>(k0, f, ks[0][x]);
          ks[1][x] = mm<1, kP>(k1, f, ks[1][x]);
          if constexpr (MODE == kForward) {
            o[0][x] = mm<1, 2>(qf[0][s], f, o[0][x]);
            o[1][x] = mm<1, 2>(qf[1][s], f, o[1][x]);
          }
        }
      }
      f32x4 dec[2], rest[2], bt[2];
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        dec[it] = rows4(m.rows.decay, it, q);
        rest[it] = rows4(m.rows.rest, it, q);
        bt[it] = rows4(m.rows.beta, it, q);
      }
      const float total = m.rows.total;
      Frag<T> t0, t1;
      get<kP>(t0, m.t, lane);
      get<kP>(t1, m.t + kOperand<T>, lane);
#pragma unroll
      for (int x = 0; x < NCT; ++x) {
        Frag<T> f;
        make<kP>(f, V[0][x] - dec[0] * ks[0][x], V[1][x] - dec[1] * ks[1][x]);
        const f32x4 u0 = mm<kP, kP>(t0, f, zero4()) * bt[0], u1 = mm<kP, kP>(t1, f, zero4()) * bt[1];
        if constexpr (MODE == kForward) {
          Frag<T> b0, b1;
          get<2>(b0, m.b, lane);
          get<2>(b1, m.b + kOperand<T>, lane);
          make<2>(f, u0, u1);
          o[0][x] = mm<2, 2>(b0, f, o[0][x] * (dec[0] * a.scale));
          o[1][x] = mm<2, 2>(b1, f, o[1][x] * (dec[1] * a.scale));
        }
        make<kP>(f, u0 * rest[0], u1 * rest[1]);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          Frag<T> kt;
          state_rows<kPitch<T, DK>>(kt, &m.k[0][0], t, lane);
          S[t][x] = mm<1, kP>(kt, f, S[t][x] * total);
        }
      }
      if constexpr (MODE == kForward)
        store_rows<NCT>(static_cast<T*>(a.o) + first * ldv + h * DV + col, o, ldv, len, q);
    }
    __syncthreads();
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
//   du = B^T dO + G_end / G . (K dS),  dR = T^T (beta . du)  (the gradient of V),
//   dS <- G_end dS + Q^T (scale G . dO) - K^T (G . dR),    B = scale D . Q K^T (lower)
//
// by the same columns, with dS in the registers. kBack: dS after every chunk is
// stored; kBackSummary: what a piece makes of the dS behind it.
enum BackMode { kBack, kBackSummary };

template <class T, int DK>
struct BackShared {
  T k[kChunk][kPitch<T, DK>];
  T q[kChunk][kPitch<T, DK>];
  u32x4 tt[2 * kOperand<T>];  // T^T
  u32x4 bt[2 * kOperand<T>];  // B^T
  Rows rows;
};

template <class T, int DK>
__device__ __forceinline__ void prepare_back(BackShared<T, DK>& sh, const Args& a, int64_t first, int len, int h,
                                             int lane) {
  const int kh = h / (a.hv / a.hk), c = lane % 16, q = lane / 16;
  const int64_t ld = (int64_t)a.hk * DK;
  stage<T, DK, 64>(&sh.k[0][0], static_cast<const T*>(a.k) + first * ld + kh * DK, ld, len, lane);
  stage<T, DK, 64>(&sh.q[0][0], static_cast<const T*>(a.q) + first * ld + kh * DK, ld, len, lane);
  const Gates gt = gates(a, first, len, h, lane);
  put_rows(sh.rows, gt, lane);
  wave_lds_order();
  const auto key = [&](Frag<T>& f, int row, int col) { row8(f, &sh.k[row + c][col]); };
  const auto query = [&](Frag<T>& f, int row, int col) { row8(f, &sh.q[row + c][col]); };
  // N by row (keys 16-31 against keys 0-15 turned round: 10 by row is 01 by column)
  Tri n{zero4(), zero4(), zero4()};
#pragma unroll
  for (int s = 0; s < DK / 32; ++s) {
    Frag<T> k0, k1;
    key(k0, 0, 32 * s + 8 * q);
    key(k1, 16, 32 * s + 8 * q);
    n.t00 = mm<1, 1>(k0, k0, n.t00);
    n.t10 = mm<1, 1>(k0, k1, n.t10);
    n.t11 = mm<1, 1>(k1, k1, n.t11);
  }
  decay_tri<false>(n, gt, true, true, 1.0f, lane);
  Tri t;
  unit_inverse(n.t00, n.t10, n.t11, t.t00, t.t10, t.t11, reinterpret_cast<float*>(sh.tt), lane);
  t.t00 = turned(t.t00, lane);
  t.t10 = turned(t.t10, lane);
  t.t11 = turned(t.t11, lane);
  put_upper<T, kWhole<T>>(sh.tt, t, lane);
  Tri w = products<1, 1, T, DK>(query, key, q);
  decay_tri<true>(w, gt, false, false, a.scale, lane);
  put_upper<T, kWhole<T>>(sh.bt, w, lane);
}

template <class T, int DK, int DV, int NCT, int W, int GC, BackMode MODE>
__global__ __launch_bounds__(64 * W, 1) void back_kernel(const Args a) {
  constexpr int kTiles = DK / 16, kSteps = DK / 32, kP = kWhole<T>;
  __shared__ BackShared<T, DK> sh[GC];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int c = lane % 16, q = lane / 16;
  const int h = blockIdx.x % a.hv;
  const int64_t sid = blockIdx.x / a.hv;
  const Piece p = find_piece(a.cu, a.nseq, a.n, a.per, sid, lane);
  if (p.seg < 0) return;
  if (MODE == kBackSummary && p.seg == 0) return;  // nothing lies before it
  const int col = (blockIdx.y * W + wave) * 16 * NCT + NCT * c;
  const bool unit = MODE == kBackSummary && col >= DV;
  if (unit && p.seg == p.segs - 1) return;  // the dS behind it is known

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

  const int64_t ldv = (int64_t)a.hv * DV;
  const int chunks = (p.len + kChunk - 1) / kChunk;
  for (int c1 = chunks; c1 > 0; c1 -= GC) {  // chunks c1 - 1, c1 - 2, ..
    if (wave < GC && c1 - 1 - wave >= 0) {
      const int at = (c1 - 1 - wave) * kChunk;
      prepare_back<T, DK>(sh[wave], a, p.first + at, min(kChunk, p.len - at), h, lane);
    }
    __syncthreads();
    for (int i = 0; i < GC && c1 - 1 - i >= 0; ++i) {
      const BackShared<T, DK>& m = sh[i];
      const int at = (c1 - 1 - i) * kChunk;
      const int64_t first = p.first + at;
      const int len = min(kChunk, p.len - at);
      if constexpr (MODE == kBack) {
        const int64_t slot = p.begin / kChunk + p.b + (first - p.begin) / kChunk;
        store_state<DK, NCT>(S, a.dstates + (slot * a.hv + h) * DK * DV + col, DV, q);
      }
      f32x4 dO[2][NCT];
      load_rows<NCT>(dO, static_cast<const T*>(a.dout) + first * ldv + h * DV + col, ldv, unit ? 0 : len, q);
      f32x4 kd[2][NCT];
#pragma unroll
      for (int it = 0; it < 2; ++it)
#pragma unroll
        for (int x = 0; x < NCT; ++x) kd[it][x] = zero4();
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        Frag<T> k0, k1;
        row8(k0, &m.k[c][32 * s + 8 * q]);
        row8(k1, &m.k[16 + c][32 * s + 8 * q]);
#pragma unroll
        for (int x = 0; x < NCT; ++x) {
          Frag<T> f;
          make<kP>(f, S[2 * s][x], S[2 * s + 1][x]);
          kd[0][x] = mm<1, kP>(k0, f, kd[0][x]);
          kd[1][x] = mm<1, kP>(k1, f, kd[1][x]);
        }
      }
      f32x4 dec[2], rest[2], bt[2];
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        dec[it] = rows4(m.rows.decay, it, q);
        rest[it] = rows4(m.rows.rest, it, q);
        bt[it] = rows4(m.rows.beta, it, q);
      }
      const float total = m.rows.total;
#pragma unroll
      for (int x = 0; x < NCT; ++x) {
        Frag<T> f, b0, b1, t0, t1;
        make<1>(f, dO[0][x], dO[1][x]);
        get<kP>(b0, m.bt, lane);
        get<kP>(b1, m.bt + kOperand<T>, lane);
        const f32x4 du0 = mm<kP, 1>(b0, f, kd[0][x] * rest[0]), du1 = mm<kP, 1>(b1, f, kd[1][x] * rest[1]);
        make<kP>(f, du0 * bt[0], du1 * bt[1]);
        get<kP>(t0, m.tt, lane);
        get<kP>(t1, m.tt + kOperand<T>, lane);
        const f32x4 dR0 = mm<kP, kP>(t0, f, zero4()), dR1 = mm<kP, kP>(t1, f, zero4());
        Frag<T> g;
        make<kP>(f, dO[0][x] * (dec[0] * a.scale), dO[1][x] * (dec[1] * a.scale));
        make<kP>(g, -dR0 * dec[0], -dR1 * dec[1]);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          Frag<T> kt, qt;
          state_rows<kPitch<T, DK>>(kt, &m.k[0][0], t, lane);
          state_rows<kPitch<T, DK>>(qt, &m.q[0][0], t, lane);
          S[t][x] = mm<1, kP>(kt, g, mm<1, kP>(qt, f, S[t][x] * total));
        }
      }
    }
    __syncthreads();
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
// piece (BACK: from the last piece to the first), one wave for 16 columns. In fp32
// products for both types: they are few.
template <int DK, int DV, bool BACK>
__global__ __launch_bounds__(64) void join_kernel(const Args a) {
  constexpr int kTiles = DK / 16, kSteps = DK / 32;
  const int lane = threadIdx.x, c = lane % 16, q = lane / 16;
  const int h = blockIdx.x % a.hv;
  const int b = blockIdx.x / a.hv;
  const int col = blockIdx.y * 16 + c;
  const int64_t begin = bound(a.cu, b, a.n), end = bound(a.cu, b + 1, a.n);
  const int64_t len = end > begin ? end - begin : 0;
  const int segs = (int)((len + a.per - 1) / a.per);
  if (segs < 2) return;
  const int64_t sid = begin / a.per + b;
  const float* from = BACK ? a.dlast : a.state;
  f32x4 S[kTiles][1];
  load_state<DK, 1>(S, from ? from + ((int64_t)b * a.hv + h) * DK * DV + col : nullptr, DV, q);
  for (int i = 0; i < segs; ++i) {
    const int seg = BACK ? segs - 1 - i : i;
    float* np = a.seg_n + ((sid + seg) * a.hv + h) * DK * DV + col;
    const float* mp = a.seg_m + ((sid + seg) * a.hv + h) * DK * DK;
    f32x4 out[kTiles][1];
    const bool more = i + 1 < segs;
    load_state<DK, 1>(out, more ? np : nullptr, DV, q);
    store_state<DK, 1>(S, np, DV, q);
    if (!more) break;
    if (i > 0) {  // the first piece was run from the given state
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          Frag<float> m, f;
          row8(m, mp + channel(t, c) * DK + 32 * s + 8 * q);
          make<1>(f, S[2 * s][0], S[2 * s + 1][0]);
          out[t][0] = mm<1, 1>(m, f, out[t][0]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t) S[t][0] = out[t][0];
  }
}

template <class T, int DK, int DV, Mode MODE>
hipError_t run_forward(const Args& a, const Plan& p, hipStream_t stream) {
  const unsigned x = (unsigned)(p.pieces * a.hv);
  if (p.split) {
    scan_kernel<T, DK, DV, 1, 4, 2, kSummary><<<dim3(x, (DV + DK) / 64), 256, 0, stream>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
    join_kernel<DK, DV, false><<<dim3((unsigned)(a.nseq * a.hv), DV / 16), 64, 0, stream>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
  }
  scan_kernel<T, DK, DV, 1, 4, 2, MODE><<<dim3(x, DV / 64), 256, 0, stream>>>(a);
  return hipGetLastError();
}

template <class T, int DK, int DV>
hipError_t run_back(const Args& a, const Plan& p, hipStream_t stream) {
  const unsigned x = (unsigned)(p.pieces * a.hv);
  if (p.split) {
    back_kernel<T, DK, DV, 1, 4, 2, kBackSummary><<<dim3(x, (DV + DK) / 64), 256, 0, stream>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
    join_kernel<DK, DV, true><<<dim3((unsigned)(a.nseq * a.hv), DV / 16), 64, 0, stream>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
  }
  back_kernel<T, DK, DV, 1, 4, 2, kBack><<<dim3(x, DV / 64), 256, 0, stream>>>(a);
  return hipGetLastError();
}

enum What { kOutputs, kKeepStates, kReverse };

template <class T, int DK, int DV>
hipError_t run(const Args& a, const Plan& p, What what, hipStream_t s) {
  if (what == kOutputs) return run_forward<T, DK, DV, kForward>(a, p, s);
  if (what == kKeepStates) return run_forward<T, DK, DV, kStates>(a, p, s);
  return run_back<T, DK, DV>(a, p, s);
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

// Pieces: as long as about 512 workgroups of 64 columns allow, at least 4 chunks;
// one for the whole sequence where that is as much work at once.
Plan plan(int64_t n, int nseq, int64_t longest, int hv, int dk, int dv) {
  const int64_t chunks = (n + kChunk - 1) / kChunk, rows = (int64_t)hv * (dv / 64);
  int64_t each = (chunks * rows + 511) / 512;
  if (each < 4) each = 4;
  Plan p;
  p.split = longest > each * kChunk;
  p.per = p.split ? each * kChunk : (n / kChunk + 1) * kChunk;
  p.pieces = n / p.per + nseq;
  return p;
}

}  // namespace delta
}  // namespace vggt3
