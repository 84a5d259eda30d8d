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
#include "delta.hpp"
#include "delta_ops.hpp"

namespace vggt3 {
namespace delta {
namespace {

enum Mode { kForward, kSummary };

constexpr float kLog2e = 1.4426950408889634f;
constexpr double kLog2eD = 1.4426950408889634074;

// What a chunk's columns share, in LDS.
template <class T, int DK>
struct Shared {
  static constexpr int kPitch = DK + 16 / sizeof(T);  // rows 16 bytes apart in the banks
  T k[kChunk][kPitch];
  u32x4 t[2][128];   // T, rows 0-15 and 16-31, as operands
  u32x4 b[2][128];   // the triangle of Q K^T
  float decay[kChunk], rest[kChunk], beta[kChunk];
  float total;
  float scratch[2 * 16 * 20];
};

// One wave prepares a chunk: rows first .. first + len - 1, len in 1 .. 32 (rows
// behind them count as zeros).
template <class T, int DK, bool QK>
__device__ __forceinline__ void prepare(Shared<T, DK>& sh, const Args& a, int64_t first, int len, int h, int lane) {
  constexpr int kSteps = DK / 32, kPiece = 16 / sizeof(T), kPieces = DK / kPiece;
  const int kh = h / (a.hv / a.hk), c = lane % 16, q = lane / 16;
  const int64_t ld = (int64_t)a.hk * DK;
  const T* kp = static_cast<const T*>(a.k) + first * ld + kh * DK;
#pragma unroll
  for (int x = 0; x < kChunk * kPieces / 64; ++x) {
    const int at = x * 64 + lane, row = at / kPieces, col = at % kPieces * kPiece;
    u32x4 w = {0, 0, 0, 0};
    if (row < len) w = ld16(kp + row * ld + col);
    st16(&sh.k[row][col], w);
  }
  // decays in powers of 2, summed in 64 bits: a difference of two sums is right
  // whatever lies before them. Below 2^-2000 a decay is 0 in either form.
  const int t = lane % 32;
  double G = 0.0;
  float bt = 0.0f;
  if (t < len) {
    if (a.g) {
      const float g = a.g[(first + t) * a.hv + h];
      G = (g < -2000.0f ? -2000.0f : g) * kLog2eD;
    }
    bt = a.beta[(first + t) * a.hv + h];
  }
#pragma unroll
  for (int off = 1; off < kChunk; off *= 2) {
    const double up = __shfl_up(G, off, 32);
    if (t >= off) G += up;
  }
  const double end = __shfl(G, 31, 32);
  if (lane < kChunk) {
    sh.decay[t] = __builtin_amdgcn_exp2f((float)G);
    sh.rest[t] = __builtin_amdgcn_exp2f((float)(end - G));
    sh.beta[t] = bt;
    if (t == 31) sh.total = __builtin_amdgcn_exp2f((float)G);
  }
  wave_lds_order();
  // products with keys as rows and keys or queries as columns: results are left
  // operands, lane (i, q) holding columns 4q .. 4q+3 of row i
  f32x4 kk[3], qk[3];
#pragma unroll
  for (int x = 0; x < 3; ++x) kk[x] = qk[x] = zero4();
  const T* qp = static_cast<const T*>(a.q) + first * ld + kh * DK + 8 * q;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    Frag<T> k0, k1, q0, q1;
    row8(k0, &sh.k[c][32 * s + 8 * q]);
    row8(k1, &sh.k[16 + c][32 * s + 8 * q]);
    kk[0] = mm<1, 1>(k0, k0, kk[0]);
    kk[1] = mm<1, 1>(k0, k1, kk[1]);
    kk[2] = mm<1, 1>(k1, k1, kk[2]);
    if constexpr (QK) {
      clear(q0);
      clear(q1);
      if (c < len) row8(q0, qp + c * ld + 32 * s);
      if (16 + c < len) row8(q1, qp + (16 + c) * ld + 32 * s);
      qk[0] = mm<1, 1>(k0, q0, qk[0]);
      qk[1] = mm<1, 1>(k0, q1, qk[1]);
      qk[2] = mm<1, 1>(k1, q1, qk[2]);
    }
  }
  // tiles: rows (keys) 0-15 x columns 0-15; 0-15 x 16-31; 16-31 x 16-31
  const double Gi[2] = {__shfl(G, c, 32), __shfl(G, 16 + c, 32)};
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int j = 4 * q + r;
    const double G0 = __shfl(G, j, 32), G1 = __shfl(G, 16 + j, 32);
    const float d0 = __builtin_amdgcn_exp2f((float)(Gi[0] - G0)), d1 = __builtin_amdgcn_exp2f((float)(Gi[1] - G0)),
                d2 = __builtin_amdgcn_exp2f((float)(Gi[1] - G1));
    const float b0 = __shfl(bt, j, 32), b1 = __shfl(bt, 16 + j, 32);
    kk[0][r] = j < c ? kk[0][r] * d0 * b0 : 0.0f;
    kk[1][r] = kk[1][r] * d1 * b0;
    kk[2][r] = j < c ? kk[2][r] * d2 * b1 : 0.0f;
    if constexpr (QK) {
      qk[0][r] = j <= c ? qk[0][r] * d0 : 0.0f;
      qk[1][r] = qk[1][r] * d1;
      qk[2][r] = j <= c ? qk[2][r] * d2 : 0.0f;
    }
  }
  f32x4 t00, t10, t11;
  unit_inverse(kk[0], kk[1], kk[2], t00, t10, t11, sh.scratch, lane);
  Frag<T> f;
  make(f, t00, zero4());
  put(sh.t[0], f, lane);
  make(f, t10, t11);
  put(sh.t[1], f, lane);
  if constexpr (QK) {
    make(f, qk[0], zero4());
    put(sh.b[0], f, lane);
    make(f, qk[1], qk[2]);
    put(sh.b[1], f, lane);
  }
}

template <class T, int DK, int DV, int NCT, int W, int GC, Mode MODE>
__global__ __launch_bounds__(64 * W, 1) void scan_kernel(const Args a) {
  constexpr int kTiles = DK / 16, kSteps = DK / 32;
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
  {
    const float* from = nullptr;
    if (MODE == kForward && p.segs > 1)
      from = a.seg_n + (sid * a.hv + h) * DK * DV;
    else if (a.state && p.seg == 0 && !unit)
      from = a.state + ((int64_t)p.b * a.hv + h) * DK * DV;
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float w[NCT];
#pragma unroll
        for (int x = 0; x < NCT; ++x) w[x] = unit && channel(t, 4 * q + r) == col - DV + x ? 1.0f : 0.0f;
        if (from) load_n<NCT>(w, from + channel(t, 4 * q + r) * DV + col);
#pragma unroll
        for (int x = 0; x < NCT; ++x) S[t][x][r] = w[x];
      }
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
      float V[2][4][NCT];
#pragma unroll
      for (int it = 0; it < 2; ++it)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * it + 4 * q + r;
#pragma unroll
          for (int x = 0; x < NCT; ++x) V[it][r][x] = 0.0f;
          if (!unit && row < len)
            load_n<NCT>(V[it][r], static_cast<const T*>(a.v) + (first + row) * ldv + h * DV + col);
        }
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
          make(f, S[2 * s][x], S[2 * s + 1][x]);
          ks[0][x] = mm<1, 2>(k0, f, ks[0][x]);
          ks[1][x] = mm<1, 2>(k1, f, ks[1][x]);
          if constexpr (MODE == kForward) {
            o[0][x] = mm<1, 2>(qf[0][s], f, o[0][x]);
            o[1][x] = mm<1, 2>(qf[1][s], f, o[1][x]);
          }
        }
      }
      f32x4 dec[2], rest[2], bt[2];
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        dec[it] = *reinterpret_cast<const f32x4*>(&m.decay[16 * it + 4 * q]);
        rest[it] = *reinterpret_cast<const f32x4*>(&m.rest[16 * it + 4 * q]);
        bt[it] = *reinterpret_cast<const f32x4*>(&m.beta[16 * it + 4 * q]);
      }
      const float total = m.total;
      Frag<T> t0, t1;
      get(t0, m.t[0], lane);
      get(t1, m.t[1], lane);
#pragma unroll
      for (int x = 0; x < NCT; ++x) {
        f32x4 R[2];
#pragma unroll
        for (int it = 0; it < 2; ++it)
#pragma unroll
          for (int r = 0; r < 4; ++r) R[it][r] = V[it][r][x] - dec[it][r] * ks[it][x][r];
        Frag<T> f;
        make(f, R[0], R[1]);
        f32x4 u0 = mm<2, 2>(t0, f, zero4()), u1 = mm<2, 2>(t1, f, zero4());
        u0 *= bt[0];
        u1 *= bt[1];
        if constexpr (MODE == kForward) {
          Frag<T> b0, b1;
          get(b0, m.b[0], lane);
          get(b1, m.b[1], lane);
          make(f, u0, u1);
          o[0][x] = mm<2, 2>(b0, f, o[0][x] * dec[0]);
          o[1][x] = mm<2, 2>(b1, f, o[1][x] * dec[1]);
        }
        make(f, u0 * rest[0], u1 * rest[1]);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          Frag<T> kt;
          columns<Shared<T, DK>::kPitch>(kt, &m.k[0][0], t, lane);
          S[t][x] = mm<1, 2>(kt, f, S[t][x] * total);
        }
      }
      if constexpr (MODE == kForward) {
#pragma unroll
        for (int it = 0; it < 2; ++it)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = 16 * it + 4 * q + r;
            float w[NCT];
#pragma unroll
            for (int x = 0; x < NCT; ++x) w[x] = o[it][x][r] * a.scale;
            if (row < len) store_n<NCT>(static_cast<T*>(a.o) + (first + row) * ldv + h * DV + col, w);
          }
      }
    }
    __syncthreads();
  }

  float* to = nullptr;
  int64_t ld = DV;
  int at = col;
  if constexpr (MODE == kForward) {
    if (a.state_out && p.seg == p.segs - 1) to = a.state_out + ((int64_t)p.b * a.hv + h) * DK * DV;
  } else if (unit) {
    to = a.seg_m + (sid * a.hv + h) * DK * DK;
    ld = DK;
    at = col - DV;
  } else {
    to = a.seg_n + (sid * a.hv + h) * DK * DV;
  }
  if (to) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float w[NCT];
#pragma unroll
        for (int x = 0; x < NCT; ++x) w[x] = S[t][x][r];
        store_n<NCT>(to + channel(t, 4 * q + r) * ld + at, w);
      }
  }
}

// First states of a sequence's pieces: S <- M S + R from piece to piece, one wave
// for 16 columns. In fp32 products for both types: they are few.
template <int DK, int DV>
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
  f32x4 S[kTiles];
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      S[t][r] = a.state ? a.state[(((int64_t)b * a.hv + h) * DK + channel(t, 4 * q + r)) * DV + col] : 0.0f;
  for (int seg = 0; seg < segs; ++seg) {
    float* np = a.seg_n + ((sid + seg) * a.hv + h) * DK * DV + col;
    const float* mp = a.seg_m + ((sid + seg) * a.hv + h) * DK * DK;
    f32x4 out[kTiles];
    const bool more = seg + 1 < segs;
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float* at = np + channel(t, 4 * q + r) * DV;
        out[t][r] = more ? *at : 0.0f;
        *at = S[t][r];
      }
    if (!more) break;
    if (seg > 0) {  // the first piece was run from the sequence's own first state
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          Frag<float> m, f;
          row8(m, mp + channel(t, c) * DK + 32 * s + 8 * q);
          make(f, S[2 * s], S[2 * s + 1]);
          out[t] = mm<1, 1>(m, f, out[t]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t) S[t] = out[t];
  }
}

template <class T, int DK, int DV>
hipError_t forward(const Args& a, const Plan& p, hipStream_t stream) {
  const dim3 grid((unsigned)(p.pieces * a.hv), DV / 64);
  if (p.split) {
    scan_kernel<T, DK, DV, 1, 4, 2, kSummary><<<dim3(grid.x, (DV + DK) / 64), 256, 0, stream>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
    join_kernel<DK, DV><<<dim3((unsigned)(a.nseq * a.hv), DV / 16), 64, 0, stream>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
  }
  scan_kernel<T, DK, DV, 1, 4, 2, kForward><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

template <class T>
hipError_t forward_of(const Args& a, const Plan& p, hipStream_t s) {
  if (a.dk == 64) return a.dv == 64 ? forward<T, 64, 64>(a, p, s) : forward<T, 64, 128>(a, p, s);
  return a.dv == 64 ? forward<T, 128, 64>(a, p, s) : forward<T, 128, 128>(a, p, s);
}

}  // namespace

hipError_t launch_forward(const Args& a, const Plan& p, bool bf16, hipStream_t stream) {
  return bf16 ? forward_of<uint16_t>(a, p, stream) : forward_of<float>(a, p, stream);
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
