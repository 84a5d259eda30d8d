// Device helpers of the gated delta rule's kernels: products of 16 x 16 tiles in
// fp32 or in split bf16, a chunk's decays, and the inverse of its unit triangle.
//
// Tiles are held as the matrix unit leaves them: lane (c = l % 16, q = l / 16)
// has rows 4q .. 4q+3 of column c. Two tiles one above the other are, register
// for register, the right operand of a product over their 32 rows, if the left
// operand takes its 32 columns in the same order: element j of lane quarter q is
// column 16 (j / 4) + 4q + j % 4. So a product's result goes into the next product
// without leaving the wave's registers.
#pragma once

#include "bf16_ops.hpp"
#include "delta.hpp"

namespace vggt3 {
namespace delta {

// Tokens of a chunk: one 32-deep product. (A chunk of 64 costs as many products a
// token at 128-wide heads and more at 64-wide ones, since the triangle's share
// grows with the chunk.)
constexpr int kChunk = 32;

// Operand of a 32-deep product. bf16: 3 parts of 8 bits each, the whole fp32 value, or
// one where the value is bf16 already; fp32: the value.
template <class T>
struct Frag;
template <>
struct Frag<uint16_t> {
  bf16x8 part[3];
};
template <>
struct Frag<float> {
  f32x4 a, b;
};

// c += A B. NA, NB: parts of A and B (bf16, 1 or 3); products of parts that lie below the
// last one kept are left out: 2^-24 relative.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mm(const Frag<uint16_t>& a, const Frag<uint16_t>& b, f32x4 c) {
  constexpr int kLast = (NA > NB ? NA : NB) - 1;
#pragma unroll
  for (int sum = kLast; sum >= 0; --sum)
#pragma unroll
    for (int i = 0; i <= sum; ++i)
      if (i < NA && sum - i < NB)
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.part[i], b.part[sum - i], c, 0, 0, 0);
  return c;
}
template <int NA, int NB>
__device__ __forceinline__ f32x4 mm(const Frag<float>& a, const Frag<float>& b, f32x4 c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.a[e], b.a[e], c, 0, 0, 0);
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.b[e], b.b[e], c, 0, 0, 0);
  return c;
}
// c += A B over 16: one tile each, in fp32.
__device__ __forceinline__ f32x4 mm16(const f32x4& a, const f32x4& b, f32x4 c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
  return c;
}

__device__ __forceinline__ f32x4 zero4() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

// x - (the pair's low or high bf16), in one instruction: the pair's dot product with
// (-1, -0) or (-0, -1), added to x. What is left of a value that was rounded to bf16
// is exact in fp32. (With +0 the pair (-1, 0) is folded into the inline constant -1,
// which the instruction takes as (0, -1).)
__device__ __forceinline__ float less_lo(float x, uint32_t pair) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), __builtin_bit_cast(bf16x2, 0x8000bf80u), x, false);
}
__device__ __forceinline__ float less_hi(float x, uint32_t pair) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), __builtin_bit_cast(bf16x2, 0xbf808000u), x, false);
}

// Two tiles as an operand of P parts.
template <int P>
__device__ __forceinline__ void make(Frag<float>& f, const f32x4& x, const f32x4& y) {
  f.a = x;
  f.b = y;
}
template <int P>
__device__ __forceinline__ void make(Frag<uint16_t>& f, f32x4 x, f32x4 y) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
      w[2 + i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
    }
    f.part[p] = as_bf16x8(w);
    if (p + 1 < P) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[2 * i] = less_lo(x[2 * i], w[i]);
        x[2 * i + 1] = less_hi(x[2 * i + 1], w[i]);
        y[2 * i] = less_lo(y[2 * i], w[2 + i]);
        y[2 * i + 1] = less_hi(y[2 * i + 1], w[2 + i]);
      }
    }
  }
}

// 8 values of a row, at a 16-byte boundary.
__device__ __forceinline__ void row8(Frag<uint16_t>& f, const uint16_t* p) { f.part[0] = ld_op(p); }
__device__ __forceinline__ void row8(Frag<float>& f, const float* p) {
  f.a = *reinterpret_cast<const f32x4*>(p);
  f.b = *reinterpret_cast<const f32x4*>(p + 4);
}

// A head's channels are the rows of its state's tiles in an order in which 8
// neighbours are an operand's 8 elements: row p of tile t is channel
// 32 (t / 2) + 8 (p / 4) + 4 (t % 2) + p % 4.
__device__ __forceinline__ int channel(int tile, int row) {
  return 32 * (tile / 2) + 8 * (row / 4) + 4 * (tile % 2) + row % 4;
}

// X^T as a left operand over the chunk's tokens, for the rows of a state's tile, from X
// [kChunk][PITCH] in LDS. bf16: transposing reads, each lane of 16 giving the address
// of 4 neighbouring channels of one token.
template <int PITCH>
__device__ __forceinline__ void state_rows(Frag<uint16_t>& f, const uint16_t* x, int tile, int lane) {
  const int s = lane % 16, q = lane / 16;
  const uint16_t* p = x + (4 * q + s / 4) * PITCH + channel(tile, 4 * (s % 4));
  f.part[0] = tr_op(p, p + 16 * PITCH);
}
template <int PITCH>
__device__ __forceinline__ void state_rows(Frag<float>& f, const float* x, int tile, int lane) {
  const float* p = x + 4 * (lane / 16) * PITCH + channel(tile, lane % 16);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    f.a[r] = p[r * PITCH];
    f.b[r] = p[(16 + r) * PITCH];
  }
}
// X as a right operand over the chunk's tokens: lane c has channel base + N c + n (of N
// neighbours). bf16: value by value, since a lane's channels are not neighbours of the
// next lane's.
template <int N, int PITCH>
__device__ __forceinline__ void token_columns(Frag<uint16_t>& f, const uint16_t* x, int base, int n, int lane) {
  const uint16_t* p = x + 4 * (lane / 16) * PITCH + base + N * (lane % 16) + n;
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t* r = p + (16 * (i / 2) + 2 * (i % 2)) * PITCH;
    w[i] = (uint32_t)r[0] | (uint32_t)r[PITCH] << 16;
  }
  f.part[0] = as_bf16x8(w);
}
template <int N, int PITCH>
__device__ __forceinline__ void token_columns(Frag<float>& f, const float* x, int base, int n, int lane) {
  const float* p = x + 4 * (lane / 16) * PITCH + base + N * (lane % 16) + n;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    f.a[r] = p[r * PITCH];
    f.b[r] = p[(16 + r) * PITCH];
  }
}

// N neighbouring values <-> fp32 (N = 1, 2 or 4, aligned to N values).
template <int N>
__device__ __forceinline__ void load_n(float* o, const uint16_t* p) {
  if constexpr (N == 1) {
    o[0] = bf16_bits_to_f32(*p);
  } else if constexpr (N == 2) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    o[0] = bf16_lo(w);
    o[1] = bf16_hi(w);
  } else {
    const u32x2 w = ld8(p);
    o[0] = bf16_lo(w[0]);
    o[1] = bf16_hi(w[0]);
    o[2] = bf16_lo(w[1]);
    o[3] = bf16_hi(w[1]);
  }
}
template <int N>
__device__ __forceinline__ void load_n(float* o, const float* p) {
  typedef float vec __attribute__((ext_vector_type(N)));
  if constexpr (N == 1) {
    o[0] = *p;
  } else {
    const vec w = *reinterpret_cast<const vec*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = w[i];
  }
}
template <int N>
__device__ __forceinline__ void store_n(uint16_t* p, const float* v) {
  if constexpr (N == 1) {
    *p = f32_to_bf16_bits(v[0]);
  } else if constexpr (N == 2) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(v[0], v[1]);
  } else {
    st8(p, u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])});
  }
}
template <int N>
__device__ __forceinline__ void store_n(float* p, const float* v) {
  typedef float vec __attribute__((ext_vector_type(N)));
  if constexpr (N == 1) {
    *p = v[0];
  } else {
    vec w;
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = v[i];
    *reinterpret_cast<vec*>(p) = w;
  }
}

// Rows of a sequence through buffer descriptors: `len` rows from `base` on, each of D
// values, `ld` apart. Reads behind the last row give 0 and writes there are dropped, by
// the descriptor's range check. Offsets are in bytes.
typedef __amdgpu_buffer_rsrc_t Window;
template <int D, class T>
__device__ __forceinline__ Window window(const T* base, int64_t ld, int len) {
  const int64_t values = len > 0 ? (len - 1) * ld + D : 0;
  return __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, (int)(values * (int)sizeof(T)), 0x00020000);
}
// 8 values of a row, as they are stored.
template <class T>
struct Raw {
  u32x4 r[sizeof(T) / 2];
};
template <class T>
__device__ __forceinline__ void load_raw(Raw<T>& f, Window w, int off) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i)
    f.r[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(w, off + 16 * i, 0, 0));
}
template <class T>
__device__ __forceinline__ void put_raw(T* p, const Raw<T>& f) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) st16(p + 16 / sizeof(T) * i, f.r[i]);
}
__device__ __forceinline__ void as_frag(Frag<uint16_t>& f, const Raw<uint16_t>& x) { f.part[0] = as_bf16x8(x.r[0]); }
__device__ __forceinline__ void as_frag(Frag<float>& f, const Raw<float>& x) {
  f.a = __builtin_bit_cast(f32x4, x.r[0]);
  f.b = __builtin_bit_cast(f32x4, x.r[1]);
}
// N neighbouring values of a row, as they are stored, and as fp32.
template <class T, int N>
struct RawN {
  uint32_t r[(N * sizeof(T) + 3) / 4];
};
template <class T, int N>
__device__ __forceinline__ void load_rawn(RawN<T, N>& f, Window w, int off) {
  constexpr int kBytes = N * (int)sizeof(T);
  if constexpr (kBytes == 2) {
    f.r[0] = __builtin_amdgcn_raw_buffer_load_b16(w, off, 0, 0);
  } else if constexpr (kBytes == 4) {
    f.r[0] = __builtin_amdgcn_raw_buffer_load_b32(w, off, 0, 0);
  } else if constexpr (kBytes == 8) {
    const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(w, off, 0, 0));
    f.r[0] = x[0];
    f.r[1] = x[1];
  } else {
    const u32x4 x = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(w, off, 0, 0));
#pragma unroll
    for (int i = 0; i < 4; ++i) f.r[i] = x[i];
  }
}
template <int N>
__device__ __forceinline__ float value_of(const RawN<uint16_t, N>& f, int i) {
  return i % 2 ? bf16_hi(f.r[i / 2]) : bf16_lo(f.r[i / 2]);
}
template <int N>
__device__ __forceinline__ float value_of(const RawN<float, N>& f, int i) {
  return __uint_as_float(f.r[i]);
}
template <class T, int N>
__device__ __forceinline__ void store_rawn(Window w, int off, const float* v) {
  constexpr int kBytes = N * (int)sizeof(T);
  uint32_t x[(kBytes + 3) / 4];
#pragma unroll
  for (int i = 0; i < (kBytes + 3) / 4; ++i) {
    if constexpr (sizeof(T) == 4)
      x[i] = __float_as_uint(v[i]);
    else if constexpr (N == 1)
      x[i] = f32_to_bf16_bits(v[0]);
    else
      x[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  }
  if constexpr (kBytes == 2)
    __builtin_amdgcn_raw_buffer_store_b16((unsigned short)x[0], w, off, 0, 0);
  else if constexpr (kBytes == 4)
    __builtin_amdgcn_raw_buffer_store_b32(x[0], w, off, 0, 0);
  else if constexpr (kBytes == 8)
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{x[0], x[1]}, w, off, 0, 0);
  else
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{x[0], x[1], x[2], x[3]}, w, off, 0, 0);
}

// Between a wave's writes to LDS and its reads of what other lanes wrote: LDS
// operations of one wave are carried out in order, so only the compiler has to
// keep it.
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// x + w * (x of lane M of the lane's 16)
template <int M>
__device__ __forceinline__ float add_from(float x, float w) {
  const float y = __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x150 + M, 0xf, 0xf, true));
  return __builtin_fmaf(w, y, x);
}
template <int M>
__device__ __forceinline__ void eliminate(f32x4& x, f32x4& y, const float* nx, const float* ny) {
  if constexpr (M < 15) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      x[r] = add_from<M>(x[r], -nx[M]);
      y[r] = add_from<M>(y[r], -ny[M]);
    }
    eliminate<M + 1>(x, y, nx, ny);
  }
}

// A strictly lower triangle N [32][32] as left-operand tiles (lane (i, q) holds
// columns 4q .. 4q+3 of row i): n00, n11 its diagonal tiles, n10 the one below.
// t00, t10, t11: (I + N)^-1 in the same form. Row by row in the diagonal tiles
// (forward substitution, stable for any N; repeated squaring of N loses digits
// where keys repeat), then t10 = -t11 n10 t00. scratch: 2 x 16 x 20 floats of LDS.
__device__ __forceinline__ void unit_inverse(const f32x4& n00, const f32x4& n10, const f32x4& n11, f32x4& t00,
                                             f32x4& t10, f32x4& t11, float* scratch, int lane) {
  const int i = lane % 16, q = lane / 16;
  float* a = scratch + i * 20;
  float* b = scratch + (16 + i) * 20;
  *reinterpret_cast<f32x4*>(a + 4 * q) = n00;
  *reinterpret_cast<f32x4*>(b + 4 * q) = n11;
  wave_lds_order();
  float nx[16], ny[16];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const f32x4 u = *reinterpret_cast<const f32x4*>(a + 4 * s), w = *reinterpret_cast<const f32x4*>(b + 4 * s);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      nx[4 * s + r] = u[r];
      ny[4 * s + r] = w[r];
    }
  }
  wave_lds_order();
  f32x4 one;
#pragma unroll
  for (int r = 0; r < 4; ++r) one[r] = 4 * q + r == i ? 1.0f : 0.0f;
  t00 = t11 = one;
  eliminate<0>(t00, t11, nx, ny);
  const f32x4 c00 = mm16(t00, one, zero4());  // t00 as a result tile: its transpose as an operand
  const f32x4 p = mm16(n10, c00, zero4());
  t10 = mm16(p, t11, zero4());
#pragma unroll
  for (int r = 0; r < 4; ++r) t10[r] = -t10[r];
}

// A value that is the same in all lanes, as the compiler sees it: descriptors and
// addresses made of it stay in scalar registers.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __builtin_amdgcn_readfirstlane(x); }

// Rows are counted in 32 bits (at most 2^31 - 1). A boundary, held inside [0, n]
// whatever cu says.
__device__ __forceinline__ uint32_t bound(const int32_t* cu, uint32_t i, uint32_t n) {
  if (cu == nullptr) return i == 0 ? 0 : n;
  const int32_t v = cu[i];
  return v < 0 ? 0 : (uint32_t)v > n ? n : (uint32_t)v;
}

// Sums over the lanes before and with each.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ uint32_t lanes_down(uint32_t x) {
  return x + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ uint32_t running_count(uint32_t x) {
  x = lanes_down<0x111>(x);  // one lane down, within 16; then 2, 4, 8
  x = lanes_down<0x112>(x);
  x = lanes_down<0x114>(x);
  x = lanes_down<0x118>(x);
  x = lanes_down<0x142, 0xa>(x);  // every first 16's sum to the second's lanes
  return lanes_down<0x143, 0xc>(x);  // the first 32's to the others
}

// Pieces of `per` tokens that a sequence has; an empty one has one of no tokens.
__device__ __forceinline__ uint32_t pieces_of(uint32_t begin, uint32_t end, uint32_t per) {
  return end > begin ? (end - begin - 1) / per + 1 : 1;
}

// A sequence: its rows begin .. end - 1, and the numbers of its first piece and chunk.
// They rise from sequence to sequence, whatever the order of their rows.
struct Sequence {
  uint32_t begin, end, piece, chunk;
  int b;
};
// Fewer than 64 K sequences, K neighbours a lane. Where no boundary is below the one
// before it, begin / per + b leaves room for every sequence's last, shorter piece; pieces
// are counted otherwise. (Counting always would do, but pieces are a wave each and start in
// the order of their numbers: 10 ragged sequences of 24 views in fp32 463 us, counted 557,
// where the last ones wait for longer pieces.)
template <int K>
struct Lanes {
  uint32_t at[K + 1], piece[K], chunk[K];
};
template <int K>
__device__ __forceinline__ Lanes<K> lanes_of(const Args& a, uint32_t per, int lane) {
  Lanes<K> s;
  bool back = false;
#pragma unroll
  for (int i = 0; i <= K; ++i) s.at[i] = bound(a.cu, min(K * lane + i, a.nseq), (uint32_t)a.n);
#pragma unroll
  for (int i = 0; i < K; ++i) back = back || s.at[i + 1] < s.at[i];
  if (!__ballot(back)) {
#pragma unroll
    for (int i = 0; i < K; ++i) {
      s.piece[i] = s.at[i] / per + K * lane + i;
      s.chunk[i] = s.at[i] / kChunk + K * lane + i;
    }
    return s;
  }
  uint32_t pieces = 0, chunks = 0;
#pragma unroll
  for (int i = 0; i < K; ++i) {
    s.piece[i] = pieces;
    s.chunk[i] = chunks;
    if (K * lane + i < a.nseq) {
      pieces += pieces_of(s.at[i], s.at[i + 1], per);
      chunks += pieces_of(s.at[i], s.at[i + 1], kChunk);
    }
  }
  pieces = running_count(pieces) - pieces;
  chunks = running_count(chunks) - chunks;
#pragma unroll
  for (int i = 0; i < K; ++i) {
    s.piece[i] += pieces;
    s.chunk[i] += chunks;
  }
  return s;
}
template <int K>
__device__ __forceinline__ Sequence sequence_of(const Lanes<K>& s, int b) {
  Lanes<1> x{{s.at[0], s.at[1]}, {s.piece[0]}, {s.chunk[0]}};
#pragma unroll
  for (int i = 1; i < K; ++i)
    if (b % K == i) x = Lanes<1>{{s.at[i], s.at[i + 1]}, {s.piece[i]}, {s.chunk[i]}};
  Sequence o;
  o.begin = __builtin_amdgcn_readlane(x.at[0], b / K);
  o.end = __builtin_amdgcn_readlane(x.at[1], b / K);
  o.piece = __builtin_amdgcn_readlane(x.piece[0], b / K);
  o.chunk = __builtin_amdgcn_readlane(x.chunk[0], b / K);
  o.b = b;
  return o;
}
// The sequence whose pieces include `sid`, or the last that begins before it.
template <int K>
__device__ __forceinline__ Sequence sequence_with(const Args& a, uint32_t per, uint32_t sid, int lane) {
  const Lanes<K> s = lanes_of<K>(a, per, lane);
  int found = 0;
#pragma unroll
  for (int i = 0; i < K; ++i) found += __popcll(__ballot(K * lane + i < a.nseq && s.piece[i] <= sid));
  return sequence_of(s, (int)uniform(found > 0 ? found - 1 : 0));
}
__device__ __forceinline__ Sequence noted_sequence(const Args& a, uint32_t per, int b) {
  Sequence s;
  s.begin = uniform(bound(a.cu, b, (uint32_t)a.n));
  s.end = uniform(bound(a.cu, b + 1, (uint32_t)a.n));
  s.chunk = uniform(a.cuts[a.nseq + b]);
  s.piece = per == kChunk ? s.chunk : uniform(a.cuts[b]);
  s.b = b;
  return s;
}
__device__ __forceinline__ Sequence sequence(const Args& a, uint32_t per, int b, int lane) {
  if (a.cu == nullptr) return Sequence{0, (uint32_t)a.n, 0, 0, 0};
  if (a.cuts) return noted_sequence(a, per, b);
  return a.nseq < 64 ? sequence_of(lanes_of<1>(a, per, lane), b) : sequence_of(lanes_of<4>(a, per, lane), b);
}

// A sequence's piece: rows first .. first + len - 1, piece `seg` of `segs` of
// sequence b, whose chunks are numbered from `slot` on. seg < 0: there is no such piece.
struct Piece {
  int64_t first, slot;
  int len, b, seg, segs;
};

// Piece `sid` of `tokens` tokens each. Up to 255 sequences are looked at at once, in one
// trip to memory; more by a 64-ary search in their noted numbers. (Where
// sequences share rows, against the rule, there may be more chunks than room for them:
// those are left out.)
__device__ __forceinline__ Piece find_piece(const Args& a, int64_t tokens, int64_t id, int lane) {
  const uint32_t per = (uint32_t)tokens, sid = (uint32_t)id;
  Sequence s;
  if (a.cu == nullptr) {
    s = Sequence{0, (uint32_t)a.n, 0, 0, 0};
  } else if (a.cuts == nullptr) {
    s = a.nseq < 64 ? sequence_with<1>(a, per, sid, lane) : sequence_with<4>(a, per, sid, lane);
  } else {
    const uint32_t* first = per == kChunk ? a.cuts + a.nseq : a.cuts;
    uint32_t lo = 0, size = a.nseq;
    while (size > 1) {
      const uint32_t stride = (size + 63) / 64, at = lo + lane * stride;
      const bool before = lane * stride < size && first[at] <= sid;
      const uint32_t found = __popcll(__ballot(before));
      lo += (found > 0 ? found - 1 : 0) * stride;
      size = size < stride ? size : stride;
      if (lo + size > (uint32_t)a.nseq) size = a.nseq - lo;
    }
    s = noted_sequence(a, per, (int)uniform(lo));
  }
  const uint32_t len = s.end > s.begin ? s.end - s.begin : 0;
  Piece p;
  p.b = s.b;
  p.seg = sid < s.piece ? -1 : (int)(sid - s.piece);
  p.segs = (int)pieces_of(s.begin, s.end, per);
  const uint32_t before = (uint32_t)p.seg * per;
  p.slot = (int64_t)s.chunk + before / kChunk;
  const int64_t room = chunk_slots(a.n, a.nseq) - p.slot;
  if (p.seg < 0 || p.seg >= p.segs || room < 1) {
    p.seg = -1;
    p.first = s.begin;
    p.len = 0;
    return p;
  }
  const uint32_t left = len - before, some = left < per ? left : per;
  p.first = (int64_t)s.begin + before;
  p.len = (int)(some < room * kChunk ? some : room * kChunk);
  return p;
}

}  // namespace delta
}  // namespace vggt3
