// Norms of queries and keys for each head, and their rotation by position, in one
// pass; and the gradient.
//
//   h = norm(x) of a head's d channels (none; x / max(|x|, eps); RMS or layer norm
//   with weight and bias), then for each rotated pair (a, b) with angle
//   t = position on the pair's axis * base^(-j / size):
//   (a, b) <- (a cos t - b sin t, b cos t + a sin t)
//
// Bound by memory: x read once, y written once. A wave takes a token with all its
// heads, so a lane's 4 pairs keep their angles over the token's heads and their
// frequencies and weights over all tokens. A lane holds both channels of 4 pairs, so
// that a rotation is its own, and the norm's sums over a head are a few DPP
// steps over 8 to 64 lanes. 100 views of 16 + 16 heads of 64 in bf16: 214 us,
// 5.3 TB/s, a copy's rate; 48 views' gradient 154 us. Angles are formed in two doubles (in
// one a position of 2^31 is off by 6 u, in 32 bits one of a million by 0.06 of a radian) and
// reduced to a turn before the sine, one pair a lane, and handed to the lanes that hold the
// pair.
#include "qk.hpp"

#include "delta_ops.hpp"

namespace vggt3 {
namespace qk {
namespace {

using delta::load_rawn;
using delta::RawN;
using delta::store_rawn;
using delta::value_of;
using delta::Window;

template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
  return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
// Sum over the head's LANES neighbouring lanes, in all of them.
template <int LANES>
__device__ __forceinline__ float head_sum(float x) {
  if constexpr (LANES >= 2) x = dpp_add<0xB1>(x);    // lane ^ 1
  if constexpr (LANES >= 4) x = dpp_add<0x4E>(x);    // lane ^ 2
  if constexpr (LANES >= 8) x = dpp_add<0x141>(x);   // 7 - lane: the other 4 of 8
  if constexpr (LANES >= 16) x = dpp_add<0x140>(x);  // 15 - lane: the other 8 of 16
  if constexpr (LANES >= 32) x += __shfl_xor(x, 16, 64);
  if constexpr (LANES >= 64) x += __shfl_xor(x, 32, 64);
  return x;
}

// How a lane's 8 channels lie: two runs of 4 (the pairs' first and second
// channels), 8 neighbours, anyhow but read and written as 8 neighbours and handed
// over through LDS, or anyhow. 100 views in bf16 with axes of 12, 10 and 10 pairs:
// runs of 2 values were 330 us, single ones 560, handed over 214.
enum Access { kFours, kNeighbours, kStaged, kSingle };

constexpr int kNowhere = 0x40000000;  // an offset behind every row's end

// A value in two doubles, to about 100 bits. (Products and their roundings' rests must not
// be contracted: the rest would count twice.)
struct Two {
  double hi, lo;
};
__device__ __forceinline__ Two operator*(const Two& x, const Two& y) {
#pragma clang fp contract(off)
  const double p = x.hi * y.hi;
  const double e = fma(x.hi, y.lo, fma(x.lo, y.hi, fma(x.hi, y.hi, -p)));
  Two z;
  z.hi = p + e;
  z.lo = e - (z.hi - p);
  return z;
}

// A rotated pair: its channels, axis and turns a position step.
struct Pair {
  int first, second, axis;
  Two turns;
};
__device__ __forceinline__ Pair pair_of(const Args& a, int at) {
  Pair p;
  int axis = 0, before = 0;
  while (axis + 1 < a.axes && at >= before + a.pairs[axis]) before += a.pairs[axis++];
  const int size = a.per_axis ? a.pairs[axis] : a.rotated;
  const int j = a.per_axis ? at - before : at, off = a.per_axis ? 2 * before : 0;
  p.first = off + (a.interleaved ? 2 * j : j);
  p.second = a.interleaved ? p.first + 1 : p.first + size;
  p.axis = axis;
  p.turns = Two{0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};  // 1 / (2 pi)
  Two step{a.step[axis][0], a.step[axis][1]};
  for (int k = j; k > 0; k /= 2) {
    if (k % 2) p.turns = p.turns * step;
    if (k > 1) step = step * step;
  }
  return p;
}

// The channels of a lane's 4 pairs (-1: past the head's end). Channels that are not
// rotated are paired so that they lie as the others do.
struct Pairs {
  int first[4], second[4];
  bool turned[4];
};
// Pair v of a lane: 4 neighbours, or where pairs lie anyhow every LANES-th, so that
// the lanes' values are neighbours.
template <Access A, int LANES>
__device__ __forceinline__ int pair_at(int lane_in_head, int v) {
  return A == kFours || A == kNeighbours ? 4 * lane_in_head + v : lane_in_head + LANES * v;
}
template <Access A, int LANES>
__device__ __forceinline__ Pairs pairs_of(const Args& a, int lane_in_head) {
  constexpr int kRun = A == kFours ? 4 : 1;
  Pairs p;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int at = pair_at<A, LANES>(lane_in_head, v);
    p.turned[v] = at < a.rotated;
    if (p.turned[v]) {
      const Pair x = pair_of(a, at);
      p.first[v] = x.first;
      p.second[v] = x.second;
    } else {
      const int base = 2 * (at - at % kRun) + at % kRun;
      p.first[v] = base < a.d ? base : -1;
      p.second[v] = base + kRun < a.d ? base + kRun : -1;
    }
  }
  return p;
}

__device__ __forceinline__ void angle_of(const Args& a, int axis, const Two& turns, int64_t token, float& c, float& s) {
#pragma clang fp contract(off)
  const double at = a.pos[token * a.axes + axis], x = at * turns.hi;
  const double rest = fma(at, turns.lo, fma(at, turns.hi, -x));
  sincospif(2.0f * (float)((x - rint(x)) + rest), &s, &c);
}

// The sines and cosines of a lane's 4 pairs at a token. Heads of up to 128 channels
// have at most 64 pairs: lane l forms those of pair l.
struct Angles {
  float c[4], s[4];
};
template <Access A, int LANES>
struct Rotation {
  static constexpr int kOwn = LANES <= 16 ? 1 : 4;
  int axis[kOwn];
  Two turns[kOwn];
  __device__ __forceinline__ Rotation(const Args& a, int lane) {
#pragma unroll
    for (int v = 0; v < kOwn; ++v) {
      axis[v] = 0;
      turns[v] = Two{0.0, 0.0};
      const int at = kOwn == 1 ? lane : pair_at<A, LANES>(lane, v);
      if (at < a.rotated) {
        const Pair x = pair_of(a, at);
        axis[v] = x.axis;
        turns[v] = x.turns;
      }
    }
  }
  __device__ __forceinline__ Angles at(const Args& a, int64_t token, int lane_in_head) const {
    Angles t;
    if (a.rotated == 0) {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        t.c[v] = 1.0f;
        t.s[v] = 0.0f;
      }
      return t;
    }
    float c[kOwn], s[kOwn];
#pragma unroll
    for (int v = 0; v < kOwn; ++v) angle_of(a, axis[v], turns[v], token, c[v], s[v]);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if constexpr (kOwn == 1) {
        t.c[v] = __shfl(c[0], pair_at<A, LANES>(lane_in_head, v), 64);
        t.s[v] = __shfl(s[0], pair_at<A, LANES>(lane_in_head, v), 64);
      } else {
        t.c[v] = c[v];
        t.s[v] = s[v];
      }
    }
    return t;
  }
};

// A pair rotated. Channels that are not have nothing to do with the one that they are
// paired with: 0 times it would be NaN where it is Inf or NaN.
__device__ __forceinline__ void turn(bool turned, float c, float s, float& a, float& b) {
  const float x = a * c - b * s, y = b * c + a * s;
  a = turned ? x : a;
  b = turned ? y : b;
}

// A lane's 8 channels of a head as runs: how many, of how many values, and where they
// start in the head's row in bytes (behind every row's end where there is none: the
// window's range check then reads zeros and drops stores, so that no access hangs on a
// branch, behind which the compiler would wait for all stores before it).
template <Access A, class T, int LANES>
struct Runs {
  static constexpr int kN = A == kFours || A == kNeighbours ? 4 : 1, kCount = 8 / kN;
  int at[kCount];
  __device__ __forceinline__ Runs(const Args&, const Pairs& p, int) {
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      const int v = A == kNeighbours ? 2 * i : i / 2 * kN;
      const int ch = A == kNeighbours || i % 2 == 0 ? p.first[v] : p.second[v];
      at[i] = ch < 0 ? kNowhere : ch * (int)sizeof(T);
    }
  }
  // Where pair v's channels are among the runs' values.
  static __device__ __forceinline__ constexpr int first(int v) { return A == kNeighbours ? 2 * v : v / kN * 2 * kN + v % kN; }
  static __device__ __forceinline__ constexpr int second(int v) { return first(v) + (A == kNeighbours ? 1 : kN); }
  typedef RawN<T, kN> Raw8[kCount];
  __device__ __forceinline__ void load(Raw8& r, Window w, int row) const {
#pragma unroll
    for (int i = 0; i < kCount; ++i) load_rawn(r[i], w, row + at[i]);
  }
  __device__ __forceinline__ void values(float* f, float* s, const Raw8& r) const {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      f[v] = value_of(r[first(v) / kN], first(v) % kN);
      s[v] = value_of(r[second(v) / kN], second(v) % kN);
    }
  }
  __device__ __forceinline__ void store(Window w, int row, const float* f, const float* s) const {
    float x[8];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      x[first(v)] = f[v];
      x[second(v)] = s[v];
    }
#pragma unroll
    for (int i = 0; i < kCount; ++i) store_rawn<T, kN>(w, row + at[i], x + i * kN);
  }
};

// A wave's own part of LDS, in which its lanes hand over heads: rows 8 values apart in
// the banks, so that 8 heads' lanes meet in none.
template <class T, int LANES>
struct Runs<kStaged, T, LANES> {
  static constexpr int kPitch = LANES * 8 + 8, kWave = 64 / LANES * kPitch;
  float* mine;  // 8 neighbours as they lie in memory
  float* head;  // the lane's head, and its pairs' channels in it
  int first[4], second[4], at;
  __device__ __forceinline__ Runs(const Args& a, const Pairs& p, int lane) {
    __shared__ float staged[4][kWave];
    head = staged[threadIdx.x / 64] + lane / LANES * kPitch;
    const int in = lane % LANES;
    mine = head + in * 8;
    at = in * 8 < a.d ? in * 8 * (int)sizeof(T) : kNowhere;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      // past the head's end: a slot of its own behind it, which holds zeros
      first[v] = p.first[v] < 0 ? 2 * pair_at<kStaged, LANES>(in, v) : p.first[v];
      second[v] = p.second[v] < 0 ? 2 * pair_at<kStaged, LANES>(in, v) + 1 : p.second[v];
    }
  }
  typedef RawN<T, 4> Raw8[2];
  __device__ __forceinline__ void load(Raw8& r, Window w, int row) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) load_rawn(r[i], w, row + at + i * 4 * (int)sizeof(T));
  }
  static __device__ __forceinline__ void handed() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  __device__ __forceinline__ void values(float* f, float* s, const Raw8& r) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) mine[i] = value_of(r[i / 4], i % 4);
    handed();
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      f[v] = head[first[v]];
      s[v] = head[second[v]];
    }
    handed();
  }
  __device__ __forceinline__ void store(Window w, int row, const float* f, const float* s) const {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      head[first[v]] = f[v];
      head[second[v]] = s[v];
    }
    handed();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 x = reinterpret_cast<const float4*>(mine)[i];
      const float y[4] = {x.x, x.y, x.z, x.w};
      store_rawn<T, 4>(w, row + at + i * 4 * (int)sizeof(T), y);
    }
    handed();
  }
};

// Weights or biases of a lane's channels (`none` where there are none).
struct Vec {
  float f[4], s[4];
};
__device__ __forceinline__ Vec vec_of(const float* w, const Pairs& p, float none) {
  Vec o;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    o.f[v] = w && p.first[v] >= 0 ? w[p.first[v]] : none;
    o.s[v] = w && p.second[v] >= 0 ? w[p.second[v]] : none;
  }
  return o;
}

// The norm's statistic: x <- x - mean (layer), and the factor of x.
template <int LANES, int NORM>
__device__ __forceinline__ float normalise(const Args& a, float* f, float* s, const Pairs& p) {
  const float inv_d = 1.0f / a.d;
  if constexpr (NORM == kLayer) {
    float m = 0.0f;
#pragma unroll
    for (int v = 0; v < 4; ++v) m += f[v] + s[v];
    m = head_sum<LANES>(m) * inv_d;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      f[v] = p.first[v] < 0 ? 0.0f : f[v] - m;
      s[v] = p.second[v] < 0 ? 0.0f : s[v] - m;
    }
  }
  float x = 0.0f;
#pragma unroll
  for (int v = 0; v < 4; ++v) x += f[v] * f[v] + s[v] * s[v];
  x = head_sum<LANES>(x);
  if constexpr (NORM == kL2) {
    const float length = sqrtf(x);
    return 1.0f / (length < a.eps ? a.eps : length);  // (the larger one, and NaN of a length that is)
  }
  return __builtin_amdgcn_rsqf(x * inv_d + a.eps);
}

// Norms with weights and biases.
template <int NORM>
constexpr bool kAffine = NORM == kRms || NORM == kLayer;

// A token's row of heads.
template <class T>
__device__ __forceinline__ Window heads_of(const void* rows, int64_t token, int64_t ld, int heads, int d) {
  const T* at = static_cast<const T*>(rows) + token * ld;
  return __builtin_amdgcn_make_buffer_rsrc((void*)at, (short)0, rows ? heads * d * (int)sizeof(T) : 0, 0x00020000);
}

// A wave's token: its heads, 2 kHeads of q's and of k's at a time, all of whose rows are
// asked for before any is computed.
template <class T, int LANES, Access A, int NORM>
__global__ __launch_bounds__(256) void forward_kernel(const Args a) {
  constexpr int kHeads = 64 / LANES, kAhead = 2;
  const int lane = threadIdx.x % 64, head = lane / LANES;
  const Pairs p = pairs_of<A, LANES>(a, lane % LANES);
  const Rotation<A, LANES> rot(a, lane);
  const Runs<A, T, LANES> runs(a, p, lane);
  Vec w[2], b[2];
  if constexpr (kAffine<NORM>) {
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      w[side] = vec_of(a.s[side].w, p, 1.0f);
      b[side] = vec_of(a.s[side].b, p, 0.0f);
    }
  }
  const int most = a.s[0].heads > a.s[1].heads ? a.s[0].heads : a.s[1].heads, row = a.d * (int)sizeof(T);
  const int64_t step = (int64_t)gridDim.x * 4;
  for (int64_t token = (int64_t)blockIdx.x * 4 + delta::uniform(threadIdx.x / 64); token < a.n; token += step) {
    Window x[2], y[2];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const Side& sd = a.s[side];
      x[side] = heads_of<T>(sd.x, token, sd.ld, sd.heads, a.d);
      y[side] = heads_of<T>(sd.y, token, (int64_t)sd.heads * a.d, sd.heads, a.d);
    }
    const Angles t = rot.at(a, token, lane % LANES);
    for (int base = 0; base < most; base += kAhead * kHeads) {
      typename Runs<A, T, LANES>::Raw8 raw[kAhead][2];
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
#pragma unroll
        for (int side = 0; side < 2; ++side) runs.load(raw[j][side], x[side], (base + j * kHeads + head) * row);
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          float u[4], z[4];
          runs.values(u, z, raw[j][side]);
          if constexpr (NORM != kNone) {
            const float r = normalise<LANES, NORM>(a, u, z, p);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              u[v] *= r;
              z[v] *= r;
              if constexpr (kAffine<NORM>) {
                u[v] = u[v] * w[side].f[v] + b[side].f[v];
                z[v] = z[v] * w[side].s[v] + b[side].s[v];
              }
            }
          }
#pragma unroll
          for (int v = 0; v < 4; ++v) turn(p.turned[v], t.c[v], t.s[v], u[v], z[v]);
          runs.store(y[side], (base + j * kHeads + head) * row, u, z);
        }
    }
  }
}

// d = the rotation back of dy; then db += d, dw += d xhat, and with e = d w
//   RMS    dx = r (e - xhat mean(e xhat)),  layer  ... - mean(e),
//   L2     dx = r (e - xhat sum(e xhat)), or e / eps where |x| < eps.
// The sums over rows are a lane's own registers until the end, then a workgroup's
// through LDS in a fixed order, and sum_kernel's.
template <class T, int LANES, Access A, int NORM>
__global__ __launch_bounds__(256) void grad_kernel(const Args a) {
  constexpr int kHeads = 64 / LANES;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, head = lane / LANES;
  const Pairs p = pairs_of<A, LANES>(a, lane % LANES);
  const Rotation<A, LANES> rot(a, lane);
  const Runs<A, T, LANES> runs(a, p, lane);
  float dw[2][8], db[2][8];
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int v = 0; v < 8; ++v) dw[side][v] = db[side][v] = 0.0f;
  Vec w[2];
  if constexpr (kAffine<NORM>) {
    w[0] = vec_of(a.s[0].w, p, 1.0f);
    w[1] = vec_of(a.s[1].w, p, 1.0f);
  }
  const float inv_d = 1.0f / a.d;
  const int most = a.s[0].heads > a.s[1].heads ? a.s[0].heads : a.s[1].heads, row = a.d * (int)sizeof(T);
  const int64_t step = (int64_t)gridDim.x * 4;
  for (int64_t token = (int64_t)blockIdx.x * 4 + delta::uniform(threadIdx.x / 64); token < a.n; token += step) {
    Window x[2], dy[2], dx[2];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const Side& sd = a.s[side];
      x[side] = heads_of<T>(sd.x, token, sd.ld, sd.heads, a.d);
      dy[side] = heads_of<T>(sd.dy, token, (int64_t)sd.heads * a.d, sd.heads, a.d);
      dx[side] = heads_of<T>(sd.y, token, (int64_t)sd.heads * a.d, sd.heads, a.d);
    }
    const Angles t = rot.at(a, token, lane % LANES);
    for (int base = 0; base < most; base += kHeads) {
      typename Runs<A, T, LANES>::Raw8 rx[2], ry[2];
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        if constexpr (NORM != kNone) runs.load(rx[side], x[side], (base + head) * row);
        runs.load(ry[side], dy[side], (base + head) * row);
      }
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        float ef[4], es[4];
        runs.values(ef, es, ry[side]);
#pragma unroll
        for (int v = 0; v < 4; ++v) turn(p.turned[v], t.c[v], -t.s[v], ef[v], es[v]);
        if constexpr (NORM != kNone) {
          float f[4], s[4];
          runs.values(f, s, rx[side]);
          float r = normalise<LANES, NORM>(a, f, s, p);
          const bool clamped = NORM == kL2 && r >= 1.0f / a.eps;
          r = base + head < a.s[side].heads ? r : 0.0f;  // no head: nothing to the sums, whatever eps
          float along = 0.0f, mean = 0.0f;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            f[v] *= r;
            s[v] *= r;
            if constexpr (kAffine<NORM>) {
              db[side][v] += ef[v];
              db[side][4 + v] += es[v];
              dw[side][v] += ef[v] * f[v];
              dw[side][4 + v] += es[v] * s[v];
              ef[v] *= w[side].f[v];
              es[v] *= w[side].s[v];
            }
            along += ef[v] * f[v] + es[v] * s[v];
            mean += ef[v] + es[v];
          }
          along = head_sum<LANES>(along);
          if constexpr (NORM != kL2) along *= inv_d;
          if (clamped) along = 0.0f;
          if constexpr (NORM == kLayer)
            mean = head_sum<LANES>(mean) * inv_d;
          else
            mean = 0.0f;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            ef[v] = (ef[v] - f[v] * along - mean) * r;
            es[v] = (es[v] - s[v] * along - mean) * r;
          }
        }
        runs.store(dx[side], (base + head) * row, ef, es);
      }
    }
  }
  if (a.part == nullptr) return;
  __shared__ float sums[4][kMaxHead];
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      float* mine = kind == 0 ? dw[side] : db[side];
#pragma unroll
      for (int v = 0; v < 8; ++v)
        for (int off = LANES; off < 64; off *= 2) mine[v] += __shfl_xor(mine[v], off, 64);
      __syncthreads();
      if (head == 0) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          if (p.first[v] >= 0) sums[wave][p.first[v]] = mine[v];
          if (p.second[v] >= 0) sums[wave][p.second[v]] = mine[4 + v];
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < a.d; i += 256)
        a.part[((int64_t)blockIdx.x * 4 + 2 * side + kind) * a.d + i] = sums[0][i] + sums[1][i] + (sums[2][i] + sums[3][i]);
    }
}

// out[channel] = the workgroups' sums, in a fixed order: 16 lanes by 16 blocks apart.
struct Outs {
  float* out[4];
};
__global__ __launch_bounds__(256) void sum_kernel(const float* part, int blocks, int d, Outs o) {
  __shared__ float s[16][17];
  const int vec = blockIdx.y, c = threadIdx.x % 16, r = threadIdx.x / 16, ch = blockIdx.x * 16 + c;
  float* out = o.out[vec];
  if (out == nullptr) return;
  float x = 0.0f;
  if (ch < d) {
#pragma unroll 8
    for (int b = r; b < blocks; b += 16) x += part[((int64_t)b * 4 + vec) * d + ch];
  }
  s[r][c] = x;
  __syncthreads();
  if (r == 0 && ch < d) {
    x = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) x += s[i][c];
    out[ch] = x;
  }
}

bool aligned(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Runs of 4 values need rows and heads that keep their alignment, and pairs a half
// apart also axes of multiples of 4 pairs.
Access access(const Args& a, size_t value) {
  bool rows = a.d % 8 == 0;
  for (int i = 0; i < 2; ++i) {
    const Side& s = a.s[i];
    if (s.heads) rows = rows && s.ld % 4 == 0 && aligned(s.x, 4 * value) && aligned(s.y, 4 * value) && aligned(s.dy, 4 * value);
  }
  if (!rows) return kSingle;
  if (a.rotated == 0 || a.interleaved) return kNeighbours;
  bool fours = a.per_axis || a.rotated % 4 == 0;
  for (int i = 0; i < a.axes && a.per_axis; ++i) fours = fours && a.pairs[i] % 4 == 0;
  return fours ? kFours : kStaged;
}

template <class T, int LANES, Access A, int NORM, bool GRAD>
void run(const Args& a, int blocks, hipStream_t s) {
  if (GRAD)
    grad_kernel<T, LANES, A, NORM><<<blocks, 256, 0, s>>>(a);
  else
    forward_kernel<T, LANES, A, NORM><<<blocks, 256, 0, s>>>(a);
}
template <class T, int LANES, Access A, bool GRAD>
void by_norm(const Args& a, int blocks, hipStream_t s) {
  if (a.norm == kNone)
    run<T, LANES, A, kNone, GRAD>(a, blocks, s);
  else if (a.norm == kL2)
    run<T, LANES, A, kL2, GRAD>(a, blocks, s);
  else if (a.norm == kRms)
    run<T, LANES, A, kRms, GRAD>(a, blocks, s);
  else
    run<T, LANES, A, kLayer, GRAD>(a, blocks, s);
}
template <class T, Access A, bool GRAD>
void by_lanes(const Args& a, int blocks, hipStream_t s) {
  if (a.d <= 64)
    by_norm<T, 8, A, GRAD>(a, blocks, s);
  else if (a.d <= 128)
    by_norm<T, 16, A, GRAD>(a, blocks, s);
  else
    by_norm<T, 64, A, GRAD>(a, blocks, s);
}
template <class T, bool GRAD>
void by_access(const Args& a, int blocks, hipStream_t s) {
  const Access how = access(a, sizeof(T));
  if (how == kFours)
    by_lanes<T, kFours, GRAD>(a, blocks, s);
  else if (how == kNeighbours)
    by_lanes<T, kNeighbours, GRAD>(a, blocks, s);
  else if (how == kStaged)
    by_lanes<T, kStaged, GRAD>(a, blocks, s);
  else
    by_lanes<T, kSingle, GRAD>(a, blocks, s);
}

}  // namespace

hipError_t launch_forward(const Args& a, bool bf16, hipStream_t stream) {
  const int64_t units = (a.n + 3) / 4;
  const int blocks = (int)(units < 2048 ? units : 2048);
  if (bf16)
    by_access<uint16_t, false>(a, blocks, stream);
  else
    by_access<float, false>(a, blocks, stream);
  return hipGetLastError();
}

int grad_blocks(int64_t n) {
  const int64_t units = (n + 3) / 4;
  return (int)(units < 768 ? units : 768);  // three waves a SIMD, as their registers allow
}

hipError_t launch_grad(const Args& a, float* const* out, bool bf16, hipStream_t stream) {
  const int blocks = grad_blocks(a.n);
  if (blocks > 0) {
    if (bf16)
      by_access<uint16_t, true>(a, blocks, stream);
    else
      by_access<float, true>(a, blocks, stream);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (out[0] || out[1] || out[2] || out[3]) {
    sum_kernel<<<dim3((a.d + 15) / 16, 4), 256, 0, stream>>>(a.part, blocks, a.d, Outs{{out[0], out[1], out[2], out[3]}});
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace qk
}  // namespace vggt3
