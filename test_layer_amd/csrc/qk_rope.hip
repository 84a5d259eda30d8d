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
// frequencies and weights over all tokens. A lane holds both channels of 4 pairs:
// no channel moves between lanes, and the norm's sums over a head are a few DPP
// steps over 8 to 64 lanes. Angles are formed in 64 bits (in 32 a position of a
// million is off by 0.06 of a radian) and reduced to a turn before the sine, one
// pair a lane, and handed to the lanes that hold the pair.
#include "qk.hpp"

#include "delta_ops.hpp"

namespace vggt3 {
namespace qk {
namespace {

using delta::load_n;
using delta::store_n;

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
// channels), two runs of 2 twice, 8 neighbours, or anyhow.
enum Access { kFours, kTwos, kNeighbours, kSingle };

// A rotated pair: its channels, axis and turns a position step.
struct Pair {
  int first, second, axis;
  double turns;
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
  p.turns = exp2(-a.log2_base * j / size) * 0.15915494309189533577;
  return p;
}

// The channels of a lane's 4 pairs (-1: past the head's end). Channels that are not
// rotated are paired so that they lie as the others do.
struct Pairs {
  int first[4], second[4];
};
template <Access A>
__device__ __forceinline__ Pairs pairs_of(const Args& a, int lane_in_head) {
  constexpr int kRun = A == kFours ? 4 : A == kTwos ? 2 : 1;
  Pairs p;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int at = 4 * lane_in_head + v;
    if (at < a.rotated) {
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

__device__ __forceinline__ void angle_of(const Args& a, int axis, double turns, int64_t token, float& c, float& s) {
  double x = a.pos[token * a.axes + axis] * turns;
  x -= rint(x);
  sincospif(2.0f * (float)x, &s, &c);
}

// The sines and cosines of a lane's 4 pairs at a token. Heads of up to 128 channels
// have at most 64 pairs: lane l forms those of pair l.
struct Angles {
  float c[4], s[4];
};
template <int LANES>
struct Rotation {
  static constexpr int kOwn = LANES <= 16 ? 1 : 4;
  int axis[kOwn];
  double turns[kOwn];
  __device__ __forceinline__ Rotation(const Args& a, int lane) {
#pragma unroll
    for (int v = 0; v < kOwn; ++v) {
      axis[v] = 0;
      turns[v] = 0.0;
      const int at = kOwn * lane + v;
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
        t.c[v] = __shfl(c[0], 4 * lane_in_head + v, 64);
        t.s[v] = __shfl(s[0], 4 * lane_in_head + v, 64);
      } else {
        t.c[v] = c[v];
        t.s[v] = s[v];
      }
    }
    return t;
  }
};

template <Access A, class T>
__device__ __forceinline__ void load8(float* f, float* s, const T* p, const Pairs& at) {
  if constexpr (A == kFours) {
    load_n<4>(f, p + at.first[0]);
    load_n<4>(s, p + at.second[0]);
  } else if constexpr (A == kTwos) {
    load_n<2>(f, p + at.first[0]);
    load_n<2>(s, p + at.second[0]);
    if (at.first[2] >= 0) {
      load_n<2>(f + 2, p + at.first[2]);
      load_n<2>(s + 2, p + at.second[2]);
    }
  } else if constexpr (A == kNeighbours) {
    float w[8];
    load_n<4>(w, p + at.first[0]);
    load_n<4>(w + 4, p + at.first[0] + 4);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      f[v] = w[2 * v];
      s[v] = w[2 * v + 1];
    }
  } else {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if (at.first[v] >= 0) load_n<1>(&f[v], p + at.first[v]);
      if (at.second[v] >= 0) load_n<1>(&s[v], p + at.second[v]);
    }
  }
}
template <Access A, class T>
__device__ __forceinline__ void store8(T* p, const float* f, const float* s, const Pairs& at) {
  if constexpr (A == kFours) {
    store_n<4>(p + at.first[0], f);
    store_n<4>(p + at.second[0], s);
  } else if constexpr (A == kTwos) {
    store_n<2>(p + at.first[0], f);
    store_n<2>(p + at.second[0], s);
    if (at.first[2] >= 0) {
      store_n<2>(p + at.first[2], f + 2);
      store_n<2>(p + at.second[2], s + 2);
    }
  } else if constexpr (A == kNeighbours) {
    float w[8];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      w[2 * v] = f[v];
      w[2 * v + 1] = s[v];
    }
    store_n<4>(p + at.first[0], w);
    store_n<4>(p + at.first[0] + 4, w + 4);
  } else {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if (at.first[v] >= 0) store_n<1>(p + at.first[v], &f[v]);
      if (at.second[v] >= 0) store_n<1>(p + at.second[v], &s[v]);
    }
  }
}

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
  if constexpr (NORM == kL2) return 1.0f / fmaxf(sqrtf(x), a.eps);
  return __builtin_amdgcn_rsqf(x * inv_d + a.eps);
}

// Norms with weights and biases.
template <int NORM>
constexpr bool kAffine = NORM == kRms || NORM == kLayer;

// A wave's token: its heads, kHeads at a time, q's and then k's. The next heads' rows
// are asked for before the current ones are computed.
template <class T, int LANES, Access A, int NORM>
__global__ __launch_bounds__(256) void forward_kernel(const Args a) {
  constexpr int kHeads = 64 / LANES;
  const int lane = threadIdx.x % 64, head = lane / LANES;
  const Pairs p = pairs_of<A>(a, lane % LANES);
  const Rotation<LANES> rot(a, lane);
  const bool live = p.first[0] >= 0;  // lanes behind a head's end
  Vec w[2], b[2];
  if constexpr (kAffine<NORM>) {
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      w[side] = vec_of(a.s[side].w, p, 1.0f);
      b[side] = vec_of(a.s[side].b, p, 0.0f);
    }
  }
  const int64_t step = (int64_t)gridDim.x * 4;
  for (int64_t token = (int64_t)blockIdx.x * 4 + threadIdx.x / 64; token < a.n; token += step) {
    const Angles t = rot.at(a, token, lane % LANES);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const Side& sd = a.s[side];
      if (sd.heads == 0) continue;
      const T* x = static_cast<const T*>(sd.x) + token * sd.ld;
      T* y = static_cast<T*>(sd.y) + token * sd.heads * a.d;
      float f[4] = {0, 0, 0, 0}, s[4] = {0, 0, 0, 0};
      if (head < sd.heads && live) load8<A>(f, s, x + head * a.d, p);
      for (int h = head;;) {
        const bool here = h < sd.heads && live, more = h - head + kHeads < sd.heads;
        float nf[4] = {0, 0, 0, 0}, ns[4] = {0, 0, 0, 0};
        if (more && h + kHeads < sd.heads && live) load8<A>(nf, ns, x + (h + kHeads) * a.d, p);
        if constexpr (NORM != kNone) {
          const float r = normalise<LANES, NORM>(a, f, s, p);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            f[v] *= r;
            s[v] *= r;
            if constexpr (kAffine<NORM>) {
              f[v] = f[v] * w[side].f[v] + b[side].f[v];
              s[v] = s[v] * w[side].s[v] + b[side].s[v];
            }
          }
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float m = f[v] * t.c[v] - s[v] * t.s[v];
          s[v] = s[v] * t.c[v] + f[v] * t.s[v];
          f[v] = m;
        }
        if (here) store8<A>(y + h * a.d, f, s, p);
        if (!more) break;
        h += kHeads;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          f[v] = nf[v];
          s[v] = ns[v];
        }
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
  const Pairs p = pairs_of<A>(a, lane % LANES);
  const Rotation<LANES> rot(a, lane);
  const bool live = p.first[0] >= 0;
  float dw[2][8], db[2][8];
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int v = 0; v < 8; ++v) dw[side][v] = db[side][v] = 0.0f;
  Vec ws[2];
  if constexpr (kAffine<NORM>) {
    ws[0] = vec_of(a.s[0].w, p, 1.0f);
    ws[1] = vec_of(a.s[1].w, p, 1.0f);
  }
  const float inv_d = 1.0f / a.d;
  for (int64_t token = (int64_t)blockIdx.x * 4 + wave; token < a.n; token += (int64_t)gridDim.x * 4) {
    const Angles t = rot.at(a, token, lane % LANES);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const Side& sd = a.s[side];
      if (sd.heads == 0) continue;
      const Vec& w = ws[side];
      const T* x = static_cast<const T*>(sd.x) + token * sd.ld;
      const T* dy = static_cast<const T*>(sd.dy) + token * sd.heads * a.d;
      T* dx = static_cast<T*>(sd.y) + token * sd.heads * a.d;
      float xf[4] = {0, 0, 0, 0}, xs[4] = {0, 0, 0, 0}, yf[4] = {0, 0, 0, 0}, ys[4] = {0, 0, 0, 0};
      if (head < sd.heads && live) {
        if constexpr (NORM != kNone) load8<A>(xf, xs, x + head * a.d, p);
        load8<A>(yf, ys, dy + head * a.d, p);
      }
      for (int h = head;;) {
        const bool here = h < sd.heads && live, more = h - head + kHeads < sd.heads;
        float f[4], s[4], ef[4], es[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          f[v] = xf[v];
          s[v] = xs[v];
          ef[v] = yf[v];
          es[v] = ys[v];
          xf[v] = xs[v] = yf[v] = ys[v] = 0.0f;
        }
        if (more && h + kHeads < sd.heads && live) {
          if constexpr (NORM != kNone) load8<A>(xf, xs, x + (h + kHeads) * a.d, p);
          load8<A>(yf, ys, dy + (h + kHeads) * a.d, p);
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float m = ef[v] * t.c[v] + es[v] * t.s[v];
          es[v] = es[v] * t.c[v] - ef[v] * t.s[v];
          ef[v] = m;
        }
        if constexpr (NORM != kNone) {
          const float r = normalise<LANES, NORM>(a, f, s, p);
          const bool clamped = NORM == kL2 && r >= 1.0f / a.eps;
          float along = 0.0f, mean = 0.0f;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            f[v] *= r;
            s[v] *= r;
            if (kAffine<NORM> && a.part && here) {
              db[side][v] += ef[v];
              db[side][4 + v] += es[v];
              dw[side][v] += ef[v] * f[v];
              dw[side][4 + v] += es[v] * s[v];
            }
            if constexpr (kAffine<NORM>) {
              ef[v] *= w.f[v];
              es[v] *= w.s[v];
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
        if (here && sd.y) store8<A>(dx + h * a.d, ef, es, p);
        if (!more) break;
        h += kHeads;
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

// Runs of 4 or 2 channels need each axis's channels, the heads and the rows to be
// multiples of them, and rows to start at a run's alignment.
Access access(const Args& a, size_t value) {
  int run = a.d % 8 == 0 ? 4 : a.d % 4 == 0 ? 2 : 1;
  const bool halves = a.rotated > 0 && !a.interleaved;
  if (halves && a.per_axis)
    for (int i = 0; i < a.axes; ++i)
      while (a.pairs[i] % run) run /= 2;
  else if (halves)
    while (a.rotated % run) run /= 2;
  for (int i = 0; i < 2; ++i) {
    const Side& s = a.s[i];
    if (s.heads == 0) continue;
    while (s.ld % run || !aligned(s.x, run * value) || !aligned(s.y, run * value) || !aligned(s.dy, run * value)) run /= 2;
  }
  if (!halves) return run == 4 ? kNeighbours : kSingle;
  return run == 4 ? kFours : run == 2 ? kTwos : kSingle;
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
  else if (how == kTwos)
    by_lanes<T, kTwos, GRAD>(a, blocks, s);
  else if (how == kNeighbours)
    by_lanes<T, kNeighbours, GRAD>(a, blocks, s);
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
