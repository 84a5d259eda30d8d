// One token of each of several streams by the gated delta rule, on states that lie
// in a cache. With S the state before it, a its decay,
//
//   p = a S^T k,  u = beta (v - p),  S' = a S + k u^T,  o = S'^T q = a S^T q + (k . q) u
//
// so one pass over S gives both sums over its rows, S^T k and S^T q, and the pass
// that stores S' needs none. Bound by the state, read once and written once. A
// workgroup holds 64 columns of one head's state in registers, 4 columns and every
// 16th row a thread (16 bytes a load, 256 contiguous a row). 256 streams of 16 heads of
// 64 x 64: 24.7 us, 5.5 TB/s, a copy's rate; one stream 9 us, a call's host time.
#include "delta.hpp"
#include "delta_ops.hpp"

namespace vggt3 {
namespace delta {
namespace {

template <class T, int DK>
__global__ __launch_bounds__(256) void step_kernel(const StepArgs a) {
  constexpr int kRows = DK / 16;
  __shared__ float sums[2][4][2][64];  // [turn][wave][k, q][column]
  __shared__ float dots[2][4];
  __shared__ int seen[4], later[2][4];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int c = lane % 16, q = lane / 16;
  const int h = blockIdx.x % a.hv;
  int row = blockIdx.x / a.hv;
  const int col = blockIdx.y * 64 + 4 * c;
  const int kh = h / (a.hv / a.hk);
  const int64_t ldk = (int64_t)a.hk * DK, ldv = (int64_t)a.hv * a.dv;
  const int64_t slot = a.slots ? a.slots[row] : row;
  if (slot < 0 || slot >= a.n_slots) {  // a row of a padded batch
    if (wave == 0 && q == 0) {
      const float none[4] = {0.f, 0.f, 0.f, 0.f};
      store_n<4>(static_cast<T*>(a.o) + row * ldv + h * a.dv + col, none);
    }
    return;
  }
  float* state = a.state + (slot * a.hv + h) * DK * a.dv + col;
  f32x4 S[kRows];
#pragma unroll
  for (int x = 0; x < kRows; ++x)
    S[x] = *reinterpret_cast<const f32x4*>(state + (int64_t)(16 * x + 4 * wave + q) * a.dv);
  // The first row of a slot serves all its rows, in their order.
  int next = a.rows;
  if (a.slots) {
    int before = 0;
    for (int i = tid; i < a.rows; i += 256)
      if (a.slots[i] == slot) {
        if (i < row) before = 1;
        if (i > row && i < next) next = i;
      }
    before = __any(before);
#pragma unroll
    for (int off = 32; off; off /= 2) next = min(next, __shfl_xor(next, off, 64));
    if (lane == 0) {
      seen[wave] = before;
      later[0][wave] = next;
    }
  }
  for (int turn = 0;; turn ^= 1) {
    const T* kp = static_cast<const T*>(a.k) + row * ldk + kh * DK;
    const T* qp = static_cast<const T*>(a.q) + row * ldk + kh * DK;
    float kv[kRows], v[4];
    const float decay = a.g ? expf(a.g[(int64_t)row * a.hv + h]) : 1.0f, beta = a.beta[(int64_t)row * a.hv + h];
    load_n<4>(v, static_cast<const T*>(a.v) + row * ldv + h * a.dv + col);
    f32x4 sk = zero4(), sq = zero4();
    float kq = 0.0f;
#pragma unroll
    for (int x = 0; x < kRows; ++x) {
      float qv;
      load_n<1>(&kv[x], kp + 16 * x + 4 * wave + q);
      load_n<1>(&qv, qp + 16 * x + 4 * wave + q);
      sk += S[x] * kv[x];
      sq += S[x] * qv;
      kq += kv[x] * qv;
    }
#pragma unroll
    for (int off = 16; off < 64; off *= 2) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sk[j] += __shfl_xor(sk[j], off, 64);
        sq[j] += __shfl_xor(sq[j], off, 64);
      }
      kq += __shfl_xor(kq, off, 64);
    }
    if (q == 0) {
      *reinterpret_cast<f32x4*>(&sums[turn][wave][0][4 * c]) = sk;
      *reinterpret_cast<f32x4*>(&sums[turn][wave][1][4 * c]) = sq;
    }
    if (lane == 0) dots[turn][wave] = kq;
    __syncthreads();
    if (a.slots) {
      if (seen[0] | seen[1] | seen[2] | seen[3]) return;  // an earlier row serves this one
      next = min(min(later[turn][0], later[turn][1]), min(later[turn][2], later[turn][3]));
    }
    sk = sq = zero4();
    kq = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      sk += *reinterpret_cast<const f32x4*>(&sums[turn][w][0][4 * c]);
      sq += *reinterpret_cast<const f32x4*>(&sums[turn][w][1][4 * c]);
      kq += dots[turn][w];
    }
    f32x4 u;
    float o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] = beta * (v[j] - decay * sk[j]);
      o[j] = a.scale * (decay * sq[j] + kq * u[j]);
    }
    if (wave == 0 && q == 0) store_n<4>(static_cast<T*>(a.o) + row * ldv + h * a.dv + col, o);
#pragma unroll
    for (int x = 0; x < kRows; ++x) S[x] = S[x] * decay + u * kv[x];
    if (next >= a.rows) break;
    row = next;
    // the other turn's buffers: the next one's reads of these lie behind its barrier
    next = a.rows;
    for (int i = row + 1 + tid; i < a.rows; i += 256)
      if (a.slots[i] == slot) {
        next = i;
        break;
      }
#pragma unroll
    for (int off = 32; off; off /= 2) next = min(next, __shfl_xor(next, off, 64));
    if (lane == 0) later[turn ^ 1][wave] = next;
  }
#pragma unroll
  for (int x = 0; x < kRows; ++x)
    *reinterpret_cast<f32x4*>(state + (int64_t)(16 * x + 4 * wave + q) * a.dv) = S[x];
}

}  // namespace

hipError_t launch_step(const StepArgs& a, bool bf16, hipStream_t stream) {
  const dim3 grid((unsigned)(a.rows * a.hv), a.dv / 64);
  if (bf16) {
    if (a.dk == 64)
      step_kernel<uint16_t, 64><<<grid, 256, 0, stream>>>(a);
    else
      step_kernel<uint16_t, 128><<<grid, 256, 0, stream>>>(a);
  } else {
    if (a.dk == 64)
      step_kernel<float, 64><<<grid, 256, 0, stream>>>(a);
    else
      step_kernel<float, 128><<<grid, 256, 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace delta
}  // namespace vggt3
