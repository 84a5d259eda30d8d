// Launchers of the block-join kernels (norm after a block, gate, residual
// scale, residual, norm before the next block; forward and gradient).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace vggt3 {
namespace join {

enum Norm { kNone = 0, kRms = 1, kLayer = 2 };

// Widest row: 512 threads of 16 values.
constexpr int kMaxChannels = 8192;

struct Args {
  const void* x;     // forward: the stream; gradient: the joined stream r
  const void* f;     // NULL: no block output (the norm of x alone)
  const void* gate;  // NULL or [ceil(n/per)][C]
  const float* scale;
  const float* post_w;
  const float* post_b;
  const float* pre_w;
  const float* pre_b;
  void* r;
  void* y;
  uint8_t* y_codes;
  uint8_t* y_scales;
  const void* dr;
  const void* dy;
  void* dx;
  void* df;
  void* dgate;
  float* part;  // gradient: per-workgroup sums over tokens, [blocks][kVecs][C]
  float* edge;  // gradient: sums of gate groups that units share, [units][2][C]
  int64_t n, per, rows_per_unit;
  int C, post, pre;
  float eps;
};

// The per-workgroup sums (see block_join.hip), and the channel gradients made of
// them.
enum Sum { kA, kB, kSumPreW, kSumPreB, kVecs };
enum Out { kDScale, kDPostW, kDPostB, kDPreW, kDPreB, kOuts };

hipError_t launch_forward(const Args& a, bool bf16, hipStream_t stream);

// The gradient: rows in units of rows_per_unit tokens, `blocks` workgroups.
struct GradPlan {
  int64_t rows_per_unit, units, blocks;
};
GradPlan grad_plan(int64_t n, int C, bool bf16);
// out[v]: NULL or fp32 [C]; zeros for n = 0.
hipError_t launch_grad(const Args& a, const GradPlan& p, float* const* out, bool bf16, hipStream_t stream);

}  // namespace join
}  // namespace vggt3
