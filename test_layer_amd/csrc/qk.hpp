// Launchers of the query/key preparation: a norm of each head and the rotation of
// its channels by positions on up to 4 axes, and the gradient of both.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace vggt3 {
namespace qk {

enum Norm { kNone = 0, kRms = 1, kLayer = 2, kL2 = 3 };

constexpr int kMaxAxes = 4;
constexpr int kMaxHead = 512;  // 64 lanes of 8 channels

struct Side {       // queries or keys
  const void* x;    // rows of heads * d values, `ld` apart
  const void* dy;   // gradient: [n][heads][d]
  void* y;          // [n][heads][d]; gradient: dx, or NULL
  const float* w;   // NULL (1) or [d]
  const float* b;   // NULL (0) or [d]
  int64_t ld;
  int heads;
};

struct Args {
  Side s[2];
  const int32_t* pos;  // [n][axes]
  float* part;         // gradient: per-workgroup sums over rows, [blocks][4][d]: q's w, q's b, k's w, k's b
  int64_t n;
  int d, norm, axes;
  int pairs[kMaxAxes];  // rotated pairs of channels of each axis
  int rotated;          // their sum
  int per_axis;         // each axis has channels and a ladder of frequencies of its own
  int interleaved;      // pairs are neighbours; otherwise a half apart
  double step[kMaxAxes][2];  // base^(-1 / size) of each axis's ladder, in two doubles
  float eps;
};

hipError_t launch_forward(const Args& a, bool bf16, hipStream_t stream);
int grad_blocks(int64_t n);
// out[v]: NULL or fp32 [d]; zeros for n = 0.
hipError_t launch_grad(const Args& a, float* const* out, bool bf16, hipStream_t stream);

}  // namespace qk
}  // namespace vggt3
