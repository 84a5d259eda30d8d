// Launchers of the gated delta rule's kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace vggt3 {
namespace delta {

struct Args {
  const void* q;  // [n][hk dk]
  const void* k;
  const void* v;      // [n][hv dv]
  const float* g;     // NULL or [n][hv]
  const float* beta;  // [n][hv]
  const int32_t* cu;  // NULL (one sequence) or [nseq + 1]
  const float* state; // NULL (zeros) or [nseq][hv][dk][dv]
  void* o;
  float* state_out;
  void* mats;  // [chunks][hv]: the chunks' shared matrices
  int keep;    // those of the gradient among them
  // pieces (segments) of a sequence that are worked on at once
  float* seg_n;  // [pieces][hv][dk][dv]: a piece's last state from none; then its first state
  float* seg_m;  // [pieces][hv][dk][dk]: what it makes of its first state
  // gradient
  const void* dout;    // of o
  const float* dlast;  // of state_out: NULL (zeros) or [nseq][hv][dk][dv]
  float* dfirst;       // of state
  float* states;       // [chunks][hv][dk][dv]: the state before each chunk
  float* dstates;      // the gradient of the state after each chunk
  void* dq;            // each NULL: not wanted
  void* dk_out;
  void* dv_out;
  float* dg;
  float* dbeta;
  float* dq_part;  // [n][hv][dk], where value heads share a key head
  float* dk_part;
  uint32_t* cuts;  // NULL or [2][nseq]: the first piece of each sequence, its first chunk
  int64_t n, per, pieces;  // per: tokens of a piece; pieces: room for
  int nseq, hk, hv, dk, dv;
  float scale;
};

// How a call's sequences are cut: pieces of `per` tokens, at most `pieces` in all;
// split: whether a sequence may have more than one.
// wide: a wave has 64 columns (32 where d_k is 128) instead of 16.
struct Plan {
  int64_t per, pieces;
  bool split, wide;
};
Plan plan(int64_t n, int nseq, int64_t longest, int hv, int dk, int dv);

struct StepArgs {
  const void* q;  // [rows][hk dk]
  const void* k;
  const void* v;         // [rows][hv dv]
  const float* g;        // NULL or [rows][hv]
  const float* beta;     // [rows][hv]
  float* state;          // [n_slots][hv][dk][dv], updated
  const int32_t* slots;  // NULL (row r: slot r) or [rows]
  void* o;
  int64_t n_slots;
  int rows, hk, hv, dk, dv;
  float scale;
};

hipError_t launch_step(const StepArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_forward(const Args& a, const Plan& p, bool bf16, hipStream_t stream);

// Bytes of a chunk's and head's shared matrices (keep: with the gradient's).
size_t matrix_bytes(bool keep);

// More sequences than a wave looks at by itself: their pieces' numbers are written down
// beforehand, a launch more (64 sequences of a token 23 us, with it 26).
inline bool needs_cuts(bool cu, int nseq) { return cu && nseq >= 256; }

// The gradient: the state before every chunk, then the gradient of the state after
// every chunk (and dfirst), then everything else chunk by chunk. A sequence has a chunk
// and a piece at least; where sequences share no rows, chunks' numbers are below this.
__host__ __device__ constexpr int64_t chunk_slots(int64_t n, int nseq) { return n / 32 + nseq; }
hipError_t launch_states(const Args& a, const Plan& p, bool bf16, hipStream_t stream);
hipError_t launch_back(const Args& a, const Plan& p, bool bf16, hipStream_t stream);
hipError_t launch_grad(const Args& a, bool bf16, hipStream_t stream);

}  // namespace delta
}  // namespace vggt3
