// ra_ffn_mma.h -- a product of the feed-forward block on the tensor cores, as
// its kernel and its launch know it (ra_ffn_mma*).
#pragma once

#include <cuda.h>

#include "ra_ffn.h"

namespace ra {

// One launch's ranks: with more, maps and addresses outgrow a kernel's arguments.
constexpr int kLaunchRanks = 16;

// Buffers of a launch by stage.  Operands, in MmaArgs::map alone (x and grad_out the same for all ranks, or not):
//   hidden       0 x, 1 gate, 2 up
//   out, grad_x  0, 1 hidden, or grad_gate and grad_up; 2, 3 their weights
//   grad_hidden  0 grad_out, 1 down
//   grad_w       0 grad_gate, 1 grad_up, 2 hidden; 3 x, 4 grad_out
// Rows written (and kept rows read), in MmaArgs::rows, and their maps from first_rows(stage) on:
//   hidden       0 hidden, 1 gate, 2 up
//   out, grad_x  0 out
//   grad_hidden  0 grad_gate, 1 grad_up, 2 hidden; 3 gate, 4 up
//   grad_w       0, 1, 2 the weights' gradients
__host__ __device__ constexpr int first_rows(int stage) {
  return stage == kFfnHidden ? 3 : stage == kFfnGradHidden ? 2 : stage == kFfnGradW ? 5 : 4;
}

struct MmaRows {
  char* p[kLaunchRanks];         // NULL: absent
  int64_t stride[kLaunchRanks];  // bytes
  int level;                     // every rank's rows on multiples of: 3, 32 bytes; 2, 16; 1, 8; 0, less
};

struct MmaArgs {
  CUtensorMap map[8][kLaunchRanks];
  MmaRows rows[5];
  float* scales[2][kLaunchRanks];
  int width[kLaunchRanks];
  int64_t tokens;
  int64_t tiles;          // of all jobs
  int tiles_m, tiles_n;   // of one
  int segments;           // products that are summed (grad_x: two)
  int dim, keep_bits;
  int act;                // ra_activation
  int grad_f32;
  ra_device_error* err;   // where a wait that gives up says so
};

// Dtype: RA_BF16 or RA_F16.  kFfnGradX runs as kFfnOut with two segments.
template <int Dtype> cudaError_t launch_ffn_mma(FfnStage stage, const MmaArgs& a, int sms, cudaStream_t st);
// The current device's record of waits that gave up (device memory).
cudaError_t ffn_error_record(ra_device_error** at);

}  // namespace ra
