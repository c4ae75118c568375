// ra_ffn_mma.h -- a product of the feed-forward block on the tensor cores, as
// its kernel and its launch know it (ra_ffn_mma*.cu).
#pragma once

#include <cuda.h>

#include "ra_ffn.h"

namespace ra {

// Which of a call's outputs (and kept inputs) have rows on 16-byte boundaries.
enum MmaVec : int { kVecHidden = 1, kVecKept = 2, kVecPre = 4, kVecOut = 8, kVecGradW = 16 };

struct MmaArgs {
  FfnArgs f;
  int64_t tiles;          // of all jobs
  int tiles_m, tiles_n;   // of one
  int segments;           // products that are summed (grad_x: two)
  int vec;                // MmaVec
  ra_device_error* err;   // where a wait that gives up says so
  CUtensorMap a[3][kMaxRanks], b[2][kMaxRanks];
};

// Dtype: RA_BF16 or RA_F16
template <int Dtype> cudaError_t launch_ffn_mma(FfnStage stage, const MmaArgs& a, int sms, cudaStream_t st);
// The current device's record of waits that gave up (device memory).
cudaError_t ffn_error_record(ra_device_error** at);

}  // namespace ra
