// ra_ffn_mma.h -- a product of the feed-forward block on the tensor cores, as
// its kernel and its launch know it (ra_ffn_mma*).
#pragma once

#include <cuda.h>

#include "ra_ffn.h"

namespace ra {

// Buffers of a launch by stage.  Operands, by their maps alone (x and grad_out the same for all ranks, or not):
//   hidden       0 x, 1 gate, 2 up
//   out, grad_x  0, 1 hidden, or grad_gate and grad_up; 2, 3 their weights
//   grad_hidden  0 grad_out, 1 down
//   grad_w       0 grad_gate, 1 grad_up, 2 hidden; 3 x, 4 grad_out
// Rows written (and kept rows read), and their maps from first_rows(stage) on:
//   hidden       0 hidden, 1 gate, 2 up
//   out, grad_x  0 out
//   grad_hidden  0 grad_gate, 1 grad_up, 2 hidden; 3 gate, 4 up
//   grad_w       0, 1, 2 the weights' gradients
__host__ __device__ constexpr int first_rows(int stage) {
  return stage == kFfnHidden ? 3 : stage == kFfnGradHidden ? 2 : stage == kFfnGradW ? 5 : 4;
}

// What a launch knows of a rank, in one place: a CTA reads one rank's alone.
template <int Maps> struct MmaRank {
  CUtensorMap map[Maps];
  char* rows[5];         // NULL: absent
  int64_t stride[5];     // bytes
  float* scales[2];
  int width;
};

// Ranks of one launch, `Ranks` at most: with more, maps and addresses outgrow a kernel's arguments.
template <int Maps, int Ranks>
struct MmaArgsOf {
  static constexpr int kMaps = Maps, kRanks = Ranks;
  int64_t tokens;
  int64_t tiles;          // of all jobs
  int tiles_m, tiles_n;   // of one; for few tokens: of the weights' rows, of the tokens
  int segments;           // products that are summed (grad_x: two)
  int dim, keep_bits;
  int act;                // ra_activation
  int grad_f32;
  int level[5];           // rows of every rank on multiples of: 2, 16 bytes (of tensor maps); 1, 8; 0, less
  // for few tokens alone
  int nt;                 // tokens of a tile, a multiple of 16, at most 128
  int split;              // CTAs that share the terms of a tile's sums: 1, 2, 4 or 8
  int early;              // the stream's kernel before this one is the call's own
  int ring;               // bytes of the operands' ring
  WaitRecord* record;     // where a wait that gives up says so
  MmaRank<Maps> rank[Ranks];
};
using MmaArgs = MmaArgsOf<8, 16>;
// For few tokens operands alone have maps; and few ranks' arguments are handed over sooner.
template <int Ranks> using FewArgs = MmaArgsOf<4, Ranks>;
constexpr int kFewRanks = 8;

// Dtype: RA_BF16 or RA_F16.  kFfnGradX runs as kFfnOut with two segments.
template <int Dtype> cudaError_t launch_ffn_mma(FfnStage stage, const MmaArgs& a, int sms, cudaStream_t st);
// All but kFfnGradW, for few tokens; the operands' maps of the tokens have boxes of a.nt rows.
template <int Dtype> cudaError_t launch_ffn_few(FfnStage stage, const FewArgs<kFewRanks>& a, cudaStream_t st);
template <int Dtype> cudaError_t launch_ffn_few(FfnStage stage, const FewArgs<kMaxRanks>& a, cudaStream_t st);
// Rings for few tokens: for one CTA an SM, or two.
constexpr int kFewRing = 104 * 1024, kFewRingAlone = 208 * 1024;
constexpr int kFewABytes = 128 * 64 * 2, kFewMostStages = 12;
__host__ __device__ constexpr int few_sums(int stage) { return stage == kFfnHidden ? 2 : 1; }   // accumulators
__host__ __device__ constexpr int few_stage_bytes(int stage, int nt) { return few_sums(stage) * kFewABytes + nt * 128; }

}  // namespace ra
