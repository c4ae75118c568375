// ra_ops.h -- what the model operators' host side (ra_ops_host.cpp) and their
// kernels (ra_norm.cu, ra_vocab.cu) share: kernel argument blocks and launch
// functions.  Nothing here is part of the public C ABI (include/ra.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ra.h"
#include "ra_internal.h"

namespace ra {

constexpr int kNormMaxDim = 16384;
constexpr int kTopMax = 32;       // alternatives per row: one per lane of a warp
constexpr int kTeacherMax = 256;  // teacher tokens per row
constexpr float kLog2e = 1.4426950408889634f;

// Block end, forward.  Strides in elements; pointers of absent tensors NULL.
struct NormForward {
  const void* in[kMaxRanks];
  void* out[kMaxRanks];
  const void* residual;
  void* residual_out;
  void* total;
  const void* weight;
  const void* post_weight;
  const void* gate;
  float* rstd;            // [2][rows]: the post norm's, then the pre norm's
  int64_t rows, in_stride, out_stride, residual_stride, residual_out_stride, total_stride;
  int64_t rows_per_gate;  // rows that share one gate row
  int R, outs, dim;
  int param_f32;          // weights and gate are binary32 (else the activations' type)
  float eps, scale;
};

// Block end, backward.
struct NormBackward {
  const void* grad_out[kMaxRanks];   // `grads` partial gradients of the normalised rows
  void* grad_in[kMaxRanks];          // `outs` copies of the partials' gradient
  const void* grad_residual_out;     // may be NULL (zero)
  const void* residual_out;
  const void* total;                 // NULL only without post norm and gate gradient
  const float* rstd;
  const void* weight;
  const void* post_weight;
  const void* gate;
  void* grad_residual;
  float* grad_weight;
  float* grad_post_weight;
  float* grad_gate;
  float* work;                       // column partials, norm_workspace_floats()
  int64_t rows, grad_out_stride, grad_in_stride, grad_residual_out_stride, residual_out_stride, total_stride,
      grad_residual_stride;
  int64_t rows_per_gate;
  int64_t groups;                    // gate rows (1 without a gate)
  int grads, outs, dim;
  int param_f32;
  float scale;
};

// The kernels that a handle has opted in to their shared memory: a forward and
// a backward one for few and for many rows, aligned or not.
struct OptedIn {
  const void* kernels[8] = {};
  int count = 0;
  bool has(const void* k) const {
    for (int i = 0; i < count; ++i)
      if (kernels[i] == k) return true;
    return false;
  }
  void add(const void* k) {
    if (count < 8) kernels[count++] = k;
  }
};

// aligned: every row of every buffer starts on a 16-byte boundary and holds whole 16-byte vectors
cudaError_t launch_norm_forward(int dtype, int residual_dtype, bool aligned, const NormForward& a, int sms,
                                OptedIn& opted, cudaStream_t st);
cudaError_t launch_norm_backward(int dtype, int residual_dtype, bool aligned, const NormBackward& a, int sms,
                                 OptedIn& opted, cudaStream_t st);
// Floats of column partials a backward call of this width may use.
size_t norm_workspace_floats(int dim, int sms);

// A row of the vocabulary: shard r holds the columns [r C, min((r+1) C, V)).
struct VocabRows {
  const void* shard[kMaxRanks];
  int64_t stride[kMaxRanks];   // elements between rows
  int64_t rows;
  int shards;                  // shards that hold a column
  int V, C;
  int slots;                   // 16-byte slots that a shard's columns touch at most
  float tau, inv_tau;
  float scale;                 // log2(e) / tau, rounded
  float unit, unit_rest;       // 1 / (tau scale) in two parts: what 1 in the scaled logits is in x / tau
};

struct VocabForward {
  VocabRows x;
  float* lse;
  // log probabilities
  const int64_t* targets;
  float* logprob;
  float* entropy;              // may be NULL
  int64_t* top_ids;            // [rows][top], NULL when top == 0
  float* top_logprobs;
  int top;
  // distillation
  const int64_t* ids;          // [rows][K]
  const void* teacher;         // [rows][K]
  float* loss;
  int K;
  int teacher_f32;             // else the logits' type
};

struct VocabBackward {
  VocabRows x;
  void* grad[kMaxRanks];
  int64_t grad_stride[kMaxRanks];
  const float* lse;
  const int64_t* targets;      // log probabilities (NULL: distillation)
  const float* entropy;
  const float* grad_entropy;   // NULL: no entropy term
  const float* g;              // gradient of the log probability or of the loss, per row
  const int64_t* ids;
  const void* teacher;
  int K;
  int teacher_f32;
  float lift, by_lift;         // a whole number and 2^-lift: see the kernel
};

cudaError_t launch_vocab_forward(int dtype, const VocabForward& a, int sms, cudaStream_t st);
cudaError_t launch_vocab_backward(int dtype, const VocabBackward& a, int sms, cudaStream_t st);

}  // namespace ra
