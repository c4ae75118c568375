// ra_ffn.h -- what the host side of the feed-forward block and of kept rows
// (ra_ffn_host.cpp) and their kernels (ra_ffn_*.cu, ra_ckpt.cu) share.
// Nothing here is part of the public C ABI (include/ra.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ra.h"
#include "ra_internal.h"

namespace ra {

constexpr int kGroup = 128;   // columns of a row that share a scale

// The products a block consists of.  Rank r holds `width(r)` inner columns;
// its weights are [width][dim].
//   hidden      [rows][width] = act(x gate^T) (x up^T)           sums over dim
//   out         [rows][dim]   = hidden down                      sums over width
//   grad_hidden [rows][width]: dh = dy down^T, and from it and the kept
//               projections grad_gate, grad_up and hidden        sums over dim
//   grad_x      [rows][dim]   = grad_gate gate + grad_up up      sums over 2 width
//   grad_w      [width][dim]  = grad_gate^T x, grad_up^T x, hidden^T dy   sums over rows
enum FfnStage : int { kFfnHidden = 0, kFfnOut = 1, kFfnGradHidden = 2, kFfnGradX = 3, kFfnGradW = 4 };

// One call's buffers; strides in elements.  Pointers of absent tensors are NULL.
struct FfnArgs {
  const void* x[kMaxRanks];          // the same for every rank where there is one
  const void* grad_out[kMaxRanks];   // so here
  const void* w[3][kMaxRanks];       // gate, up, down
  void* hidden[kMaxRanks];
  void* out[kMaxRanks];              // partial products, or partial gradients of x
  void* kept[2][kMaxRanks];          // gate, up
  float* scales[2][kMaxRanks];       // contiguous
  void* grad_pre[2][kMaxRanks];      // gate, up
  void* grad_w[3][kMaxRanks];        // gate, up, down
  int64_t x_stride, grad_out_stride, out_stride;
  int64_t w_stride[3][kMaxRanks], hidden_stride[kMaxRanks], kept_stride[2][kMaxRanks], grad_pre_stride[2][kMaxRanks],
      grad_w_stride[3][kMaxRanks];
  int64_t rows;
  int R, dim, inner, C;              // C: columns of a full rank
  int keep_bits;                     // 0, 8, 16
  int act;                           // ra_activation
  int grad_f32;                      // the weights' gradients are binary32
#ifdef __CUDACC__
  __host__ __device__
#endif
  int width(int r) const {
    const int64_t left = (int64_t)inner - (int64_t)r * C;
    return left < 0 ? 0 : left < C ? (int)left : C;
  }
};

// Waits of the products that gave up, in device memory, one record a device:
// the first since the host took it last, and how many there have been.
struct WaitRecord {
  ra_device_error first;
  uint32_t count;
};
// The current device's.
cudaError_t ffn_wait_record(WaitRecord** at);
#ifdef RA_DEBUG_BOUNDS
cudaError_t launch_ffn_give_up(WaitRecord* record, cudaStream_t st);   // writes one down
#endif

// On the CUDA cores: any start and stride.
cudaError_t launch_ffn_simple(int dtype, FfnStage stage, const FfnArgs& a, int sms, cudaStream_t st);

// Rows kept in 8 bits.
struct CkptArgs {
  void* values;         // stored: read, loaded: written; may be NULL then
  int8_t* codes;
  float* scales;        // [rows][groups]
  const float* rstd;
  const void* weight;
  void* normed;         // may be NULL
  int64_t rows, stride, codes_stride, normed_stride;
  int dim;
  uint32_t by;          // n / groups = (mulhi(n, by) + n) >> shift for n below 2^31
  int shift;
  // Groups of a row, and by and shift for them.
  int set_groups() {
    const int groups = (dim + kGroup - 1) / kGroup;
    shift = 0;
    while (((int64_t)1 << shift) < groups) ++shift;
    by = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << shift) - (uint64_t)groups)) / (uint64_t)groups + 1);
    return groups;
  }
};
// wide: rows of every buffer start on 16-byte boundaries (codes: 8) and hold whole groups of 8 columns
cudaError_t launch_ckpt_store(int dtype, bool wide, const CkptArgs& a, int sms, cudaStream_t st);
cudaError_t launch_ckpt_load(int dtype, int normed_dtype, int param_dtype, bool wide, const CkptArgs& a, int sms,
                             cudaStream_t st);

}  // namespace ra
