// ra_ffn_simple.cu -- the feed-forward block's products on the CUDA cores, for
// operands whose rows do not start on 16-byte boundaries, which the tensor
// cores' copies cannot fetch.
//
// A CTA takes a tile of 64 x 128 of one rank's product, through shared memory
// 16 terms at a time; a thread accumulates 4 x 8 sums in binary32 registers
// (the gated projections: two sets), columns 16 apart, so that its half warp
// holds the 128 columns that share a scale.  Right for every call, and slow: 17
// TFLOP/s, loads of single elements and their addresses (2048 tokens, 2047 x
// 8191 in two ranks, forward: 12.5 ms, where 2048 x 8192 takes 0.12 on the tensor cores;
// one token of 4095 x 16383 in eight: 2.0 ms and 0.07).
#include "ra_ffn.cuh"
#include "ra_ffn_mma.h"
#include "ra_tensor.cuh"

namespace ra {

namespace {

constexpr int kTileM = 64, kTileN = 128, kTileK = 16, kThreads = 256;

// Element (i, k) of an operand: k runs along a row, or i does.
template <class T, bool KMajor> struct Matrix {
  const T* p;
  int64_t stride, n, k;   // n x k
  __device__ T at(int64_t i, int64_t j) const {
    return i < n && j < k ? ld_g(p + (KMajor ? i * stride + j : j * stride + i)) : T(0);
  }
};

template <class D, bool KMajor, int Rows>
__device__ void fill(float (*to)[Rows + 1], const Matrix<typename D::T, KMajor>& m, int64_t i0, int64_t k0) {
#pragma unroll
  for (int e = threadIdx.x; e < Rows * kTileK; e += kThreads) {
    const int i = KMajor ? e / kTileK : e % Rows, k = KMajor ? e % kTileK : e / Rows;
    to[k][i] = widen<D>(m.at(i0 + i, k0 + k));
  }
}

template <class D, int Stage, int Act>
__global__ void __launch_bounds__(kThreads) ffn_simple_kernel(const __grid_constant__ FfnArgs a) {
  using T = typename D::T;
  constexpr bool kDual = Stage == kFfnHidden;
  constexpr bool kAK = Stage != kFfnGradW, kBK = Stage == kFfnHidden || Stage == kFfnGradHidden;
  __shared__ float sa[kTileK][kTileM + 1], sb[kDual ? 2 : 1][kTileK][kTileN + 1];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  // full ranks' tiles; those of a short rank that lie beyond it are passed over
  const int64_t M = Stage == kFfnGradW ? a.C : a.rows;
  const int64_t N = Stage == kFfnHidden || Stage == kFfnGradHidden ? a.C : a.dim;
  const int64_t tm = (M + kTileM - 1) / kTileM, tn = (N + kTileN - 1) / kTileN;
  const int jobs = Stage == kFfnGradW ? 3 * a.R : a.R;
  for (int64_t tile = blockIdx.x; tile < tm * tn * jobs; tile += gridDim.x) {
    const int job = (int)(tile / (tm * tn)), r = Stage == kFfnGradW ? job / 3 : job, which = job % 3;
    const int64_t i0 = tile % (tm * tn) / tn * kTileM, j0 = tile % tn * kTileN;
    const int width = a.width(r);
    if (Stage == kFfnGradW && !a.grad_w[which][r]) continue;
    const int64_t m = Stage == kFfnGradW ? width : a.rows;
    const int64_t n = Stage == kFfnHidden || Stage == kFfnGradHidden ? width : a.dim;
    if (i0 >= m || j0 >= n) continue;
    float acc[kDual ? 2 : 1][4][8] = {};
    for (int seg = 0; seg < (Stage == kFfnGradX ? 2 : 1); ++seg) {
      Matrix<T, kAK> A;
      Matrix<T, kBK> B, B2;
      if constexpr (Stage == kFfnHidden) {
        A = {(const T*)a.x[r], a.x_stride, m, a.dim};
        B = {(const T*)a.w[0][r], a.w_stride[0][r], n, a.dim};
        B2 = {(const T*)a.w[1][r], a.w_stride[1][r], n, a.dim};
      } else if constexpr (Stage == kFfnOut) {
        A = {(const T*)a.hidden[r], a.hidden_stride[r], m, width};
        B = {(const T*)a.w[2][r], a.w_stride[2][r], n, width};
      } else if constexpr (Stage == kFfnGradHidden) {
        A = {(const T*)a.grad_out[r], a.grad_out_stride, m, a.dim};
        B = {(const T*)a.w[2][r], a.w_stride[2][r], n, a.dim};
      } else if constexpr (Stage == kFfnGradX) {
        A = {(const T*)a.grad_pre[seg][r], a.grad_pre_stride[seg][r], m, width};
        B = {(const T*)a.w[seg][r], a.w_stride[seg][r], n, width};
      } else {
        const bool down = which == 2;
        A = {(const T*)(down ? a.hidden[r] : a.grad_pre[which & 1][r]),
             down ? a.hidden_stride[r] : a.grad_pre_stride[which & 1][r], m, a.rows};
        B = {(const T*)(down ? a.grad_out[r] : a.x[r]), down ? a.grad_out_stride : a.x_stride, n, a.rows};
      }
      for (int64_t k0 = 0; k0 < A.k; k0 += kTileK) {
        __syncthreads();
        fill<D, kAK, kTileM>(sa, A, i0, k0);
        fill<D, kBK, kTileN>(sb[0], B, j0, k0);
        if constexpr (kDual) fill<D, kBK, kTileN>(sb[1], B2, j0, k0);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kTileK; ++k) {
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = sa[k][ty + 16 * i];
#pragma unroll
          for (int b = 0; b < (kDual ? 2 : 1); ++b)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float y = sb[b][k][tx + 16 * j];
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[b][i][j] = __fmaf_rn(x[i], y, acc[b][i][j]);
            }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = i0 + ty + 16 * i;
      float scale[2] = {}, by[2] = {};
      if constexpr (Stage == kFfnHidden) {
        if (a.keep_bits == 8) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float most = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) most = max_nan(most, fabsf(acc[b % (kDual ? 2 : 1)][i][j]));   // beyond the width: 0
#pragma unroll
            for (int s = 8; s > 0; s >>= 1) most = max_nan(most, __shfl_xor_sync(0xFFFFFFFFu, most, s));
            group_scale(most, &scale[b], &by[b]);
            if (tx == 0 && row < m) st_g(a.scales[b][r] + row * ((width + kGroup - 1) / kGroup) + j0 / kGroup, scale[b]);
          }
        }
      }
      if (row >= m) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t col = j0 + tx + 16 * j;
        if (col >= n) continue;
        const float v = acc[0][i][j];
        if constexpr (Stage == kFfnHidden) {
          const float u = acc[1 % (kDual ? 2 : 1)][i][j];
          float2 act, slope;
          activate<Act, false>(both(v), &act, &slope);
          st_g((T*)a.hidden[r] + row * a.hidden_stride[r] + col, narrow<D>(act.x * u));
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int64_t at = row * a.kept_stride[b][r] + col;
            if (a.keep_bits == 8) st_g((int8_t*)a.kept[b][r] + at, code_of(b ? u : v, by[b]));
            if (a.keep_bits == 16) st_g((T*)a.kept[b][r] + at, narrow<D>(b ? u : v));
          }
        } else if constexpr (Stage == kFfnGradHidden) {
          float kept[2];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int64_t at = row * a.kept_stride[b][r] + col;
            if (a.keep_bits == 8)
              kept[b] = (float)ld_g((const int8_t*)a.kept[b][r] + at) *
                        ld_g(a.scales[b][r] + row * ((width + kGroup - 1) / kGroup) + col / kGroup);
            else
              kept[b] = widen<D>(ld_g((const T*)a.kept[b][r] + at));
          }
          float2 act, slope;
          activate<Act, true>(both(kept[0]), &act, &slope);
          st_g((T*)a.grad_pre[0][r] + row * a.grad_pre_stride[0][r] + col, narrow<D>(v * kept[1] * slope.x));
          st_g((T*)a.grad_pre[1][r] + row * a.grad_pre_stride[1][r] + col, narrow<D>(v * act.x));
          if (a.hidden[r]) st_g((T*)a.hidden[r] + row * a.hidden_stride[r] + col, narrow<D>(act.x * kept[1]));
        } else if constexpr (Stage == kFfnGradW) {
          const int64_t at = row * a.grad_w_stride[which][r] + col;
          if (a.grad_f32)
            st_g((float*)a.grad_w[which][r] + at, v);
          else
            st_g((T*)a.grad_w[which][r] + at, narrow<D>(v));
        } else {
          st_g((T*)a.out[r] + row * a.out_stride + col, narrow<D>(v));
        }
      }
    }
  }
}

template <class D, int Stage> cudaError_t launch(const FfnArgs& a, int sms, cudaStream_t st) {
  const dim3 grid((unsigned)(4 * sms));
  if (a.act == RA_SILU || Stage == kFfnOut || Stage == kFfnGradX || Stage == kFfnGradW)
    ffn_simple_kernel<D, Stage, RA_SILU><<<grid, kThreads, 0, st>>>(a);
  else
    ffn_simple_kernel<D, Stage, RA_GELU><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <class D> cudaError_t by_stage(FfnStage stage, const FfnArgs& a, int sms, cudaStream_t st) {
  switch (stage) {
    case kFfnHidden: return launch<D, kFfnHidden>(a, sms, st);
    case kFfnOut: return launch<D, kFfnOut>(a, sms, st);
    case kFfnGradHidden: return launch<D, kFfnGradHidden>(a, sms, st);
    case kFfnGradX: return launch<D, kFfnGradX>(a, sms, st);
    default: return launch<D, kFfnGradW>(a, sms, st);
  }
}

}  // namespace

__device__ WaitRecord g_ffn_waits;

cudaError_t ffn_wait_record(WaitRecord** at) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(at), g_ffn_waits);
}

#ifdef RA_DEBUG_BOUNDS
namespace {
__global__ void give_up_kernel(WaitRecord* record) { record_give_up(record, 0, 0, 1u); }
}  // namespace

cudaError_t launch_ffn_give_up(WaitRecord* record, cudaStream_t st) {
  const cudaError_t e = debug_upload(st);
  if (e != cudaSuccess) return e;
  give_up_kernel<<<1, 1, 0, st>>>(record);
  return cudaGetLastError();
}
#endif

cudaError_t launch_ffn_simple(int dtype, FfnStage stage, const FfnArgs& a, int sms, cudaStream_t st) {
  const cudaError_t e = debug_upload(st);
  if (e != cudaSuccess) return e;
  return dtype == RA_BF16 ? by_stage<DBF16>(stage, a, sms, st) : by_stage<DF16>(stage, a, sms, st);
}

}  // namespace ra
