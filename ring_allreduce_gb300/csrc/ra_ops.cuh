// ra_ops.cuh -- device building blocks of the model operators: conversions
// between the activations' types and binary32, groups of a row's columns, and
// sums over a block.
#pragma once

#include <float.h>
#include <math.h>

#include "ra_device.cuh"
#include "ra_ops.h"

namespace ra {

template <class D> __device__ __forceinline__ float widen(typename D::T v);
template <> __device__ __forceinline__ float widen<DF32>(float v) { return v; }
template <> __device__ __forceinline__ float widen<DBF16>(uint16_t v) { return bf16_widen(v); }
template <> __device__ __forceinline__ float widen<DF16>(uint16_t v) {
  return __half2float(__ushort_as_half(v));
}

// One rounding to the activations' type, to nearest even.
template <class D> __device__ __forceinline__ typename D::T narrow(float v);
template <> __device__ __forceinline__ float narrow<DF32>(float v) { return v; }
template <> __device__ __forceinline__ uint16_t narrow<DBF16>(float v) { return bf16_round(v); }
template <> __device__ __forceinline__ uint16_t narrow<DF16>(float v) {
  return __half_as_ushort(__float2half_rn(v));
}

// Two 16-bit elements of a word as binary32.
template <class D> __device__ __forceinline__ void unpack2(uint32_t w, float* x);
template <> __device__ __forceinline__ void unpack2<DBF16>(uint32_t w, float* x) {
  x[0] = __uint_as_float(w << 16);
  x[1] = __uint_as_float(w & 0xFFFF0000u);
}
template <> __device__ __forceinline__ void unpack2<DF16>(uint32_t w, float* x) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  x[0] = f.x;
  x[1] = f.y;
}

// The elements of one 16-byte vector as binary32, and back.
template <class D> __device__ __forceinline__ void unpack(uint4 v, float* x) {
  if constexpr (sizeof(typename D::T) == 4) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  } else {
    unpack2<D>(v.x, x);
    unpack2<D>(v.y, x + 2);
    unpack2<D>(v.z, x + 4);
    unpack2<D>(v.w, x + 6);
  }
}

template <class D> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<DBF16>(float lo, float hi) {
  __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&p);
}
template <> __device__ __forceinline__ uint32_t pack2<DF16>(float lo, float hi) {
  __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&p);
}
template <> __device__ __forceinline__ uint32_t pack2<DF32>(float lo, float) { return __float_as_uint(lo); }

template <class D> __device__ __forceinline__ uint4 pack(const float* x) {
  if (sizeof(typename D::T) == 4)
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  return make_uint4(pack2<D>(x[0], x[1]), pack2<D>(x[2], x[3]), pack2<D>(x[4 % D::kVec], x[5 % D::kVec]),
                    pack2<D>(x[6 % D::kVec], x[7 % D::kVec]));
}

// A vector that many rows read: cached.
__device__ __forceinline__ uint4 ld_plain(const uint4* p) {
  if (!RA_ACCESS_OK(p, 16u, 1u)) return make_uint4(0u, 0u, 0u, 0u);
  return *p;
}

// The operators' kernels are launched with programmatic stream serialisation:
// a call's kernel may be set up while the one before it in the stream still
// runs.  Each begins with this, before it touches any memory, so that
// everything before it is complete and visible; its own successor may then be
// set up in turn.  Back to back, calls of a few microseconds come 1 to 3 us
// sooner after each other.
__device__ __forceinline__ void after_predecessor() {
  griddep_wait();
  griddep_launch_dependents();
}

// One such launch, in clusters of `cluster` CTAs along x.
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, int cluster,
                         const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, s);
  return v;
}

// The larger value; NaN when either is (a masked place that holds NaN must
// not vanish from a maximum).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, s));
  return v;
}

// 2^x, to about 2 ulp (ex2.approx: 0 for arguments below the subnormals).
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

}  // namespace ra
