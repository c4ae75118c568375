// ra_ckpt.cu -- rows kept in 8 bits (ra_ckpt_store) and brought back
// (ra_ckpt_load), with the normalised rows of a kept residual stream.
//
// A half warp takes a group of 128 columns, a lane eight of them side by side:
// the group's largest magnitude is found by four shuffles, and every group is
// read and written once.
#include "ra_ffn.cuh"

namespace ra {

namespace {

constexpr int kThreads = 256, kHalf = 16, kItems = 4;   // groups that a half warp has in flight

// The columns of group g that a lane holds: eight side by side, or (rows off
// the 16-byte grid) every 16th.
template <bool Wide> __device__ __forceinline__ int column(int g, int lane, int j) {
  return g * kGroup + (Wide ? lane * 8 + j : lane + kHalf * j);
}

template <class D, bool Wide>
__device__ __forceinline__ void get8(const typename D::T* row, int g, int lane, int dim, float* v) {
  if constexpr (Wide) {
    const bool in = column<true>(g, lane, 0) < dim;
    const uint4* p = reinterpret_cast<const uint4*>(row + column<true>(g, lane, 0));
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    unpack<D>(in ? ld_stream(p) : zero, v);
    if constexpr (D::kVec == 4) unpack<D>(in ? ld_stream(p + 1) : zero, v + 4);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<false>(g, lane, j);
      v[j] = c < dim ? widen<D>(ld_g(row + c)) : 0.0f;
    }
  }
}

template <class D, bool Wide>
__device__ __forceinline__ void put8(typename D::T* row, int g, int lane, int dim, const float* v) {
  if constexpr (Wide) {
    if (column<true>(g, lane, 0) >= dim) return;
    uint4* p = reinterpret_cast<uint4*>(row + column<true>(g, lane, 0));
    st_stream(p, pack<D>(v));
    if constexpr (D::kVec == 4) st_stream(p + 1, pack<D>(v + 4));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<false>(g, lane, j);
      if (c < dim) st_g(row + c, narrow<D>(v[j]));
    }
  }
}

// Group `i` of all rows'.
struct Place {
  int64_t row;
  int group;
  __device__ __forceinline__ Place(int64_t i, int groups) {
    if (i <= 0x7FFFFFFF) {
      const uint32_t n = (uint32_t)i, q = n / (uint32_t)groups;
      row = q;
      group = (int)(n - q * (uint32_t)groups);
    } else {
      row = i / groups;
      group = (int)(i - row * groups);
    }
  }
};

template <class D, bool Wide>
__global__ void __launch_bounds__(kThreads) ckpt_store_kernel(const CkptArgs a) {
  using T = typename D::T;
  after_predecessor();
  const int lane = threadIdx.x % kHalf, groups = (a.dim + kGroup - 1) / kGroup;
  const int64_t total = a.rows * groups, step = (int64_t)gridDim.x * (kThreads / kHalf);
  const int64_t whole = (total + step - 1) / step * step;   // a warp's halves stay together for the shuffles
  for (int64_t i0 = blockIdx.x * (int64_t)(kThreads / kHalf) + threadIdx.x / kHalf; i0 < whole; i0 += kItems * step) {
    float v[kItems][8];
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      const int64_t i = i0 + u * step;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[u][j] = 0.0f;
      if (i < total) {
        const Place p(i, groups);
        get8<D, Wide>((const T*)a.values + p.row * a.stride, p.group, lane, a.dim, v[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      const int64_t i = i0 + u * step;
      float most = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) most = max_nan(most, fabsf(v[u][j]));
#pragma unroll
      for (int s = kHalf / 2; s > 0; s >>= 1) most = max_nan(most, __shfl_xor_sync(0xFFFFFFFFu, most, s));
      if (i >= total) continue;
      float scale, by;
      group_scale(most, &scale, &by);
      const Place p(i, groups);
      if (lane == 0) st_g(a.scales + i, scale);
      int8_t* codes = a.codes + p.row * a.codes_stride;
      if constexpr (Wide) {
        const int c = column<true>(p.group, lane, 0);
        if (c < a.dim) st_g(reinterpret_cast<uint2*>(codes + c), make_uint2(codes4(v[u], by), codes4(v[u] + 4, by)));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = column<false>(p.group, lane, j);
          if (c < a.dim) st_g(codes + c, code_of(v[u][j], by));
        }
      }
    }
  }
}

template <class D, class N, class P, bool Wide>
__global__ void __launch_bounds__(kThreads) ckpt_load_kernel(const CkptArgs a) {
  using T = typename D::T;
  using TN = typename N::T;
  using TP = typename P::T;
  after_predecessor();
  const int lane = threadIdx.x % kHalf, groups = (a.dim + kGroup - 1) / kGroup;
  const int64_t total = a.rows * groups, step = (int64_t)gridDim.x * (kThreads / kHalf);
  for (int64_t i0 = blockIdx.x * (int64_t)(kThreads / kHalf) + threadIdx.x / kHalf; i0 < total; i0 += kItems * step) {
    uint2 q[kItems];
    float scale[kItems], rstd[kItems];
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      const int64_t i = i0 + u * step;
      q[u] = make_uint2(0u, 0u);
      scale[u] = rstd[u] = 0.0f;
      if (i >= total) continue;
      const Place p(i, groups);
      const int8_t* codes = a.codes + p.row * a.codes_stride;
      if constexpr (Wide) {
        const int c = column<true>(p.group, lane, 0);
        if (c < a.dim) q[u] = ld_g(reinterpret_cast<const uint2*>(codes + c));
      } else {
        uint32_t w[2] = {};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = column<false>(p.group, lane, j);
          if (c < a.dim) w[j / 4] |= (uint32_t)(uint8_t)ld_g(codes + c) << (8 * (j % 4));
        }
        q[u] = make_uint2(w[0], w[1]);
      }
      scale[u] = ld_g(a.scales + i);
      if (a.normed) rstd[u] = ld_g(a.rstd + p.row);
    }
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      const int64_t i = i0 + u * step;
      if (i >= total) continue;
      const Place p(i, groups);
      float v[8];
      const uint32_t lo = bias_codes(q[u].x), hi = bias_codes(q[u].y);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = code_value(j < 4 ? lo : hi, j % 4) * scale[u];
      if (a.values) put8<D, Wide>((T*)a.values + p.row * a.stride, p.group, lane, a.dim, v);
      if (!a.normed) continue;
      float w[8];
      if constexpr (Wide) {
        const int c = column<true>(p.group, lane, 0);
        if (c < a.dim) {
          const uint4* at = reinterpret_cast<const uint4*>((const TP*)a.weight + c);
          unpack<P>(ld_plain(at), w);
          if constexpr (P::kVec == 4) unpack<P>(ld_plain(at + 1), w + 4);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = column<false>(p.group, lane, j);
          w[j] = c < a.dim ? widen<P>(ld_g((const TP*)a.weight + c)) : 0.0f;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = v[j] * rstd[u] * w[j];
      put8<N, Wide>((TN*)a.normed + p.row * a.normed_stride, p.group, lane, a.dim, w);
    }
  }
}

int ctas(const CkptArgs& a, int sms) {
  const int64_t groups = (a.dim + kGroup - 1) / kGroup;
  const int64_t need = (a.rows * groups + kThreads / kHalf - 1) / (kThreads / kHalf);
  return (int)(need < 8 * sms ? need : 8 * sms);
}

template <class F> cudaError_t with_float(int dtype, F&& f) {
  return dtype == RA_F32 ? f(DF32{}) : dtype == RA_BF16 ? f(DBF16{}) : f(DF16{});
}

}  // namespace

cudaError_t launch_ckpt_store(int dtype, bool wide, const CkptArgs& a, int sms, cudaStream_t st) {
  const cudaError_t e = debug_upload(st);
  if (e != cudaSuccess) return e;
  return with_float(dtype, [&](auto d) {
    using D = decltype(d);
    return launch_after(wide ? ckpt_store_kernel<D, true> : ckpt_store_kernel<D, false>, dim3(ctas(a, sms)),
                        dim3(kThreads), 0, st, 1, a);
  });
}

cudaError_t launch_ckpt_load(int dtype, int normed_dtype, int param_dtype, bool wide, const CkptArgs& a, int sms,
                             cudaStream_t st) {
  const cudaError_t e = debug_upload(st);
  if (e != cudaSuccess) return e;
  return with_float(dtype, [&](auto d) {
    return with_float(normed_dtype, [&](auto n) {
      using D = decltype(d);
      using N = decltype(n);
      const bool f32 = param_dtype == RA_F32;
      const auto kernel = f32 ? (wide ? ckpt_load_kernel<D, N, DF32, true> : ckpt_load_kernel<D, N, DF32, false>)
                              : (wide ? ckpt_load_kernel<D, N, N, true> : ckpt_load_kernel<D, N, N, false>);
      return launch_after(kernel, dim3(ctas(a, sms)), dim3(kThreads), 0, st, 1, a);
    });
  });
}

}  // namespace ra
