// ra_norm.cu -- the end of a tensor-parallel block, forward and backward: the
// R ranks' partial products summed, normalised, gated, added to the residual
// stream and normalised again for the next block.
//
//   S = sum_r P_r;  y = S r1 w1,  r1 = (mean S^2 + eps)^-1/2   (no post norm: y = S)
//   h' = h + a g y; r2 = (mean h'^2 + eps)^-1/2;  z = h' r2 w
//
//   dz = sum_r dz_r;  x2 = h' r2;  c2 = mean(w dz x2)
//   e = dh' + r2 (w dz - x2 c2);   dw = sum_t dz x2;   dh = e
//   dy = a g e;  dg = sum a y e;   x1 = S r1;  dw1 = sum_t dy x1
//   c1 = mean(w1 dy x1);  dS = r1 (w1 dy - x1 c1)      (no post norm: dS = dy)
//
// Everything between the loads and the stores is binary32: the sum over the
// ranks in rank order, both statistics, the residual; each output is rounded
// once.  A row's columns stay in the registers of the threads that loaded
// them (one warp a row for narrow rows, one CTA for wide ones), so every
// input is read once and every output written once: the kernels are bound by
// memory traffic, few rows by the latency of two sums over a block.
#include "ra_ops.cuh"

namespace ra {
namespace {

constexpr int kWarpRows = 8;   // rows per CTA where one warp takes a row

// Sum over the threads of a row, the same value in all of them.  `red`
// alternates between calls: a buffer is written again only after the barrier
// of the call between.
__device__ __forceinline__ float row_sum(float v, float (*red)[32], int& turn) {
  v = warp_sum(v);
  const int warps = (int)(blockDim.x + 31) >> 5;
  if (warps == 1) return v;
  float* buf = red[turn];
  turn ^= 1;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  if (lane == 0) buf[w] = v;
  __syncthreads();
  return warp_sum(lane < warps ? buf[lane] : 0.0f);
}

// Group j of a thread's columns.  Aligned rows: V neighbouring columns, whole
// 16-byte vectors.  Other rows (an odd width or stride): V columns a row's
// threads apart, so that a warp's scalar accesses stay side by side.
template <bool AL, int V> struct Group {
  int first, step;
  __device__ __forceinline__ Group(int j) {
    const int n = blockDim.x;
    first = AL ? (j * n + (int)threadIdx.x) * V : j * V * n + (int)threadIdx.x;
    step = AL ? 1 : n;
  }
};

template <class E, bool AL, int V>
__device__ __forceinline__ void load_cols(const void* base, int64_t at, int j, int dim, float (&x)[V]) {
  const typename E::T* row = static_cast<const typename E::T*>(base) + at;
  const Group<AL, V> g(j);
  if (AL) {
    if (g.first < dim) {
#pragma unroll
      for (int k = 0; k < V / E::kVec; ++k)
        unpack<E>(ld_stream(reinterpret_cast<const uint4*>(row + g.first) + k), x + k * E::kVec);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = 0.0f;
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int c = g.first + e * g.step;
      x[e] = c < dim ? widen<E>(ld_stream_scalar(row + c)) : 0.0f;
    }
  }
}

template <class E, bool AL, int V>
__device__ __forceinline__ void store_cols(void* base, int64_t at, int j, int dim, const float (&x)[V]) {
  typename E::T* row = static_cast<typename E::T*>(base) + at;
  const Group<AL, V> g(j);
  if (AL) {
    if (g.first < dim) {
#pragma unroll
      for (int k = 0; k < V / E::kVec; ++k)
        st_stream(reinterpret_cast<uint4*>(row + g.first) + k, pack<E>(x + k * E::kVec));
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int c = g.first + e * g.step;
      if (c < dim) st_g(row + c, narrow<E>(x[e]));
    }
  }
}

// Weights and gate: binary32 or the activations' type; cached, every row reads them.
template <class D, bool AL, int V>
__device__ __forceinline__ void load_params(const void* base, int64_t at, bool f32, int j, int dim, float (&x)[V]) {
  if (f32)
    load_cols<DF32, AL, V>(base, at, j, dim, x);
  else
    load_cols<D, AL, V>(base, at, j, dim, x);
}

// Sum of `count` rank buffers' columns in rank order.
template <class D, bool AL, int V, int VPT>
__device__ __forceinline__ void sum_ranks(const void* const* in, int count, int64_t at, int dim,
                                          float (&acc)[VPT][V]) {
#pragma unroll
  for (int j = 0; j < VPT; ++j) load_cols<D, AL, V>(in[0], at, j, dim, acc[j]);
#pragma unroll 4
  for (int r = 1; r < count; ++r) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float x[V];
      load_cols<D, AL, V>(in[r], at, j, dim, x);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[j][e] = __fadd_rn(acc[j][e], x[e]);
    }
  }
}

template <class D, class RD, int VPT, bool AL>
__global__ void __launch_bounds__(1024) norm_forward_kernel(const __grid_constant__ NormForward a) {
  constexpr int V = D::kVec;
  __shared__ float red[2][32];
  int turn = 0;
  const float inv_dim = 1.0f / (float)a.dim;
  for (int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; row < a.rows;
       row += (int64_t)gridDim.x * blockDim.y) {
    float s[VPT][V], h[VPT][V];
    sum_ranks<D, AL, V, VPT>(a.in, a.R, row * a.in_stride, a.dim, s);
#pragma unroll
    for (int j = 0; j < VPT; ++j) load_cols<RD, AL, V>(a.residual, row * a.residual_stride, j, a.dim, h[j]);
    if (a.total) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) store_cols<D, AL, V>(a.total, row * a.total_stride, j, a.dim, s[j]);
    }
    float r1 = 0.0f;
    if (a.post_weight) {
      float sq = 0.0f;
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) sq = __fmaf_rn(s[j][e], s[j][e], sq);
      r1 = rsqrtf(row_sum(sq, red, turn) * inv_dim + a.eps);
    }
    float sq = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (a.post_weight) {
        float w[V];
        load_params<D, AL, V>(a.post_weight, 0, a.param_f32, j, a.dim, w);
#pragma unroll
        for (int e = 0; e < V; ++e) s[j][e] = s[j][e] * r1 * w[e];
      }
      if (a.gate) {
        float g[V];
        load_params<D, AL, V>(a.gate, row / a.rows_per_gate * a.dim, a.param_f32, j, a.dim, g);
#pragma unroll
        for (int e = 0; e < V; ++e) s[j][e] *= g[e];
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        h[j][e] = __fmaf_rn(a.scale, s[j][e], h[j][e]);
        sq = __fmaf_rn(h[j][e], h[j][e], sq);
      }
      store_cols<RD, AL, V>(a.residual_out, row * a.residual_out_stride, j, a.dim, h[j]);
    }
    const float r2 = rsqrtf(row_sum(sq, red, turn) * inv_dim + a.eps);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float w[V];
      load_params<D, AL, V>(a.weight, 0, a.param_f32, j, a.dim, w);
#pragma unroll
      for (int e = 0; e < V; ++e) h[j][e] = h[j][e] * r2 * w[e];
      for (int q = 0; q < a.outs; ++q) store_cols<D, AL, V>(a.out[q], row * a.out_stride, j, a.dim, h[j]);
    }
    if (a.rstd && threadIdx.x == 0) {
      st_g(a.rstd + row, r1);
      st_g(a.rstd + a.rows + row, r2);
    }
  }
}

// How the rows of a backward call are dealt: units of rows that share a gate
// row (`parts` units per gate row), each worker (CTA, or warp of narrow rows)
// taking unit w, w + workers, ...
struct Deal {
  int64_t units, parts, rows_per_part;
  int64_t workers;
};

template <class D, class RD, int VPT, bool AL>
__global__ void __launch_bounds__(1024) norm_backward_kernel(const __grid_constant__ NormBackward a, const Deal d) {
  constexpr int V = D::kVec;
  __shared__ float red[2][32];
  int turn = 0;
  const float inv_dim = 1.0f / (float)a.dim;
  const int64_t worker = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  float dw[VPT][V], dp[VPT][V];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) dw[j][e] = dp[j][e] = 0.0f;
  for (int64_t u = worker; u < d.units; u += d.workers) {
    const int64_t group = u / d.parts, part = u % d.parts;
    const int64_t lo = group * a.rows_per_gate + part * d.rows_per_part;
    const int64_t end = (group + 1) * a.rows_per_gate;
    const int64_t hi = lo + d.rows_per_part < end ? lo + d.rows_per_part : end;
    float dg[VPT][V];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) dg[j][e] = 0.0f;
    for (int64_t row = lo; row < hi; ++row) {
      float z[VPT][V], x2[VPT][V];
      sum_ranks<D, AL, V, VPT>(a.grad_out, a.grads, row * a.grad_out_stride, a.dim, z);
      const float r2 = ld_g(a.rstd + a.rows + row);
      float c = 0.0f;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        float w[V];
        load_cols<RD, AL, V>(a.residual_out, row * a.residual_out_stride, j, a.dim, x2[j]);
        load_params<D, AL, V>(a.weight, 0, a.param_f32, j, a.dim, w);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          x2[j][e] *= r2;
          dw[j][e] = __fmaf_rn(z[j][e], x2[j][e], dw[j][e]);
          z[j][e] *= w[e];
          c = __fmaf_rn(z[j][e], x2[j][e], c);
        }
      }
      const float c2 = row_sum(c, red, turn) * inv_dim;
      const float r1 = a.post_weight ? ld_g(a.rstd + row) : 1.0f;
      float c1 = 0.0f;
      // e in z, then the gradient of y in z; x1 in x2
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (a.grad_residual_out) {
          float t[V];
          load_cols<RD, AL, V>(a.grad_residual_out, row * a.grad_residual_out_stride, j, a.dim, t);
#pragma unroll
          for (int e = 0; e < V; ++e) z[j][e] = __fmaf_rn(r2, __fmaf_rn(-c2, x2[j][e], z[j][e]), t[e]);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) z[j][e] = r2 * __fmaf_rn(-c2, x2[j][e], z[j][e]);
        }
        store_cols<RD, AL, V>(a.grad_residual, row * a.grad_residual_stride, j, a.dim, z[j]);
        if (a.total) load_cols<D, AL, V>(a.total, row * a.total_stride, j, a.dim, x2[j]);
        float w[V], g[V];
        if (a.post_weight) load_params<D, AL, V>(a.post_weight, 0, a.param_f32, j, a.dim, w);
        if (a.gate) load_params<D, AL, V>(a.gate, group * a.dim, a.param_f32, j, a.dim, g);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float x1 = x2[j][e] * r1, ae = a.scale * z[j][e];
          if (a.grad_gate) dg[j][e] = __fmaf_rn(a.post_weight ? x1 * w[e] : x1, ae, dg[j][e]);
          z[j][e] = a.gate ? ae * g[e] : ae;
          if (a.post_weight) {
            dp[j][e] = __fmaf_rn(z[j][e], x1, dp[j][e]);
            z[j][e] *= w[e];
            c1 = __fmaf_rn(z[j][e], x1, c1);
          }
          x2[j][e] = x1;
        }
      }
      if (a.post_weight) c1 = row_sum(c1, red, turn) * inv_dim;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (a.post_weight) {
#pragma unroll
          for (int e = 0; e < V; ++e) z[j][e] = r1 * __fmaf_rn(-c1, x2[j][e], z[j][e]);
        }
        for (int q = 0; q < a.outs; ++q) store_cols<D, AL, V>(a.grad_in[q], row * a.grad_in_stride, j, a.dim, z[j]);
      }
    }
    if (a.grad_gate) {
      // one unit per gate row: its gradient is whole; else a partial per unit
      float* to = d.parts == 1 ? a.grad_gate : a.work + 2 * d.workers * a.dim;
#pragma unroll
      for (int j = 0; j < VPT; ++j) store_cols<DF32, AL, V>(to, u * a.dim, j, a.dim, dg[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if (a.grad_weight) store_cols<DF32, AL, V>(a.work, worker * a.dim, j, a.dim, dw[j]);
    if (a.grad_post_weight) store_cols<DF32, AL, V>(a.work, (d.workers + worker) * a.dim, j, a.dim, dp[j]);
  }
}

// The workers' column partials joined, in worker order: blockIdx.y 0 the pre
// norm's weight, 1 the post norm's, 2.. the gate rows.
constexpr int kJoinSlices = 32;
__global__ void norm_join_kernel(const __grid_constant__ NormBackward a, const Deal d) {
  __shared__ float part[kJoinSlices][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  const float* from;
  float* to;
  int64_t count;
  if (blockIdx.y < 2) {
    from = a.work + blockIdx.y * d.workers * a.dim;
    to = blockIdx.y == 0 ? a.grad_weight : a.grad_post_weight;
    count = d.workers;
  } else {
    const int64_t g = blockIdx.y - 2;
    from = a.work + (2 * d.workers + g * d.parts) * a.dim;
    to = a.grad_gate + g * a.dim;
    count = d.parts;
  }
  if ((blockIdx.y < 2 && !to) || (blockIdx.y >= 2 && !a.grad_gate)) return;
  float s = 0.0f;
  if (c < a.dim) {
    for (int64_t i = threadIdx.y; i < count; i += kJoinSlices) s += ld_g(from + i * a.dim + c);
  }
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < a.dim) {
    for (int k = 1; k < kJoinSlices; ++k) s += part[k][threadIdx.x];
    st_g(to + c, s);
  }
}

// Threads per row and 16-byte groups per thread for a row of `dim` columns.
struct Shape {
  int threads, groups, rows;
};
Shape row_shape(int dim, int vec) {
  const int vectors = (dim + vec - 1) / vec;
  Shape s;
  s.groups = 1;
  while (vectors > 512 * s.groups && s.groups < 2) s.groups *= 2;
  while (vectors > 1024 * s.groups) s.groups *= 2;
  s.threads = ((vectors + s.groups - 1) / s.groups + 31) / 32 * 32;
  s.rows = s.threads == 32 ? kWarpRows : 1;
  return s;
}

// CTAs of a row's threads to fill the SMs: 2048 threads each at most.
int64_t most_ctas(const Shape& s, int sms) {
  const int per_sm = 2048 / (s.threads * s.rows);
  return (int64_t)sms * (per_sm < 1 ? 1 : per_sm > 2 ? 2 : per_sm);
}

template <class F> cudaError_t with_types(int dtype, int rdtype, F&& f) {
  if (dtype == RA_F32 && rdtype == RA_F32) return f(DF32{}, DF32{});
  if (dtype == RA_BF16 && rdtype == RA_BF16) return f(DBF16{}, DBF16{});
  if (dtype == RA_BF16 && rdtype == RA_F32) return f(DBF16{}, DF32{});
  if (dtype == RA_F16 && rdtype == RA_F16) return f(DF16{}, DF16{});
  if (dtype == RA_F16 && rdtype == RA_F32) return f(DF16{}, DF32{});
  return cudaErrorInvalidValue;
}

// f(IntC<groups per thread>) for the widths a type has: at most 16384 columns
// in 1024 threads.
template <class D, class F> cudaError_t with_groups(int groups, F&& f) {
  if (groups == 1) return f(IntC<1>{});
  if (groups == 2) return f(IntC<2>{});
  if constexpr (D::kVec == 4) {
    if (groups == 4) return f(IntC<4>{});
  }
  return cudaErrorInvalidValue;
}

int vec_of(int dtype) { return dtype == RA_F32 ? 4 : 8; }

Deal make_deal(const NormBackward& a, const Shape& s, int sms) {
  Deal d;
  const int64_t most = most_ctas(s, sms) * s.rows;
  d.parts = (most + a.groups - 1) / a.groups;
  if (d.parts > a.rows_per_gate) d.parts = a.rows_per_gate;
  d.rows_per_part = (a.rows_per_gate + d.parts - 1) / d.parts;
  d.parts = (a.rows_per_gate + d.rows_per_part - 1) / d.rows_per_part;
  d.units = d.parts * a.groups;
  d.workers = d.units < most ? (d.units + s.rows - 1) / s.rows * s.rows : most;
  return d;
}

}  // namespace

size_t norm_workspace_floats(int dim, int sms) {
  // two weights' partials per worker, and fewer than two gate partials per
  // worker (`parts` > 1 only where there are fewer gate rows than workers)
  size_t most = 0;
  for (int vec : {4, 8}) {
    const Shape s = row_shape(dim, vec);
    const size_t w = (size_t)most_ctas(s, sms) * s.rows;
    if (w > most) most = w;
  }
  return 4 * most * (size_t)dim;
}

cudaError_t launch_norm_forward(int dtype, int rdtype, bool aligned, const NormForward& a, int sms,
                                cudaStream_t st) {
  cudaError_t e = debug_upload(st);
  if (e != cudaSuccess) return e;
  const Shape s = row_shape(a.dim, vec_of(dtype));
  const int64_t want = (a.rows + s.rows - 1) / s.rows, most = most_ctas(s, sms);
  const dim3 block(s.threads, s.rows);
  const unsigned grid = (unsigned)(want < most ? want : most);
  return with_types(dtype, rdtype, [&](auto d, auto r) {
    using D = decltype(d);
    using RD = decltype(r);
    return with_groups<D>(s.groups, [&](auto g) {
      if (aligned)
        norm_forward_kernel<D, RD, decltype(g)::value, true><<<grid, block, 0, st>>>(a);
      else
        norm_forward_kernel<D, RD, decltype(g)::value, false><<<grid, block, 0, st>>>(a);
      return cudaGetLastError();
    });
  });
}

cudaError_t launch_norm_backward(int dtype, int rdtype, bool aligned, const NormBackward& a, int sms,
                                 cudaStream_t st) {
  cudaError_t e = debug_upload(st);
  if (e != cudaSuccess) return e;
  const Shape s = row_shape(a.dim, vec_of(dtype));
  const Deal dl = make_deal(a, s, sms);
  const dim3 block(s.threads, s.rows);
  const unsigned grid = (unsigned)(dl.workers / s.rows);
  e = with_types(dtype, rdtype, [&](auto d, auto r) {
    using D = decltype(d);
    using RD = decltype(r);
    return with_groups<D>(s.groups, [&](auto g) {
      if (aligned)
        norm_backward_kernel<D, RD, decltype(g)::value, true><<<grid, block, 0, st>>>(a, dl);
      else
        norm_backward_kernel<D, RD, decltype(g)::value, false><<<grid, block, 0, st>>>(a, dl);
      return cudaGetLastError();
    });
  });
  if (e != cudaSuccess) return e;
  const bool gates = a.grad_gate && dl.parts > 1;
  if (!a.grad_weight && !a.grad_post_weight && !gates) return cudaSuccess;
  const dim3 join((a.dim + 31) / 32, 2 + (gates ? (unsigned)a.groups : 0u));
  norm_join_kernel<<<join, dim3(32, kJoinSlices), 0, st>>>(a, dl);
  return cudaGetLastError();
}

}  // namespace ra
