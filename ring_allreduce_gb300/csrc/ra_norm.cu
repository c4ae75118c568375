// ra_norm.cu -- the block end's launches (kernels: ra_norm.cuh, instantiated
// in ra_norm_inst.cu) and the sum of the weights' gradients over the workers.
#include "ra_norm.cuh"

namespace ra {
namespace norm {

#define RA_NORM_EXTERN(D, RD)                                                                                      \
  extern template cudaError_t run_forward<D, RD>(const Shape&, bool, const NormForward&, OptedIn&, unsigned,        \
                                                 cudaStream_t);                                                     \
  extern template cudaError_t run_backward<D, RD>(const Shape&, bool, const NormBackward&, const Deal&, OptedIn&,   \
                                                  unsigned, cudaStream_t);
RA_NORM_EXTERN(DF32, DF32)
RA_NORM_EXTERN(DBF16, DBF16)
RA_NORM_EXTERN(DBF16, DF32)
RA_NORM_EXTERN(DF16, DF16)
RA_NORM_EXTERN(DF16, DF32)

}  // namespace norm

namespace {

using namespace norm;

// The CTAs' column partials joined, in their order (a gate row's: the units'): blockIdx.y 0 the pre
// norm's weight, 1 the post norm's, 2.. the gate rows.
// Warp w of a CTA's 32 columns sums every blockDim.y-th partial, then a column's slices are summed by a warp.
// 147 partials of 8192 columns, two weights and a gate: 13 us with nothing in L2, 14 MB of reads; a few us
// behind the kernel that wrote them.
__global__ void __launch_bounds__(1024) norm_join_kernel(const __grid_constant__ NormBackward a,
                                                         const __grid_constant__ Deal d) {
  __shared__ float part[32][33];
  after_predecessor();
  const int c = blockIdx.x * 32 + threadIdx.x;
  const float* from;
  float* to;
  int64_t count;
  if (blockIdx.y < 2) {
    from = a.work + blockIdx.y * d.ctas * a.dim;
    to = blockIdx.y == 0 ? a.grad_weight : a.grad_post_weight;
    count = d.ctas;
  } else {
    const int64_t g = blockIdx.y - 2;
    from = a.work + (2 * d.ctas + g * d.parts) * a.dim;
    to = a.grad_gate + g * a.dim;
    count = d.parts;
  }
  if ((blockIdx.y < 2 && !to) || (blockIdx.y >= 2 && !a.grad_gate)) return;
  float s = 0.0f;
  if (c < a.dim) {
#pragma unroll 4
    for (int64_t i = threadIdx.y; i < count; i += blockDim.y) s += ld_g(from + i * a.dim + c);
  }
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  for (int k = threadIdx.y; k < 32; k += blockDim.y) {
    s = warp_sum(threadIdx.x < blockDim.y ? part[threadIdx.x][k] : 0.0f);
    if (threadIdx.x == 0 && blockIdx.x * 32 + k < a.dim) st_g(to + blockIdx.x * 32 + k, s);
  }
}

template <class F> cudaError_t with_types(int dtype, int rdtype, F&& f) {
  if (dtype == RA_F32 && rdtype == RA_F32) return f(DF32{}, DF32{});
  if (dtype == RA_BF16 && rdtype == RA_BF16) return f(DBF16{}, DBF16{});
  if (dtype == RA_BF16 && rdtype == RA_F32) return f(DBF16{}, DF32{});
  if (dtype == RA_F16 && rdtype == RA_F16) return f(DF16{}, DF16{});
  if (dtype == RA_F16 && rdtype == RA_F32) return f(DF16{}, DF32{});
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
  d.ctas = d.workers / s.rows;
  return d;
}

}  // namespace

size_t norm_workspace_floats(int dim, int sms) {
  // two weights' partials per worker, and fewer than two gate partials per
  // worker (`parts` > 1 only where there are fewer gate rows than workers)
  size_t most = 0;
  for (int vec : {4, 8}) {
    for (bool deep : {false, true}) {
      const Shape s = backward_shape(dim, vec, deep);
      const size_t w = (size_t)most_ctas(s, sms) * s.rows;
      if (w > most) most = w;
    }
  }
  return 4 * most * (size_t)dim;
}

cudaError_t launch_norm_forward(int dtype, int rdtype, bool aligned, const NormForward& a, int sms, OptedIn& opted,
                                cudaStream_t st) {
  const Shape s = forward_shape(a.dim, vec_of(dtype), a.rows >= 2 * (int64_t)sms);
  const int64_t per = s.rows * (aligned ? s.packs : 1), want = (a.rows + per - 1) / per, most = most_ctas(s, sms);
  const unsigned grid = (unsigned)(want < most ? want : most);
  return with_types(dtype, rdtype, [&](auto d, auto r) {
    return run_forward<decltype(d), decltype(r)>(s, aligned, a, opted, grid, st);
  });
}

cudaError_t launch_norm_backward(int dtype, int rdtype, bool aligned, const NormBackward& a, int sms, OptedIn& opted,
                                 cudaStream_t st) {
  const Shape s = backward_shape(a.dim, vec_of(dtype), a.rows >= 2 * (int64_t)sms);
  const Deal dl = make_deal(a, s, sms);
  const unsigned grid = (unsigned)dl.ctas;
  cudaError_t e = with_types(dtype, rdtype, [&](auto d, auto r) {
    return run_backward<decltype(d), decltype(r)>(s, aligned, a, dl, opted, grid, st);
  });
  if (e != cudaSuccess) return e;
  const bool gates = a.grad_gate && dl.parts > 1;
  if (!a.grad_weight && !a.grad_post_weight && !gates) return cudaSuccess;
  e = debug_upload(st);
  if (e != cudaSuccess) return e;
  const dim3 join((a.dim + 31) / 32, 2 + (gates ? (unsigned)a.groups : 0u));
  // eight slices where a handful of partials each is left, else as many as there can be
  return launch_after(norm_join_kernel, join, dim3(32, dl.ctas <= 128 ? 8 : 32), 0, st, 1, a, dl);
}

}  // namespace ra
