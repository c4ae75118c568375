// ra_norm.cuh -- the end of a tensor-parallel block, forward and backward: the
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
// once.  A row's columns stay with the threads that loaded them (one warp a
// row for narrow rows, one CTA for wide ones), so every input is read once
// and every output written once: the kernels are bound by memory traffic, few
// rows by the latency of two sums over a block.
//
// The rows reach the registers through a ring of kDepth slots in shared
// memory: a slot holds one tensor's part of a row, every thread copies its own
// columns into it (cp.async) kDepth - 1 slots ahead and reads them back
// itself, so the copies need no barrier and run on through the sums over the
// block and into the next row.
#pragma once

#include "ra_ops.cuh"

namespace ra {
namespace norm {

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

__device__ __forceinline__ void copy_async(uint32_t smem, const void* p, int bytes) {
  if (!RA_ACCESS_OK(p, (unsigned)bytes, 1u)) return;
  if (bytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(p) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem), "l"(p) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The columns of one thread, for rows of type D: kEach of them in pieces of U
// neighbouring columns, a row's threads side by side.  GRAIN is what every
// row of every buffer of the call is aligned to, and whole multiples of:
//   16 bytes  pieces of one 16-byte vector
//   4 bytes   pieces of 4 bytes (two columns of a 16-bit type)
//   2 bytes   single columns of a 16-bit type, loaded without the ring
//             (cp.async copies no less than 4 bytes)
template <class D, int VPT, int GRAIN, int MAXT> struct Cols {
  using T = typename D::T;
  static constexpr int kEach = D::kVec * VPT;
  static constexpr int U = GRAIN / (int)sizeof(T);
  static constexpr int kPieces = kEach / U;
  static constexpr bool kRing = GRAIN >= 4;
  static constexpr int kSlotBytes = kEach * (int)sizeof(T);   // per thread
  // slots of the ring: 8, or what 192 KB hold for a row of MAXT threads
  static constexpr int kDepth = 192 * 1024 / (MAXT * kSlotBytes) < 8 ? 192 * 1024 / (MAXT * kSlotBytes) : 8;

  static __device__ __forceinline__ int column(int k) { return (k * (int)blockDim.x + (int)threadIdx.x) * U; }

  // `half` of E's elements of each piece (a residual stream of binary32 beside
  // a 16-bit type takes two slots)
  template <class E>
  static __device__ __forceinline__ void fetch(uint32_t slot, const void* base, int64_t at, int half, int dim) {
    const char* row = static_cast<const char*>(base) + at * (int64_t)sizeof(typename E::T);
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int c = column(k);
      if (c < dim)
        copy_async(slot + (uint32_t)((k * blockDim.x + threadIdx.x) * GRAIN),
                   row + (int64_t)c * (int)sizeof(typename E::T) + half * GRAIN, GRAIN);
    }
  }

  // a slot's columns (of E; the half of each piece that it holds)
  template <class E>
  static __device__ __forceinline__ void read(uint32_t slot, int half, int dim, float (&x)[kEach]) {
    constexpr int n = GRAIN / (int)sizeof(typename E::T);   // elements of a piece that one slot holds
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      float v[n];
      const uint32_t at = slot + (uint32_t)((k * blockDim.x + threadIdx.x) * GRAIN);
      if (GRAIN == 16) {
        uint4 w;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at));
        float u[E::kVec];
        unpack<E>(w, u);
#pragma unroll
        for (int e = 0; e < n; ++e) v[e] = u[e];
      } else {
        uint32_t w;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(at));
        if (sizeof(typename E::T) == 4) {
          v[0] = __uint_as_float(w);
        } else {
          v[0] = widen<E>((typename E::T)(w & 0xFFFFu));
          v[n - 1] = widen<E>((typename E::T)(w >> 16));
        }
      }
      const bool some = column(k) < dim;
#pragma unroll
      for (int e = 0; e < n; ++e) x[k * U + half * n + e] = some ? v[e] : 0.0f;
    }
  }

  // straight from memory: weights and gates, which every row reads, and rows without the ring
  template <class E>
  static __device__ __forceinline__ void load_piece(const void* base, int64_t at, int k, int dim, float (&x)[U]) {
    const typename E::T* row = static_cast<const typename E::T*>(base) + at;
    const int c = column(k);
    if (c >= dim) {
#pragma unroll
      for (int e = 0; e < U; ++e) x[e] = 0.0f;
      return;
    }
    if constexpr (GRAIN == 16) {
#pragma unroll
      for (int q = 0; q < U / E::kVec; ++q)
        unpack<E>(ld_plain(reinterpret_cast<const uint4*>(row + c) + q), x + q * E::kVec);
    } else if constexpr (U == 2 && sizeof(typename E::T) == 2) {
      const uint32_t w = ld_g(reinterpret_cast<const uint32_t*>(row + c));
      x[0] = widen<E>((typename E::T)(w & 0xFFFFu));
      x[1] = widen<E>((typename E::T)(w >> 16));
    } else {
#pragma unroll
      for (int e = 0; e < U; ++e) x[e] = widen<E>(ld_g(row + c + e));
    }
  }
  // weights and gates are binary32 or of type D
  static __device__ __forceinline__ void load_param(const void* base, int64_t at, bool f32, int k, int dim,
                                                    float (&x)[U]) {
    if (f32)
      load_piece<DF32>(base, at, k, dim, x);
    else
      load_piece<D>(base, at, k, dim, x);
  }

  template <class E>
  static __device__ __forceinline__ void store_piece(void* base, int64_t at, int k, int dim, const float* x) {
    typename E::T* row = static_cast<typename E::T*>(base) + at;
    const int c = column(k);
    if (c >= dim) return;
    if constexpr (GRAIN == 16) {
#pragma unroll
      for (int q = 0; q < U / E::kVec; ++q)
        st_stream(reinterpret_cast<uint4*>(row + c) + q, pack<E>(x + q * E::kVec));
    } else if constexpr (U == 2 && sizeof(typename E::T) == 2) {
      st_g(reinterpret_cast<uint32_t*>(row + c), pack2<E>(x[0], x[1]));
    } else {
#pragma unroll
      for (int e = 0; e < U; ++e) st_g(row + c + e, narrow<E>(x[e]));
    }
  }
  template <class E>
  static __device__ __forceinline__ void store(void* base, int64_t at, int dim, const float (&x)[kEach]) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k) store_piece<E>(base, at, k, dim, x + k * U);
  }
};

extern __shared__ uint4 g_ring[];

// The ring of one thread: its slots' addresses, the next slot to fill and to
// read.  Every step commits one group of copies, so kDepth - 1 of them are in
// flight; the slot that is filled is the one read in the step before.
template <class C> struct Ring {
  uint32_t base;
  int fill, take;
  __device__ __forceinline__ Ring() {
    // a CTA's slots one after another, the rows of a CTA of narrow rows apart
    base = smem_addr(g_ring) + threadIdx.y * (uint32_t)(C::kDepth * C::kSlotBytes) * blockDim.x;
    fill = take = 0;
  }
  __device__ __forceinline__ uint32_t slot(int i) const {
    return base + (uint32_t)i * (uint32_t)C::kSlotBytes * blockDim.x;
  }
  // Rows: what the kernel reads, in its order; next(slot) starts the next copy
  template <class Rows> __device__ __forceinline__ void start(Rows& rows) {
    if (C::kRing)
      for (int i = 0; i < C::kDepth - 1; ++i) refill(rows);
  }
  template <class Rows> __device__ __forceinline__ void refill(Rows& rows) {
    rows.next(slot(fill));
    copy_commit();
    fill = fill + 1 == C::kDepth ? 0 : fill + 1;
  }
  // the oldest copy, complete
  __device__ __forceinline__ uint32_t oldest() {
    copy_wait<C::kDepth - 2>();
    const uint32_t at = slot(take);
    take = take + 1 == C::kDepth ? 0 : take + 1;
    return at;
  }
};

// One tensor's columns of the current row, next in the ring's order (or
// straight from memory).
template <class C, class E, class D, class Rows>
__device__ __forceinline__ void take(Ring<C>& ring, Rows& rows, const void* base, int64_t at, int dim,
                                     float (&x)[C::kEach]) {
  if constexpr (C::kRing) {
    constexpr int halves = (int)(sizeof(typename E::T) / sizeof(typename D::T));
#pragma unroll
    for (int half = 0; half < halves; ++half) {
      C::template read<E>(ring.oldest(), half, dim, x);
      ring.refill(rows);
    }
  } else {
#pragma unroll
    for (int k = 0; k < C::kPieces; ++k) {
      float v[C::U];
      C::template load_piece<E>(base, at, k, dim, v);
#pragma unroll
      for (int e = 0; e < C::U; ++e) x[k * C::U + e] = v[e];
    }
  }
}

template <class C, class D, class Rows>
__device__ __forceinline__ void take_sum(Ring<C>& ring, Rows& rows, const void* const* in, int count, int64_t at,
                                         int dim, float (&acc)[C::kEach]) {
  take<C, D, D>(ring, rows, in[0], at, dim, acc);
#pragma unroll 4
  for (int r = 1; r < count; ++r) {
    float x[C::kEach];
    take<C, D, D>(ring, rows, in[r], at, dim, x);
#pragma unroll
    for (int e = 0; e < C::kEach; ++e) acc[e] = __fadd_rn(acc[e], x[e]);
  }
}

// What forward reads: every row's R partials, then its residual.
template <class C, class D, class RD> struct ForwardRows {
  const NormForward& a;
  int64_t row, step;
  int item;
  __device__ __forceinline__ ForwardRows(const NormForward& args, int64_t first, int64_t by)
      : a(args), row(first), step(by), item(0) {}
  __device__ __forceinline__ void next(uint32_t slot) {
    constexpr int halves = (int)(sizeof(typename RD::T) / sizeof(typename D::T));
    if (row >= a.rows) return;
    if (item < a.R)
      C::template fetch<D>(slot, a.in[item], row * a.in_stride, 0, a.dim);
    else
      C::template fetch<RD>(slot, a.residual, row * a.residual_stride, item - a.R, a.dim);
    if (++item == a.R + halves) {
      item = 0;
      row += step;
    }
  }
};

template <class D, class RD, int VPT, int GRAIN, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_forward_kernel(const __grid_constant__ NormForward a) {
  using C = Cols<D, VPT, GRAIN, MAXT>;
  constexpr int U = C::U;
  __shared__ float red[2][32];
  int turn = 0;
  const float inv_dim = 1.0f / (float)a.dim;
  const int64_t first = (int64_t)blockIdx.x * blockDim.y + threadIdx.y, step = (int64_t)gridDim.x * blockDim.y;
  ForwardRows<C, D, RD> rows(a, first, step);
  Ring<C> ring;
  ring.start(rows);
  for (int64_t row = first; row < a.rows; row += step) {
    float s[C::kEach], h[C::kEach];
    take_sum<C, D>(ring, rows, a.in, a.R, row * a.in_stride, a.dim, s);
    if (a.total) C::template store<D>(a.total, row * a.total_stride, a.dim, s);
    float r1 = 0.0f;
    if (a.post_weight) {
      float sq = 0.0f;
#pragma unroll
      for (int e = 0; e < C::kEach; ++e) sq = __fmaf_rn(s[e], s[e], sq);
      r1 = rsqrtf(row_sum(sq, red, turn) * inv_dim + a.eps);
    }
    take<C, RD, D>(ring, rows, a.residual, row * a.residual_stride, a.dim, h);
    float sq = 0.0f;
#pragma unroll
    for (int k = 0; k < C::kPieces; ++k) {
      if (a.post_weight) {
        float w[U];
        C::load_param(a.post_weight, 0, a.param_f32, k, a.dim, w);
#pragma unroll
        for (int e = 0; e < U; ++e) s[k * U + e] = s[k * U + e] * r1 * w[e];
      }
      if (a.gate) {
        float g[U];
        C::load_param(a.gate, row / a.rows_per_gate * a.dim, a.param_f32, k, a.dim, g);
#pragma unroll
        for (int e = 0; e < U; ++e) s[k * U + e] *= g[e];
      }
#pragma unroll
      for (int e = 0; e < U; ++e) {
        h[k * U + e] = __fmaf_rn(a.scale, s[k * U + e], h[k * U + e]);
        sq = __fmaf_rn(h[k * U + e], h[k * U + e], sq);
      }
    }
    C::template store<RD>(a.residual_out, row * a.residual_out_stride, a.dim, h);
    const float r2 = rsqrtf(row_sum(sq, red, turn) * inv_dim + a.eps);
#pragma unroll
    for (int k = 0; k < C::kPieces; ++k) {
      float w[U];
      C::load_param(a.weight, 0, a.param_f32, k, a.dim, w);
#pragma unroll
      for (int e = 0; e < U; ++e) h[k * U + e] = h[k * U + e] * r2 * w[e];
    }
    for (int q = 0; q < a.outs; ++q) C::template store<D>(a.out[q], row * a.out_stride, a.dim, h);
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

// The rows of one worker, in order.
struct Dealt {
  int64_t u, row, hi;
  __device__ __forceinline__ void open(const NormBackward& a, const Deal& d) {
    if (u >= d.units) return;
    const int64_t group = u / d.parts, part = u - group * d.parts;
    const int64_t end = (group + 1) * a.rows_per_gate;
    row = group * a.rows_per_gate + part * d.rows_per_part;
    hi = row + d.rows_per_part < end ? row + d.rows_per_part : end;
  }
};

// What backward reads: every row's partial gradients, what forward's residual
// was, the residual's gradient where there is one, and the sum where it is needed.
template <class C, class D, class RD> struct BackwardRows {
  const NormBackward& a;
  const Deal& d;
  Dealt at;
  int item, items;
  static constexpr int kHalves = (int)(sizeof(typename RD::T) / sizeof(typename D::T));
  __device__ __forceinline__ BackwardRows(const NormBackward& args, const Deal& deal, int64_t worker)
      : a(args), d(deal), item(0) {
    at.u = worker;
    at.open(a, d);
    items = a.grads + kHalves + (a.grad_residual_out ? kHalves : 0) + (a.total ? 1 : 0);
  }
  __device__ __forceinline__ void next(uint32_t slot) {
    if (at.u >= d.units) return;
    int i = item;
    if (i < a.grads) {
      C::template fetch<D>(slot, a.grad_out[i], at.row * a.grad_out_stride, 0, a.dim);
    } else if ((i -= a.grads) < kHalves) {
      C::template fetch<RD>(slot, a.residual_out, at.row * a.residual_out_stride, i, a.dim);
    } else if (a.grad_residual_out && (i -= kHalves) < kHalves) {
      C::template fetch<RD>(slot, a.grad_residual_out, at.row * a.grad_residual_out_stride, i, a.dim);
    } else {
      C::template fetch<D>(slot, a.total, at.row * a.total_stride, 0, a.dim);
    }
    if (++item == items) {
      item = 0;
      if (++at.row == at.hi) {
        at.u += d.workers;
        at.open(a, d);
      }
    }
  }
};

template <class D, class RD, int VPT, int GRAIN, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_backward_kernel(const __grid_constant__ NormBackward a,
                                                             const __grid_constant__ Deal d) {
  using C = Cols<D, VPT, GRAIN, MAXT>;
  constexpr int U = C::U, N = C::kEach;
  __shared__ float red[2][32];
  int turn = 0;
  const float inv_dim = 1.0f / (float)a.dim;
  const int64_t worker = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  BackwardRows<C, D, RD> rows(a, d, worker);
  Ring<C> ring;
  ring.start(rows);
  float dw[N], dp[N];
#pragma unroll
  for (int e = 0; e < N; ++e) dw[e] = dp[e] = 0.0f;
  Dealt at;
  for (at.u = worker; at.u < d.units; at.u += d.workers) {
    at.open(a, d);
    const int64_t group = at.u / d.parts;
    float dg[N];
#pragma unroll
    for (int e = 0; e < N; ++e) dg[e] = 0.0f;
    for (int64_t row = at.row; row < at.hi; ++row) {
      float z[N], x[N];
      take_sum<C, D>(ring, rows, a.grad_out, a.grads, row * a.grad_out_stride, a.dim, z);
      take<C, RD, D>(ring, rows, a.residual_out, row * a.residual_out_stride, a.dim, x);
      const float r2 = ld_g(a.rstd + a.rows + row);
      const float r1 = a.post_weight ? ld_g(a.rstd + row) : 1.0f;
      float c = 0.0f;
#pragma unroll
      for (int k = 0; k < C::kPieces; ++k) {
        float w[U];
        C::load_param(a.weight, 0, a.param_f32, k, a.dim, w);
#pragma unroll
        for (int e = 0; e < U; ++e) {
          const int i = k * U + e;
          x[i] *= r2;                                   // x2
          dw[i] = __fmaf_rn(z[i], x[i], dw[i]);
          z[i] *= w[e];
          c = __fmaf_rn(z[i], x[i], c);
        }
      }
      const float c2 = row_sum(c, red, turn) * inv_dim;
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = r2 * __fmaf_rn(-c2, x[i], z[i]);
      if (a.grad_residual_out) {
        float t[N];
        take<C, RD, D>(ring, rows, a.grad_residual_out, row * a.grad_residual_out_stride, a.dim, t);
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] += t[i];       // e
      }
      C::template store<RD>(a.grad_residual, row * a.grad_residual_stride, a.dim, z);
      if (a.total) take<C, D, D>(ring, rows, a.total, row * a.total_stride, a.dim, x);
      c = 0.0f;
#pragma unroll
      for (int k = 0; k < C::kPieces; ++k) {
        float w[U], g[U];
        if (a.post_weight) C::load_param(a.post_weight, 0, a.param_f32, k, a.dim, w);
        if (a.gate) C::load_param(a.gate, group * a.dim, a.param_f32, k, a.dim, g);
#pragma unroll
        for (int e = 0; e < U; ++e) {
          const int i = k * U + e;
          x[i] *= r1;                                   // x1 (S without a post norm)
          z[i] *= a.scale;
          if (a.grad_gate) dg[i] = __fmaf_rn(a.post_weight ? x[i] * w[e] : x[i], z[i], dg[i]);
          if (a.gate) z[i] *= g[e];                     // the gradient of y
          if (a.post_weight) {
            dp[i] = __fmaf_rn(z[i], x[i], dp[i]);
            z[i] *= w[e];
            c = __fmaf_rn(z[i], x[i], c);
          }
        }
      }
      if (a.post_weight) {
        const float c1 = row_sum(c, red, turn) * inv_dim;
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = r1 * __fmaf_rn(-c1, x[i], z[i]);
      }
      for (int q = 0; q < a.outs; ++q) C::template store<D>(a.grad_in[q], row * a.grad_in_stride, a.dim, z);
    }
    // one unit per gate row: its gradient is whole; else a partial per unit
    if (a.grad_gate)
      C::template store<DF32>(d.parts == 1 ? a.grad_gate : a.work + 2 * d.workers * a.dim, at.u * a.dim, a.dim, dg);
  }
  if (a.grad_weight) C::template store<DF32>(a.work, worker * a.dim, a.dim, dw);
  if (a.grad_post_weight) C::template store<DF32>(a.work, (d.workers + worker) * a.dim, a.dim, dp);
}

// How a row of `dim` columns is spread: threads, 16-byte vectors per thread,
// rows per CTA, and the kernel's most threads.
struct Shape {
  int threads, groups, rows, most;
};

inline Shape spread(int dim, int vec, int groups, int most) {
  const int vectors = (dim + vec - 1) / vec;
  Shape s;
  s.groups = groups;
  s.most = most;
  s.threads = ((vectors + groups - 1) / groups + 31) / 32 * 32;
  s.rows = s.threads == 32 ? kWarpRows : 1;
  return s;
}

// Forward: one vector a thread up to 1024 threads.
inline Shape forward_shape(int dim, int vec) {
  int groups = 1;
  while (dim > vec * 1024 * groups) groups *= 2;
  return spread(dim, vec, groups, 1024);
}

// Backward keeps three sums per column in registers: at 128 registers a
// thread, up to 512 threads, sixteen columns fit; wider rows take 1024
// threads of 64.
inline Shape backward_shape(int dim, int vec) {
  int groups = 1;
  while (dim > vec * 512 * groups && vec * groups < 16) groups *= 2;
  return spread(dim, vec, groups, dim > vec * 512 * groups ? 1024 : 512);
}

// CTAs that the SMs hold: 64 K registers each.
inline int64_t most_ctas(const Shape& s, int sms) {
  const int per_sm = s.most / (s.threads * s.rows);
  return (int64_t)sms * (per_sm < 1 ? 1 : per_sm > 4 ? 4 : per_sm);
}

// f(IntC<GRAIN>) for what every row is aligned to.
template <class D, class F> cudaError_t with_grain(int grain, F&& f) {
  if (grain == 16) return f(IntC<16>{});
  if (grain == 4) return f(IntC<4>{});
  if constexpr (sizeof(typename D::T) == 2) {
    if (grain == 2) return f(IntC<2>{});
  }
  return cudaErrorInvalidValue;
}

// f(IntC<groups per thread>)
template <class D, class F> cudaError_t with_groups(int groups, F&& f) {
  if (groups == 1) return f(IntC<1>{});
  if (groups == 2) return f(IntC<2>{});
  if constexpr (D::kVec == 4) {
    if (groups == 4) return f(IntC<4>{});
  }
  return cudaErrorInvalidValue;
}

// The ring's shared memory, opted in to.
template <class C, class K> cudaError_t ring_bytes(K kernel, const Shape& s, size_t* bytes) {
  *bytes = C::kRing ? (size_t)C::kDepth * C::kSlotBytes * s.threads * s.rows : 0;
  if (*bytes <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)*bytes);
}

template <class D, class RD>
cudaError_t run_forward(const Shape& s, int grain, const NormForward& a, unsigned grid, cudaStream_t st) {
  cudaError_t e = debug_upload(st);
  if (e != cudaSuccess) return e;
  return with_groups<D>(s.groups, [&](auto g) {
    return with_grain<D>(grain, [&](auto al) {
      constexpr int kGroups = decltype(g)::value, kGrain = decltype(al)::value;
      auto kernel = norm_forward_kernel<D, RD, kGroups, kGrain, 1024>;
      size_t smem;
      const cudaError_t e2 = ring_bytes<Cols<D, kGroups, kGrain, 1024>>(kernel, s, &smem);
      if (e2 != cudaSuccess) return e2;
      kernel<<<grid, dim3(s.threads, s.rows), smem, st>>>(a);
      return cudaGetLastError();
    });
  });
}

template <class D, class RD>
cudaError_t run_backward(const Shape& s, int grain, const NormBackward& a, const Deal& d, unsigned grid,
                         cudaStream_t st) {
  cudaError_t e = debug_upload(st);
  if (e != cudaSuccess) return e;
  return with_groups<D>(s.groups, [&](auto g) {
    return with_grain<D>(grain, [&](auto al) {
      constexpr int kGroups = decltype(g)::value, kGrain = decltype(al)::value;
      auto launch = [&](auto kernel, auto cols) {
        size_t smem;
        const cudaError_t e2 = ring_bytes<decltype(cols)>(kernel, s, &smem);
        if (e2 != cudaSuccess) return e2;
        kernel<<<grid, dim3(s.threads, s.rows), smem, st>>>(a, d);
        return cudaGetLastError();
      };
      if constexpr (kGroups * D::kVec == 16) {
        if (s.most == 1024)
          return launch(norm_backward_kernel<D, RD, kGroups, kGrain, 1024>, Cols<D, kGroups, kGrain, 1024>{});
      }
      return launch(norm_backward_kernel<D, RD, kGroups, kGrain, 512>, Cols<D, kGroups, kGrain, 512>{});
    });
  });
}

}  // namespace norm
}  // namespace ra
