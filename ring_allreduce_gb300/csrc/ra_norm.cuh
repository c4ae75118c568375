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
// The rows reach the registers through a ring of kDepth steps in shared
// memory: a step holds up to kQ tensors' parts of a row, every warp copies its
// own columns into its part of it (cp.async) kDepth - 1 steps ahead and reads
// them back itself, so the copies need no barrier of the block and run on
// through the sums over it and into the next row.  What binds next is the
// instructions per column: arithmetic is done on pairs of columns
// (fma.rn.f32x2 and its like), a warp's columns lie side by side, so that all
// addresses within a row are constants away from the warp's first one, and a
// step of four tensors waits, counts and commits once (one at a time, that
// took 40 to 60 instructions a tensor beside the 13 a vector needs).
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

__device__ __forceinline__ void copy_async(uint32_t smem, const char* p) {
  if (!RA_ACCESS_OK(p, 16u, 1u)) return;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(p) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A value that is the same in the whole warp, in a form the compiler can see to be.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// The columns of one thread, for rows of type D: kEach of them (as pairs), of
// a warp's 32 kEach neighbouring columns.
//   AL   every row of every buffer of the call starts on a 16-byte boundary
//        and holds whole 16-byte vectors: a thread has whole vectors, the
//        warp's side by side.
//   else rows may start on any element: a thread has every 32nd column, and a
//        slot holds the 16-byte vectors that cover the warp's columns, shifted
//        as they lie in memory (bytes of the neighbouring rows come along and
//        are not used).
//   PK   AL, and a row has sixteen vectors at most: as many rows as fit share a
//        warp, a power of two of lanes each (65536 x 128 bf16, eight ranks:
//        37 us forward, 63 backward; a warp a row 67 and 100).
template <class D, int VPT, bool AL, int MAXT, bool PK = false> struct Cols {
  static_assert(!PK || (AL && VPT == 1), "rows that share a warp");
  using T = typename D::T;
  static constexpr bool kPacked = PK;
  static constexpr int V = D::kVec;
  static constexpr int kEach = V * VPT, kPairs = kEach / 2;
  static constexpr int kWarpBytes = 32 * kEach * (int)sizeof(T) + (AL ? 0 : 16);   // of a slot
  // tensors of a step, and steps of the ring: 128 KB for 1024 threads of one
  // vector each (the L1 cache keeps the rest, for the weights)
  static constexpr int kFits = 33 * 1024 / (MAXT / 32 * kWarpBytes);
  static constexpr int kQ = kFits >= 4 ? 4 : kFits >= 2 ? 2 : 1;
  static constexpr int kSteps = 198 * 1024 / (MAXT / 32 * kWarpBytes * kQ);
  static constexpr int kDepth = kSteps < 4 ? kSteps : 4;

  int lane, base;   // the thread among its row's lanes of the warp; the warp's first column
  int all, left;    // columns of the row from the thread's first on (left: none where its row is past the end)
  int dim;
  int lanes, sub, packs;   // a row's lanes, the thread's row among the warp's, and those
  bool whole;       // all of the warp's columns are in the row
  __device__ __forceinline__ explicit Cols(int columns) : dim(columns), lanes(32), sub(0), packs(1) {
    lane = threadIdx.x & 31;
    if constexpr (PK) {
      while (lanes / 2 * V >= dim) lanes /= 2;
      packs = 32 / lanes;
      sub = lane / lanes;
      lane &= lanes - 1;
    }
    base = uniform((int)(threadIdx.x >> 5)) * 32 * kEach;
    all = left = dim - base - (AL ? lane * V : lane);
    whole = base + lanes * kEach <= dim;
  }
  __device__ __forceinline__ void live(bool is) {
    if constexpr (PK) left = is ? all : 0;
  }
  // Sum over the threads of a row, the same value in all of them.
  __device__ __forceinline__ float sum(float v, float (*red)[32], int& turn) const {
    if constexpr (PK) {
      for (int o = lanes / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      return v;
    } else {
      return row_sum(v, red, turn);
    }
  }
  // pieces: AL a vector, else a column
  static constexpr int kPieces = AL ? VPT : kEach;
  static constexpr bool kZeroed = AL;
  static constexpr int kUnroll = AL ? 4 : 1;
  // Columns one by one are loaded and stored without a test each by the warps
  // that are whole, which doubles that code: so only where there are many rows
  // (sixteen columns a thread).  4096 x 5001 bf16 of three ranks takes 67 us so, 83
  // without; for few rows it is nearly one (96 x 5001: 6.3 us, 6.0 with it; 96 x 1538
  // fp16 of two ranks backward: 9.3 and 9.1).
  static constexpr bool kTwice = !AL && kEach == 16;
  static constexpr int kStep = AL ? 32 * V : 32;   // columns from a thread's piece to its next
  __device__ __forceinline__ bool has(int k) const { return k * kStep < left; }
  __device__ __forceinline__ uint32_t place() const { return (threadIdx.x & 31u) * 16; }   // in a slot
  __device__ __forceinline__ int first() const { return base + (AL ? lane * V : lane); }

  // Buffers are addressed by a row's offset in elements; the warp's (else) or
  // the thread's (AL) first column of that row:
  template <class E> __device__ __forceinline__ int64_t offset(int64_t elements) const {
    return (elements + (AL ? first() : base)) * (int64_t)sizeof(typename E::T);
  }

  // Copies of E take sizeof(E) / sizeof(D) slots: `half` of each vector of
  // columns (AL) or of the warp's columns (else).
  template <class E> static __host__ __device__ constexpr int halves() { return (int)(sizeof(typename E::T) / sizeof(T)); }

  // One tensor's part of a row into a slot.  lo: where the buffer begins;
  // elements: its row's offset; inner: 16 bytes on both sides of the row are
  // the buffer's, else rows and stride say what is.
  template <class E>
  __device__ __forceinline__ void fetch(uint32_t slot, const void* buffer, int64_t elements, int half, bool inner,
                                        int64_t rows, int64_t stride) const {
    constexpr int es = (int)sizeof(typename E::T);
    const char* lo = static_cast<const char*>(buffer);
    const char* p = lo + offset<E>(elements);
    if constexpr (AL) {
#pragma unroll
      for (int k = 0; k < VPT; ++k)
        if (k * kStep < all) copy_async(slot + k * 512 + place(), p + half * 16 + k * kStep * es);
    } else {
      constexpr int most = 32 * kEach / halves<E>();   // columns in a slot
      p += half * most * es;
      const int columns = min(most, dim - base - half * most);
      if (columns <= 0) return;
      const int shift = (int)(reinterpret_cast<uintptr_t>(p) & 15u);
      const char* v0 = p - shift;
      const int vectors = (shift + columns * es + 15) >> 4;
      bool inside = inner;   // nothing but the buffer is read
      if (!inner) inside = v0 >= lo && v0 + 16 * vectors <= lo + ((rows - 1) * stride + dim) * es;
#pragma unroll
      for (int i = 0; i < (most * es / 16 + 1 + 31) / 32; ++i) {
        const int v = lane + 32 * i;
        if (v < vectors && (inside || (v > 0 && v < vectors - 1))) copy_async(slot + v * 16, v0 + v * 16);
      }
      if (inside) return;
      // the vectors at the ends, an element a lane (16 and shift are multiples of its size)
      constexpr int each = 16 / es;
      const int at = lane < each ? lane : lane - each + (vectors - 1) * each;   // in elements from v0
      const int c = at - shift / es;
      if (lane < (vectors > 1 ? 2 * each : each) && c >= 0 && c < columns) {
        const typename E::T x = ld_g(reinterpret_cast<const typename E::T*>(p) + c);
        if constexpr (es == 4)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(slot + at * es), "f"(x) : "memory");
        else
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(slot + at * es), "h"(x) : "memory");
      }
    }
  }

  // A slot's columns of E; p as in fetch.  Columns past the row come back as
  // anything (AL: 0), see clear().
  template <class E>
  __device__ __forceinline__ void read(uint32_t slot, const char* p, int half, float2 (&x)[kPairs]) const {
    constexpr int es = (int)sizeof(typename E::T), n = halves<E>();
    if constexpr (AL) {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        uint4 w;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                     : "r"(slot + k * 512 + place())
                     : "memory");
        unpack<E>(w, reinterpret_cast<float*>(&x[k * (V / 2)]) + half * (V / n));
      }
    } else {
      p += half * (32 * kEach / n) * es;
      const uint32_t at = slot + (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u) + lane * es;
      float* to = reinterpret_cast<float*>(x) + half * (kEach / n);
#pragma unroll
      for (int e = 0; e < kEach / n; ++e) {
        if constexpr (es == 4) {
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(to[e]) : "r"(at + e * 32 * es) : "memory");
        } else {
          unsigned short w;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w) : "r"(at + e * 32 * es) : "memory");
          to[e] = widen<E>(w);
        }
      }
    }
  }

  // 0 in the columns past the row, and in rows past the end
  __device__ __forceinline__ void clear(float2 (&x)[kPairs]) const {
    if ((AL && !PK) || (!PK && whole)) return;
    float* f = reinterpret_cast<float*>(x);
#pragma unroll
    for (int e = 0; e < kEach; ++e) f[e] = has(PK ? 0 : e) ? f[e] : 0.0f;
  }

  // The rows of a warp (PK) summed, for its first one.
  __device__ __forceinline__ void fold(float2 (&x)[kPairs]) {
    if constexpr (PK) {
      for (int o = lanes; o < 32; o *= 2) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
          x[i] = add2(x[i], make_float2(__shfl_xor_sync(0xFFFFFFFFu, x[i].x, o), __shfl_xor_sync(0xFFFFFFFFu, x[i].y, o)));
      }
      left = sub == 0 ? all : 0;
    }
  }

  // The warp's columns, binary32, into shared memory, `to` the row's first.
  __device__ __forceinline__ void keep(float* to, const float2 (&x)[kPairs]) const {
    const float* f = reinterpret_cast<const float*>(x);
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      if (!has(k)) continue;
#pragma unroll
      for (int e = 0; e < kEach / kPieces; ++e) to[first() + k * kStep + e] = f[k * (kEach / kPieces) + e];
    }
  }

  // Weights and gates, binary32 or of type D, which every row reads; 1 where there are none, 0 past the row.
  template <class E> __device__ __forceinline__ void load_as(const void* from, int64_t elements, float2 (&x)[kPairs]) const {
    const typename E::T* p = static_cast<const typename E::T*>(from) + elements + first();
    float* f = reinterpret_cast<float*>(x);
    if constexpr (kTwice) {
      if (whole) {
#pragma unroll
        for (int k = 0; k < kPieces; ++k) f[k] = widen<E>(ld_g(p + k * kStep));
        return;
      }
    }
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      if constexpr (AL) {
        if (has(k)) {
#pragma unroll
          for (int q = 0; q < V / E::kVec; ++q)
            unpack<E>(ld_plain(reinterpret_cast<const uint4*>(p + k * kStep) + q), f + k * V + q * E::kVec);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) f[k * V + e] = 0.0f;
        }
      } else {
        f[k] = has(k) ? widen<E>(ld_g(p + k * kStep)) : 0.0f;
      }
    }
  }
  __device__ __forceinline__ void param(const void* from, int64_t elements, bool f32, float2 (&x)[kPairs]) const {
    if (!from) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) x[i] = splat(1.0f);
    } else if (f32) {
      load_as<DF32>(from, elements, x);
    } else {
      load_as<D>(from, elements, x);
    }
  }

  template <class E> __device__ __forceinline__ void store(void* to, int64_t elements, const float2 (&x)[kPairs]) const {
    typename E::T* p = static_cast<typename E::T*>(to) + elements + first();
    const float* f = reinterpret_cast<const float*>(x);
    if constexpr (kTwice) {
      if (whole) {
#pragma unroll
        for (int k = 0; k < kPieces; ++k) st_g(p + k * kStep, narrow<E>(f[k]));
        return;
      }
    }
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      if (!has(k)) continue;
      if constexpr (AL) {
#pragma unroll
        for (int q = 0; q < V / E::kVec; ++q)
          st_stream(reinterpret_cast<uint4*>(p + k * kStep) + q, pack<E>(f + k * V + q * E::kVec));
      } else {
        st_g(p + k * kStep, narrow<E>(f[k]));
      }
    }
  }
};

extern __shared__ uint4 g_ring[];

// The ring of one warp: the next step to fill and the one being read.  Every
// step commits one group of copies; a step is filled again as soon as the
// warp has gone on to the next one.
template <class C> struct Ring {
  uint32_t base, fill, now, end;
  uint32_t part, step;   // bytes of a tensor's slot in a step, and of a step, for the row's warps
  __device__ __forceinline__ explicit Ring(const C& cols) {
    // a CTA's slots one after another; the rows of a CTA of narrow rows apart
    part = (uint32_t)C::kWarpBytes * (blockDim.x >> 5);
    step = part * C::kQ;
    base = smem_addr(g_ring) + (uint32_t)uniform((int)threadIdx.y) * (uint32_t)C::kDepth * step +
           (uint32_t)uniform((int)(threadIdx.x >> 5)) * (uint32_t)C::kWarpBytes;
    end = base + (uint32_t)C::kDepth * step;
    // vectors past the row are never copied: 0 for good (rows anywhere: see clear())
    if (C::kZeroed && !cols.whole)
      for (uint32_t at = base + cols.place(); at < end; at += part)
        for (uint32_t k = 0; k + cols.place() < C::kWarpBytes; k += 512)
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at + k), "r"(0) : "memory");
    __syncwarp();
    fill = base;
    now = end - step;    // the first advance() goes on to `base`
  }
  // Rows: what the kernel reads, in its order
  template <class Rows> __device__ __forceinline__ void start(Rows& rows) {
    for (int i = 0; i < C::kDepth - 1; ++i) refill(rows);
  }
  template <class Rows> __device__ __forceinline__ void refill(Rows& rows) {
    rows.fetch(fill, part);
    copy_commit();
    fill += step;
    fill = fill == end ? base : fill;
  }
  // On to the next step, complete for the whole warp; the one before is filled again.
  template <class Rows> __device__ __forceinline__ void advance(Rows& rows) {
    copy_wait<C::kDepth - 2>();
    __syncwarp();
    now += step;
    now = now == end ? base : now;
    refill(rows);
  }
};

// The tensors of a row in their order; the first one opens a step.
template <class E, class C, class Rows>
__device__ __forceinline__ void take(const C& cols, Ring<C>& ring, Rows& rows, int item, const char* p,
                                     float2 (&x)[C::kPairs]) {
#pragma unroll
  for (int half = 0; half < C::template halves<E>(); ++half) {
    const int q = (item + half) & (C::kQ - 1);
    if (q == 0) ring.advance(rows);
    cols.template read<E>(ring.now + (uint32_t)q * ring.part, p, half, x);
  }
}

template <class D, class C, class Rows>
__device__ __forceinline__ void take_sum(const C& cols, Ring<C>& ring, Rows& rows, const void* const* in, int count,
                                         int64_t elements, float2 (&acc)[C::kPairs]) {
  const int64_t at = cols.template offset<D>(elements);
#pragma unroll 1
  for (int r = 0; r < count; r += C::kQ) {
    ring.advance(rows);
#pragma unroll
    for (int q = 0; q < C::kQ; ++q) {
      if (r + q >= count) break;
      float2 x[C::kPairs];
      cols.template read<D>(ring.now + (uint32_t)q * ring.part, static_cast<const char*>(in[r + q]) + at, 0, x);
      if (q == 0 && r == 0) {
#pragma unroll
        for (int i = 0; i < C::kPairs; ++i) acc[i] = x[i];
      } else {
#pragma unroll
        for (int i = 0; i < C::kPairs; ++i) acc[i] = add2(acc[i], x[i]);
      }
    }
  }
  cols.clear(acc);
}

// Rows between others, of 16 bytes at least, have that much of their buffer on both sides.
template <class D> __device__ __forceinline__ bool inner_row(int64_t row, int64_t rows, int dim) {
  return row > 0 && row < rows - 1 && dim * (int)sizeof(typename D::T) >= 16;
}

// What forward reads: every row's R partials, then its residual.  (fetch()
// stands in the kernel once for every place that goes on to the next step, so
// it is kept short: one copy of the code for all tensors of a type.)
template <class C, class D, class RD> struct ForwardRows {
  static constexpr int kHalves = C::template halves<RD>();
  const NormForward& a;
  const C& cols;
  int64_t row, step;
  int item, items;
  __device__ __forceinline__ ForwardRows(const NormForward& args, const C& c, int64_t first, int64_t every)
      : a(args), cols(c), row(first), step(every), item(0), items(args.R + kHalves) {}
  // the next step's tensors, `part` bytes apart
  __device__ __forceinline__ void fetch(uint32_t slot, uint32_t part) {
    const int64_t mine = row + (C::kPacked ? cols.sub : 0);
    if (row >= a.rows) return;
    const bool inner = inner_row<D>(row, a.rows, a.dim);
#pragma unroll(C::kUnroll)
    for (int q = 0; q < C::kQ; ++q, slot += part) {
      const int i = item + q;
      if (i >= items || (C::kPacked && mine >= a.rows)) break;
      const bool rank = i < a.R;
      const void* buffer = rank ? a.in[i] : a.residual;
      const int64_t stride = rank ? a.in_stride : a.residual_stride;
      if (kHalves == 1 || rank)
        cols.template fetch<D>(slot, buffer, mine * stride, 0, inner, a.rows, stride);
      else
        cols.template fetch<RD>(slot, buffer, mine * stride, i - a.R, inner, a.rows, stride);
    }
    item += C::kQ;
    if (item < items) return;
    item = 0;
    row += step;
  }
};

// Measured, as parts of a copy's 6.8 TB/s for the bytes that have to move:
// 8192 x 4096, four ranks, bf16 with a binary32 residual, post norm, gate, the
// sum kept and four copies out: 143 us, 0.90; 1023 x 5001 binary32, three
// ranks, no row aligned: 30 us, 0.71 (seven rows an SM, the last ones alone);
// one row of 4096 from eight ranks: 4.5 us, two dependent reads and two sums
// over a block after the launch.
template <class D, class RD, int VPT, bool AL, int MAXT, bool PK = false>
__global__ void __launch_bounds__(MAXT) norm_forward_kernel(const __grid_constant__ NormForward a) {
  using C = Cols<D, VPT, AL, MAXT, PK>;
  constexpr int N = C::kPairs;
  __shared__ float red[2][32];
  after_predecessor();
  int turn = 0;
  const float inv_dim = 1.0f / (float)a.dim;
  C cols(a.dim);
  const int64_t first = ((int64_t)blockIdx.x * blockDim.y + uniform((int)threadIdx.y)) * cols.packs,
                step = (int64_t)gridDim.x * blockDim.y * cols.packs;
  ForwardRows<C, D, RD> rows(a, cols, first, step);
  Ring<C> ring(cols);
  ring.start(rows);
  for (int64_t warp_row = first; warp_row < a.rows; warp_row += step) {
    const int64_t row = warp_row + (PK ? cols.sub : 0);
    cols.live(row < a.rows);
    float2 s[N], h[N], w[N];
    take_sum<D>(cols, ring, rows, a.in, a.R, row * a.in_stride, s);
    if (a.total) cols.template store<D>(a.total, row * a.total_stride, s);
    float r1 = 0.0f, f = 1.0f;
    if (a.post_weight) {
      float2 sq = splat(0.0f);
#pragma unroll
      for (int i = 0; i < N; ++i) sq = fma2(s[i], s[i], sq);
      f = r1 = rsqrtf(cols.sum(sq.x + sq.y, red, turn) * inv_dim + a.eps);
      cols.param(a.post_weight, 0, a.param_f32, w);
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] = mul2(mul2(s[i], splat(f)), w[i]);
    }
    if (a.gate) {
      cols.param(a.gate, row / a.rows_per_gate * a.dim, a.param_f32, w);
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] = mul2(s[i], w[i]);
    }
    take<RD>(cols, ring, rows, a.R,
             static_cast<const char*>(a.residual) + cols.template offset<RD>(row * a.residual_stride), h);
    cols.clear(h);
    float2 sq = splat(0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      h[i] = fma2(splat(a.scale), s[i], h[i]);
      sq = fma2(h[i], h[i], sq);
    }
    cols.template store<RD>(a.residual_out, row * a.residual_out_stride, h);
    const float r2 = rsqrtf(cols.sum(sq.x + sq.y, red, turn) * inv_dim + a.eps);
    cols.param(a.weight, 0, a.param_f32, w);
#pragma unroll
    for (int i = 0; i < N; ++i) h[i] = mul2(mul2(h[i], splat(r2)), w[i]);
    for (int q = 0; q < a.outs; ++q) cols.template store<D>(a.out[q], row * a.out_stride, h);
    if (a.rstd && (PK ? cols.lane == 0 && cols.left > 0 : threadIdx.x == 0)) {
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
  int64_t workers, ctas;
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
  static constexpr int kHalves = C::template halves<RD>();
  const NormBackward& a;
  const Deal& d;
  const C& cols;
  Dealt row;
  int item, residuals, items;
  __device__ __forceinline__ BackwardRows(const NormBackward& args, const Deal& deal, const C& c, int64_t worker)
      : a(args), d(deal), cols(c), item(0) {
    row.u = worker;
    row.open(a, d);
    residuals = a.grads + kHalves * (a.grad_residual_out ? 2 : 1);
    items = residuals + (a.total ? 1 : 0);
  }
  __device__ __forceinline__ void fetch(uint32_t slot, uint32_t part) {
    if (row.u >= d.units) return;
    const int64_t mine = row.row + (C::kPacked ? cols.sub : 0);
    const bool inner = inner_row<D>(row.row, a.rows, a.dim);
#pragma unroll(C::kUnroll)
    for (int q = 0; q < C::kQ; ++q, slot += part) {
      const int i = item + q;
      if (i >= items || (C::kPacked && mine >= row.hi)) break;
      const bool residual = i >= a.grads && i < residuals;
      const void* buffer;
      int64_t stride;
      if (i < a.grads) {
        buffer = a.grad_out[i];
        stride = a.grad_out_stride;
      } else if (!residual) {
        buffer = a.total;
        stride = a.total_stride;
      } else {
        const bool grad = i - a.grads >= kHalves;
        buffer = grad ? a.grad_residual_out : a.residual_out;
        stride = grad ? a.grad_residual_out_stride : a.residual_out_stride;
      }
      if (kHalves == 1 || !residual)
        cols.template fetch<D>(slot, buffer, mine * stride, 0, inner, a.rows, stride);
      else
        cols.template fetch<RD>(slot, buffer, mine * stride, (i - a.grads) & (kHalves - 1), inner, a.rows, stride);
    }
    item += C::kQ;
    if (item < items) return;
    item = 0;
    row.row += cols.packs;
    if (row.row >= row.hi) {
      row.u += d.workers;
      row.open(a, d);
    }
  }
};

// Measured: 4096 x 8192 bf16, eight partial gradients, post norm and gate:
// 162 us with the join of the column sums, 0.79 of the copy bandwidth.  The
// registers bound it: a row's values and three sums per column leave one
// CTA of 16 warps to an SM, whose waits for its own sums nothing else fills
// (DRAM 63 % busy, each scheduler with four warps to choose from).  96 x 1538
// fp16, two ranks, eight gate rows: 9.7 us, two launches' latency.  Above 8192
// columns 64 registers a thread spill: 4096 x 16384 551 us, 0.47.
template <class D, class RD, int VPT, bool AL, int MAXT, bool PK = false>
__global__ void __launch_bounds__(MAXT) norm_backward_kernel(const __grid_constant__ NormBackward a,
                                                             const __grid_constant__ Deal d) {
  using C = Cols<D, VPT, AL, MAXT, PK>;
  constexpr int N = C::kPairs, kHalves = C::template halves<RD>();
  __shared__ float red[2][32];
  after_predecessor();
  int turn = 0;
  const float inv_dim = 1.0f / (float)a.dim;
  const int64_t worker = (int64_t)blockIdx.x * blockDim.y + uniform((int)threadIdx.y);
  C cols(a.dim);
  BackwardRows<C, D, RD> rows(a, d, cols, worker);
  Ring<C> ring(cols);
  ring.start(rows);
  float2 dw[N], dp[N];
#pragma unroll
  for (int i = 0; i < N; ++i) dw[i] = dp[i] = splat(0.0f);
  Dealt at;
  for (at.u = worker; at.u < d.units; at.u += d.workers) {
    at.open(a, d);
    const int64_t group = at.u / d.parts;
    float2 dg[N];
#pragma unroll
    for (int i = 0; i < N; ++i) dg[i] = splat(0.0f);
    for (int64_t warp_row = at.row; warp_row < at.hi; warp_row += cols.packs) {
      const int64_t row = warp_row + (PK ? cols.sub : 0);
      const bool live = !PK || row < at.hi;
      cols.live(live);
      float2 z[N], x[N], w[N];
      take_sum<D>(cols, ring, rows, a.grad_out, a.grads, row * a.grad_out_stride, z);
      take<RD>(cols, ring, rows, a.grads,
               static_cast<const char*>(a.residual_out) + cols.template offset<RD>(row * a.residual_out_stride), x);
      cols.clear(x);
      const float r2 = live ? ld_g(a.rstd + a.rows + row) : 0.0f;
      const float r1 = !a.post_weight ? 1.0f : live ? ld_g(a.rstd + row) : 0.0f;
      cols.param(a.weight, 0, a.param_f32, w);
      float2 c = splat(0.0f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        x[i] = mul2(x[i], splat(r2));         // x2
        dw[i] = fma2(z[i], x[i], dw[i]);
        z[i] = mul2(z[i], w[i]);
        c = fma2(z[i], x[i], c);
      }
      const float c2 = cols.sum(c.x + c.y, red, turn) * inv_dim;
      if (a.grad_residual_out) {
        take<RD>(cols, ring, rows, a.grads + kHalves,
                 static_cast<const char*>(a.grad_residual_out) +
                     cols.template offset<RD>(row * a.grad_residual_out_stride), w);
        cols.clear(w);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = splat(0.0f);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = fma2(splat(r2), fma2(splat(-c2), x[i], z[i]), w[i]);   // e
      cols.template store<RD>(a.grad_residual, row * a.grad_residual_stride, z);
      if (a.total) {
        take<D>(cols, ring, rows, a.grads + kHalves * (a.grad_residual_out ? 2 : 1),
                static_cast<const char*>(a.total) + cols.template offset<D>(row * a.total_stride), x);
        cols.clear(x);
      }
      cols.param(a.post_weight, 0, a.param_f32, w);
      // without a post norm w and r1 are 1: dp then counts for nothing, and c1 is 0
#pragma unroll
      for (int i = 0; i < N; ++i) {
        x[i] = mul2(x[i], splat(r1));         // x1
        dg[i] = fma2(mul2(x[i], w[i]), z[i], dg[i]);
      }
      if (a.gate) {
        float2 g[N];
        cols.param(a.gate, group * a.dim, a.param_f32, g);
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = mul2(z[i], g[i]);
      }
      c = splat(0.0f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        z[i] = mul2(z[i], splat(a.scale));    // the gradient of y
        dp[i] = fma2(z[i], x[i], dp[i]);
        z[i] = mul2(z[i], w[i]);
        c = fma2(z[i], x[i], c);
      }
      if (a.post_weight) {
        const float c1 = cols.sum(c.x + c.y, red, turn) * inv_dim;
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = mul2(splat(r1), fma2(splat(-c1), x[i], z[i]));
      }
      for (int q = 0; q < a.outs; ++q) cols.template store<D>(a.grad_in[q], row * a.grad_in_stride, z);
    }
    // one unit per gate row: its gradient is whole; else a partial per unit
    if (a.grad_gate) {
#pragma unroll
      for (int i = 0; i < N; ++i) dg[i] = mul2(dg[i], splat(a.scale));
      cols.fold(dg);
      cols.template store<DF32>(d.parts == 1 ? a.grad_gate : a.work + 2 * d.ctas * a.dim, at.u * a.dim, dg);
    }
  }
  cols.fold(dw);
  cols.fold(dp);
  if (blockDim.y == 1) {
    if (a.grad_weight) cols.template store<DF32>(a.work, (int64_t)blockIdx.x * a.dim, dw);
    if (a.grad_post_weight) cols.template store<DF32>(a.work, (d.ctas + blockIdx.x) * a.dim, dp);
    return;
  }
  // a warp a row, or several: the warps' sums are added here, each warp's in its own ring
  static_assert(C::kDepth * C::kQ * C::kWarpBytes >= 2 * 32 * C::kEach * 4, "two binary32 rows");
  const int ring_floats = (int)(C::kDepth * ring.step / 4);
  float* shared = reinterpret_cast<float*>(g_ring);
  __syncwarp();
  cols.keep(shared + threadIdx.y * ring_floats, dw);
  cols.keep(shared + threadIdx.y * ring_floats + a.dim, dp);
  __syncthreads();
  for (int c = threadIdx.y * 32 + threadIdx.x; c < 2 * a.dim; c += 32 * blockDim.y) {
    const bool post = c >= a.dim;
    if (!(post ? a.grad_post_weight : a.grad_weight)) continue;
    float s = 0.0f;
    for (int y = 0; y < (int)blockDim.y; ++y) s += shared[y * ring_floats + c];
    st_g(a.work + (post ? d.ctas + blockIdx.x : (int64_t)blockIdx.x) * a.dim + (post ? c - a.dim : c), s);
  }
}

// How a row of `dim` columns is spread: threads, 16-byte vectors per thread,
// warps of rows per CTA, the kernel's most threads, and the rows that share a
// warp where all rows are aligned (Cols: PK).
struct Shape {
  int threads, groups, rows, most, packs;
};

inline Shape spread(int dim, int vec, int groups, int most) {
  const int vectors = (dim + vec - 1) / vec;
  Shape s;
  s.groups = groups;
  s.most = most;
  s.threads = ((vectors + groups - 1) / groups + 31) / 32 * 32;
  s.rows = s.threads == 32 ? kWarpRows : 1;
  s.packs = 1;
  while (s.packs < 32 && vectors * 2 * s.packs <= 32) s.packs *= 2;
  return s;
}

// With rows enough for every SM (`deep`) a thread takes up to sixteen columns,
// so that what a warp does once a row counts for more of them and several
// CTAs share an SM, one's sums over the block beside another's loads; a few
// rows are spread over as many threads as there are vectors.
inline int groups_for(int dim, int vec, bool deep) {
  int groups = 1;
  while (deep && vec * groups < 16 && dim >= 64 * vec * groups) groups *= 2;
  return groups;
}

inline Shape forward_shape(int dim, int vec, bool deep) {
  int groups = groups_for(dim, vec, deep);
  while (dim > vec * 1024 * groups) groups *= 2;
  return spread(dim, vec, groups, 1024);
}

// Backward keeps three sums per column in registers: sixteen columns fit into
// the 128 registers of 512 threads, eight into the 102 of 640.  Sixteen where
// an SM then holds two rows, or a row needs them; wider rows take 1024
// threads of 64 registers.
constexpr int backward_most(int each, bool wide) { return wide ? 1024 : each == 16 ? 512 : 640; }

inline Shape backward_shape(int dim, int vec, bool deep) {
  int groups = groups_for(dim, vec, deep);
  if (vec * groups == 16 && dim > 16 * 256) groups /= 2;
  while (vec * groups < 16 && dim > vec * groups * backward_most(vec * groups, false)) groups *= 2;
  return spread(dim, vec, groups, backward_most(vec * groups, dim > vec * groups * 512 && vec * groups == 16));
}

// CTAs that the SMs hold: 64 K registers each.
inline int64_t most_ctas(const Shape& s, int sms) {
  const int per_sm = s.most / (s.threads * s.rows);
  return (int64_t)sms * (per_sm < 1 ? 1 : per_sm > 16 ? 16 : per_sm);
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

// One launch, with the ring's shared memory.  The kernel is opted in to the
// most that its CTAs may ask for, once a handle, and never to less: the
// attribute is the kernel's, and calls of other widths may be on their way from
// other host threads.
template <class C, class... P, class... A>
cudaError_t launch_ring(void (*kernel)(P...), const Shape& s, int most, OptedIn& opted, unsigned grid, cudaStream_t st,
                        const A&... args) {
  constexpr size_t warp = (size_t)C::kDepth * C::kQ * C::kWarpBytes;
  const size_t bytes = warp * (s.threads / 32) * s.rows;
  if (bytes > 40 * 1024 && !opted.has((const void*)kernel)) {   // 48 KB, the static part included, need no opt-in
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(warp * (most / 32)));
    if (e != cudaSuccess) return e;
    opted.add((const void*)kernel);
  }
  return launch_after(kernel, dim3(grid), dim3(s.threads, s.rows), bytes, st, 1, args...);
}

template <class D, class RD>
cudaError_t run_forward(const Shape& s, bool aligned, const NormForward& a, OptedIn& opted, unsigned grid,
                        cudaStream_t st) {
  cudaError_t e = debug_upload(st);
  if (e != cudaSuccess) return e;
  return with_groups<D>(s.groups, [&](auto g) {
    constexpr int kGroups = decltype(g)::value;
    auto launch = [&](auto kernel, auto al) {   // (a packed row's slots are a vector a lane, too)
      return launch_ring<Cols<D, kGroups, decltype(al)::value != 0, 1024>>(kernel, s, 1024, opted, grid, st, a);
    };
    if constexpr (kGroups == 1)
      if (aligned && s.packs > 1) return launch(norm_forward_kernel<D, RD, 1, true, 1024, true>, IntC<1>{});
    if (aligned) return launch(norm_forward_kernel<D, RD, kGroups, true, 1024>, IntC<1>{});
    return launch(norm_forward_kernel<D, RD, kGroups, false, 1024>, IntC<0>{});
  });
}

template <class D, class RD>
cudaError_t run_backward(const Shape& s, bool aligned, const NormBackward& a, const Deal& d, OptedIn& opted,
                         unsigned grid, cudaStream_t st) {
  cudaError_t e = debug_upload(st);
  if (e != cudaSuccess) return e;
  return with_groups<D>(s.groups, [&](auto g) {
    constexpr int kGroups = decltype(g)::value;
    auto launch = [&](auto kernel, auto al, auto most) {
      constexpr int kMost = decltype(most)::value;
      return launch_ring<Cols<D, kGroups, decltype(al)::value != 0, kMost>>(kernel, s, kMost, opted, grid, st, a, d);
    };
    if constexpr (kGroups * D::kVec == 16) {
      if (s.most == 1024) {
        if (aligned) return launch(norm_backward_kernel<D, RD, kGroups, true, 1024>, IntC<1>{}, IntC<1024>{});
        return launch(norm_backward_kernel<D, RD, kGroups, false, 1024>, IntC<0>{}, IntC<1024>{});
      }
    }
    constexpr int kMost = backward_most(kGroups * D::kVec, false);
    if constexpr (kGroups == 1)
      if (aligned && s.packs > 1)
        return launch(norm_backward_kernel<D, RD, 1, true, kMost, true>, IntC<1>{}, IntC<kMost>{});
    if (aligned) return launch(norm_backward_kernel<D, RD, kGroups, true, kMost>, IntC<1>{}, IntC<kMost>{});
    return launch(norm_backward_kernel<D, RD, kGroups, false, kMost>, IntC<0>{}, IntC<kMost>{});
  });
}

}  // namespace norm
}  // namespace ra
