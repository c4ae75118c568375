// ra_ckpt.cu -- rows kept in 8 bits (ra_ckpt_store) and brought back
// (ra_ckpt_load), with the normalised rows of a kept residual stream.
//
// A half warp takes a group of 128 columns, a lane eight of them side by side:
// the group's largest magnitude is found by four shuffles, and every group is
// read and written once.  DRAM bounds it where rows start on 16-byte boundaries: 16384 x 8192 f32 kept in 101 us (0.98 of the
// copy bandwidth), brought back with bf16 normalised rows in 149 (0.93); 8192 x
// 5120 bf16 brought back in 21.6 (0.87).  Two groups a half warp in flight and
// 32 CTAs an SM over the kernel's time: more groups held more registers (eight: 119
// and 96 us for the 101 and, 16384 x 4096 bf16, 37), fewer CTAs left a tail (eight: 121, 60).
// Further off: f32 rows brought back without or with f32 normalised rows (131 and 258 us, 0.76 and 0.69: a lane's 32
// bytes go as two accesses, each of which fills half of its sectors), and rows off the 8-column grid, an element a
// lane (65536 x 2047 bf16 kept in 108 us, 0.56, brought back in 107, with normalised rows in 179).
#include "ra_ffn.cuh"

namespace ra {

namespace {

constexpr int kThreads = 256, kHalf = 16, kItems = 2;   // groups that a half warp has in flight
constexpr int kCtas = 32;                               // an SM, over the kernel's time

// How the rows lie: anywhere (a lane takes every 16th column of a group, an
// element at a time); on 16-byte boundaries and whole groups of 8 columns
// (eight columns a lane); and so one after the other, in whole groups of 128.
enum RowForm : int { kAnywhere = 0, kWide = 1, kFlat = 2 };

// Group `i` of all rows'; the row by a product instead of a quotient.
struct Place {
  int64_t row;
  int group;
  __device__ __forceinline__ Place(int64_t i, const CkptArgs& a, int groups) {
    if (i <= 0x7FFFFFFF) {
      const uint32_t n = (uint32_t)i, q = (__umulhi(n, a.by) + n) >> a.shift;
      row = q;
      group = (int)(n - q * (uint32_t)groups);
    } else {
      row = i / groups;
      group = (int)(i - row * groups);
    }
  }
};

// A lane's eight columns of group i: where they start, and how many there are.
template <int Form> struct Columns {
  int64_t row;
  int first, count;
  __device__ __forceinline__ Columns(int64_t i, const CkptArgs& a, int groups, int lane) {
    if constexpr (Form == kFlat) {
      row = 0;
      first = 0;
      count = 8;
    } else {
      const Place p(i, a, groups);
      row = p.row;
      first = p.group * kGroup + (Form == kWide ? lane * 8 : lane);
      const int left = a.dim - first;
      count = Form == kWide ? (left > 0 ? 8 : 0) : (left + kHalf - 1) / kHalf;
    }
  }
  template <class T> __device__ __forceinline__ T* at(T* p, int64_t stride, int64_t i, int lane) const {
    return Form == kFlat ? p + i * kGroup + lane * 8 : p + row * stride + first;
  }
};

// Eight columns as words: 16-bit ones in pairs, 32-bit ones each.
template <class D, int Form>
__device__ __forceinline__ void get8(const typename D::T* p, int count, uint32_t* w) {
  constexpr int kPer = D::kVec / 4;
  if constexpr (Form != kAnywhere) {
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int q = 0; q < 2 / kPer; ++q) {
      const uint4 x = count ? ld_stream(reinterpret_cast<const uint4*>(p) + q) : zero;
      w[4 * q] = x.x, w[4 * q + 1] = x.y, w[4 * q + 2] = x.z, w[4 * q + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8 / kPer; ++j) w[j] = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= count) continue;
      if constexpr (kPer == 2) w[j / 2] |= (uint32_t)ld_g(p + kHalf * j) << (16 * (j % 2));
      else w[j] = __float_as_uint(ld_g(p + kHalf * j));
    }
  }
}

template <class D, int Form>
__device__ __forceinline__ void put8(typename D::T* p, int count, const float2* v) {
  if constexpr (Form != kAnywhere) {
    if (!count) return;
    const float* x = reinterpret_cast<const float*>(v);
    uint4* to = reinterpret_cast<uint4*>(p);
    st_stream(to, pack<D>(x));
    if constexpr (D::kVec == 4) st_stream(to + 1, pack<D>(x + 4));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < count) st_g(p + kHalf * j, narrow<D>(j % 2 ? v[j / 2].y : v[j / 2].x));
  }
}

// Columns 2 j and 2 j + 1.
template <class D> __device__ __forceinline__ float2 pair_of(const uint32_t* w, int j) {
  float2 v;
  if constexpr (D::kVec == 8) unpack2<D>(w[j], reinterpret_cast<float*>(&v));
  else v = make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
  return v;
}

template <class D, int Form>
__global__ void __launch_bounds__(kThreads) ckpt_store_kernel(const CkptArgs a) {
  using T = typename D::T;
  constexpr int kWords = 32 / D::kVec;   // of eight columns
  after_predecessor();
  const int lane = threadIdx.x % kHalf, groups = (a.dim + kGroup - 1) / kGroup;
  const int64_t total = a.rows * groups, step = (int64_t)gridDim.x * (kThreads / kHalf);
  const int64_t whole = (total + step - 1) / step * step;   // a warp's halves stay together for the shuffles
  for (int64_t i0 = blockIdx.x * (int64_t)(kThreads / kHalf) + threadIdx.x / kHalf; i0 < whole; i0 += kItems * step) {
    uint32_t w[kItems][kWords];
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      const int64_t i = i0 + u * step;
#pragma unroll
      for (int j = 0; j < kWords; ++j) w[u][j] = 0u;
      if (i < total) {
        const Columns<Form> c(i, a, groups, lane);
        get8<D, Form>(c.at((const T*)a.values, a.stride, i, lane), c.count, w[u]);
      }
    }
    // magnitudes order as their bits do, NaN last, 16-bit ones two at a time;
    // a lane's quotients are those of one of the groups in flight
    uint32_t mine = 0;
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      uint32_t most = 0;
#pragma unroll
      for (int j = 0; j < kWords; ++j)
        most = D::kVec == 8 ? __vmaxu2(most, w[u][j] & 0x7FFF7FFFu) : max(most, w[u][j] & 0x7FFFFFFFu);
#pragma unroll
      for (int s = kHalf / 2; s > 0; s >>= 1) {
        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, most, s);
        most = D::kVec == 8 ? __vmaxu2(most, other) : max(most, other);
      }
      if (D::kVec == 8) most = max(most & 0xFFFFu, most >> 16);
      if (lane == u) mine = most;
    }
    float scale, own;
    if constexpr (D::kVec == 8) group_scale(widen<D>((uint16_t)mine), &scale, &own);
    else group_scale(__uint_as_float(mine), &scale, &own);
    if (lane < kItems && i0 + lane * step < total) st_g(a.scales + i0 + lane * step, scale);
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      const int64_t i = i0 + u * step;
      const float by = __shfl_sync(0xFFFFFFFFu, own, u, kHalf);
      if (i >= total) continue;
      const Columns<Form> c(i, a, groups, lane);
      int8_t* const to = c.at(a.codes, a.codes_stride, i, lane);
      uint32_t q[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 x = code_sum(pair_of<D>(w[u], 2 * k), by), y = code_sum(pair_of<D>(w[u], 2 * k + 1), by);
        q[k] = codes4(x, y);
      }
      if constexpr (Form != kAnywhere) {
        if (c.count) st_g(reinterpret_cast<uint2*>(to), make_uint2(q[0], q[1]));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < c.count) st_g(to + kHalf * j, (int8_t)(q[j / 4] >> (8 * (j % 4))));
      }
    }
  }
}

template <class D, class N, class P, int Form>
__global__ void __launch_bounds__(kThreads) ckpt_load_kernel(const CkptArgs a) {
  using T = typename D::T;
  using TN = typename N::T;
  using TP = typename P::T;
  after_predecessor();
  const int lane = threadIdx.x % kHalf, groups = (a.dim + kGroup - 1) / kGroup;
  const int64_t total = a.rows * groups, step = (int64_t)gridDim.x * (kThreads / kHalf);
  for (int64_t i0 = blockIdx.x * (int64_t)(kThreads / kHalf) + threadIdx.x / kHalf; i0 < total; i0 += kItems * step) {
    uint2 q[kItems];
    float scale[kItems];
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      const int64_t i = i0 + u * step;
      q[u] = make_uint2(0u, 0u);
      scale[u] = 0.0f;
      if (i >= total) continue;
      const Columns<Form> c(i, a, groups, lane);
      const int8_t* const from = c.at((const int8_t*)a.codes, a.codes_stride, i, lane);
      if constexpr (Form != kAnywhere) {
        if (c.count) q[u] = ld_g(reinterpret_cast<const uint2*>(from));
      } else {
        uint32_t w[2] = {};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < c.count) w[j / 4] |= (uint32_t)(uint8_t)ld_g(from + kHalf * j) << (8 * (j % 4));
        q[u] = make_uint2(w[0], w[1]);
      }
      scale[u] = ld_g(a.scales + i);
    }
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      const int64_t i = i0 + u * step;
      if (i >= total) continue;
      const Columns<Form> c(i, a, groups, lane);
      const uint32_t lo = bias_codes(q[u].x), hi = bias_codes(q[u].y);
      float2 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __fmul2_rn(code_pair(j < 2 ? lo : hi, 2 * (j % 2)), both(scale[u]));
      if (a.values) put8<D, Form>(c.at((T*)a.values, a.stride, i, lane), c.count, v);
      if (!a.normed) continue;
      const Place p(i, a, groups);
      const float rstd = ld_g(a.rstd + p.row);
      const int first = p.group * kGroup + (Form == kAnywhere ? lane : lane * 8);
      const TP* const from = (const TP*)a.weight + first;
      uint32_t w[32 / P::kVec] = {};
      if constexpr (Form != kAnywhere) {
        if (c.count) {
#pragma unroll
          for (int k = 0; k < 8 / P::kVec; ++k) {
            const uint4 x = ld_plain(reinterpret_cast<const uint4*>(from) + k);
            w[4 * k] = x.x, w[4 * k + 1] = x.y, w[4 * k + 2] = x.z, w[4 * k + 3] = x.w;
          }
        }
      } else {
        get8<P, kAnywhere>(from, c.count, w);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __fmul2_rn(__fmul2_rn(v[j], both(rstd)), pair_of<P>(w, j));
      put8<N, Form>(c.at((TN*)a.normed, a.normed_stride, i, lane), c.count, v);
    }
  }
}

int ctas(const CkptArgs& a, int sms) {
  const int64_t groups = (a.dim + kGroup - 1) / kGroup;
  const int64_t need = (a.rows * groups + kThreads / kHalf - 1) / (kThreads / kHalf);
  return (int)(need < kCtas * sms ? need : kCtas * sms);
}

template <class F> cudaError_t with_float(int dtype, F&& f) {
  return dtype == RA_F32 ? f(DF32{}) : dtype == RA_BF16 ? f(DBF16{}) : f(DF16{});
}
template <class F> cudaError_t with_form(bool wide, bool flat, F&& f) {
  return flat ? f(IntC<kFlat>{}) : wide ? f(IntC<kWide>{}) : f(IntC<kAnywhere>{});
}

}  // namespace

cudaError_t launch_ckpt_store(int dtype, bool wide, const CkptArgs& a, int sms, cudaStream_t st) {
  const cudaError_t e = debug_upload(st);
  if (e != cudaSuccess) return e;
  const bool flat = wide && a.dim % kGroup == 0 && a.stride == a.dim && a.codes_stride == a.dim;
  return with_float(dtype, [&](auto d) {
    return with_form(wide, flat, [&](auto form) {
      return launch_after(ckpt_store_kernel<decltype(d), decltype(form)::value>, dim3(ctas(a, sms)), dim3(kThreads), 0, st,
                          1, a);
    });
  });
}

cudaError_t launch_ckpt_load(int dtype, int normed_dtype, int param_dtype, bool wide, const CkptArgs& a, int sms,
                             cudaStream_t st) {
  const cudaError_t e = debug_upload(st);
  if (e != cudaSuccess) return e;
  const bool flat = wide && a.dim % kGroup == 0 && a.codes_stride == a.dim && (!a.values || a.stride == a.dim) &&
                    (!a.normed || a.normed_stride == a.dim);
  return with_float(dtype, [&](auto d) {
    return with_float(normed_dtype, [&](auto n) {
      return with_form(wide, flat, [&](auto form) {
        using D = decltype(d);
        using N = decltype(n);
        const auto kernel = param_dtype == RA_F32 ? ckpt_load_kernel<D, N, DF32, decltype(form)::value>
                                                  : ckpt_load_kernel<D, N, N, decltype(form)::value>;
        return launch_after(kernel, dim3(ctas(a, sms)), dim3(kThreads), 0, st, 1, a);
      });
    });
  });
}

}  // namespace ra
