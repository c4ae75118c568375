// ra_ffn.cuh -- device pieces of the feed-forward block and of rows kept in 8
// bits: activations with their derivatives, and the codes.
#pragma once

#include "ra_ffn.h"
#include "ra_ops.cuh"

namespace ra {

// The activation act(a) and, with Slope, its derivative: sigmoid-weighted
// (act = a p, act' = p + a p (1 - p), p = 1 / (1 + e^-a)) or by the normal
// distribution (act = a P(a), act' = P(a) + a e^(-a^2/2) / sqrt(2 pi)).
//
// P(-z) = e^(-z^2/2) R(z), z >= 0, where R falls smoothly from 1/2: a
// polynomial of degree 8 in t = 1 / (1 + 0.23 z), fitted to R's values at
// Chebyshev points by reweighted least squares until its largest relative
// error stood still: 6.2e-8 up to z = 13.3, beyond which e^(-z^2/2) is below
// binary32's normal numbers (8.0e-8 with binary32's 0.23); 7 units of 2^-24
// evaluated in binary32.  Nothing cancels, as it does in 1 + erf; but the
// exponent is rounded twice, so that P is off by up to 7 + 1.2 z^2 units of 2^-24
// (23 by z = 5, 45 by z = 8): less than a hundredth of the 16-bit outputs' own
// rounding.  Twenty instructions with the derivative, which takes the same
// exponential.
//
// Arithmetic is on pairs, two binary32 operations an instruction.
__device__ __forceinline__ float reciprocal(float x) {   // 0 from 2^126 on
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

template <int Act, bool Slope> __device__ __forceinline__ void activate(float2 a, float2* act, float2* slope) {
  if constexpr (Act == RA_SILU) {
    const float2 x = __fmul2_rn(a, both(-1.4426950408889634f));
    const float2 y = __fadd2_rn(make_float2(exp2_fast(x.x), exp2_fast(x.y)), both(1.0f));
    const float2 p = make_float2(reciprocal(y.x), reciprocal(y.y));
    *act = __fmul2_rn(a, p);
    if constexpr (Slope) *slope = __ffma2_rn(*act, __ffma2_rn(p, both(-1.0f), both(1.0f)), p);
  } else {
    const float2 d = __ffma2_rn(make_float2(fabsf(a.x), fabsf(a.y)), both(0.23f), both(1.0f));
    const float2 t = make_float2(reciprocal(d.x), reciprocal(d.y));
    const float2 x = __fmul2_rn(__fmul2_rn(a, a), both(-0.7213475204444817f));
    const float2 e = make_float2(exp2_fast(x.x), exp2_fast(x.y));
    float2 R = both(-0.07840986549854279f);
    R = __ffma2_rn(R, t, both(0.2901213765144348f));
    R = __ffma2_rn(R, t, both(-0.2774907052516937f));
    R = __ffma2_rn(R, t, both(0.3007018566131592f));
    R = __ffma2_rn(R, t, both(-0.032351523637771606f));
    R = __ffma2_rn(R, t, both(0.1192530021071434f));
    R = __ffma2_rn(R, t, both(0.08583563566207886f));
    R = __ffma2_rn(R, t, both(0.09236723184585571f));
    R = __ffma2_rn(R, t, both(-2.7028399927075952e-05f));
    const float2 q = __fmul2_rn(e, R), u = __ffma2_rn(q, both(-1.0f), both(1.0f));
    const float2 p = make_float2(a.x > 0.0f ? u.x : q.x, a.y > 0.0f ? u.y : q.y);
    *act = __fmul2_rn(a, p);
    if constexpr (Slope) *slope = __ffma2_rn(__fmul2_rn(a, both(0.3989422804014327f)), e, p);
  }
}

// Groups with nothing above this are kept as zeros: 127 / m stays finite.
constexpr float kKeepLowest = 7.703719777548943e-34f;   // 2^-110

// The largest scale whose 127th multiple is a number: that of binary32's largest
// number would be rounded up to 8454660 * 2^98, and 127 of those are infinite.
constexpr float kMostScale = 0x1.020406p+121f;   // 8454659 * 2^98

// A group's scale and the factor to its codes, from its largest magnitude (NaN
// where a value is NaN).  Infinite and NaN groups come back as NaN.
__device__ __forceinline__ void group_scale(float most, float* scale, float* by) {
  if (!(most <= FLT_MAX)) {
    *scale = __uint_as_float(0x7FC00000u);
    *by = 0.0f;
  } else if (most > kKeepLowest) {
    *scale = fminf(__fdiv_rn(most, 127.0f), kMostScale);
    *by = __fdiv_rn(127.0f, most);
  } else {
    *scale = *by = 0.0f;
  }
}

// v * by to the nearest whole number: adding 1.5 * 2^23 leaves it, to even, in
// the low bits (|v * by| < 128).  0 * infinity, NaN, leaves whatever: the scale is NaN then.
// (Products one by one: of two at a time the compiler makes one operation with
// the sums, and a product that is not rounded before goes the other way at a half.)
__device__ __forceinline__ float2 code_sum(float2 v, float by) {
  return __fadd2_rn(make_float2(__fmul_rn(v.x, by), __fmul_rn(v.y, by)), both(12582912.0f));
}
__device__ __forceinline__ int8_t code_of(float v, float by) {
  return (int8_t)(__float_as_uint(__fadd_rn(__fmul_rn(v, by), 12582912.0f)) & 0xFFu);
}
// Four of them as a word.
__device__ __forceinline__ uint32_t codes4(float2 x, float2 y) {
  return __byte_perm(__byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x0040),
                     __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x0040), 0x5410);
}
__device__ __forceinline__ uint32_t codes4(const float* v, float by) {
  return codes4(code_sum(make_float2(v[0], v[1]), by), code_sum(make_float2(v[2], v[3]), by));
}

// Code k of four in a word, as a number: the biased byte as the low bits of 2^23 + ...
__device__ __forceinline__ float code_raised(uint32_t biased, int k) {
  return __uint_as_float(__byte_perm(biased, 0x4B000000u, 0x7440u + (uint32_t)k));
}
// codes k and k + 1
__device__ __forceinline__ float2 code_pair(uint32_t biased, int k) {
  return __fadd2_rn(make_float2(code_raised(biased, k), code_raised(biased, k + 1)), both(-8388736.0f));
}
// ... of the word with every byte's sign bit turned over
__device__ __forceinline__ uint32_t bias_codes(uint32_t w) { return w ^ 0x80808080u; }

}  // namespace ra
