// ra_ffn.cuh -- device pieces of the feed-forward block and of rows kept in 8
// bits: activations with their derivatives, and the codes.
#pragma once

#include "ra_ffn.h"
#include "ra_ops.cuh"

namespace ra {

// The activation act(a) and, with Slope, its derivative: sigmoid-weighted
// (act = a p, act' = p + a p (1 - p), p = 1 / (1 + e^-a)) or by the normal
// distribution (act = a P(a), act' = P(a) + a e^(-a^2/2) / sqrt(2 pi)).  P
// comes from normcdff, which keeps its relative accuracy where 1 + erf cancels.
template <int Act, bool Slope> __device__ __forceinline__ void activate(float a, float* act, float* slope) {
  if constexpr (Act == RA_SILU) {
    const float p = __fdividef(1.0f, __fadd_rn(1.0f, exp2_fast(-1.4426950408889634f * a)));
    *act = a * p;
    if constexpr (Slope) *slope = __fmaf_rn(*act, 1.0f - p, p);
  } else {
    const float p = normcdff(a);
    *act = a * p;
    if constexpr (Slope) *slope = __fmaf_rn(a * 0.3989422804014327f, exp2_fast(-0.7213475204444817f * a * a), p);
  }
}

// Groups with nothing above this are kept as zeros: 127 / m stays finite.
constexpr float kKeepLowest = 7.703719777548943e-34f;   // 2^-110

// A group's scale and the factor to its codes, from its largest magnitude (NaN
// where a value is NaN).  Infinite and NaN groups come back as NaN.
__device__ __forceinline__ void group_scale(float most, float* scale, float* by) {
  if (!(most <= FLT_MAX)) {
    *scale = __uint_as_float(0x7FC00000u);
    *by = 0.0f;
  } else if (most > kKeepLowest) {
    *scale = __fdiv_rn(most, 127.0f);
    *by = __fdiv_rn(127.0f, most);
  } else {
    *scale = *by = 0.0f;
  }
}

// v * by to the nearest whole number: adding 1.5 * 2^23 leaves it, to even, in
// the low bits (|v * by| < 128).  0 * infinity, NaN, leaves whatever: the scale is NaN then.
__device__ __forceinline__ uint32_t code_bits(float v, float by) {
  return __float_as_uint(__fadd_rn(__fmul_rn(v, by), 12582912.0f)) & 0xFFu;
}
__device__ __forceinline__ int8_t code_of(float v, float by) { return (int8_t)code_bits(v, by); }

__device__ __forceinline__ uint32_t codes4(const float* v, float by) {
  return __byte_perm(__byte_perm(code_bits(v[0], by), code_bits(v[1], by), 0x0040),
                     __byte_perm(code_bits(v[2], by), code_bits(v[3], by), 0x0040), 0x5410);
}

// Code k of four in a word, as a number: the biased byte as the low bits of 2^23 + ...
__device__ __forceinline__ float code_value(uint32_t biased, int k) {
  return __uint_as_float(__byte_perm(biased, 0x4B000000u, 0x7440u + (uint32_t)k)) - 8388736.0f;
}
// ... of the word with every byte's sign bit turned over
__device__ __forceinline__ uint32_t bias_codes(uint32_t w) { return w ^ 0x80808080u; }

}  // namespace ra
