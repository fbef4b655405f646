// MX (microscaling) encoding shared by the MX quantizer and the gate+up
// epilogues that quantize H or Y1: the E8M0 shared exponent of a block and the
// encodings of its elements.  The rule (the published microscaling one;
// the pages do not define MX): for a block with amax a > 0 the shared scale
// is X = 2^(floor(log2 a) - emax) (emax = 8 for E4M3, 2 for E2M1), clamped
// to 2^[-127, 127], and 2^-127 for an all-zero block; every element is V / X
// rounded to nearest even, saturated to 448 (E4M3).
#pragma once

#include "common.hpp"

namespace nvfp4moe {

typedef __attribute__((ext_vector_type(2))) short s16x2_t;

// Unbiased shared exponent of a block with amax a: floor(log2 a) - emax,
// clamped to [-127, 127]; -127 when a == 0 (also when a is an fp32
// subnormal, whose exponent is below -126: the clamp gives -127 there).
template <int EMAX>
__device__ __forceinline__ int shared_exp(float a) {
  if (!(a > 0.0f)) return -127;
  const int e = __builtin_amdgcn_frexp_expf(a) - 1 - EMAX;  // a = m * 2^(e+1), m in [0.5, 1)
  return e < -127 ? -127 : e > 127 ? 127 : e;
}

// 4 fp32 values to E4M3 codes (one word, element i in byte i): scaled by
// 2^-se (exact), clamped to +-448 (the format saturates; the converter would
// otherwise overflow), then rounded to nearest even by the hardware
// converter with a unit scale.
__device__ __forceinline__ uint32_t encode4_e4m3(const float* v, int se) {
  float r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float s = __builtin_ldexpf(v[i], -se);
    r[i] = __builtin_copysignf(fminf(fabsf(s), 448.0f), s);
  }
  s16x2_t p = {0, 0};
  p = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(p, r[0], r[1], 1.0f, false);
  p = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(p, r[2], r[3], 1.0f, true);
  return __builtin_bit_cast(uint32_t, p);
}

// 8 fp32 values to E2M1 codes (one word, element 2j in the low nibble of pair
// j): scaled by 2^-se (exact), rounded to nearest even and saturated to 6 by
// the hardware converter with a unit scale, sign kept.
__device__ __forceinline__ uint32_t encode8_e2m1(const float* v, int se) {
  uint32_t w = 0u;
#define MXQ_PAIR(I, SEL)                                                                              \
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __builtin_ldexpf(v[I], -se),                         \
                                               __builtin_ldexpf(v[(I) + 1], -se), 1.0f, SEL)
  MXQ_PAIR(0, 0);
  MXQ_PAIR(2, 1);
  MXQ_PAIR(4, 2);
  MXQ_PAIR(6, 3);
#undef MXQ_PAIR
  return w;
}

// MXINT8, the form of activations kept for the backward pass: a block of 32
// shares S, an element is a whole number q in [-127, 127] and stands for
// q * 2^(S - 133).  With the block's amax a, S is the exponent field of a
// (2^(S-127) <= a < 2^(S-126); 0 for a subnormal or zero a), so that a / step is
// in [64, 128): rounding is off by half a step, 2^-7 of a, and by less than a
// step where it would give 128.  S = 255 (a block that holds an infinity or a
// NaN) reads back as NaN, so a gradient shows what the forward pass met.

// S of a block from the greatest of its elements' bits without their signs.
__device__ __forceinline__ int int8_scale(uint32_t amax_bits) { return (int)(amax_bits >> 23); }

// The greater of two bf16 pairs' bits without their signs, half by half.
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t m, uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, m),
                                                                __builtin_bit_cast(u16x2_t, w & 0x7FFF7FFFu)));
}
// The greatest of a pair as fp32 bits.
__device__ __forceinline__ uint32_t max_of_pair(uint32_t m) { return max(m << 16, m & 0xFFFF0000u); }

// Codes of a block with S, four elements at a time (element i in byte i).
// v * 2^(133 - S) is exact or far below a half, so adding 1.5 * 2^23 in the same
// step rounds to nearest even and leaves the whole number's low byte in the
// sum's.  Blocks below 2^-120, whose power is no fp32 number, take another way.
struct Int8Encoder {
  float scale;
  int exponent;
  bool tiny;
};
__device__ __forceinline__ Int8Encoder int8_encoder(uint32_t amax_bits) {
  const int s = int8_scale(amax_bits);
  return {__uint_as_float((uint32_t)(260 - s) << 23), 133 - s, s < 7 && amax_bits != 0};  // (zeros: any scale)
}
template <bool TINY>
__device__ __forceinline__ uint32_t encode4_int8(const float* v, const Int8Encoder& e) {
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float n = TINY ? __builtin_ldexpf(v[i], e.exponent) + 12582912.0f : __builtin_fmaf(v[i], e.scale, 12582912.0f);
    b[i] = __float_as_uint(__builtin_amdgcn_fmed3f(n, 12582912.0f - 127.0f, 12582912.0f + 127.0f));
  }
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400u), __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u),
                               0x05040100u);
}
// Whether any lane's block needs the other way (the same answer in every lane).
__device__ __forceinline__ bool any_tiny(const Int8Encoder& e) { return __any(e.tiny); }

// What a block's codes are multiplied with: 2^(S - 133), or NaN.
__device__ __forceinline__ float int8_step(int s) { return s == 255 ? __builtin_nanf("") : __builtin_ldexpf(1.0f, s - 133); }
__device__ __forceinline__ float decode_int8(int q, float step) { return (float)q * step; }

}  // namespace nvfp4moe
