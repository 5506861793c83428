// MXFP4 on gfx950: groups of 32 consecutive inputs of a row hold 4-bit floats (sign,
// two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) under one power
// of two, 2^(byte - 127); byte 255 makes the whole group NaN.  Two codes a byte, the
// even input low.
#pragma once

#include <stdint.h>

#include "wq_device.hpp"

namespace wq {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kMxGroup = 32;
// Weights of one call: the quantiser and its inverse take a thread for 32, and a grid's axis
// holds less than 2^32 threads.
constexpr int64_t kMxMost = ((int64_t)1 << 37) - (1 << 13);

// 16 bytes of codes as the matrix instructions' operand, whose other half they do not read.
typedef int i32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i32x8 mx_operand(u32x4 v) {
  const i32x4 q = __builtin_bit_cast(i32x4, v);
  return __builtin_shufflevector(q, q, 0, 1, 2, 3, -1, -1, -1, -1);
}

// A constant index for a generic lambda.
template <int V>
struct At {
  static constexpr int value = V;
};

// Scale byte `j` of a word, as the fp32 operand of the conversions below.  They look
// at its exponent field only, so byte 0 stands for 2^-127 and 255 for NaN.
__device__ __forceinline__ float mx_scale(uint32_t word, int j) {
  return __uint_as_float(((word >> (8 * j)) & 0xFFu) << 23);
}

// The eight codes of a word times the scale as bf16, in order: exact where the result
// is one (scale bytes up to 252; beyond, products past the largest bf16 are infinite).
__device__ __forceinline__ bf16x8 mx_bf16(uint32_t w, float scale) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  const u4 r = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3))};
  return __builtin_bit_cast(bf16x8, r);
}

// The scale byte of a group whose largest absolute value has the fp32 bits `top`:
// 2^(floor(log2) - 2), so that the largest code's range covers it (values in
// (6, 8) scales saturate at 6), not below 2^-127; infinities and NaN give 255.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
  const uint32_t e = top >> 23;
  return e == 255u ? 255u : e < 2u ? 0u : e - 2u;
}

// Eight values in codes, each the nearest (ties to the even code, saturating at 6);
// zeros where the group is NaN.
__device__ __forceinline__ uint32_t mx_codes(const float (&v)[8], uint32_t byte) {
  // byte 0: the conversion takes the exponent field of a subnormal, 2^-127
  const float scale = __uint_as_float(byte ? byte << 23 : 0x00400000u);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], scale, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], scale, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], scale, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], scale, 3);
  return byte == 255u ? 0u : r;
}

// Largest of four lanes' values (bits of non-negative floats compare as they do).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false);
  v = v > o ? v : o;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false);
  return v > o ? v : o;
}

}  // namespace wq
