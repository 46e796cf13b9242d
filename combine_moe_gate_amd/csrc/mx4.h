// Microscaled 4-bit floating point on gfx950.
//
// A row is cut into blocks of 32 values. A block has a scale byte E, which stands for 2^(E - 127)
// (255: not a number), and each value four bits, a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6
// (two exponent bits, one mantissa bit): it stands for their product. Two values to a byte, the
// first in the low half. A block of 16 code bytes is what one lane of a 4-bit matrix instruction
// takes, with the block's scale.
//
// Quantising: E = floor(log2 top) - 2 + 127 for the block's largest magnitude `top`, at least 0,
// which is top's exponent field less 2; values divided by the scale (exact) and rounded to the
// nearest of the eight, half-way cases to the even code, past 6 to 6. A block that holds an
// infinity or a NaN gets E = 255 and codes 0: it reads back as NaN. A block of zeros gets E = 0.
#pragma once

#include "moe_device.h"

namespace moe {

typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kMx4 = 3;       // beside the element types: rows of 4-bit values
constexpr int kMx4Block = 32;

// The scale as the conversion instructions take it: 2^(E - 127) in float32 (a subnormal for
// E = 0); E = 255 gives an infinity's bits, which they read as "not a number".
__device__ __forceinline__ float mx4_scale(uint32_t E) { return __uint_as_float(E != 0u ? E << 23 : 0x00400000u); }

// A block's scale byte, from the bits of its largest magnitude.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t top) {
  const uint32_t field = top >> 23;
  return field == 255u ? 255u : field > 2u ? field - 2u : 0u;
}

// Eight values' codes (0 in a block with E = 255), the first in the low half of the low byte.
__device__ __forceinline__ uint32_t mx4_codes8(const float (&v)[8], uint32_t E) {
  const float s = mx4_scale(E);
  uint32_t c = 0u;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
  return E == 255u ? 0u : c;
}

// Eight values of a block whose 32 lie in four neighbouring lanes (lane % 4 = 0..3, all active):
// their codes, and the block's scale byte in every lane.
__device__ __forceinline__ uint32_t mx4_quantize8(const float (&v)[8], uint32_t* E) {
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;  // as whole numbers NaN > inf > finite
    top = b > top ? b : top;
  }
  uint32_t other = __builtin_amdgcn_update_dpp(0, static_cast<int>(top), 0xb1, 0xf, 0xf, false);  // quad_perm [1,0,3,2]
  top = other > top ? other : top;
  other = __builtin_amdgcn_update_dpp(0, static_cast<int>(top), 0x4e, 0xf, 0xf, false);           // quad_perm [2,3,0,1]
  top = other > top ? other : top;
  *E = mx4_scale_byte(top);
  return mx4_codes8(v, *E);
}

// Eight codes as eight values of a 16-bit element type: bf16 holds every value of a scale up to 2^125;
// f16 those of scales from 2^-23 to 2^13, others are rounded to nearest, past its range to infinity.
template <int DT>
__device__ __forceinline__ chunk_t mx4_values8(uint32_t codes, float scale) {
  chunk_t o;
  if constexpr (DT == kBF16) {
    o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
    o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
    o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
    o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
  } else {
    o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 0));
    o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 1));
    o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 2));
    o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 3));
  }
  return o;
}

}  // namespace moe
