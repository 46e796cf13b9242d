// What the products with 4-bit weights share: 16-bit matrix instructions and the exact forms in
// which 4-bit weights meet f16 rows.
#pragma once

#include "gemm_common.h"
#include "mx4.h"

namespace moe {

typedef float f32x4_t __attribute__((ext_vector_type(4)));

template <int DT>
__device__ __forceinline__ f32x4_t mfma_16x16x32(const chunk_t& a, const chunk_t& b, f32x4_t c) {
  if constexpr (DT == kBF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                    0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c,
                                                   0, 0, 0);
}

// Whether every value of a block with scale byte E is an f16 value: 0.5 2^(E - 127) is a multiple
// of f16's smallest, 2^-24, and 6 2^(E - 127) is within its range.
__device__ __forceinline__ bool mx4_fits_f16(uint32_t E) { return E - 104u <= 36u; }

// Eight f16 values as the sums of two bf16 values each: the upper 8 of the 11 significant bits, and
// the other 3. An infinity or NaN is all in the first.
__device__ __forceinline__ void split_f16(const chunk_t& a, chunk_t& hi, chunk_t& lo) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h[2], l[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float f = f16_bits_to_f32(q ? a[i] >> 16 : a[i] & 0xffffu);
      h[q] = __float_as_uint(f) & 0xffff0000u;
      l[q] = (h[q] & 0x7f800000u) == 0x7f800000u ? 0u : __float_as_uint(f - __uint_as_float(h[q]));
    }
    hi[i] = (h[0] >> 16) | h[1];
    lo[i] = (l[0] >> 16) | (l[1] & 0xffff0000u);
  }
}

}  // namespace moe
