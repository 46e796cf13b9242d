// What the products with 4-bit weights share: matrix instructions, the exact forms in which 4-bit
// weights meet f16 rows, and the ends of the epilogue.
#pragma once

#include "expert_act.h"
#include "mx4.h"

namespace moe {

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
constexpr uint32_t kMx4F16Reach = 36u;
__device__ __forceinline__ uint32_t mx4_f16_reach(uint32_t E) { return E - 104u; }
__device__ __forceinline__ bool mx4_fits_f16(uint32_t E) { return mx4_f16_reach(E) <= kMx4F16Reach; }
// Zeros are f16 values under any scale (the quantiser gives a block of them 0; under 255 they are widened to
// NaN, which f16 holds too). The scales alone are looked at first: codes matter only where they do not fit.
__device__ __forceinline__ bool mx4_zeros(const chunk_t& codes) { return ((codes.x | codes.y | codes.z | codes.w) & 0x77777777u) == 0u; }

// Whether blocks `first` .. + count - 1 hold values that f16 does not.
__device__ __forceinline__ bool mx4_misfits_f16(const chunk_t* codes, const uint8_t* scales, size_t first, int count) {
  typedef uint64_t __attribute__((aligned(1), may_alias)) bytes8_t;
  bool bad = false;
  for (int at = 0; at < count; at += 32) {
    uint64_t E[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      E[i] = 0x7f7f7f7f7f7f7f7full;
      if (at + 8 * i + 8 <= count) {
        E[i] = *reinterpret_cast<const bytes8_t*>(scales + first + at + 8 * i);
      } else {
        for (int b = 0; at + 8 * i + b < count; ++b)
          E[i] = (E[i] & ~(255ull << (8 * b))) | static_cast<uint64_t>(scales[first + at + 8 * i + b]) << (8 * b);
      }
    }
#pragma unroll
    for (int b = 0; b < 32; ++b)
      if (!mx4_fits_f16(static_cast<uint32_t>(E[b / 8] >> (8 * (b % 8))) & 255u)) bad = bad || !mx4_zeros(codes[first + at + b]);
  }
  return bad;
}

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

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// A block of 4-bit codes per lane on each side, lane l's of row l % 16 and K block l / 16, with the
// scales in byte SA of sa and byte SB of sb.
template <int SA = 0, int SB = 0>
__device__ __forceinline__ f32x4_t mfma_mx4(const chunk_t& a, uint32_t sa, const chunk_t& b, uint32_t sb, f32x4_t c) {
  const i32x8_t va = {static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w), 0, 0, 0, 0};
  const i32x8_t vb = {static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z), static_cast<int>(b.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, c, 4, 4, SA, static_cast<int>(sa), SB, static_cast<int>(sb));
}

// The route weight of buffer row r (token t): that of the route placed there. The token's routes are
// read eight at a time, all their loads in flight together: one after another they would hold a
// workgroup up at its start or end (24 tokens of 64 experts, weighted: 38.0 us, not 36.3).
__device__ __forceinline__ float route_weight_wide(const ExpertAct& p, int r, int t) {
  float w = 1.0f;
  if (p.route_w == nullptr) return w;
  const size_t first = static_cast<size_t>(t) * p.k;
  for (int j0 = 0; j0 < p.k; j0 += 8) {
    int d[8];
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const size_t at = first + (j0 + j < p.k ? j0 + j : p.k - 1);
      d[j] = p.dst[at];
      v[j] = p.route_w[at];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) w = d[j] == r ? v[j] : w;  // the last one twice at worst
  }
  return w;
}

// Eight output features, finished and stored: rounded to 16 bits, or to 4 with the block's other
// 24 in the lane's group of four (lanes 4 i .. 4 i + 3 hold features c - c % 32 .. + 31 of a row).
template <int DT>
__device__ __forceinline__ void finish8_mx4(const Mx4Act& p, int x, int r, int t, float w, int c, float (&v)[8],
                                            float (&u)[8]) {
  epilogue8<DT>(p, x, r, t, w, c, v, u);
  const size_t at = static_cast<size_t>(r) * p.n + c;
  if (p.out_scales != nullptr) {
    uint32_t E;
    static_cast<uint32_t*>(p.out)[at / 8] = mx4_quantize8(v, &E);
    if (c % 32 == 0) p.out_scales[at / 32] = static_cast<uint8_t>(E);
  } else {
    *reinterpret_cast<chunk_t*>(static_cast<uint16_t*>(p.out) + at) = pack<DT>(v);
  }
}

__device__ __forceinline__ void zero_unfilled_mx4(const Mx4Act& p, int b, int nb) {
  if (p.out_scales == nullptr) {
    zero_unfilled(p, b, nb);
    return;
  }
  each_unfilled(p, b, nb, [&](int r) {
    const int blocks = p.n / kMx4Block;
    chunk_t* o = static_cast<chunk_t*>(p.out) + static_cast<size_t>(r) * blocks;
    uint8_t* s = p.out_scales + static_cast<size_t>(r) * blocks;
    for (int c = lane_id(); c < blocks; c += kWave) {
      o[c] = chunk_t{0u, 0u, 0u, 0u};
      s[c] = 0;
    }
    clear_preact(p, r);
  });
}

}  // namespace moe
