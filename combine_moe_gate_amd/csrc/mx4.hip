// Rows to microscaled 4-bit values and back, on gfx950 (the format stands in mx4.h).
//
// Rows are whole blocks, so a tensor is one flat run of blocks. A lane takes eight values (16 bytes
// of a 16-bit type), four neighbouring lanes a block: the block's largest magnitude meets over two
// DPP moves, and loads and stores are whole lines of the wave. Bound by memory: 2 (float32: 4) bytes
// read and 0.53 written a value, or the reverse.
#include "mx4.h"
#include "ops.h"

namespace moe {

constexpr int kMxThreads = 256;
constexpr int64_t kMxWorkgroups = 4096;  // of a launch at most; each takes piece after piece

typedef float f32x4_t __attribute__((ext_vector_type(4)));

template <int DT>
__device__ __forceinline__ void mx4_load8(const void* x, int64_t piece, float (&v)[8]) {
  if constexpr (DT == kF32) {
    const chunk_t* p = static_cast<const chunk_t*>(x) + 2 * piece;
    const chunk_t a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(a[i]);
      v[4 + i] = __uint_as_float(b[i]);
    }
  } else {
    unpack<DT>(static_cast<const chunk_t*>(x)[piece], v);
  }
}

template <int DT>
__global__ __launch_bounds__(kMxThreads) void mx4_quantize_kernel(const void* __restrict__ x, int64_t pieces,
                                                                  uint32_t* __restrict__ codes,
                                                                  uint8_t* __restrict__ scales) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * kMxThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kMxThreads + threadIdx.x; i < pieces; i += step) {
    float v[8];
    mx4_load8<DT>(x, i, v);
    uint32_t E;
    const uint32_t c = mx4_quantize8(v, &E);  // pieces is a multiple of 4: a block's four lanes stay together
    codes[i] = c;
    if (i % 4 == 0) scales[i / 4] = static_cast<uint8_t>(E);
  }
}

template <int DT>
__global__ __launch_bounds__(kMxThreads) void mx4_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                                    const uint8_t* __restrict__ scales, int64_t pieces,
                                                                    void* __restrict__ out) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * kMxThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kMxThreads + threadIdx.x; i < pieces; i += step) {
    const uint32_t c = codes[i];
    const float s = mx4_scale(scales[i / 4]);
    if constexpr (DT == kF32) {
      typedef float f32x2 __attribute__((ext_vector_type(2)));
      const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
      const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2), e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
      f32x4_t* o = static_cast<f32x4_t*>(out) + 2 * i;
      o[0] = f32x4_t{a[0], a[1], b[0], b[1]};
      o[1] = f32x4_t{d[0], d[1], e[0], e[1]};
    } else {
      static_cast<chunk_t*>(out)[i] = mx4_values8<DT>(c, s);
    }
  }
}

static unsigned mx4_grid(int64_t pieces) {
  const int64_t all = (pieces + kMxThreads - 1) / kMxThreads;
  return static_cast<unsigned>(all < kMxWorkgroups ? all : kMxWorkgroups);
}

hipError_t launch_mx4_quantize(const void* x, int64_t blocks, int dtype, void* codes, void* scales, hipStream_t stream) {
  if (blocks == 0) return hipSuccess;
  const int64_t pieces = 4 * blocks;
  auto* c = static_cast<uint32_t*>(codes);
  auto* s = static_cast<uint8_t*>(scales);
  const unsigned grid = mx4_grid(pieces);
  if (dtype == kBF16) mx4_quantize_kernel<kBF16><<<grid, kMxThreads, 0, stream>>>(x, pieces, c, s);
  else if (dtype == kF16) mx4_quantize_kernel<kF16><<<grid, kMxThreads, 0, stream>>>(x, pieces, c, s);
  else mx4_quantize_kernel<kF32><<<grid, kMxThreads, 0, stream>>>(x, pieces, c, s);
  return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const void* codes, const void* scales, int64_t blocks, int dtype, void* out,
                                 hipStream_t stream) {
  if (blocks == 0) return hipSuccess;
  const int64_t pieces = 4 * blocks;
  auto* c = static_cast<const uint32_t*>(codes);
  auto* s = static_cast<const uint8_t*>(scales);
  const unsigned grid = mx4_grid(pieces);
  if (dtype == kBF16) mx4_dequantize_kernel<kBF16><<<grid, kMxThreads, 0, stream>>>(c, s, pieces, out);
  else if (dtype == kF16) mx4_dequantize_kernel<kF16><<<grid, kMxThreads, 0, stream>>>(c, s, pieces, out);
  else mx4_dequantize_kernel<kF32><<<grid, kMxThreads, 0, stream>>>(c, s, pieces, out);
  return hipGetLastError();
}

}  // namespace moe
