// Rows to microscaled 4-bit values and back, on gfx950 (the format stands in mx4.h).
//
// Rows are whole blocks, so a tensor is one flat run of blocks. A lane takes eight values (16 bytes
// of a 16-bit type), four neighbouring lanes a block: the block's largest magnitude meets over two
// DPP moves, and loads and stores are whole lines of the wave. Bound by memory: 2 (float32: 4) bytes
// read and 0.53 written a value, or the reverse; 6.5 and 7.1 TB/s on 507 MB of bf16, 5.2 and 4.6 on float32.
#include "mx4.h"
#include "ops.h"

namespace moe {

constexpr int kMxThreads = 256;
constexpr int kMxUnroll = 4;                        // pieces of a lane whose loads are in flight together
constexpr int kMxTile = kMxThreads * kMxUnroll;    // pieces of a workgroup's turn
constexpr int64_t kMxWorkgroups = 1 << 20;         // of a launch at most; past them each takes another turn

// A piece: eight values, one chunk of a 16-bit type or two of float32. Rows are loaded with the
// nontemporal hint, and 16-bit values stored with it: 253 million bf16 values take 99 us to 4 bits and
// 91 back, without the hint 113 and 117 (with one load of a lane in flight and 4096 workgroups, 127
// both ways). Float32 values are not: a lane's two chunks lie side by side, each a half of a 32-byte
// piece, and 123 million take 207 us with the hint, 120 without.
template <int DT>
constexpr int kMxChunks = DT == kF32 ? 2 : 1;

template <int DT>
__device__ __forceinline__ void mx4_load(const void* x, int64_t piece, chunk_t (&c)[kMxChunks<DT>]) {
#pragma unroll
  for (int i = 0; i < kMxChunks<DT>; ++i)
    c[i] = __builtin_nontemporal_load(static_cast<const chunk_t*>(x) + kMxChunks<DT> * piece + i);
}

template <int DT>
__device__ __forceinline__ void mx4_quantize_piece(const chunk_t (&c)[kMxChunks<DT>], int64_t piece,
                                                   uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  float v[8];
  if constexpr (DT == kF32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(c[i / 4][i % 4]);
  } else {
    unpack<DT>(c[0], v);
  }
  uint32_t E;
  const uint32_t q = mx4_quantize8(v, &E);
  codes[piece] = q;
  if (piece % 4 == 0) scales[piece / 4] = static_cast<uint8_t>(E);
}

// `pieces` is a multiple of 4, and so is a turn: a block's four lanes stay together.
template <int DT>
__global__ __launch_bounds__(kMxThreads) void mx4_quantize_kernel(const void* __restrict__ x, int64_t pieces,
                                                                  uint32_t* __restrict__ codes,
                                                                  uint8_t* __restrict__ scales) {
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kMxTile; t < pieces; t += static_cast<int64_t>(gridDim.x) * kMxTile) {
    const int64_t at = t + threadIdx.x;
    chunk_t c[kMxUnroll][kMxChunks<DT>];
    if (t + kMxTile <= pieces) {  // uniform
#pragma unroll
      for (int u = 0; u < kMxUnroll; ++u) mx4_load<DT>(x, at + u * kMxThreads, c[u]);
#pragma unroll
      for (int u = 0; u < kMxUnroll; ++u) mx4_quantize_piece<DT>(c[u], at + u * kMxThreads, codes, scales);
    } else {
#pragma unroll 1
      for (int64_t i = at; i < pieces; i += kMxThreads) {
        mx4_load<DT>(x, i, c[0]);
        mx4_quantize_piece<DT>(c[0], i, codes, scales);
      }
    }
  }
}

template <int DT>
__device__ __forceinline__ void mx4_dequantize_piece(uint32_t c, uint32_t E, int64_t piece, void* __restrict__ out) {
  const float s = mx4_scale(E);
  if constexpr (DT == kF32) {
    const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
    const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2), e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
    f32x4_t* o = static_cast<f32x4_t*>(out) + 2 * piece;
    o[0] = f32x4_t{a[0], a[1], b[0], b[1]};
    o[1] = f32x4_t{d[0], d[1], e[0], e[1]};
  } else {
    __builtin_nontemporal_store(mx4_values8<DT>(c, s), static_cast<chunk_t*>(out) + piece);
  }
}

template <int DT>
__global__ __launch_bounds__(kMxThreads) void mx4_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                                    const uint8_t* __restrict__ scales, int64_t pieces,
                                                                    void* __restrict__ out) {
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kMxTile; t < pieces; t += static_cast<int64_t>(gridDim.x) * kMxTile) {
    const int64_t at = t + threadIdx.x;
    uint32_t c[kMxUnroll], E[kMxUnroll];
    if (t + kMxTile <= pieces) {  // uniform
#pragma unroll
      for (int u = 0; u < kMxUnroll; ++u) {
        c[u] = codes[at + u * kMxThreads];
        E[u] = scales[(at + u * kMxThreads) / 4];
      }
#pragma unroll
      for (int u = 0; u < kMxUnroll; ++u) mx4_dequantize_piece<DT>(c[u], E[u], at + u * kMxThreads, out);
    } else {
#pragma unroll 1
      for (int64_t i = at; i < pieces; i += kMxThreads) mx4_dequantize_piece<DT>(codes[i], scales[i / 4], i, out);
    }
  }
}

static unsigned mx4_grid(int64_t pieces) {
  const int64_t all = (pieces + kMxTile - 1) / kMxTile;
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
