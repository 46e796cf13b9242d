// Input-row gradient of the products with microscaled 4-bit weights, on gfx950 matrix cores.
//
// For each placed row r of expert x: out[r] = a[r] @ W[x], a the 16-bit gradient rows [rows, nz], W
// [nz, m] the values the codes stand for. The sum runs along the weights' rows, each with scales of
// its own, so the weights are widened (to bf16, exact) before they are multiplied; f16 gradients are
// split into two bf16 values each, exact as well.
//
// A workgroup of four waves takes 64 rows by 64 input features, each wave 16 of the rows: 32 weight
// rows at a time are widened into LDS.
#include "mx4_product.h"

namespace moe {

constexpr int kMxdThreads = 256, kMxdRows = 64, kMxdCols = 64, kMxdK = 32, kMxdPitch = 72, kMxdBand = 8;

template <int DT>
__global__ __launch_bounds__(kMxdThreads) void mx4_dgrad_kernel(Mx4Act p, int col_blocks, int tile_grid) {
  __shared__ __attribute__((aligned(16))) uint16_t wt[kMxdK][kMxdPitch];
  if (static_cast<int>(blockIdx.x) >= tile_grid) {
    zero_unfilled(p, blockIdx.x - tile_grid, gridDim.x - tile_grid);
    return;
  }
  const SegmentTile tc = segment_tile(blockIdx.x, p.e, p.kept, p.offsets, col_blocks, kMxdBand,
                                      [](int r) { return (r + kMxdRows - 1) / kMxdRows; });
  if (tc.expert < 0) return;
  const int lane = lane_id(), wv = wave_in_block(), g = lane >> 4;
  const int row0 = tc.offset + tc.rb * kMxdRows;
  const int rem = tc.rows - tc.rb * kMxdRows;
  const int nrows = rem < kMxdRows ? rem : kMxdRows;
  const int col0 = tc.cb * kMxdCols, kb = p.n / kMx4Block;
  const int K = p.m;  // weight rows
  const int row = wv * 16 + (lane & 15);
  const chunk_t* a_row = static_cast<const chunk_t*>(p.a) + static_cast<size_t>(row0 + (row < nrows ? row : 0)) * (K / 8);
  const size_t w0 = static_cast<size_t>(tc.expert) * K;
  f32x4_t acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  for (int k0 = 0; k0 < K; k0 += kMxdK) {
    __syncthreads();
    if (threadIdx.x < 2 * kMxdK) {  // a block of 32 weights per thread; past the last row or column: zeros
      const int k = threadIdx.x / 2, b = col0 / kMx4Block + threadIdx.x % 2;
      chunk_t c = {0u, 0u, 0u, 0u};
      uint32_t E = 127u;
      if (k0 + k < K && b < kb) {
        const size_t at = (w0 + k0 + k) * kb + b;
        c = static_cast<const chunk_t*>(p.w)[at];
        E = p.w_scales[at];
      }
      chunk_t* to = reinterpret_cast<chunk_t*>(&wt[k][(threadIdx.x % 2) * kMx4Block]);
#pragma unroll
      for (int q = 0; q < 4; ++q) to[q] = mx4_values8<kBF16>(c[q], mx4_scale(E));
    }
    __syncthreads();
    chunk_t a = {0u, 0u, 0u, 0u};
    if (k0 + 8 * g < K) a = a_row[k0 / 8 + g];
    chunk_t hi = a, lo = a;
    if constexpr (DT == kF16) split_f16(a, hi, lo);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      chunk_t w;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = wt[8 * g + 2 * q][16 * j + (lane & 15)] | (static_cast<uint32_t>(wt[8 * g + 2 * q + 1][16 * j + (lane & 15)]) << 16);
      if constexpr (DT == kF16) acc[j] = mfma_16x16x32<kBF16>(w, lo, acc[j]);
      acc[j] = mfma_16x16x32<kBF16>(w, hi, acc[j]);
    }
  }
  if (row >= nrows) return;
  uint16_t* out = static_cast<uint16_t*>(p.out) + static_cast<size_t>(row0 + row) * p.n + col0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = 16 * j + 4 * g;
    if (col0 + c < p.n)
      *reinterpret_cast<uint2*>(out + c) = uint2{narrow2<DT>(acc[j][0], acc[j][1]), narrow2<DT>(acc[j][2], acc[j][3])};
  }
}

static int64_t mx4_dgrad_grid(const LayoutView& L, int m, int64_t* col_blocks) {
  *col_blocks = (static_cast<int64_t>(m) + kMxdCols - 1) / kMxdCols;
  const int64_t tiles = L.s == 0 ? 0 : row_tiles(L, kMxdRows) * *col_blocks;
  return (tiles + kXcds - 1) / kXcds * kXcds + kZeroBlocks;
}

bool mx4_dgrad_fits(const LayoutView& L, int m) {
  int64_t cb;
  return mx4_dgrad_grid(L, m, &cb) <= most_workgroups(kMxdThreads);
}

hipError_t launch_mx4_dgrad(const LayoutView& L, const Mx4Act& p, int dtype, hipStream_t stream) {
  if (p.rows == 0) return hipSuccess;
  int64_t cb;
  const int64_t grid = mx4_dgrad_grid(L, p.n, &cb);
  const int tiles = static_cast<int>(grid) - kZeroBlocks;
  if (dtype == kBF16)
    mx4_dgrad_kernel<kBF16><<<static_cast<unsigned>(grid), kMxdThreads, 0, stream>>>(p, static_cast<int>(cb), tiles);
  else
    mx4_dgrad_kernel<kF16><<<static_cast<unsigned>(grid), kMxdThreads, 0, stream>>>(p, static_cast<int>(cb), tiles);
  return hipGetLastError();
}

}  // namespace moe
