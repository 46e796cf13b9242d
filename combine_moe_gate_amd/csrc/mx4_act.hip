// The experts' products with microscaled 4-bit weights (the format stands in mx4.h) and the
// epilogue of expert_act.h, on gfx950 matrix cores.
//
// For each placed row r of expert x, z = A(r) @ W[x]^T + b[x], W the values the codes stand for;
// out[r] = w_r u + residual(r), u = act(z) or act(z_gate) * z_up, rounded once to 16 bits or to 4.
// Rows A(r) are 16-bit or 4-bit.
//
// 4-bit rows meet 4-bit weights in v_mfma_scale_f32_16x16x128_f8f6f4, which takes the scales. For
// bf16 rows the codes are widened to bf16 with their scale, which is exact. For f16 rows they are
// widened to f16 where the scales of the step in hand allow that exactly (2^-23 to 2^13, what
// weights have in earnest); elsewhere each row value is split into two bf16 values, the upper 8
// bits of its 11 and the rest, both products exact again.
//
// Two kernels, chosen by the rows an expert has on average: the tiles of mx4_tile.hip, and few rows:
// a workgroup of four waves multiplies up to 16 F rows by 16 FB weight rows, each wave a
// quarter of the K steps of four blocks: codes, scales and rows go from memory straight to the
// registers, several steps ahead, and the four partial sums meet in LDS.
#include <atomic>

#include "mx4_product.h"

namespace moe {

// ---------------------------------------------------------------------------------
// few rows

constexpr int kMxFewThreads = 256, kMxFewWaves = 4, kMxFewBand = 8;

// RT: the rows' type (kBF16, kF16 or kMx4); DT: the element type of bias, residual and results.
template <int RT, int DT, int F, int FB>
__global__ __launch_bounds__(kMxFewThreads, 2) void mx4_few_kernel(Mx4Act p, int col_blocks, int tile_grid) {
  constexpr bool kQ = RT == kMx4;
  constexpr int kAChunks = kQ ? 1 : 4;                  // 16-byte pieces of a row's block
  constexpr int kStepRegs = FB * 5 + F * (kQ ? 5 : 16);
  constexpr int kDepth = kStepRegs <= 26 ? 4 : kStepRegs <= 40 ? 2 : 1;  // K steps in flight per wave
  constexpr int kCols = 16 * FB;                        // weight rows per workgroup
  constexpr int kPitch = kCols * 4 + 16;                // bytes per row of a wave's float32 sums
  extern __shared__ __attribute__((aligned(1024))) char lds[];  // [wave][16 F rows][kPitch]
  if (static_cast<int>(blockIdx.x) >= tile_grid) {
    zero_unfilled_mx4(p, blockIdx.x - tile_grid, gridDim.x - tile_grid);
    return;
  }
  const SegmentTile tc = segment_tile(blockIdx.x, p.e, p.kept, p.offsets, col_blocks, kMxFewBand,
                                      [](int r) { return (r + 16 * F - 1) / (16 * F); });
  const int x = tc.expert;
  if (x < 0) return;
  const int lane = lane_id(), wv = wave_in_block(), g = lane >> 4;
  const int row0 = tc.offset + tc.rb * 16 * F;
  const int rem = tc.rows - tc.rb * 16 * F;
  const int nrows = rem < 16 * F ? rem : 16 * F;
  const int out_cols = p.gated ? kCols / 2 : kCols;
  const int col0 = tc.cb * out_cols;
  const int kb = p.m / kMx4Block;

  // lane l takes block 4 step + l / 16 of row l % 16 of each fragment; rows past the segment repeat
  // its first one, whose results are not stored
  const chunk_t* a_row[F];
  const uint8_t* a_scale[F];
#pragma unroll
  for (int i = 0; i < F; ++i) {
    const int r = i * 16 + (lane & 15);
    const int rr = row0 + (r < nrows ? r : 0);
    const size_t block = static_cast<size_t>(p.gather ? p.src[rr] : rr) * kb + g;
    a_row[i] = static_cast<const chunk_t*>(p.a) + block * kAChunks;
    a_scale[i] = p.a_scales + block;  // read for 4-bit rows only
  }
  // The first half of the fragments are gate rows and the second the up rows that meet them, or all
  // are plain; each fragment by a uniform base and a lane's own offset in its 16 rows.
  const chunk_t* b_base[FB];
  const uint8_t* s_base[FB];
  uint32_t b_off[FB];
#pragma unroll
  for (int j = 0; j < FB; ++j) {
    int f = p.gated ? col0 + j % (FB / 2) * 16 : col0 + j * 16;
    f = f < p.n ? f : 0;  // past the last feature: any rows, their sums are not stored
    const int have = p.n - f < 16 ? p.n - f : 16;
    const int first = p.gated && j >= FB / 2 ? p.n + f : f;
    const size_t block = (static_cast<size_t>(x) * p.nz + first) * kb;
    b_base[j] = static_cast<const chunk_t*>(p.w) + block;
    s_base[j] = p.w_scales + block;
    b_off[j] = static_cast<uint32_t>((lane & 15) < have ? lane & 15 : 0) * kb + g;
  }

  f32x4_t acc[F][FB];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  chunk_t fb[kDepth][FB], fa[kDepth][F][kAChunks];
  uint32_t sb[kDepth][FB], sa[kDepth][F];
  auto load = [&](int step, int d) {
#pragma unroll
    for (int j = 0; j < FB; ++j) {
      fb[d][j] = __builtin_nontemporal_load(b_base[j] + 4 * static_cast<size_t>(step) + b_off[j]);
      sb[d][j] = s_base[j][4 * static_cast<size_t>(step) + b_off[j]];
    }
#pragma unroll
    for (int i = 0; i < F; ++i) {
#pragma unroll
      for (int q = 0; q < kAChunks; ++q) fa[d][i][q] = a_row[i][(4 * static_cast<size_t>(step)) * kAChunks + q];
      if constexpr (kQ) sa[d][i] = a_scale[i][4 * static_cast<size_t>(step)];
    }
  };
  auto multiply = [&](int d) {
    if constexpr (kQ) {
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j) acc[i][j] = mfma_mx4(fb[d][j], sb[d][j], fa[d][i][0], sa[d][i], acc[i][j]);
    } else {
      bool split = false;
      if constexpr (RT == kF16) {
        bool fits = true;
#pragma unroll
        for (int j = 0; j < FB; ++j) fits = fits && mx4_fits_f16(sb[d][j]);
        split = !__all(fits);
      }
      if (RT == kBF16 || !split) {
#pragma unroll
        for (int j = 0; j < FB; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const chunk_t w = mx4_values8<RT == kF16 ? kF16 : kBF16>(fb[d][j][q], mx4_scale(sb[d][j]));
#pragma unroll
            for (int i = 0; i < F; ++i) acc[i][j] = mfma_16x16x32<RT == kF16 ? kF16 : kBF16>(w, fa[d][i][kQ ? 0 : q], acc[i][j]);
          }
      } else {
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            chunk_t hi, lo;
            split_f16(fa[d][i][kQ ? 0 : q], hi, lo);
#pragma unroll
            for (int j = 0; j < FB; ++j) {
              const chunk_t w = mx4_values8<kBF16>(fb[d][j][q], mx4_scale(sb[d][j]));
              acc[i][j] = mfma_16x16x32<kBF16>(w, lo, acc[i][j]);
              acc[i][j] = mfma_16x16x32<kBF16>(w, hi, acc[i][j]);
            }
          }
      }
    }
  };
  const int full = kb / 4;  // whole K steps; wave wv takes steps wv, wv + 4, ...
#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (wv + d * kMxFewWaves < full) load(wv + d * kMxFewWaves, d);  // uniform
  int step = wv;
  for (; step + (2 * kDepth - 1) * kMxFewWaves < full; step += kDepth * kMxFewWaves) {  // every refill is a real step
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      multiply(d);
      load(step + (d + kDepth) * kMxFewWaves, d);
    }
  }
  for (; step < full; step += kDepth * kMxFewWaves) {  // what is left: at most two rounds
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {  // uniform conditions
      if (step + d * kMxFewWaves < full) multiply(d);
      if (step + (d + kDepth) * kMxFewWaves < full) load(step + (d + kDepth) * kMxFewWaves, d);
    }
  }
  if (kb % 4 != 0 && wv == full % kMxFewWaves) {  // the last, partial step: zeros past the rows' end
    const chunk_t z = {0u, 0u, 0u, 0u};
    const bool in = 4 * full + g < kb;
    const size_t at = 4 * static_cast<size_t>(full);
#pragma unroll
    for (int j = 0; j < FB; ++j) {
      fb[0][j] = in ? b_base[j][at + b_off[j]] : z;
      sb[0][j] = in ? s_base[j][at + b_off[j]] : 127u;
    }
#pragma unroll
    for (int i = 0; i < F; ++i) {
#pragma unroll
      for (int q = 0; q < kAChunks; ++q) fa[0][i][q] = in ? a_row[i][at * kAChunks + q] : z;
      if constexpr (kQ) sa[0][i] = in ? a_scale[i][at] : 127u;
    }
    multiply(0);
  }

#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j)
      *reinterpret_cast<f32x4_t*>(lds + (wv * 16 * F + i * 16 + (lane & 15)) * kPitch + j * 64 + (lane >> 4) * 16) =
          acc[i][j];
  __syncthreads();
  // a thread per row and eight features of each half
  constexpr int kPieces = FB;  // 16 FB / 2 / 8
  const int row = threadIdx.x / kPieces, q8 = 8 * (threadIdx.x % kPieces);
  if (row >= nrows) return;
  float v[8], u[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = u[q] = 0.0f;
  for (int w = 0; w < kMxFewWaves; ++w) {
    const float* part = reinterpret_cast<const float*>(lds + (w * 16 * F + row) * kPitch) + q8;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      v[q] += part[q];
      u[q] += part[8 * FB + q];
    }
  }
  const int r = row0 + row, t = p.src[r];
  const float w = p.route_w != nullptr ? route_weight(p, r, t) : 1.0f;
  const int c = col0 + q8;
  if (c < p.n) finish8_mx4<DT>(p, x, r, t, w, c, v, u);
  if (!p.gated && c + 8 * FB < p.n) finish8_mx4<DT>(p, x, r, t, w, c + 8 * FB, u, v);
}

// ---------------------------------------------------------------------------------
// launches

// How a launch is shaped: F of its row tiles (16 F rows; 0: the large tiles), the weight rows
// per workgroup, and its workgroups.
struct Mx4Shape {
  int few, cols;
  int64_t col_blocks, tiles;
};

static Mx4Shape mx4_shape(const LayoutView& L, const Mx4Act& p) {
  auto shape = [&](int few) {
    // 64 weight rows, so that a 4-bit block of 32 gated results lies in one workgroup
    Mx4Shape a{few, few ? 64 : 256, 0, 0};
    a.col_blocks = (static_cast<int64_t>(p.nz) + a.cols - 1) / a.cols;
    a.tiles = L.s == 0 ? 0 : row_tiles(L, few ? 16 * few : mx4_tile_rows()) * a.col_blocks;
    return a;
  };
  const int64_t routes = static_cast<int64_t>(L.s) * L.k;
  int64_t mean = (routes + L.e - 1) / L.e;
  if (L.capacity > 0 && mean > L.capacity) mean = L.capacity;
  return shape(mean <= 16 ? 1 : 0);
}

static int64_t mx4_grid(const Mx4Shape& a) { return (a.tiles + kXcds - 1) / kXcds * kXcds + kZeroBlocks; }

bool mx4_act_fits(const LayoutView& L, const Mx4Act& p, int) {
  const Mx4Shape a = mx4_shape(L, p);
  return mx4_grid(a) <= most_workgroups(a.few ? kMxFewThreads : kMx4TileThreads);
}

template <int RT, int DT, int F, int FB>
static hipError_t launch_few(const Mx4Act& p, int col_blocks, int64_t grid, hipStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr int kBytes = kMxFewWaves * 16 * F * (16 * FB * 4 + 16);
  auto kern = mx4_few_kernel<RT, DT, F, FB>;
  if (kBytes > 65536) {
    const hipError_t err = allow_lds(reinterpret_cast<const void*>(kern), kBytes, done);
    if (err != hipSuccess) return err;
  }
  kern<<<static_cast<unsigned>(grid), kMxFewThreads, kBytes, stream>>>(p, col_blocks, static_cast<int>(grid) - kZeroBlocks);
  return hipGetLastError();
}

template <int RT, int DT>
static hipError_t launch_rt(const LayoutView& L, const Mx4Act& p, hipStream_t stream) {
  const Mx4Shape a = mx4_shape(L, p);
  const int col_blocks = static_cast<int>(a.col_blocks);
  if (a.few == 0) return launch_mx4_tiles(p, DT, col_blocks, mx4_grid(a), stream);
  return launch_few<RT, DT, 1, 4>(p, col_blocks, mx4_grid(a), stream);
}

hipError_t launch_mx4_act(const LayoutView& L, const Mx4Act& p, int dtype, hipStream_t stream) {
  if (p.rows == 0) return hipSuccess;
  if (p.a_scales != nullptr)
    return dtype == kBF16 ? launch_rt<kMx4, kBF16>(L, p, stream) : launch_rt<kMx4, kF16>(L, p, stream);
  return dtype == kBF16 ? launch_rt<kBF16, kBF16>(L, p, stream) : launch_rt<kF16, kF16>(L, p, stream);
}

}  // namespace moe
