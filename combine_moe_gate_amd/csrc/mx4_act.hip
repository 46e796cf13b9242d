// The experts' products with microscaled 4-bit weights (the format stands in mx4.h) and the
// epilogue of expert_act.h, on gfx950 matrix cores.
//
// For each placed row r of expert x, z = A(r) @ W[x]^T + b[x], W the values the codes stand for;
// out[r] = w_r u + residual(r), u = act(z) or act(z_gate) * z_up, rounded once to 16 bits or to 4.
// Rows A(r) are 16-bit or 4-bit.
//
// 4-bit rows meet 4-bit weights in v_mfma_scale_f32_16x16x128_f8f6f4, which takes the scales. For
// bf16 rows the codes are widened to bf16 with their scale, which is exact. For f16 rows they are
// widened to f16 where the scales of the step in hand allow that exactly (2^-23 to 2^13, which is what
// weights in use have, and any over zeros); elsewhere each row value is split into two bf16 values, the
// upper 8 bits of its 11 and the rest, both products exact again.
//
// Three kernels, chosen by the rows an expert has on average, the workgroups there would be and the
// scales' alignment (mx4_shape() below): the tiles of mx4_tile.hip, the streams of mx4_stream.hip, and
// here the form that takes rows and scales of any alignment: a workgroup of four waves multiplies up
// to 16 F rows by 64 weight rows, each wave a quarter of the K steps of four blocks: codes, scales
// and rows go from memory straight to the registers, and the four partial sums meet in LDS.
#include "mx4_product.h"

namespace moe {

// ---------------------------------------------------------------------------------
// few rows

constexpr int kMxFewThreads = 256, kMxFewWaves = 4, kMxFewBand = 8;

// RT: the rows' type (kBF16, kF16 or kMx4); DT: the element type of bias, residual and results; kDepth:
// the K steps in flight per wave.
template <int RT, int DT, int F, int kDepth, int kOcc>
__global__ __launch_bounds__(kMxFewThreads, kOcc) void mx4_few_kernel(Mx4Act p, int col_blocks, int tile_grid) {
  constexpr bool kQ = RT == kMx4;
  constexpr int kAChunks = kQ ? 1 : 4;                  // 16-byte pieces of a row's block
  constexpr int FB = 4;
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
  auto load_b = [&](int step, int d) {
#pragma unroll
    for (int j = 0; j < FB; ++j) {
      fb[d][j] = __builtin_nontemporal_load(b_base[j] + 4 * static_cast<size_t>(step) + b_off[j]);
      sb[d][j] = s_base[j][4 * static_cast<size_t>(step) + b_off[j]];
    }
  };
  const int full = kb / 4;  // whole K steps; wave wv takes steps wv, wv + 4, ...
#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (wv + d * kMxFewWaves < full) load_b(wv + d * kMxFewWaves, d);  // uniform
  __builtin_amdgcn_sched_barrier(0);

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
  auto load_a = [&](int step, int d) {
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
        if (split) {  // uniform
          fits = true;
#pragma unroll
          for (int j = 0; j < FB; ++j) fits = fits && (mx4_fits_f16(sb[d][j]) || mx4_zeros(fb[d][j]));
          split = !__all(fits);
        }
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
  auto load = [&](int step, int d) {
    load_b(step, d);
    load_a(step, d);
  };
#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (wv + d * kMxFewWaves < full) load_a(wv + d * kMxFewWaves, d);  // uniform
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
  const float w = route_weight_wide(p, r, t);
  const int c = col0 + q8;
  if (c < p.n) finish8_mx4<DT>(p, x, r, t, w, c, v, u);
  if (!p.gated && c + 8 * FB < p.n) finish8_mx4<DT>(p, x, r, t, w, c + 8 * FB, u, v);
}

// ---------------------------------------------------------------------------------
// launches

// How a launch is formed: the tiles, streams of 16 `few` rows, or this file's kernel, the weight rows
// per workgroup, and its workgroups.
enum class Mx4Form { tiles, stream, few };
struct Mx4Shape {
  Mx4Form form;
  int few;             // row tiles of 16 of a workgroup
  int64_t col_blocks, tiles;
};

// Streams read weights best (5.5 TB/s where the tiles reach 4.3); the tiles multiply best, once an
// expert has rows to fill them and there are enough of them for the CUs. Microseconds, random rows,
// bf16 and 4-bit (`mean` per expert; `tiles` as counted below):
//                                          bf16: stream of           4-bit: stream of
//   experts, weight rows x length   mean    16     32    tiles        16     32     64    tiles  (tiles)
//   128, 4096 x 4096                1/16    17     21     61          14     14     15     20
//   128, 4096 x 4096                16     289    265    465         276    231    233    253
//   128, 2816 x 2816                32     212    168    260         179    137    121    141
//   128, 2816 x 2816                64     337    255    285         287    190    151    158
//   128, 2816 x 2816                72     375    289    291         315    213    168    162
//   128, 2816 x 2816                128    608    446    348         520    321    226    186
//   64, 2816 x 1408                 8       30     37     68          28     29     30     39
//   64, 2816 x 1408                 16      37     39     69          32     30     31     40
//   64, 2816 x 1408                 72     102     95     87          78     64     55     55
//   8, 1024 x 1024                  16     6.9    8.0     17         5.8    6.4    7.3    8.2
//   16, 1024 x 1024                 256     25     24     38          19     15     13     20    (120)
//   8, 1024 x 2048                  1024    72     60     65          54     36     27     29    (144)
//   16, 1024 x 4096                 512    154    100    117         107     66     51     45    (176)
//   8, 512 x 512                    4000    59     50     29          42     32     24     20    (238)
// Rows that are no multiple of 128 elements, or unaligned scales, take this file's kernel in place of a
// stream (16 experts, 576 x 544, mean 125 in 9.1 and 7.2, tiles 19 and 12). It takes 32 rows at a time, of f16
// rows 16 where experts have few: beside 32, the split form leaves registers for one K step in flight, not
// two. As an expert's rows pass that its time doubles, and the tiles' grows little; of short rows its start costs
// less. With 16 rows / with 32 / the tiles:
//   experts, weight rows x length   mean          bf16               f16               4-bit
//   128, 2880 x 2880                1        121 / 128 / 174    125 / 140 / 185    117 / 113 / 105
//   128, 2880 x 2880                8        197 / 205 / 263    199 / 216 / 280    195 / 187 / 164
//   128, 2880 x 2880                16       304 / 243 / 265    280 / 236 / 281    292 / 207 / 166
//   128, 2880 x 2880                24       421 / 285 / 270    374 / 265 / 285    403 / 228 / 170
//   128, 2880 x 2880                32       459 / 390 / 279    432 / 351 / 291    445 / 294 / 174
//   64, 2880 x 1440                 16        72 / 69 / 71       82 / 75 / 79       69 / 56 / 41
//   64, 2880 x 1440                 24        94 / 76 / 74      109 / 81 / 80       89 / 60 / 41
//   128, 1088 x 544                 8         21 / 23 / 37       29 / 32 / 41       19 / 20 / 23
//   128, 1088 x 544                 24        38 / 29 / 38       52 / 37 / 42       30 / 24 / 24
//   128, 1088 x 544                 32        45 / 39 / 41       63 / 49 / 44       36 / 33 / 26
//   60, 1408 x 288                  24        17 / 13 / 19       23 / 16 / 21       13 / 11 / 14
// With streams 2816 x 2816 of these takes 73, 112, 130, 133 and 163 in bf16: rows of any length, or scales at any
// address, cost up to twice that.
constexpr int kMx4Mean = 72;                         // mean rows from which the tiles are worth while
constexpr int64_t kMx4Tiles16 = 200, kMx4Tiles4 = 128;
constexpr int kMx4Long = 1024;                       // elements of a row that is not short
static Mx4Shape mx4_shape(const LayoutView& L, const Mx4Act& p, int dtype) {
  const bool q = p.a_scales != nullptr;
  auto shape = [&](Mx4Form form, int few, int height, int cols) {
    Mx4Shape a{form, few, (static_cast<int64_t>(p.nz) + cols - 1) / cols, 0};
    a.tiles = L.s == 0 ? 0 : row_tiles(L, height) * a.col_blocks;
    return a;
  };
  const Mx4Shape large = shape(Mx4Form::tiles, 0, mx4_tile_rows(), 256);
  const int64_t routes = static_cast<int64_t>(L.s) * L.k;
  int64_t mean = (routes + L.e - 1) / L.e;
  if (L.capacity > 0 && mean > L.capacity) mean = L.capacity;
  const bool many = large.tiles >= (q ? kMx4Tiles4 : kMx4Tiles16);
  if (many && mean >= kMx4Mean) return large;
  const uintptr_t scales = reinterpret_cast<uintptr_t>(p.w_scales) | reinterpret_cast<uintptr_t>(p.a_scales);
  if (p.m % 128 == 0 && scales % 4 == 0) {
    const int few = mean <= (q ? 8 : 12) ? 1 : q && mean > 24 ? 4 : 2;
    return shape(Mx4Form::stream, few, 16 * few, 128);
  }
  const bool longer = p.m >= kMx4Long;
  if (many && mean > (q ? (longer ? 0 : 24) : longer ? 20 : 32)) return large;
  const int few = !q && dtype == kF16 && mean <= 12 ? 1 : 2;
  // 64 weight rows, so that a 4-bit block of 32 gated results lies in one workgroup
  return shape(Mx4Form::few, few, 16 * few, 64);
}

static int64_t mx4_grid(const Mx4Shape& a) { return (a.tiles + kXcds - 1) / kXcds * kXcds + kZeroBlocks; }

bool mx4_act_fits(const LayoutView& L, const Mx4Act& p, int dtype) {
  const Mx4Shape a = mx4_shape(L, p, dtype);
  static_assert(kMxFewThreads == kMx4StreamThreads);
  return mx4_grid(a) <= most_workgroups(a.form == Mx4Form::tiles ? kMx4TileThreads : kMxFewThreads);
}

template <int RT, int DT, int F, int kDepth, int kOcc>
static hipError_t launch_few(const Mx4Act& p, int col_blocks, int64_t grid, hipStream_t stream) {
  constexpr int kBytes = kMxFewWaves * 16 * F * (64 * 4 + 16);
  static_assert(kBytes <= 65536);
  mx4_few_kernel<RT, DT, F, kDepth, kOcc><<<static_cast<unsigned>(grid), kMxFewThreads, kBytes, stream>>>(
      p, col_blocks, static_cast<int>(grid) - kZeroBlocks);
  return hipGetLastError();
}

hipError_t launch_mx4_act(const LayoutView& L, const Mx4Act& p, int dtype, hipStream_t stream) {
  if (p.rows == 0) return hipSuccess;
  const Mx4Shape a = mx4_shape(L, p, dtype);
  const int64_t grid = mx4_grid(a);
  const int col_blocks = static_cast<int>(a.col_blocks);
  if (a.form == Mx4Form::tiles) return launch_mx4_tiles(p, dtype, col_blocks, grid, stream);
  if (a.form == Mx4Form::stream) return launch_mx4_stream(p, dtype, a.few, col_blocks, grid, stream);
  if (p.a_scales != nullptr)
    return dtype == kBF16 ? launch_few<kMx4, kBF16, 2, 2, 3>(p, col_blocks, grid, stream)
                          : launch_few<kMx4, kF16, 2, 2, 3>(p, col_blocks, grid, stream);
  if (dtype == kBF16) return launch_few<kBF16, kBF16, 2, 1, 3>(p, col_blocks, grid, stream);
  return a.few == 1 ? launch_few<kF16, kF16, 1, 2, 2>(p, col_blocks, grid, stream)
                    : launch_few<kF16, kF16, 2, 1, 2>(p, col_blocks, grid, stream);
}

}  // namespace moe
