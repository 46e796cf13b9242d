// The products with 4-bit weights for segments of few rows, on gfx950 matrix cores (mx4_act.hip
// chooses): what they cost is reading the weights.
//
// A workgroup of four waves multiplies up to 16 FR rows (16 or 32, of 4 bits 64) by 128 weight rows of one
// expert, 32 of them each wave. Both sides stream through LDS in stages of 256 elements (codes and 16-bit rows in
// XOR-swizzled 16-byte pieces, scales in 4-byte words), all loaded directly, S - 1 of S stages ahead: every
// wave issues the same number of loads a stage, so that it can wait for the oldest stage alone. Lane
// group g = lane / 16 multiplies block 4 p + g of a stage in its half p. Rows past the segment repeat
// its first row (their results are not stored). The sums meet in LDS, and a thread finishes eight
// features of a row.
//
// Measured: one token, 8 of 128 experts, 4096 -> 2 x 2048, bf16 rows, 71 MB in 17 us; 32 tokens, 4-bit
// rows, 2816 -> 2 x 1408, 460 MB in 84 us (5.5 TB/s) and 1408 -> 2816, 243 MB in 51 (4.8): the shorter
// the rows, the more of a workgroup's time is its start and end.
//
// Scales load as words: rows must be a multiple of 128 elements and scales 4-byte aligned.
#include <atomic>

#include "mx4_product.h"

namespace moe {

constexpr int kMsThreads = kMx4StreamThreads;
constexpr int kMsBN = 128;                         // weight rows per workgroup
constexpr int kMsBand = 8;                         // row-blocks per band of the tile order
constexpr int kMsPitch = kMsBN * 4 + 16;           // bytes per row of the float32 sums

// Stages in LDS: as many as two workgroups of a CU have room for, or for short rows two, so that up to four
// workgroups lie on a CU: of a few stages' time in LDS a workgroup's start and end are much, and the
// others' loads cover them. Microseconds with two stages and with more, 32 tokens (16-bit rows: 24):
//   4-bit rows: 1408 -> 2816  50 and 54    2048 -> 4096  88 and 89    2816 -> 2816  84 and 82    4096 -> 4096  180 and 175
//   16-bit rows: 1408 -> 2816  31 and 36   4 tokens, 4096 -> 4096  62 and 55
// With no more workgroups than CUs, more stages: 4-bit rows, one token, 6 of 64, 1408 -> 2816, 7.7 and 7.1.
constexpr int kMsShort = 2048;                     // elements of the longest short row
constexpr int kMsCus = 256;
constexpr int ms_stages(int RT, int FR, bool few) { return few ? 2 : RT == kMx4 ? (FR == 1 ? 4 : 3) : FR == 1 ? 3 : 2; }

template <int RT, int FR, int S>
struct MsLds {
  static constexpr bool kQ = RT == kMx4;
  static constexpr int kStages = S;
  static constexpr int kRowBytes = kQ ? 128 : 512;                   // 256 elements of a row
  static constexpr int kA = 16 * FR * kRowBytes;
  static constexpr int kAScales = kQ ? (FR == 4 ? 512 : 256) : 0;    // whole wave loads of words
  static constexpr int kB = kA + kAScales, kBScales = kB + kMsBN * 128;
  static constexpr int kStage = kBScales + kMsBN * 8;
  static constexpr int kRows = kStages * kStage > 16 * FR * kMsPitch ? kStages * kStage : 16 * FR * kMsPitch;
  static constexpr int kBytes = kRows + 16 * FR * 8;                 // per row its token and route weight
  // loads of a stage that each wave issues
  static constexpr int kALoads = kQ ? (FR == 4 ? 2 : 1) : 2 * FR;
  static constexpr int kLoads = kALoads + (kQ ? 1 : 0) + 4 + 1;
  static_assert(kBytes <= 160 * 1024 && (kStages - 2) * kLoads < 64);
};

template <int RT, int DT, int FR, int S>
__global__ __launch_bounds__(kMsThreads) void mx4_stream_kernel(Mx4Act p, int col_blocks, int tile_grid) {
  using Lds = MsLds<RT, FR, S>;
  constexpr bool kQ = Lds::kQ;
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  if (static_cast<int>(blockIdx.x) >= tile_grid) {
    zero_unfilled_mx4(p, blockIdx.x - tile_grid, gridDim.x - tile_grid);
    return;
  }
  const SegmentTile tc = segment_tile(blockIdx.x, p.e, p.kept, p.offsets, col_blocks, kMsBand,
                                      [](int r) { return (r + 16 * FR - 1) / (16 * FR); });
  const int x = tc.expert;
  if (x < 0) return;
  const int lane = lane_id(), wv = wave_in_block(), grp = lane >> 4;
  const int row0 = tc.offset + tc.rb * 16 * FR;
  const int rem = tc.rows - tc.rb * 16 * FR;
  const int nrows = rem < 16 * FR ? rem : 16 * FR;
  const int out_cols = p.gated ? kMsBN / 2 : kMsBN;
  const int col0 = tc.cb * out_cols;
  const int kb = p.m / kMx4Block;
  const int achunks = kQ ? kb : 4 * kb;                // 16-byte pieces of a row
  const int nu = (kb + 7) / 8;

  // rows: 16-bit ones fill two of 512 bytes a load, piece slot ^ a_swizzle(row % 16) of 32 at each slot
  // (lanes of rows 0-3 and 12-15 of one group and 4-11 of the next read together, four pieces apart:
  // the order of the rows' fours keeps them on different banks); 4-bit ones eight of 128 bytes,
  // swizzled as the codes. Rows past the segment repeat its first. They are
  // looked up before any load to LDS starts: the wait for them would be one for those as well.
  auto a_swizzle = [](int r) { return 4 * ((0x78 >> (r / 4 * 2)) & 3) + r % 4; };
  auto input_row = [&](int r) {
    const int rr = row0 + (r < nrows ? r : 0);
    return static_cast<size_t>(p.gather ? p.src[rr] : rr);
  };
  const chunk_t* a_row[Lds::kALoads];
  int a_load[Lds::kALoads], a_piece[Lds::kALoads];
#pragma unroll
  for (int q = 0; q < Lds::kALoads; ++q) {
    a_load[q] = kQ ? (q * 4 + wv) % (2 * FR) : q * 4 + wv;  // fewer loads than waves: some are issued twice
    const int r = kQ ? a_load[q] * 8 + lane / 8 : a_load[q] * 2 + lane / 32;
    a_piece[q] = kQ ? (lane % 8) ^ (r / 2 % 8) : (lane % 32) ^ a_swizzle(r % 16);
    a_row[q] = static_cast<const chunk_t*>(p.a) + input_row(r) * achunks;
  }
  const int as_load = kQ ? wv % (FR == 4 ? 2 : 1) : 0;
  int my_token = static_cast<int>(threadIdx.x) < nrows ? p.src[row0 + threadIdx.x] : 0;
  const uint32_t* as_row = nullptr;
  if constexpr (kQ) as_row = reinterpret_cast<const uint32_t*>(p.a_scales + input_row((as_load * 32 + lane / 2) % (16 * FR)) * kb);
  asm volatile("" : "+v"(my_token));

  // weight row of staged row r: gated, 64 gate rows and the 64 up rows that meet them; rows past the
  // last repeat it: they reach only results never stored
  auto weight_row = [&](int r) {
    int j;
    if (p.gated) {
      const int f = col0 + r % 64;
      j = (f < p.n ? f : p.n - 1) + (r >= 64 ? p.n : 0);
    } else {
      j = col0 + r < p.n ? col0 + r : p.n - 1;
    }
    return static_cast<size_t>(x) * p.nz + j;
  };
  // codes: load q of wave wv fills staged rows 8 (4 q + wv) .. + 7, slot lane % 8 of staged row R with
  // piece slot ^ (R / 2 % 8)
  const int b_piece = (lane % 8) ^ (4 * (wv % 2) + lane / 16);
  const chunk_t* b_row[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    b_row[q] = static_cast<const chunk_t*>(p.w) + weight_row((q * 4 + wv) * 8 + lane / 8) * kb;
  // scales: two words a row
  const uint32_t* bs_row = reinterpret_cast<const uint32_t*>(p.w_scales + weight_row(wv * 32 + lane / 2) * kb);
  auto issue_b = [&](int u) __attribute__((always_inline)) {
    char* st = lds + (u % S) * Lds::kStage;
    const int at = u * 8 + b_piece < kb ? u * 8 + b_piece : 0;  // past the row's end: any codes, zeros meet them
#pragma unroll
    for (int q = 0; q < 4; ++q)
      __builtin_amdgcn_global_load_lds(static_cast<const void*>(b_row[q] + at),
                                       (lds_void_t*)(st + Lds::kB + (q * 4 + wv) * 1024), 16, 0, 0);
    // past the row's end: its first word, set to scales of 1 once landed
    const int word = 2 * u + lane % 2 < kb / 4 ? 2 * u + lane % 2 : 0;
    __builtin_amdgcn_global_load_lds(static_cast<const void*>(bs_row + word), (lds_void_t*)(st + Lds::kBScales + wv * 256), 4, 0, 0);
  };
  constexpr int kPieces = kQ ? 8 : 32;                 // of a stage of a row
  auto issue_a = [&](int u) __attribute__((always_inline)) {
    char* st = lds + (u % S) * Lds::kStage;
#pragma unroll
    for (int q = 0; q < Lds::kALoads; ++q) {
      const int at = u * kPieces + a_piece[q] < achunks ? u * kPieces + a_piece[q] : 0;  // past the end: cleared once landed
      __builtin_amdgcn_global_load_lds(static_cast<const void*>(a_row[q] + at), (lds_void_t*)(st + a_load[q] * 1024), 16, 0, 0);
    }
    if constexpr (kQ) {
      const int word = 2 * u + lane % 2 < kb / 4 ? 2 * u + lane % 2 : 0;
      __builtin_amdgcn_global_load_lds(static_cast<const void*>(as_row + word), (lds_void_t*)(st + Lds::kA + as_load * 256), 4, 0, 0);
    }
  };
#pragma unroll
  for (int u = 0; u < S - 1; ++u) {
    if (u < nu) {  // uniform
      issue_b(u);
      issue_a(u);
    }
  }

  int* row_token = reinterpret_cast<int*>(lds + Lds::kRows);
  float* row_weight = reinterpret_cast<float*>(lds + Lds::kRows + 16 * FR * 4);
  if (static_cast<int>(threadIdx.x) < nrows) {
    row_token[threadIdx.x] = my_token;
    row_weight[threadIdx.x] = route_weight_wide(p, row0 + threadIdx.x, my_token);
  }

  f32x4_t acc[FR][2];
#pragma unroll
  for (int i = 0; i < FR; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  const int lrow = lane & 15, a_swz = a_swizzle(lrow);
  const int word_at = wv * 32 + lrow;  // staged weight row of this lane's first fragment
  for (int u = 0; u < nu; ++u) {
    // stage u has landed; up to S - 2 later ones may be in flight
    if (u + S - 2 < nu) __builtin_amdgcn_s_waitcnt(wait_vm((S - 2) * Lds::kLoads));
    else __builtin_amdgcn_s_waitcnt(wait_vm(0));
    char* st = lds + (u % S) * Lds::kStage;
    if ((u + 1) * 8 > kb) {  // only in the last stage
#pragma unroll
      for (int q = 0; q < Lds::kALoads; ++q)
        if (u * kPieces + a_piece[q] >= achunks)
          *reinterpret_cast<chunk_t*>(st + a_load[q] * 1024 + lane * 16) = chunk_t{0u, 0u, 0u, 0u};
      // any codes times other blocks' scales could pass bf16's range, and zeros then make no zero of them
      if (2 * u + lane % 2 >= kb / 4) *reinterpret_cast<uint32_t*>(st + Lds::kBScales + wv * 256 + lane * 4) = 0x7f7f7f7fu;
      __builtin_amdgcn_s_waitcnt(kWaitLdsOnly);
    }
    stage_barrier();  // and every wave has read out the stage before it
    if (u + S - 1 < nu) {
      issue_b(u + S - 1);
      issue_a(u + S - 1);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      chunk_t codes[2];
      uint32_t sb[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = word_at + 16 * j;
        codes[j] = *reinterpret_cast<const chunk_t*>(st + Lds::kB + r * 128 + (((4 * h + grp) ^ (r / 2 % 8)) << 4));
        sb[j] = *reinterpret_cast<const uint32_t*>(st + Lds::kBScales + r * 8 + 4 * h) >> (8 * grp);
      }
      if constexpr (kQ) {
#pragma unroll
        for (int i = 0; i < FR; ++i) {
          const int r = 16 * i + lrow;
          const chunk_t a = *reinterpret_cast<const chunk_t*>(st + r * 128 + (((4 * h + grp) ^ (r / 2 % 8)) << 4));
          const uint32_t sa = *reinterpret_cast<const uint32_t*>(st + Lds::kA + r * 8 + 4 * h) >> (8 * grp);
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = mfma_mx4(codes[j], sb[j], a, sa, acc[i][j]);
        }
      } else {
        chunk_t a[FR][4];
#pragma unroll
        for (int i = 0; i < FR; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            a[i][q] = *reinterpret_cast<const chunk_t*>(st + (16 * i + lrow) * 512 + (((4 * (4 * h + grp) + q) ^ a_swz) << 4));
        bool split = false;
        if constexpr (RT == kF16) {
          const bool fit0 = mx4_fits_f16(sb[0] & 255u), fit1 = mx4_fits_f16(sb[1] & 255u);
          split = !__all(fit0 && fit1);
          if (split) split = !__all((fit0 || mx4_zeros(codes[0])) && (fit1 || mx4_zeros(codes[1])));  // uniform
        }
        constexpr int kWide = RT == kF16 ? kF16 : kBF16;
        if (!split) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const chunk_t w = mx4_values8<kWide>(codes[j][q], mx4_scale(sb[j] & 255u));
#pragma unroll
              for (int i = 0; i < FR; ++i) acc[i][j] = mfma_16x16x32<kWide>(w, a[i][q], acc[i][j]);
            }
        } else {
#pragma unroll
          for (int i = 0; i < FR; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              chunk_t hi, lo;
              split_f16(a[i][q], hi, lo);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const chunk_t w = mx4_values8<kBF16>(codes[j][q], mx4_scale(sb[j] & 255u));
                acc[i][j] = mfma_16x16x32<kBF16>(w, lo, acc[i][j]);
                acc[i][j] = mfma_16x16x32<kBF16>(w, hi, acc[i][j]);
              }
            }
        }
      }
    }
  }

  __syncthreads();  // the sums reuse the stages
#pragma unroll
  for (int i = 0; i < FR; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      *reinterpret_cast<f32x4_t*>(lds + (16 * i + lrow) * kMsPitch + (wv * 32 + 16 * j + 4 * grp) * 4) = acc[i][j];
  __syncthreads();
  const int pieces = out_cols / 8;                     // 16, or gated 8: a block's four threads are neighbours
  for (int i = threadIdx.x; i < nrows * pieces; i += kMsThreads) {
    const int row = i / pieces, c8 = 8 * (i % pieces), c = col0 + c8;
    if (c >= p.n) continue;
    float v[8], u[8];
    const float* at = reinterpret_cast<const float*>(lds + row * kMsPitch) + c8;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      v[q] = at[q];
      u[q] = p.gated ? at[64 + q] : 0.0f;
    }
    const int t = row_token[row];
    const float w = row_weight[row];
    finish8_mx4<DT>(p, x, row0 + row, t, w, c, v, u);
  }
}

template <int RT, int DT, int FR, int S>
static hipError_t launch_stages(const Mx4Act& p, int col_blocks, int64_t grid, hipStream_t stream) {
  static std::atomic<uint64_t> done{0};
  auto kern = mx4_stream_kernel<RT, DT, FR, S>;
  constexpr int kBytes = MsLds<RT, FR, S>::kBytes;
  const hipError_t err = allow_lds(reinterpret_cast<const void*>(kern), kBytes, done);
  if (err != hipSuccess) return err;
  kern<<<static_cast<unsigned>(grid), kMsThreads, kBytes, stream>>>(p, col_blocks, static_cast<int>(grid) - kZeroBlocks);
  return hipGetLastError();
}

template <int RT, int DT, int FR>
static hipError_t launch(const Mx4Act& p, int col_blocks, int64_t grid, hipStream_t stream) {
  return p.m <= kMsShort && grid - kZeroBlocks > kMsCus ? launch_stages<RT, DT, FR, ms_stages(RT, FR, true)>(p, col_blocks, grid, stream)
                                                        : launch_stages<RT, DT, FR, ms_stages(RT, FR, false)>(p, col_blocks, grid, stream);
}

template <int RT, int DT>
static hipError_t launch_rows(const Mx4Act& p, int few, int col_blocks, int64_t grid, hipStream_t stream) {
  if (few == 1) return launch<RT, DT, 1>(p, col_blocks, grid, stream);
  if constexpr (RT == kMx4)
    if (few == 4) return launch<RT, DT, 4>(p, col_blocks, grid, stream);
  return launch<RT, DT, 2>(p, col_blocks, grid, stream);
}

hipError_t launch_mx4_stream(const Mx4Act& p, int dtype, int few, int col_blocks, int64_t grid, hipStream_t stream) {
  if (p.a_scales != nullptr)
    return dtype == kBF16 ? launch_rows<kMx4, kBF16>(p, few, col_blocks, grid, stream)
                          : launch_rows<kMx4, kF16>(p, few, col_blocks, grid, stream);
  return dtype == kBF16 ? launch_rows<kBF16, kBF16>(p, few, col_blocks, grid, stream)
                        : launch_rows<kF16, kF16>(p, few, col_blocks, grid, stream);
}

}  // namespace moe
