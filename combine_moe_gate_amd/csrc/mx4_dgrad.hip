// Input-row gradient of the products with microscaled 4-bit weights, on gfx950 matrix cores.
//
// For each placed row r of expert x: out[r] = a[r] @ W[x], a the 16-bit gradient rows [rows, nz], W
// [nz, m] the values the codes stand for. The sum runs along the weights' rows, each with scales of
// its own, so the weights are widened on their way to LDS: to bf16, which is exact, or for f16 gradients
// to f16, exact for scales from 2^-23 to 2^13. A tile that met others, over values that are not zeros, is
// formed again from gradients in two parts (split_f16) and bf16 weights, straight from memory: slower, and
// in few registers.
// Gradient rows that come in two bf16 parts are multiplied part by part, the second's steps after the
// first's, on the same weights: twice the steps. Results are rounded to 16 bits or stay float32.
//
// Tiles of up to 256 rows by 256 input features, eight waves, as in mx4_tile.hip: a step is 64 weight
// rows. Each thread has one block of 32 weights of a step: loaded two steps ahead, widened and written
// to LDS under the step before its own (64-byte pieces, their 16-byte parts in an order that keeps the
// sixteen lanes of a write on different banks), and read through LDS's transposing reads. Gradient rows
// go to LDS directly.
//
// Measured, 49152 routes, 64 experts: 2816 -> 2048 561 us and 2048 -> 1408 326 us (1.01 and 0.87 PFLOP/s;
// the product with bf16 weights takes 600 and 370); rows in parts, to float32, 1071 and 639. Bound by
// the main loop, matrix units busy 38 to 44%: its matrix instruction alone reaches 1.95.
#include <atomic>

#include "mx4_product.h"

namespace moe {

constexpr int kMdThreads = 512;
constexpr int kMdUnits = 8;                        // a tile's most units of 32 rows
constexpr int kMdBN = 256;                         // input features per tile
constexpr int kMdBand = 8;                         // row-blocks per band of the tile order
constexpr int kMdRowBytes = 128;                   // a staged gradient row: 64 elements
constexpr int kMdAStage = 32 * kMdUnits * kMdRowBytes, kMdBStage = 64 * kMdBN * 2;
constexpr int kMdB = 2 * kMdAStage;
constexpr int kMdVotes = kMdB + 2 * kMdBStage;
constexpr int kMdLds = kMdVotes + 32;
constexpr int kMdSlabPitch = 64 * 4 + 16;          // bytes per row of a wave's 16 x 64 float32 slab
static_assert(8 * 2 * 16 * kMdSlabPitch <= kMdVotes, "the slabs reuse the stages");

// Eight results. Of 16-bit gradient rows they are float32 or of the same type; of rows in parts, of any.
template <int DT, int PARTS>
__device__ __forceinline__ void mx4_dgrad_store(const Mx4Dgrad& p, size_t at, const float (&v)[8]) {
  if (p.out_type == DT) *reinterpret_cast<chunk_t*>(static_cast<uint16_t*>(p.out) + at) = pack<DT>(v);
  else if (p.out_type == kF32) store8<DT>(p.out, at, true, v);
  else if (PARTS == 2) *reinterpret_cast<chunk_t*>(static_cast<uint16_t*>(p.out) + at) = pack<kF16>(v);
}

// A tile of 32 FM rows; false if it is left to mx4_dgrad_split (f16 alone).
template <int DT, int PARTS, int FM>
__device__ __forceinline__ bool mx4_dgrad_body(const Mx4Dgrad& p, const UnitTile& tc, char* lds) {
  constexpr int FN = 4;
  // A step's products in order: (k32 half, row tile), 2 FM slots of FN MFMAs, cut into groups of up to
  // four slots whose fragments are read together; the last group lies in the second half.
  constexpr int kSlots = 2 * FM, kGroups = FM <= 4 ? 2 : (kSlots + 3) / 4;
  auto first_slot = [](int g) constexpr { return g * kSlots / kGroups; };
  constexpr int kALoads = (4 * FM + 7) / 8;            // direct-to-LDS loads of 8 rows, per wave
  const int lane = lane_id(), wv = wave_in_block(), grp = lane >> 4, tid = threadIdx.x;
  const int wm = wv / 4, wn = wv % 4;
  const int row0 = tc.offset + tc.unit0 * 32;
  const int rem = tc.rows - tc.unit0 * 32;
  const int nrows = rem < 32 * FM ? rem : 32 * FM;
  const int col0 = tc.cb * kMdBN;
  const int K = p.m, achunks = K / 8, kb = p.n / kMx4Block;
  const int part_steps = (achunks + 7) / 8, nk = part_steps * PARTS;
  auto in_part = [&](int kt) { return PARTS == 1 || kt < part_steps ? kt : kt - part_steps; };  // a step's number in its part

  // this thread's block of a step: weight row tid / 8, input features 32 (tid % 8) .. + 31; past the
  // last feature any block (its sums are not stored), past the last row one that is all finite
  const int b_row = tid / 8, b_col = tid % 8;
  const int my_block = col0 / kMx4Block + b_col < kb ? col0 / kMx4Block + b_col : kb - 1;
  const size_t w0 = static_cast<size_t>(tc.expert) * K * kb + my_block;
  chunk_t breg;
  uint32_t sreg;
  uint32_t reach = 0;  // f16: the largest distance from the least scale that fits
  auto load_b = [&](int kt) __attribute__((always_inline)) {
    const int r = in_part(kt) * 64 + b_row;
    const size_t at = w0 + static_cast<size_t>(r < K ? r : K - 1) * kb;
    breg = static_cast<const chunk_t*>(p.w)[at];
    sreg = p.w_scales[at];
  };
  // the staged row's 16-byte piece i lies at slot i ^ swizzle(row)
  auto kn_swizzle = [](int row) { return 4 * (row % 4) + 2 * ((row >> 3) & 1); };
  const int turn = (b_col >> 2) | ((b_row & 1) << 1);  // part q goes out as q ^ turn
  const int b_to = b_row * 512 + (((4 * b_col) ^ kn_swizzle(b_row) ^ turn) << 4);
  auto write_b = [&](int kt) __attribute__((always_inline)) {
    const uint32_t E = in_part(kt) * 64 + b_row < K ? sreg : 127u;
    const float s = mx4_scale(E);
    reach = mx4_f16_reach(E) > reach ? mx4_f16_reach(E) : reach;
    chunk_t c = breg;
    c = turn & 1 ? chunk_t{c.y, c.x, c.w, c.z} : c;
    c = turn & 2 ? chunk_t{c.z, c.w, c.x, c.y} : c;
    char* st = lds + kMdB + (kt % 2) * kMdBStage;
#pragma unroll
    for (int q = 0; q < 4; ++q) *reinterpret_cast<chunk_t*>(st + (b_to ^ (q << 4))) = mx4_values8<DT>(c[q], s);
  };
  load_b(0);

  // slot lane % 8 of staged row R takes piece slot ^ (R / 2 % 8); the loads' first rows are
  // multiples of 8, so R / 2 % 8 = 4 (load % 2) + lane / 16. Rows past the segment repeat its first.
  const int chunk = (lane % 8) ^ (4 * (wv % 2) + lane / 16);
  const chunk_t* a_row[kALoads];
#pragma unroll
  for (int q = 0; q < kALoads; ++q) {
    const int r = (q * 8 + wv) * 8 + lane / 8;
    a_row[q] = static_cast<const chunk_t*>(p.a) + static_cast<size_t>(row0 + (r < nrows ? r : 0)) * (achunks * PARTS);
  }
  auto issue_a = [&](int kt) __attribute__((always_inline)) {
    const int piece = in_part(kt) * 8 + chunk;
    const int at = (piece < achunks ? piece : 0) + (PARTS == 1 || kt < part_steps ? 0 : achunks);  // past the row's end: cleared once landed
#pragma unroll
    for (int q = 0; q < kALoads; ++q)
      if (q * 8 + wv < 4 * FM)  // uniform
        __builtin_amdgcn_global_load_lds(static_cast<const void*>(a_row[q] + at),
                                         (lds_void_t*)(lds + (kt % 2) * kMdAStage + (q * 8 + wv) * 1024), 16, 0, 0);
  };
  issue_a(0);
  if (nk > 1) issue_a(1);
  __builtin_amdgcn_sched_barrier(0);
  write_b(0);
  __builtin_amdgcn_sched_barrier(0);
  if (nk > 1) load_b(1);  // the newest loads at the first publish
  __builtin_amdgcn_sched_barrier(0);

  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // row fragments: row lane % 16 of a 16-row MFMA tile, piece 4 half + grp at slot piece ^ (row / 2 % 8)
  const int frag_swz = (lane & 15) >> 1;
  const int a_base = wm * 16 * FM * kMdRowBytes + (lane & 15) * kMdRowBytes;
  auto read_a = [&](int kt, int g, chunk_t (&f)[4]) __attribute__((always_inline)) {  // the fragments of group g
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int slot = first_slot(g) + q;
      if (slot < first_slot(g + 1))
        f[q] = *reinterpret_cast<const chunk_t*>(lds + (kt % 2) * kMdAStage + a_base + (slot % FM) * 16 * kMdRowBytes +
                                                 (((4 * (slot / FM) + grp) ^ frag_swz) << 4));
    }
  };
  // gfx950's transposing LDS read hands lane i of each 16-lane group column i of the four K rows its
  // lanes point at, lane i at row i / 4, columns 4 (i % 4) .. + 3; two reads make the lane's eight K
  // rows. The swizzle puts the 32 lanes served together on 32 different 8-byte pieces of the 256-byte
  // bank row.
  const uint32_t lds_at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void_t*)lds));
  const int kn_at = (8 * grp + ((lane & 15) >> 2)) * 512 + (lane & 1) * 8;
  const int kn_slot = (8 * wn + ((lane & 3) >> 1)) ^ kn_swizzle(8 * grp + ((lane & 15) >> 2));
  auto read_b = [&](int kt, int half, chunk_t (&b)[FN]) __attribute__((always_inline)) {
    const uint32_t st = lds_at + kMdB + (kt % 2) * kMdBStage + half * 32 * 512 + kn_at;
    uint32_t at[4];
#pragma unroll
    for (int j = 0; j < FN; ++j) at[j] = st + ((kn_slot ^ (2 * j)) << 4);
    read_tr16(at, b);
  };
  // step kt is whole in LDS and every wave has read out the step before it; the loads of a block for
  // the step after it may be in flight (two, the newest)
  auto publish = [&](int kt) __attribute__((always_inline)) {
    if (kt + 1 < nk) __builtin_amdgcn_s_waitcnt(wait_vm(2) & ~0xF00);
    else __builtin_amdgcn_s_waitcnt(wait_vm(0) & ~0xF00);
    if ((in_part(kt) + 1) * 8 > achunks) {
      if (in_part(kt) * 8 + chunk >= achunks) {
#pragma unroll
        for (int q = 0; q < kALoads; ++q)
          if (q * 8 + wv < 4 * FM)
            *reinterpret_cast<chunk_t*>(lds + (kt % 2) * kMdAStage + (q * 8 + wv) * 1024 + lane * 16) = chunk_t{0u, 0u, 0u, 0u};
      }
      __builtin_amdgcn_s_waitcnt(kWaitLdsOnly);
    }
    stage_barrier();
  };

  publish(0);
  chunk_t fa[2][4], fb[2][FN];
  read_a(0, 0, fa[0]);
  read_b(0, 0, fb[0]);

  // Under each group's MFMAs the next group's fragments are read, and with the group before the first
  // one of the second half the weights' of that half. After the first group's MFMAs the next step's
  // weights are written to LDS and the loads of those after them start. Before the last group's MFMAs
  // the next step is published (by then every fragment of this step is in registers), the loads of the
  // rows of the step after it start, and the next step's first fragments are read; after the last step
  // these find old contents, which nothing uses.
  for (int kt = 0; kt < nk; ++kt) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      __builtin_amdgcn_s_waitcnt(kWaitLdsOnly);  // this group's fragments have landed
      __builtin_amdgcn_sched_barrier(0);
      if (g + 1 < kGroups) {
        read_a(kt, g + 1, fa[(g + 1) % 2]);
        if (first_slot(g + 1) <= FM && first_slot(g + 2) > FM) read_b(kt, 1, fb[1]);
      } else {
        if (kt + 1 < nk) {
          publish(kt + 1);
          if (kt + 2 < nk) issue_a(kt + 2);
        }
        __builtin_amdgcn_sched_barrier(0);
        read_a(kt + 1, 0, fa[(g + 1) % 2]);
        read_b(kt + 1, 0, fb[0]);  // the last group is all of the second half
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int slot = first_slot(g) + q;
        if (slot < first_slot(g + 1)) {
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[slot % FM][j] = mfma_16x16x32<DT>(fb[slot / FM][j], fa[g % 2][q], acc[slot % FM][j]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if (g == 0 && kt + 1 < nk) {
        write_b(kt + 1);
        if (kt + 2 < nk) load_b(kt + 2);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (kGroups % 2 != 0) {
#pragma unroll
      for (int q = 0; q < 4; ++q) fa[0][q] = fa[1][q];
    }
  }

  if constexpr (DT == kF16) {
    int* votes = reinterpret_cast<int*>(lds + kMdVotes);
    auto vote = [&](bool mine) {
      if (lane == 0) votes[wv] = mine;
      __syncthreads();
      int any = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) any |= votes[i];
      return __builtin_amdgcn_readfirstlane(any) != 0;
    };
    if (vote(__any(reach > kMx4F16Reach))) {
      // the sums are right if only zeros lie under the scales that do not fit: a thread a weight row looks at
      // the tile's blocks. 65536 routes, 128 experts, 4096 -> 4096: 2.03 ms without zeros, 2.03 with a block of
      // them in 256 weight rows, 2.21 with a quarter of the rows zero; with the codes looked at in the loop 2.46.
      const int first = col0 / kMx4Block, count = kb - first < kMdBN / kMx4Block ? kb - first : kMdBN / kMx4Block;
      bool bad = false;
      for (int r = tid; r < K; r += kMdThreads)
        bad = bad || mx4_misfits_f16(static_cast<const chunk_t*>(p.w), p.w_scales, (static_cast<size_t>(tc.expert) * K + r) * kb + first, count);
      __syncthreads();  // every wave has read the votes
      if (vote(__any(bad))) return false;
    }
  }
  __syncthreads();

  // each 16-row tile's sums through one of the wave's two slabs: lane l holds row l % 16, features
  // 16 j + 4 (l / 16) .. + 3 of its 64; it takes back row l / 4, features 8 (l % 4) .. + 7 of each 32
  char* slabs = lds + wv * 2 * 16 * kMdSlabPitch;
  const int below = nrows - wm * 16 * FM;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    if (i * 16 < below) {  // uniform
      char* slab = slabs + (i % 2) * 16 * kMdSlabPitch;
#pragma unroll
      for (int j = 0; j < FN; ++j)
        *reinterpret_cast<f32x4_t*>(slab + (lane & 15) * kMdSlabPitch + j * 64 + grp * 16) = acc[i][j];
      const float* back = reinterpret_cast<const float*>(slab + (lane >> 2) * kMdSlabPitch) + 8 * (lane & 3);
      const int row = wm * 16 * FM + i * 16 + (lane >> 2);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = back[32 * h + q];
        const int c = col0 + wn * 64 + 32 * h + 8 * (lane & 3);
        if (row < nrows && c < p.n) mx4_dgrad_store<DT, PARTS>(p, static_cast<size_t>(row0 + row) * p.n + c, v);
      }
    }
  }
  return true;
}

// A tile whose weights f16 does not hold, 16 rows by 16 features of a wave at a time: 56 ms where the loop takes
// 2.03, were all tiles such.
__device__ __forceinline__ void mx4_dgrad_split(const Mx4Dgrad& p, const UnitTile& tc) {
  const int lane = lane_id(), wv = wave_in_block(), grp = lane >> 4, lrow = lane & 15;
  const int row0 = tc.offset + tc.unit0 * 32;
  const int rem = tc.rows - tc.unit0 * 32;
  const int nrows = rem < 32 * tc.units ? rem : 32 * tc.units;
  const int K = p.m, kb = p.n / kMx4Block;
  const uint8_t* codes = static_cast<const uint8_t*>(p.w);
  for (int item = wv; item < 2 * tc.units * (kMdBN / 16); item += kMdThreads / kWave) {
    const int first = item / (kMdBN / 16) * 16, col = tc.cb * kMdBN + item % (kMdBN / 16) * 16;
    if (first >= nrows || col >= p.n) continue;  // uniform; p.n is a multiple of 32
    const int row = first + lrow;
    const chunk_t* a_row = static_cast<const chunk_t*>(p.a) + static_cast<size_t>(row0 + (row < nrows ? row : 0)) * (K / 8);
    const int c = col + lrow;
    f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k = 0; k < K; k += 32) {
      const int k8 = k + 8 * grp;  // this lane's eight weight rows; K is a multiple of 8
      chunk_t a = {0u, 0u, 0u, 0u}, w = a, hi, lo;
      if (k8 < K) {
        a = a_row[k8 / 8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const size_t block = (static_cast<size_t>(tc.expert) * K + k8 + i) * kb + c / kMx4Block;
          const uint32_t code = (codes[block * 16 + c % kMx4Block / 2] >> (4 * (c % 2))) & 15u;
          const f32x2_t v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, mx4_scale(p.w_scales[block]), 0);
          w[i / 2] |= (__float_as_uint(v[0]) >> 16) << (16 * (i % 2));  // a bf16 value
        }
      }
      split_f16(a, hi, lo);
      acc = mfma_16x16x32<kBF16>(w, lo, acc);
      acc = mfma_16x16x32<kBF16>(w, hi, acc);
    }
    const size_t at = static_cast<size_t>(row0 + row) * p.n + col + 4 * grp;
    if (row < nrows) {
      if (p.out_type == kF32) *reinterpret_cast<f32x4_t*>(static_cast<float*>(p.out) + at) = acc;
      else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = uint2{narrow2<kF16>(acc[0], acc[1]), narrow2<kF16>(acc[2], acc[3])};
    }
  }
}

template <int DT, int PARTS>
__global__ __launch_bounds__(kMdThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void mx4_dgrad_kernel(
    Mx4Dgrad p, int col_blocks, int tile_grid) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  if (static_cast<int>(blockIdx.x) >= tile_grid) {
    each_unfilled(p, blockIdx.x - tile_grid, gridDim.x - tile_grid, [&](int r) {
      const size_t chunks = p.n / (p.out_type == kF32 ? 4 : 8);
      chunk_t* o = static_cast<chunk_t*>(p.out) + static_cast<size_t>(r) * chunks;
      for (size_t c = lane_id(); c < chunks; c += kWave) o[c] = chunk_t{0u, 0u, 0u, 0u};
    });
    return;
  }
  const UnitTile tc = unit_tile<kMdUnits>(blockIdx.x, p.e, p.kept, p.offsets, col_blocks, kMdBand);
  if (tc.expert < 0) return;
  bool done = true;
  switch (tc.units) {
    case 1: done = mx4_dgrad_body<DT, PARTS, 1>(p, tc, lds); break;
    case 2: done = mx4_dgrad_body<DT, PARTS, 2>(p, tc, lds); break;
    case 3: done = mx4_dgrad_body<DT, PARTS, 3>(p, tc, lds); break;
    case 4: done = mx4_dgrad_body<DT, PARTS, 4>(p, tc, lds); break;
    case 5: done = mx4_dgrad_body<DT, PARTS, 5>(p, tc, lds); break;
    case 6: done = mx4_dgrad_body<DT, PARTS, 6>(p, tc, lds); break;
    case 7: done = mx4_dgrad_body<DT, PARTS, 7>(p, tc, lds); break;
    default: done = mx4_dgrad_body<DT, PARTS, 8>(p, tc, lds); break;
  }
  if constexpr (DT == kF16)
    if (!done) mx4_dgrad_split(p, tc);
}

static int64_t mx4_dgrad_grid(const LayoutView& L, int m, int64_t* col_blocks) {
  *col_blocks = (static_cast<int64_t>(m) + kMdBN - 1) / kMdBN;
  const int64_t tiles = L.s == 0 ? 0 : row_tiles(L, 32 * kMdUnits) * *col_blocks;
  return (tiles + kXcds - 1) / kXcds * kXcds + kZeroBlocks;
}

bool mx4_dgrad_fits(const LayoutView& L, int m) {
  int64_t cb;
  return mx4_dgrad_grid(L, m, &cb) <= most_workgroups(kMdThreads);
}

template <int DT, int PARTS>
static hipError_t launch_dt(const LayoutView& L, const Mx4Dgrad& p, hipStream_t stream) {
  static std::atomic<uint64_t> done{0};
  auto kern = mx4_dgrad_kernel<DT, PARTS>;
  const hipError_t err = allow_lds(reinterpret_cast<const void*>(kern), kMdLds, done);
  if (err != hipSuccess) return err;
  int64_t cb;
  const int64_t grid = mx4_dgrad_grid(L, p.n, &cb);
  kern<<<static_cast<unsigned>(grid), kMdThreads, kMdLds, stream>>>(p, static_cast<int>(cb),
                                                                   static_cast<int>(grid) - kZeroBlocks);
  return hipGetLastError();
}

hipError_t launch_mx4_dgrad(const LayoutView& L, const Mx4Dgrad& p, int dtype, hipStream_t stream) {
  if (p.rows == 0) return hipSuccess;
  if (p.parts == 2) return launch_dt<kBF16, 2>(L, p, stream);
  return dtype == kBF16 ? launch_dt<kBF16, 1>(L, p, stream) : launch_dt<kF16, 1>(L, p, stream);
}

}  // namespace moe
