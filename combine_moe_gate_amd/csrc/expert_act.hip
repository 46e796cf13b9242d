// The experts' products with bias, activation (plain or gated), route weight and residual
// applied to the float32 sums before their one rounding, on gfx950 matrix cores.
//
// For each placed row r of expert x, with z = A(r) @ W[x]^T + b[x] (A(r) = a[src[r]] or
// a[r]):   out[r] = w_r u + residual(r),   u = act(z), or act(z_gate) * z_up for a gated
// projection, whose weights hold the n gate rows, then the n up rows. Kept apart from the
// plain product, the activation would read and write every [rows, n] value again.
//
// Two kernels, chosen by the rows an expert has on average and by the workgroups there would
// be (act_shape() below):
//
// Tiles (long segments; bound by the matrix cores). A workgroup of eight waves, 2 along the
// rows by 4 along the columns, multiplies up to 288 rows by 256 weight rows of one expert
// (v_mfma_f32_16x16x32, float32 accumulators). A segment of R rows is cut into the fewest
// tiles of at most 288 rows, of heights that differ by at most 32: tiles of a fixed 256
// would leave a segment of 530 rows a third tile of 18, and a quarter of a uniform batch's
// products on rows that are not there; this way fewer than 32 rows per expert are. The
// height is a multiple of 32 rows (FM 16-row MFMA tiles for each of the two waves along the
// rows), and the main loop is compiled for each of the nine. Operands go to LDS directly
// (64-element K steps, two stages, XOR-swizzled: conflict-free 16-byte fragment reads, whole
// 128-byte lines from memory). Fragments are read a group of up to four MFMA row tiles ahead
// of their use, across the K step's border: the next stage is published, by the step's one
// barrier, before its last group's MFMAs, and the loads of the stage after it start there.
// For a gated projection a wave's 64 weight rows are 32 gate rows and the 32 up rows that
// meet them, so both products of an output are in one wave. The finished sums leave through
// a piece of LDS of the wave's own, 16 rows at a time, and come back as eight consecutive
// features per lane: bias, residual and results then move as 16-byte pieces.
//
// Few rows (decoding; bound by reading the weights). A workgroup of four waves multiplies
// up to 16 F rows by 16 FB weight rows, each wave a quarter of the K steps: weights go from
// memory straight to the registers the MFMA reads, several steps ahead (nothing is reused,
// so LDS would only add a stop), and the four partial sums meet in LDS.
//
// The input-row gradient runs the tiles on the same weights, which are [K][N] to it: pieces
// of 64 K rows by 256 features are staged as they lie and read through LDS's transposing
// reads, and a tile has at most 256 rows (nine units would spill). 49152 rows of 64 experts
// from 2816 to 2048 features take 600 us, from 2048 to 1408 370; moe_expert_gemm_dgrad's
// kernel, with tiles of a fixed 256 rows, 738 and 503.
//
// Measured (bf16, random routing): 65536 rows of 128 experts by 4096 x 4096 (gated, 2.2
// TFLOP) with bias and kept pre-activations 2.05 ms, 1070 TFLOP/s, the matrix cores busy in 54%
// of the cycles; one dense expert 1250 TFLOP/s, where the same loop without loads from memory
// reaches 1530 and a library product of that size 1340. 32768 rows by 2816 x 2816, weights 2.0
// of 2.3 GB read: 0.57 ms, 4.2 TB/s, 45%. One token, 8 experts of 128, 201 MB of weights: 41 us,
// 4.9 TB/s of them, where loads alone reach 6.8.
#include <atomic>

#include "expert_act.h"

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

// ---------------------------------------------------------------------------------
// tiles

constexpr int kActUnits = 9;                       // a tile's most units of 32 rows
constexpr int kActBM = 32 * kActUnits;
constexpr int kActBN = 256;                        // weight rows per tile
constexpr int kActThreads = 512;
constexpr int kActBand = 8;                        // row-blocks per band of the tile order
constexpr int kActRowBytes = 128;                  // a staged row: 64 elements
constexpr int kActAStage = kActBM * kActRowBytes, kActBStage = kActBN * kActRowBytes;
constexpr int kActStage = kActAStage + kActBStage;
constexpr int kSlabPitch = 64 * 4 + 16;            // bytes per row of a wave's 16 x 64 float32 slab
constexpr int kActLds = 2 * kActStage + kActBM * 8;
static_assert(8 * 2 * 16 * kSlabPitch <= 2 * kActStage, "the slabs reuse the stages");

// The most units of a tile: with [K][N] weights nine would not fit the registers.
template <bool KN>
constexpr int act_units = KN ? kActUnits - 1 : kActUnits;

// The tile's products and its epilogue, for a height of 32 FM rows. KN: weights stored
// [K][N] per expert (the input gradient).
template <int DT, bool KN, int FM>
__device__ __forceinline__ void act_tile_body(const ExpertAct& p, const UnitTile& tc, char* lds) {
  constexpr int FN = 4;
  // A K step's products in order: (k32 half, row tile), 2 FM slots of FN MFMAs, cut into
  // groups of up to four slots whose fragments are read together; the last group lies in
  // the second half.
  constexpr int kSlots = 2 * FM, kGroups = FM <= 4 ? 2 : (kSlots + 3) / 4;
  auto first_slot = [](int g) constexpr { return g * kSlots / kGroups; };
  constexpr int kALoads = (4 * FM + 7) / 8;            // direct-to-LDS loads of 8 rows, per wave
  const int lane = lane_id(), wv = wave_in_block();
  const int wm = wv / 4, wn = wv % 4;
  const int x = tc.expert;
  const int row0 = tc.offset + tc.unit0 * 32;
  const int rem = tc.rows - tc.unit0 * 32;
  const int nrows = rem < 32 * FM ? rem : 32 * FM;
  const int out_cols = p.gated ? kActBN / 2 : kActBN;
  const int col0 = tc.cb * out_cols;                   // first output feature
  const int kchunks = p.m / 8, nk = (p.m + 63) / 64;

  // staged row and chunk of each load of this lane. Rows past the segment repeat its first
  // one and weight rows past the last repeat it: both reach only results never stored.
  const chunk_t* a_row[kALoads];
  const chunk_t* b_row[4];
  const chunk_t* wx = static_cast<const chunk_t*>(p.w) + static_cast<size_t>(x) * p.nz * kchunks;
  const int nchunks = p.n / 8;
  // [K][N]: lane l of a load fills slot l % 32 of staged K row 2 (load) + l / 32 with chunk
  // slot ^ kn_swizzle(row); columns past the last repeat its chunk. A wave's loads are 16 rows
  // apart, which changes neither the swizzle nor the chunk: b_row[0] serves them all.
  auto kn_swizzle = [](int row) { return 4 * (row % 4) + 2 * ((row >> 3) & 1); };
  auto kn_row = [&](int q) { return (q * 8 + wv) * 2 + lane / 32; };
  if constexpr (KN) {
    const int c = col0 / 8 + ((lane % 32) ^ kn_swizzle(kn_row(0)));
    b_row[0] = wx + static_cast<size_t>(kn_row(0)) * nchunks + (c < nchunks ? c : nchunks - 1);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = (q * 8 + wv) * 8 + lane / 8;
      int j;
      if (p.gated) {  // 32 gate rows, then the 32 up rows of the same features
        const int f = col0 + (r / 64) * 32 + r % 32;
        j = (f < p.n ? f : p.n - 1) + (r % 64 >= 32 ? p.n : 0);
      } else {
        j = col0 + r < p.n ? col0 + r : p.n - 1;
      }
      b_row[q] = wx + static_cast<size_t>(j) * kchunks;
    }
  }
  // slot lane % 8 of staged row R takes chunk slot ^ (R / 2 % 8); the loads' first rows are
  // multiples of 8, so R / 2 % 8 = 4 (load % 2) + lane / 16
  const int swz = 4 * (wv % 2) + lane / 16;
  const int chunk = (lane % 8) ^ swz;
  auto chunk_at = [&](int kt) {
    const int kq = kt * 8 + chunk;
    return kq < kchunks ? kq : 0;  // past the row's end: its first chunk, cleared once landed
  };
  auto issue_b = [&](int kt) {
    char* st = lds + (kt % 2) * kActStage + kActAStage;
    if constexpr (KN) {
      const int64_t step = static_cast<int64_t>(kt) * 64 * nchunks;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        int64_t at = step + q * 16 * static_cast<int64_t>(nchunks);
        if ((kt + 1) * 64 > p.m) {  // uniform: K rows past the end load the last one, cleared once landed
          const int over = kt * 64 + kn_row(0) + 16 * q - (p.m - 1);
          if (over > 0) at -= static_cast<int64_t>(over) * nchunks;
        }
        __builtin_amdgcn_global_load_lds(static_cast<const void*>(b_row[0] + at),
                                         (lds_void_t*)(st + (q * 8 + wv) * 1024), 16, 0, 0);
      }
    } else {
      const int at = chunk_at(kt);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        __builtin_amdgcn_global_load_lds(static_cast<const void*>(b_row[q] + at),
                                         (lds_void_t*)(st + (q * 8 + wv) * 1024), 16, 0, 0);
    }
  };
  // the weights' first loads start before the rows' addresses are read from the layout
  issue_b(0);
  if (nk > 1) issue_b(1);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int q = 0; q < kALoads; ++q) {
    const int r = (q * 8 + wv) * 8 + lane / 8;
    const int rr = row0 + (r < nrows ? r : 0);
    a_row[q] = static_cast<const chunk_t*>(p.a) + static_cast<size_t>(p.gather ? p.src[rr] : rr) * kchunks;
  }
  auto issue_a = [&](int kt) {
    char* st = lds + (kt % 2) * kActStage;
    const int at = chunk_at(kt);
#pragma unroll
    for (int q = 0; q < kALoads; ++q)
      if (q * 8 + wv < 4 * FM)  // uniform
        __builtin_amdgcn_global_load_lds(static_cast<const void*>(a_row[q] + at),
                                         (lds_void_t*)(st + (q * 8 + wv) * 1024), 16, 0, 0);
  };
  issue_a(0);
  if (nk > 1) issue_a(1);
  // per tile row: its token and route weight, for the epilogue
  int* row_token = reinterpret_cast<int*>(lds + 2 * kActStage);
  float* row_weight = reinterpret_cast<float*>(lds + 2 * kActStage + kActBM * 4);
  if (static_cast<int>(threadIdx.x) < nrows) {
    const int r = row0 + threadIdx.x;
    const int t = p.src[r];
    row_token[threadIdx.x] = t;
    row_weight[threadIdx.x] = p.route_w != nullptr ? route_weight(p, r, t) : 1.0f;
  }

  auto clear_tail = [&](int kt) {
    char* st = lds + (kt % 2) * kActStage;
    const chunk_t z = {0u, 0u, 0u, 0u};
    const bool past = kt * 8 + chunk >= kchunks;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (KN ? kt * 64 + kn_row(0) + 16 * q >= p.m : past)
        *reinterpret_cast<chunk_t*>(st + kActAStage + (q * 8 + wv) * 1024 + lane * 16) = z;
#pragma unroll
    for (int q = 0; q < kALoads; ++q)
      if (q * 8 + wv < 4 * FM && past) *reinterpret_cast<chunk_t*>(st + (q * 8 + wv) * 1024 + lane * 16) = z;
  };

  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // fragments: row lane % 16 of a 16-row MFMA tile, chunk 4 half + lane / 16, at slot
  // chunk ^ (row / 2 % 8)
  const int frag_row = (lane & 15) * kActRowBytes;
  const int frag_swz = (lane & 15) >> 1;
  const int a_base = wm * 16 * FM * kActRowBytes + frag_row;
  const int b_base = kActAStage + wn * 64 * kActRowBytes + frag_row;
  auto read_a = [&](int kt, int g, chunk_t (&f)[4]) {  // the fragments of group g
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int slot = first_slot(g) + q;
      if (slot < first_slot(g + 1))
        f[q] = *reinterpret_cast<const chunk_t*>(lds + (kt % 2) * kActStage + a_base + (slot % FM) * 16 * kActRowBytes +
                                                 (((4 * (slot / FM) + (lane >> 4)) ^ frag_swz) << 4));
    }
  };
  // [K][N]: gfx950's transposing LDS read hands lane i of each 16-lane group column i of the
  // four K rows its lanes point at, lane i at row i / 4, columns 4 (i % 4) .. + 3; two reads
  // make the lane's eight K rows. The swizzle puts the 32 lanes served together on 32
  // different 8-byte pieces of the 256-byte bank row.
  const uint32_t lds_at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void_t*)lds));
  const int kn_at = (8 * (lane >> 4) + ((lane & 15) >> 2)) * 512 + (lane & 1) * 8;
  const int kn_slot = (8 * wn + ((lane & 3) >> 1)) ^ kn_swizzle(8 * (lane >> 4) + ((lane & 15) >> 2));
  auto read_b = [&](int kt, int half, chunk_t (&b)[FN]) {
    if constexpr (KN) {
      const uint32_t st = lds_at + (kt % 2) * kActStage + kActAStage + half * 32 * 512 + kn_at;
      uint32_t at[4];
#pragma unroll
      for (int j = 0; j < FN; ++j) at[j] = st + ((kn_slot ^ (2 * j)) << 4);
      read_tr16(at, b);
      return;
    }
#pragma unroll
    for (int j = 0; j < FN; ++j)
      b[j] = *reinterpret_cast<const chunk_t*>(lds + (kt % 2) * kActStage + b_base + j * 16 * kActRowBytes +
                                               (((4 * half + (lane >> 4)) ^ frag_swz) << 4));
  };
  // step kt is whole in LDS and every wave has read out the step before it
  auto publish = [&](int kt) {
    __builtin_amdgcn_s_waitcnt(wait_vm(0) & ~0xF00);  // all loads and LDS operations
    if ((kt + 1) * 8 > kchunks) {
      clear_tail(kt);
      __builtin_amdgcn_s_waitcnt(kWaitLdsOnly);
    }
    stage_barrier();
  };

  publish(0);
  chunk_t fa[2][4], fb[2][FN];
  read_a(0, 0, fa[0]);
  read_b(0, 0, fb[0]);

  // Under each group's MFMAs the next group's fragments are read, and with the group before
  // the first one of the second k32 half the weights' of that half. Before the last group's
  // MFMAs the next step is published (by then every fragment of this step is in registers),
  // the loads of the one after it start into this step's stage, and the next step's first
  // fragments are read; after the last step these find old contents, which nothing uses.
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
          if (kt + 2 < nk) {
            issue_b(kt + 2);
            issue_a(kt + 2);
          }
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
    }
    if (kGroups % 2 != 0) {
#pragma unroll
      for (int q = 0; q < 4; ++q) fa[0][q] = fa[1][q];
    }
  }

  // epilogue: each 16-row tile's sums through one of the wave's two slabs. Lane l holds token
  // row l % 16, features 16 j + 4 (l / 16) .. + 3 of its 64; it takes back row l / 4, features
  // 8 (l % 4) .. + 7 of each 32 (gated: the gate's and the up's). The next tile goes through
  // LDS while one is finished.
  __syncthreads();
  char* slabs = lds + wv * 2 * 16 * kSlabPitch;
  const int below = nrows - wm * 16 * FM;
  const int tiles = below <= 0 ? 0 : below < 16 * FM ? (below + 15) / 16 : FM;
  auto pass = [&](int i, float (&v)[8], float (&u)[8]) __attribute__((always_inline)) {
    char* slab = slabs + (i % 2) * 16 * kSlabPitch;
    static_for(std::make_integer_sequence<int, FM>{}, [&](auto ii) __attribute__((always_inline)) {
      if (ii == i) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
          *reinterpret_cast<f32x4_t*>(slab + (lane & 15) * kSlabPitch + j * 64 + (lane >> 4) * 16) = acc[ii][j];
        // the empty asm keeps the branches apart: with their stores folded into one, they
        // would index the accumulators dynamically and so move them to memory
        asm volatile("" ::"i"(decltype(ii)::value) : "memory");
      }
    });
    const float* back = reinterpret_cast<const float*>(slab + (lane >> 2) * kSlabPitch) + 8 * (lane & 3);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      v[q] = back[q];
      u[q] = back[32 + q];
    }
  };
  auto finish = [&](int i, float (&v)[8], float (&u)[8]) __attribute__((always_inline)) {
    const int row = wm * 16 * FM + i * 16 + (lane >> 2);
    if (row >= nrows) return;
    const int r = row0 + row, t = row_token[row];
    const float w = row_weight[row];
    const int c = col0 + wn * (out_cols / 4) + 8 * (lane & 3);
    if (c < p.n) finish8<DT>(p, x, r, t, w, c, v, u);
    if (!p.gated && c + 32 < p.n) finish8<DT>(p, x, r, t, w, c + 32, u, v);
  };
  float v[2][8], u[2][8];
  if (tiles > 0) pass(0, v[0], u[0]);
#pragma unroll 1
  for (int i = 0; i < tiles; i += 2) {  // uniform conditions
    if (i + 1 < tiles) pass(i + 1, v[1], u[1]);
    finish(i, v[0], u[0]);
    if (i + 2 < tiles) pass(i + 2, v[0], u[0]);
    if (i + 1 < tiles) finish(i + 1, v[1], u[1]);
  }
}

template <int DT, bool KN>
__global__ __launch_bounds__(kActThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void expert_act_kernel(
    ExpertAct p, int col_blocks, int tile_grid) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  if (static_cast<int>(blockIdx.x) >= tile_grid) {
    zero_unfilled(p, blockIdx.x - tile_grid, gridDim.x - tile_grid);
    return;
  }
  const UnitTile tc = unit_tile<act_units<KN>>(blockIdx.x, p.e, p.kept, p.offsets, col_blocks, kActBand);
  if (tc.expert < 0) return;
  switch (tc.units) {
    case 1: act_tile_body<DT, KN, 1>(p, tc, lds); break;
    case 2: act_tile_body<DT, KN, 2>(p, tc, lds); break;
    case 3: act_tile_body<DT, KN, 3>(p, tc, lds); break;
    case 4: act_tile_body<DT, KN, 4>(p, tc, lds); break;
    case 5: act_tile_body<DT, KN, 5>(p, tc, lds); break;
    case 6: act_tile_body<DT, KN, 6>(p, tc, lds); break;
    case 7: act_tile_body<DT, KN, 7>(p, tc, lds); break;
    case 8: act_tile_body<DT, KN, 8>(p, tc, lds); break;
    default:
      if constexpr (!KN) act_tile_body<DT, KN, 9>(p, tc, lds);
      break;
  }
}

// ---------------------------------------------------------------------------------
// few rows

constexpr int kFewThreads = 256, kFewWaves = 4;

template <int DT, int F, int FB>
__global__ __launch_bounds__(kFewThreads, F == 4 ? 2 : 4) void expert_act_few_kernel(ExpertAct p, int col_blocks,
                                                                                     int tile_grid) {
  constexpr int kDepth = F == 4 ? 1 : 4;  // K steps of 64 elements in flight per wave
  constexpr int kCols = 16 * FB;                        // weight rows per workgroup
  constexpr int kPitch = kCols * 4 + 16;                // bytes per row of a wave's float32 sums
  extern __shared__ __attribute__((aligned(1024))) char lds[];  // [wave][16 F rows][kPitch]
  if (static_cast<int>(blockIdx.x) >= tile_grid) {
    zero_unfilled(p, blockIdx.x - tile_grid, gridDim.x - tile_grid);
    return;
  }
  const SegmentTile tc =
      segment_tile(blockIdx.x, p.e, p.kept, p.offsets, col_blocks, kActBand, [](int r) { return (r + 16 * F - 1) / (16 * F); });
  const int x = tc.expert;
  if (x < 0) return;
  const int lane = lane_id(), wv = wave_in_block();
  const int row0 = tc.offset + tc.rb * 16 * F;
  const int rem = tc.rows - tc.rb * 16 * F;
  const int nrows = rem < 16 * F ? rem : 16 * F;
  const int out_cols = p.gated ? kCols / 2 : kCols;
  const int col0 = tc.cb * out_cols;
  const int kchunks = p.m / 8;

  const chunk_t* a_row[F];
#pragma unroll
  for (int i = 0; i < F; ++i) {
    const int r = i * 16 + (lane & 15);
    const int rr = row0 + (r < nrows ? r : 0);
    a_row[i] = static_cast<const chunk_t*>(p.a) + static_cast<size_t>(p.gather ? p.src[rr] : rr) * kchunks + (lane >> 4);
  }
  // The first half of the fragments are gate rows and the second the up rows that meet them,
  // or all are plain; each fragment by a uniform base and a lane's own offset in its 16 rows.
  const char* b_base[FB];
  uint32_t b_off[FB];
#pragma unroll
  for (int j = 0; j < FB; ++j) {
    int f = p.gated ? col0 + j % (FB / 2) * 16 : col0 + j * 16;
    f = f < p.n ? f : 0;  // past the last feature: any rows, their sums are not stored
    const int have = p.n - f < 16 ? p.n - f : 16;
    const int first = p.gated && j >= FB / 2 ? p.n + f : f;
    b_base[j] = static_cast<const char*>(p.w) + (static_cast<size_t>(x) * p.nz + first) * kchunks * 16;
    b_off[j] = static_cast<uint32_t>((lane & 15) < have ? lane & 15 : 0) * kchunks * 16u + (lane >> 4) * 16u;
  }

  f32x4_t acc[F][FB];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  chunk_t fa[kDepth][2][F], fb[kDepth][2][FB];
  const int full = kchunks / 8;  // whole K steps; wave wv takes steps wv, wv + 4, ...
  auto load = [&](int step, int d) {
    const size_t at = static_cast<size_t>(step) * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < FB; ++j)
        fb[d][h][j] = __builtin_nontemporal_load(
            reinterpret_cast<const chunk_t*>(b_base[j] + static_cast<size_t>(step) * 128 + 64 * h + b_off[j]));
#pragma unroll
      for (int i = 0; i < F; ++i) fa[d][h][i] = a_row[i][at + 4 * h];
    }
  };
  auto multiply = [&](int d) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j) acc[i][j] = mfma_16x16x32<DT>(fb[d][h][j], fa[d][h][i], acc[i][j]);
  };
#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (wv + d * kFewWaves < full) load(wv + d * kFewWaves, d);  // uniform
  int step = wv;
  for (; step + (2 * kDepth - 1) * kFewWaves < full; step += kDepth * kFewWaves) {  // every refill is a real step
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      multiply(d);
      load(step + (d + kDepth) * kFewWaves, d);
    }
  }
  for (; step < full; step += kDepth * kFewWaves) {  // what is left: at most two rounds
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {  // uniform conditions
      if (step + d * kFewWaves < full) multiply(d);
      if (step + (d + kDepth) * kFewWaves < full) load(step + (d + kDepth) * kFewWaves, d);
    }
  }
  if (kchunks % 8 != 0 && wv == full % kFewWaves) {  // the last, partial step: zeros past the rows' end
    const chunk_t z = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = full * 8 + 4 * h + (lane >> 4) < kchunks;
      const size_t at = static_cast<size_t>(full) * 8 + 4 * h;
#pragma unroll
      for (int j = 0; j < FB; ++j)
        fb[0][h][j] = in ? *reinterpret_cast<const chunk_t*>(b_base[j] + at * 16 + b_off[j]) : z;
#pragma unroll
      for (int i = 0; i < F; ++i) fa[0][h][i] = in ? a_row[i][at] : z;
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
  for (int w = 0; w < kFewWaves; ++w) {
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
  if (c < p.n) finish8<DT>(p, x, r, t, w, c, v, u);
  if (!p.gated && c + 8 * FB < p.n) finish8<DT>(p, x, r, t, w, c + 8 * FB, u, v);
}

// ---------------------------------------------------------------------------------
// launches

int64_t row_tiles(const LayoutView& L, int height) {
  const int64_t routes = static_cast<int64_t>(L.s) * L.k;
  const int64_t with_rows = routes < L.e ? routes : L.e;
  if (L.capacity > 0) {
    const int64_t most = L.capacity < L.s ? L.capacity : L.s;
    const int64_t each = with_rows * ((most + height - 1) / height);
    const int64_t all = routes / height + with_rows;
    return each < all ? each : all;
  }
  return routes / height + with_rows;
}

// How a launch is shaped: F of its row tiles (16 F rows; 0: the large tiles), the weight rows
// per workgroup, and its workgroups.
struct ActShape {
  int few, cols;
  int64_t col_blocks, tiles;
};

// The large tiles move the most once there are enough of them to fill the CUs several times;
// until then the last of few rounds is mostly idle. F = 1 is for experts with a handful of
// rows, its 32 weight rows per workgroup (against 64: 40 us to 51 for one token's 8 of 128
// experts, 1536 x 4096 gated; 89 to 92 for 24 tokens of 64 experts, 2816 x 1408). F = 4, 64
// weight rows wide, is for small products, where all its workgroups are resident at once
// (two per CU) and each is short. Microseconds, bf16, random rows (`mean` per expert):
//   experts, weight rows x length   mean    F = 1   F = 4   large tiles
//   128, 4096 x 4096                4       816             735   (2064 of them)
//   64, 2816 x 1408                 4       101     105     109   (704)
//   64, 2816 x 1408                 12      115     113     107
//   64, 2816 x 1408                 64              235     127
//   8, 1024 x 1024                  12      7.5     10      11    (32)
//   8, 1024 x 4096                  24      33      32      47
//   16, 528 x 520                   64      11      8.2     12.5  (57)
//   16, 528 x 520                   128     17      11      16
//   8, 2048 x 1024                  64      33      22      18    (F = 4 would be 512)
constexpr int64_t kActMany = 1024, kActFewMost = 448;
constexpr int kActOneMean = 8, kActOneSmall = 12;
static ActShape act_shape(const LayoutView& L, int n, bool gated, bool kn) {
  auto shape = [&](int few) {
    ActShape a{few, few == 1 ? 32 : few == 4 ? 64 : kActBN, 0, 0};
    a.col_blocks = (static_cast<int64_t>(n) * (gated ? 2 : 1) + a.cols - 1) / a.cols;
    a.tiles = L.s == 0 ? 0 : row_tiles(L, few ? 16 * few : kn ? 32 * act_units<true> : kActBM) * a.col_blocks;
    return a;
  };
  const ActShape large = shape(0);
  if (kn || large.tiles >= kActMany) return large;
  const int64_t routes = static_cast<int64_t>(L.s) * L.k;
  int64_t mean = (routes + L.e - 1) / L.e;
  if (L.capacity > 0 && mean > L.capacity) mean = L.capacity;
  const ActShape small = shape(4);
  const bool fits = small.tiles <= kActFewMost;
  if (mean <= (fits ? kActOneSmall : kActOneMean)) return shape(1);
  return fits ? small : large;
}

static int64_t act_grid(const ActShape& a) { return (a.tiles + kXcds - 1) / kXcds * kXcds + kZeroBlocks; }

static bool act_fits(const ActShape& a) { return act_grid(a) <= most_workgroups(a.few ? kFewThreads : kActThreads); }

bool expert_act_fits(const LayoutView& L, int n, bool gated) { return act_fits(act_shape(L, n, gated, false)); }

bool expert_act_dgrad_fits(const LayoutView& L, int m) { return act_fits(act_shape(L, m, false, true)); }

hipError_t allow_lds(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return err;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit) != 0) return hipSuccess;
  err = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err == hipSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return err;
}

template <int DT, int F, int FB>
static hipError_t launch_few(const ExpertAct& p, int col_blocks, int64_t grid, hipStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr int kBytes = kFewWaves * 16 * F * (16 * FB * 4 + 16);
  auto kern = expert_act_few_kernel<DT, F, FB>;
  if (kBytes > 65536) {
    const hipError_t err = allow_lds(reinterpret_cast<const void*>(kern), kBytes, done);
    if (err != hipSuccess) return err;
  }
  kern<<<static_cast<unsigned>(grid), kFewThreads, kBytes, stream>>>(p, col_blocks, static_cast<int>(grid) - kZeroBlocks);
  return hipGetLastError();
}

template <int DT, bool KN>
static hipError_t launch_tiles(const ExpertAct& p, int col_blocks, int64_t grid, hipStream_t stream) {
  static std::atomic<uint64_t> done{0};
  auto kern = expert_act_kernel<DT, KN>;
  const hipError_t err = allow_lds(reinterpret_cast<const void*>(kern), kActLds, done);
  if (err != hipSuccess) return err;
  kern<<<static_cast<unsigned>(grid), kActThreads, kActLds, stream>>>(p, col_blocks,
                                                                     static_cast<int>(grid) - kZeroBlocks);
  return hipGetLastError();
}

template <int DT>
static hipError_t launch_dt(const LayoutView& L, const ExpertAct& p, hipStream_t stream) {
  const ActShape a = act_shape(L, p.n, p.gated, false);
  const int64_t grid = act_grid(a);
  const int col_blocks = static_cast<int>(a.col_blocks);
  if (a.few == 1) return launch_few<DT, 1, 2>(p, col_blocks, grid, stream);
  if (a.few == 4) return launch_few<DT, 4, 4>(p, col_blocks, grid, stream);
  return launch_tiles<DT, false>(p, col_blocks, grid, stream);
}

hipError_t launch_expert_act(const LayoutView& L, const ExpertAct& p, int dtype, hipStream_t stream) {
  if (p.rows == 0) return hipSuccess;
  return dtype == kBF16 ? launch_dt<kBF16>(L, p, stream) : launch_dt<kF16>(L, p, stream);
}

hipError_t launch_expert_act_dgrad(const LayoutView& L, const ExpertAct& p, int dtype, hipStream_t stream) {
  if (p.rows == 0) return hipSuccess;
  const ActShape a = act_shape(L, p.n, false, true);
  const int64_t grid = act_grid(a);
  const int col_blocks = static_cast<int>(a.col_blocks);
  return dtype == kBF16 ? launch_tiles<kBF16, true>(p, col_blocks, grid, stream)
                        : launch_tiles<kF16, true>(p, col_blocks, grid, stream);
}

}  // namespace moe
