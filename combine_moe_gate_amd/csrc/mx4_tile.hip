// The products with 4-bit weights for long segments, on gfx950 matrix cores (mx4_act.hip chooses).
//
// A workgroup of eight waves, 2 along the rows by 4 along the columns, multiplies up to 32 U rows by
// 256 weight rows of one expert; a segment is cut into the fewest tiles of nearly equal height (a
// multiple of 32 rows), and the main loop is compiled for each height. Codes and 16-bit rows go to
// LDS directly, in rows of 128 bytes: 256 4-bit values or 64 16-bit ones, XOR-swizzled in 16-byte
// pieces, two stages of each. Fragments are read a group of up to four row tiles ahead of their use;
// the next stage is published by the step's one barrier before its last group's products, and the
// loads of the stage after it start there.
//
// 4-bit rows: a step is 256 elements of both sides. In the products of half h lane group g = lane / 16
// multiplies block 4 h + g of the step.
// 16-bit rows: a step is 64 elements of the rows and a quarter of a 256-element stage of the weights;
// in half h of step p group g takes elements 8 g .. + 7 of the stage's block 2 p + h, and widens its
// weights after they are read from LDS.
// (With block 2 g + h, and elements 16 g + 8 h, an LDS read of rows would meet every bank twice.)
//
// Scales go through registers (a row's may start at any byte) to LDS, 8 bytes a staged row and 256
// elements, a step later than loaded and a step before they are read. For 4-bit rows they lie there as
// the matrix instructions take them: a lane's word holds both halves' scales of a row and of the row 16
// further on, its next MFMA tile, and an instruction names the byte.
//
// Measured, 8192 tokens, 8 of 128 experts, 4096 -> 2 x 2048 gated: 4-bit rows 746 us (2.9 PFLOP/s, matrix
// units busy 32%; the loop without its loads and epilogue 4.2, the scaled instruction alone on random codes
// 6.9); without the loop's loads 130 us less, without the epilogue 58. bf16 rows 1.94 ms (1.13 PFLOP/s, busy
// 48%, where their instruction alone reaches 1.95 and a large library product 1.5).
#include <atomic>

#include "mx4_product.h"

namespace moe {

constexpr int kMtThreads = kMx4TileThreads;
constexpr int kMtBN = 256;                         // weight rows per tile
constexpr int kMtBand = 8;                         // row-blocks per band of the tile order
constexpr int kMtRowBytes = 128;                   // a staged row
constexpr int kMtBStage = kMtBN * kMtRowBytes;
constexpr int kMtSlabPitch = 64 * 4 + 16;          // bytes per row of a wave's 16 x 64 float32 slab

// The most units of 32 rows of a tile, its LDS in order: rows, weights, scales (two stages each), and
// per row its token and route weight.
template <int RT>
struct MtLds {
  static constexpr int kUnits = 9;
  static constexpr int kBM = 32 * kUnits;
  static constexpr int kAStage = kBM * kMtRowBytes;
  static constexpr int kScaleStage = (kMtBN + (RT == kMx4 ? kBM + 32 : 0)) * 8;  // an odd tile takes a pair's room
  static constexpr int kB = 2 * kAStage;
  static constexpr int kScales = kB + 2 * kMtBStage;
  static constexpr int kRows = kScales + 2 * kScaleStage;
  static constexpr int kVotes = kRows + kBM * 8;
  static constexpr int kBytes = kVotes + (RT == kF16 ? 32 : 0);
  static_assert(8 * 2 * 16 * kMtSlabPitch <= kScales, "the slabs reuse the stages");
  static_assert(kBytes <= 160 * 1024);
};

// The tile's float32 sums, for a height of 32 FM rows. f16 rows: true if some scale that this wave met
// does not let f16 hold the weights.
template <int RT, int FM>
__device__ __forceinline__ bool mx4_tile_products(const Mx4Act& p, const UnitTile& tc, char* lds, f32x4_t (&acc)[FM][4]) {
  using Lds = MtLds<RT>;
  constexpr bool kQ = RT == kMx4;
  constexpr int FN = 4;
  // A step's products in order: (half, row tile), 2 FM slots of FN MFMAs, cut into groups of up to
  // four slots whose fragments are read together; the last group lies in the second half.
  constexpr int kSlots = 2 * FM, kGroups = FM <= 4 ? 2 : FM > 8 ? 6 : (kSlots + 3) / 4;
  auto first_slot = [](int g) constexpr { return g * kSlots / kGroups; };
  constexpr int kALoads = (4 * FM + 7) / 8;            // direct-to-LDS loads of 8 rows, per wave
  constexpr bool kMoreScales = kQ && FM > 8;           // rows whose scales have no thread of their own
  const int lane = lane_id(), wv = wave_in_block(), grp = lane >> 4;
  const int wm = wv / 4, wn = wv % 4;
  const int x = tc.expert;
  const int row0 = tc.offset + tc.unit0 * 32;
  const int rem = tc.rows - tc.unit0 * 32;
  const int nrows = rem < 32 * FM ? rem : 32 * FM;
  const int out_cols = p.gated ? kMtBN / 2 : kMtBN;
  const int col0 = tc.cb * out_cols;                   // first output feature
  const int kb = p.m / kMx4Block;
  const int achunks = kQ ? kb : 4 * kb;                // 16-byte pieces of a row
  const int nk = (achunks + 7) / 8, nu = (kb + 7) / 8; // steps of the rows, 256-element stages of the weights

  // weight row of staged row 64 q + r, r < 64; rows past the last repeat it: they reach only results never
  // stored. Addresses are formed where they are used: pointers would take the registers that the
  // tallest tiles need for their sums.
  auto weight_row = [&](uint32_t r, uint32_t q) __attribute__((always_inline)) {
    const uint32_t n = p.n, c = col0;
    if (p.gated) {  // 32 gate rows, then the 32 up rows of the same features
      const uint32_t f = c + q * 32 + r % 32;
      return (f < n ? f : n - 1) + (r >= 32 ? n : 0);
    }
    return c + q * 64 + r < n ? c + q * 64 + r : n - 1;
  };
  // buffer or token row of staged row r; rows past the segment repeat its first
  auto input_row = [&](int r) __attribute__((always_inline)) {
    const int rr = row0 + (r < nrows ? r : 0);
    return static_cast<uint32_t>(p.gather ? p.src[rr] : rr);
  };
  // slot lane % 8 of staged row R takes piece slot ^ (R / 2 % 8); the loads' first rows are
  // multiples of 8, so R / 2 % 8 = 4 (load % 2) + lane / 16
  const int chunk = (lane % 8) ^ (4 * (wv % 2) + lane / 16);
  const chunk_t* wx = static_cast<const chunk_t*>(p.w) + static_cast<size_t>(x) * p.nz * kb;
  auto issue_b = [&](int u, int q) __attribute__((always_inline)) {  // 64 rows of weight stage u
    const int at = u * 8 + chunk < kb ? u * 8 + chunk : 0;  // past the row's end: any codes, the rows' zeros meet them
    uint32_t r = wv * 8 + lane / 8;
    asm volatile("" : "+v"(r));  // not a value to keep from step to step
    const chunk_t* from = wx + static_cast<uint64_t>(weight_row(r, q)) * static_cast<uint32_t>(kb) + at;
    __builtin_amdgcn_global_load_lds(static_cast<const void*>(from),
                                     (lds_void_t*)(lds + Lds::kB + (u % 2) * kMtBStage + (q * 8 + wv) * 1024), 16, 0, 0);
  };
#pragma unroll
  for (int q = 0; q < 4; ++q) issue_b(0, q);
  if (kQ && nk > 1) {
#pragma unroll
    for (int q = 0; q < 4; ++q) issue_b(1, q);
  }
  __builtin_amdgcn_sched_barrier(0);
  // the rows are looked up before any load to LDS starts: the wait for them would be one for those as well
  uint32_t a_row[kALoads];
#pragma unroll
  for (int q = 0; q < kALoads; ++q) a_row[q] = input_row((q * 8 + wv) * 8 + lane / 8);
  auto issue_a = [&](int kt) __attribute__((always_inline)) {
    const int at = kt * 8 + chunk < achunks ? kt * 8 + chunk : 0;  // past the row's end: cleared once landed
#pragma unroll
    for (int q = 0; q < kALoads; ++q)
      if (q * 8 + wv < 4 * FM) {  // uniform
        uint32_t r = a_row[q];
        asm volatile("" : "+v"(r));
        __builtin_amdgcn_global_load_lds(static_cast<const chunk_t*>(p.a) +
                                             static_cast<uint64_t>(r) * static_cast<uint32_t>(achunks) + at,
                                         (lds_void_t*)(lds + (kt % 2) * Lds::kAStage + (q * 8 + wv) * 1024), 16, 0, 0);
      }
  };
  issue_a(0);
  if (nk > 1) issue_a(1);

  // scales: thread t < 256 those of weight row t; with 4-bit rows thread 256 + t those of row t, and
  // threads t < 32 those of row 256 + t besides. Past a row's end 127 (the codes there are zeros, or
  // meet zeros).
  const int tid = threadIdx.x;
  const bool has_scale = tid < kMtBN || (kQ && tid - kMtBN < 32 * FM);
  const uint8_t* s_from = p.w_scales + (static_cast<size_t>(x) * p.nz + weight_row(tid % 64, tid / 64 % 4)) * kb;
  if (kQ && tid >= kMtBN) s_from = p.a_scales + static_cast<size_t>(input_row(tid - kMtBN)) * kb;
  const uint8_t* s_more = kMoreScales ? p.a_scales + static_cast<size_t>(input_row(256 + tid % 32)) * kb : nullptr;
  typedef uint64_t __attribute__((aligned(1), may_alias)) bytes8_t;
  // stage u's eight bytes of a row lie in the eight from first(u) on (a row of less has them one by one)
  auto first = [&](int u) { return 8 * u + 8 <= kb ? 8 * u : kb - 8; };
  uint64_t sreg = 0, smore = 0;
  auto load_scales = [&](int u) __attribute__((always_inline)) {
    if (u >= nu) return;  // uniform
    if (has_scale) sreg = *reinterpret_cast<const bytes8_t*>(s_from + first(u));
    if (kMoreScales && tid < 32) smore = *reinterpret_cast<const bytes8_t*>(s_more + first(u));
  };
  // of staged row R's bytes, those of lane group i (blocks i and 4 + i) go to scale_at(R) + 4 i; 16-bit
  // rows: the weights' as they are, row by row
  auto pair_row = [](int region, int tile, int row) { return ((region + tile / 2) * 16 + row) * 16 + (tile % 2) * 2; };
  auto scale_at = [&](int R) {
    if (!kQ) return R * 8;
    if (R < kMtBN) return pair_row(0, R / 16, R % 16);
    const int a = R - kMtBN, w = a >= 16 * FM;
    return pair_row(kMtBN / 32 + w * ((FM + 1) / 2), a / 16 - w * FM, a % 16);
  };
  auto put = [&](int u, uint64_t v, int R) __attribute__((always_inline)) {
    const int over = 8 * (8 * u - first(u));  // bits before the stage's first byte, only in the last stage
    if (over != 0) v = v >> over | 0x7f7f7f7f7f7f7f7full << (64 - over);
    char* to = lds + Lds::kScales + (u % 2) * Lds::kScaleStage + scale_at(R);
    if constexpr (kQ) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        reinterpret_cast<uint16_t*>(to)[2 * i] = static_cast<uint16_t>((v >> (8 * i) & 255u) | (v >> (24 + 8 * i) & 0xff00u));
    } else {
      *reinterpret_cast<uint64_t*>(to) = v;
    }
  };
  auto write_scales = [&](int u) __attribute__((always_inline)) {
    if (u >= nu) return;
    if (has_scale) put(u, sreg, tid);
    if (kMoreScales && tid < 32) put(u, smore, 512 + tid);
  };
  if (kb >= 8) {
    load_scales(0);
  } else {  // the only stage
    uint64_t v = 0, more = 0;
    for (int i = 0; i < 8; ++i) {
      v |= static_cast<uint64_t>(has_scale && i < kb ? s_from[i] : 127) << (8 * i);
      if (kMoreScales) more |= static_cast<uint64_t>(tid < 32 && i < kb ? s_more[i] : 127) << (8 * i);
    }
    // as if they had been loaded from first(0) < 0 on
    sreg = v << (8 * (8 - kb));
    smore = more << (8 * (8 - kb));
  }
  {  // the second stage's loads start before the first's are waited for
    const uint64_t s0 = sreg, more0 = smore;
    load_scales(1);
    if (has_scale) put(0, s0, tid);
    if (kMoreScales && tid < 32) put(0, more0, 512 + tid);
  }

  // per tile row: its token and route weight, for the epilogue
  int* row_token = reinterpret_cast<int*>(lds + Lds::kRows);
  float* row_weight = reinterpret_cast<float*>(lds + Lds::kRows + Lds::kBM * 4);
  if (tid < nrows) {
    const int r = row0 + tid;
    const int t = p.src[r];
    row_token[tid] = t;
    row_weight[tid] = route_weight_wide(p, r, t);
  }

#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // fragments: row lane % 16 of a 16-row MFMA tile, piece 4 half + grp at slot piece ^ (row / 2 % 8)
  const int frag_row = (lane & 15) * kMtRowBytes, frag_swz = (lane & 15) >> 1;
  const int a_base = wm * 16 * FM * kMtRowBytes + frag_row;
  const int b_base = Lds::kB + wn * 64 * kMtRowBytes + frag_row;
  const int bs_base = Lds::kScales + (kQ ? wn * 2 * 256 + (lane & 15) * 16 + grp * 4 : (wn * 64 + (lane & 15)) * 8);
  const int as_base = Lds::kScales + kMtBN * 8 + wm * ((FM + 1) / 2) * 256 + (lane & 15) * 16 + grp * 4;
  auto read_a = [&](int kt, int g, chunk_t (&f)[4]) __attribute__((always_inline)) {  // the fragments of group g
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int slot = first_slot(g) + q;
      if (slot < first_slot(g + 1))
        f[q] = *reinterpret_cast<const chunk_t*>(lds + (kt % 2) * Lds::kAStage + a_base + (slot % FM) * 16 * kMtRowBytes +
                                                 (((4 * (slot / FM) + grp) ^ frag_swz) << 4));
    }
  };
  // 4-bit rows: the weights' fragments of a half
  auto read_b = [&](int kt, int half, chunk_t (&b)[FN]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
      b[j] = *reinterpret_cast<const chunk_t*>(lds + (kt % 2) * kMtBStage + b_base + j * 16 * kMtRowBytes +
                                               (((4 * half + grp) ^ frag_swz) << 4));
  };
  // and a step's scales, of both sides
  constexpr int kPairs = (FM + 1) / 2;
  auto read_scales = [&](int kt, uint32_t (&a)[kPairs], uint32_t (&b)[2]) __attribute__((always_inline)) {
    const char* st = lds + (kt % 2) * Lds::kScaleStage;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) a[i] = *reinterpret_cast<const uint32_t*>(st + as_base + i * 256);
#pragma unroll
    for (int i = 0; i < 2; ++i) b[i] = *reinterpret_cast<const uint32_t*>(st + bs_base + i * 256);
  };
  // 16-bit rows: the eight codes of each half of a step, and both halves' scales
  auto read_codes = [&](int kt, uint2 (&c)[FN], uint32_t (&sc)[FN]) __attribute__((always_inline)) {
    const int u = kt / 4, block = 2 * (kt % 4);
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const char* row = lds + (u % 2) * kMtBStage + b_base + j * 16 * kMtRowBytes + 4 * grp;
      c[j].x = *reinterpret_cast<const uint32_t*>(row + ((block ^ frag_swz) << 4));
      c[j].y = *reinterpret_cast<const uint32_t*>(row + (((block + 1) ^ frag_swz) << 4));
      sc[j] = *reinterpret_cast<const uint16_t*>(lds + (u % 2) * Lds::kScaleStage + bs_base + j * 128 + block);
    }
  };
  // step kt is whole in LDS and every wave has read out the step before it
  auto publish = [&](int kt) __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(wait_vm(0) & ~0xF00);  // all loads and LDS operations
    if ((kt + 1) * 8 > achunks) {
      if (kt * 8 + chunk >= achunks) {
#pragma unroll
        for (int q = 0; q < kALoads; ++q)
          if (q * 8 + wv < 4 * FM)
            *reinterpret_cast<chunk_t*>(lds + (kt % 2) * Lds::kAStage + (q * 8 + wv) * 1024 + lane * 16) = chunk_t{0u, 0u, 0u, 0u};
      }
      __builtin_amdgcn_s_waitcnt(kWaitLdsOnly);
    }
    stage_barrier();
  };
  // what starts once step t is published, into what the step before it has left
  auto start = [&](int t) __attribute__((always_inline)) {
    if constexpr (kQ) {
      write_scales(t + 1);
      load_scales(t + 2);
      if (t > 0 && t + 1 < nk) {
#pragma unroll
        for (int q = 0; q < 4; ++q) issue_b(t + 1, q);
      }
    } else {
      const int u = t / 4;
      if (t % 4 == 0) {
        write_scales(u + 1);
        load_scales(u + 2);
      }
      if (u + 1 < nu) {  // all landed a step before their own: their first codes are read under the step before
        switch (t % 4) {  // uniform
          case 0: issue_b(u + 1, 0); issue_b(u + 1, 1); break;
          case 1: issue_b(u + 1, 2); break;
          case 2: issue_b(u + 1, 3); break;
          default: break;
        }
      }
    }
    if (t > 0 && t + 1 < nk) issue_a(t + 1);
  };

  publish(0);
  start(0);
  chunk_t fa[2][4], fb[2][FN];
  uint32_t sa[2][kPairs], sb[2][2];  // 4-bit rows: the scales of this step and the next
  uint2 codes[FN];                   // 16-bit rows: the weights of a step, and their scales
  uint32_t sc[FN];
  read_a(0, 0, fa[0]);
  if constexpr (kQ) {
    read_b(0, 0, fb[0]);
    read_scales(0, sa[0], sb[0]);
  } else {
    read_codes(0, codes, sc);
  }
  uint32_t reach = 0;  // f16 rows: the largest distance from the least scale that fits f16
  constexpr int kWide = RT == kF16 ? kF16 : kBF16;  // 16-bit rows: what the weights are widened to
  auto widen = [&](int half) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[half][j] = mx4_values8<kWide>(half == 0 ? codes[j].x : codes[j].y, mx4_scale(sc[j] >> (8 * half) & 255u));
  };
  if constexpr (!kQ) {
    __builtin_amdgcn_s_waitcnt(kWaitLdsOnly);
    widen(0);
  }

  // Under each group's MFMAs the next group's fragments are read, and with the group before the
  // first one of the second half the weights' of that half. Before the last group's MFMAs the next
  // step is published (by then every fragment of this step is in registers), the loads of the one
  // after it start, and the next step's first fragments are read; after the last step these find old
  // contents, which nothing uses. 16-bit rows: the second half's weights are widened among the first
  // group's MFMAs, the next step's first among the last group's, from codes read after the first.
  for (int kt = 0; kt < nk; ++kt) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      __builtin_amdgcn_s_waitcnt(kWaitLdsOnly);  // this group's fragments have landed
      __builtin_amdgcn_sched_barrier(0);
      if (g + 1 < kGroups) {
        read_a(kt, g + 1, fa[(g + 1) % 2]);
        if (kQ && first_slot(g + 1) <= FM && first_slot(g + 2) > FM) read_b(kt, 1, fb[1]);
      } else {
        if (kt + 1 < nk) {
          publish(kt + 1);
          start(kt + 1);
        }
        __builtin_amdgcn_sched_barrier(0);
        read_a(kt + 1, 0, fa[(g + 1) % 2]);
        if constexpr (kQ) {
          read_b(kt + 1, 0, fb[0]);  // the last group is all of the second half
          read_scales(kt + 1, sa[1], sb[1]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (kQ) {
        static_for(std::make_integer_sequence<int, 4>{}, [&](auto qq) __attribute__((always_inline)) {
          constexpr int q = decltype(qq)::value;
          const int slot = first_slot(g) + q;
          if (slot < first_slot(g + 1)) {
#pragma unroll
            for (int j = 0; j < FN; ++j) {
              const int i = slot % FM;
              const chunk_t& w = fb[slot / FM][j];
              f32x4_t& c = acc[i][j];
              // the byte of each word: 2 (tile % 2) + half
              switch ((slot / FM) * 4 + (j % 2) * 2 + i % 2) {  // constant once unrolled
                case 0: c = mfma_mx4<0, 0>(w, sb[0][j / 2], fa[g % 2][q], sa[0][i / 2], c); break;
                case 1: c = mfma_mx4<0, 2>(w, sb[0][j / 2], fa[g % 2][q], sa[0][i / 2], c); break;
                case 2: c = mfma_mx4<2, 0>(w, sb[0][j / 2], fa[g % 2][q], sa[0][i / 2], c); break;
                case 3: c = mfma_mx4<2, 2>(w, sb[0][j / 2], fa[g % 2][q], sa[0][i / 2], c); break;
                case 4: c = mfma_mx4<1, 1>(w, sb[0][j / 2], fa[g % 2][q], sa[0][i / 2], c); break;
                case 5: c = mfma_mx4<1, 3>(w, sb[0][j / 2], fa[g % 2][q], sa[0][i / 2], c); break;
                case 6: c = mfma_mx4<3, 1>(w, sb[0][j / 2], fa[g % 2][q], sa[0][i / 2], c); break;
                default: c = mfma_mx4<3, 3>(w, sb[0][j / 2], fa[g % 2][q], sa[0][i / 2], c); break;
              }
              // the scaled instruction may be moved past the step's barrier and branches, next to the use
              // of its result: the empty asm keeps it in its group
              asm volatile("" : "+v"(c));
            }
          }
        });
      } else {
        if (g == 0) {
          widen(1);
          if (RT == kF16) {
#pragma unroll
            for (int j = 0; j < FN; ++j) {
              const uint32_t r0 = mx4_f16_reach(sc[j] & 255u), r1 = mx4_f16_reach(sc[j] >> 8 & 255u);
              const uint32_t r = r0 > r1 ? r0 : r1;
              reach = r > reach ? r : reach;
            }
          }
        } else if (g + 1 == kGroups) {
          widen(0);  // the next step's
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int slot = first_slot(g) + q;
          if (slot < first_slot(g + 1)) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
              acc[slot % FM][j] = mfma_16x16x32<kWide>(fb[slot / FM][j], fa[g % 2][q], acc[slot % FM][j]);
          }
        }
        if (g == 0 || g + 1 == kGroups) {  // the widening goes between the products
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a matrix instruction
            __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);  // two others
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if (!kQ && g == 0) {
        read_codes(kt + 1, codes, sc);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (kGroups % 2 != 0) {
#pragma unroll
      for (int q = 0; q < 4; ++q) fa[0][q] = fa[1][q];
    }
    if constexpr (kQ) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) sa[0][i] = sa[1][i];
#pragma unroll
      for (int i = 0; i < 2; ++i) sb[0][i] = sb[1][i];
    }
  }
  return __any(reach > kMx4F16Reach);
}

// A tile of 32 FM rows; false if it is left to mx4_tile_split (f16 rows alone).
template <int RT, int DT, int FM>
__device__ __forceinline__ bool mx4_tile_body(const Mx4Act& p, const UnitTile& tc, char* lds) {
  using Lds = MtLds<RT>;
  constexpr int FN = 4;
  const int lane = lane_id(), wv = wave_in_block(), grp = lane >> 4;
  const int wm = wv / 4, wn = wv % 4;
  const int x = tc.expert;
  const int row0 = tc.offset + tc.unit0 * 32;
  const int rem = tc.rows - tc.unit0 * 32;
  const int nrows = rem < 32 * FM ? rem : 32 * FM;
  const int out_cols = p.gated ? kMtBN / 2 : kMtBN;
  const int col0 = tc.cb * out_cols;
  int* row_token = reinterpret_cast<int*>(lds + Lds::kRows);
  float* row_weight = reinterpret_cast<float*>(lds + Lds::kRows + Lds::kBM * 4);
  f32x4_t acc[FM][FN];
  const bool misfit = mx4_tile_products<RT, FM>(p, tc, lds, acc);
  if constexpr (RT == kF16) {  // weights in use have zeros at most under such scales: what it costs others is the vote
    int* votes = reinterpret_cast<int*>(lds + Lds::kVotes);
    auto vote = [&](bool mine) {
      if (lane == 0) votes[wv] = mine;
      __syncthreads();
      int any = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) any |= votes[i];
      return __builtin_amdgcn_readfirstlane(any) != 0;
    };
    if (vote(misfit)) {
      // the sums are right if only zeros lie under the scales that do not fit. Two threads a weight row look, half
      // a row each: of the same product 1.96 ms with a block of zeros in each tile, 1.99 with a quarter of the
      // weight rows zero. Looking at the codes within the loop would take registers from it: 2.00 with or without.
      const int kb = p.m / kMx4Block, half = (kb + 1) / 2, from = (threadIdx.x % 2) * half;
      const int R = threadIdx.x / 2;  // staged row, as the tile stages them: gated, 32 gate rows and their up rows
      const int f = p.gated ? col0 + R / 64 * 32 + R % 32 : col0 + R;
      const int row = (f < p.n ? f : p.n - 1) + (p.gated && R % 64 >= 32 ? p.n : 0);
      const bool bad = mx4_misfits_f16(static_cast<const chunk_t*>(p.w), p.w_scales,
                                       (static_cast<size_t>(x) * p.nz + row) * kb + from, kb - from < half ? kb - from : half);
      __syncthreads();  // every wave has read the votes
      if (vote(__any(bad))) return false;
    }
  }

  // epilogue: each 16-row tile's sums through one of the wave's two slabs. Lane l holds token
  // row l % 16, features 16 j + 4 (l / 16) .. + 3 of its 64; it takes back row l / 4, features
  // 8 (l % 4) .. + 7 of each 32 (gated: the gate's and the up's). The next tile goes through
  // LDS while one is finished.
  __syncthreads();
  char* slabs = lds + wv * 2 * 16 * kMtSlabPitch;
  const int below = nrows - wm * 16 * FM;
  const int tiles = below <= 0 ? 0 : below < 16 * FM ? (below + 15) / 16 : FM;
  auto pass = [&](int i, float (&v)[8], float (&u)[8]) __attribute__((always_inline)) {
    char* slab = slabs + (i % 2) * 16 * kMtSlabPitch;
    static_for(std::make_integer_sequence<int, FM>{}, [&](auto ii) __attribute__((always_inline)) {
      if (ii == i) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
          *reinterpret_cast<f32x4_t*>(slab + (lane & 15) * kMtSlabPitch + j * 64 + grp * 16) = acc[ii][j];
        // the empty asm keeps the branches apart: with their stores folded into one, they
        // would index the accumulators dynamically and so move them to memory
        asm volatile("" ::"i"(decltype(ii)::value) : "memory");
      }
    });
    const float* back = reinterpret_cast<const float*>(slab + (lane >> 2) * kMtSlabPitch) + 8 * (lane & 3);
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
    if (c < p.n) finish8_mx4<DT>(p, x, r, t, w, c, v, u);
    if (!p.gated && c + 32 < p.n) finish8_mx4<DT>(p, x, r, t, w, c + 32, u, v);
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
  return true;
}

// A tile of f16 rows whose weights f16 does not hold: each row value in two parts (split_f16) times the
// weights in bf16, 16 rows by 64 weight rows of a wave at a time, straight from memory, in few registers. Seven
// times slower than the tile's own loop (8192 tokens, 8 of 128 experts, 4096 -> 2 x 2048: 13.2 ms where that takes
// 1.92): a second loop of that kind, next to the first, would take registers from it (2.5 ms where 2.0 are).
// Only tiles with values, other than zeros, under scales below 2^-23 or above 2^13 come here.
template <int DT>
__device__ __forceinline__ void mx4_tile_split(const Mx4Act& p, const UnitTile& tc, char* lds) {
  using Lds = MtLds<kF16>;
  const int lane = lane_id(), wv = wave_in_block(), grp = lane >> 4, lrow = lane & 15;
  const int wm = wv / 4, wn = wv % 4;
  const int row0 = tc.offset + tc.unit0 * 32;
  const int rem = tc.rows - tc.unit0 * 32;
  const int nrows = rem < 32 * tc.units ? rem : 32 * tc.units;
  const int out_cols = p.gated ? kMtBN / 2 : kMtBN;
  const int col0 = tc.cb * out_cols, kb = p.m / kMx4Block;
  const int* row_token = reinterpret_cast<const int*>(lds + Lds::kRows);
  const float* row_weight = reinterpret_cast<const float*>(lds + Lds::kRows + Lds::kBM * 4);
  char* slab = lds + wv * 16 * kMtSlabPitch;
  size_t block[4];  // of this lane's weight rows, as the tile stages them: gated, 32 gate rows and their up rows
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    int f = p.gated ? col0 + wn * 32 + (j % 2) * 16 + lrow : col0 + wn * 64 + j * 16 + lrow;
    f = (f < p.n ? f : p.n - 1) + (p.gated && j >= 2 ? p.n : 0);
    block[j] = (static_cast<size_t>(tc.expert) * p.nz + f) * kb + grp;
  }
  for (int i = 0; i < tc.units; ++i) {
    const int first = (wm * tc.units + i) * 16;
    if (first >= nrows) return;  // uniform
    const int rr = row0 + (first + lrow < nrows ? first + lrow : 0);
    const chunk_t* a_row = static_cast<const chunk_t*>(p.a) + (static_cast<size_t>(p.gather ? p.src[rr] : rr) * kb + grp) * 4;
    f32x4_t acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int b = 0; b < kb; b += 4) {
      const bool in = b + grp < kb;  // past the row's end: zeros
      chunk_t codes[4], a[4];
      uint32_t E[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        codes[j] = in ? static_cast<const chunk_t*>(p.w)[block[j] + b] : chunk_t{0u, 0u, 0u, 0u};
        E[j] = in ? p.w_scales[block[j] + b] : 127u;
        a[j] = in ? a_row[4 * b + j] : chunk_t{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        chunk_t hi, lo;
        split_f16(a[q], hi, lo);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const chunk_t w = mx4_values8<kBF16>(codes[j][q], mx4_scale(E[j]));
          acc[j] = mfma_16x16x32<kBF16>(w, lo, acc[j]);
          acc[j] = mfma_16x16x32<kBF16>(w, hi, acc[j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<f32x4_t*>(slab + lrow * kMtSlabPitch + j * 64 + grp * 16) = acc[j];
    const float* back = reinterpret_cast<const float*>(slab + (lane >> 2) * kMtSlabPitch) + 8 * (lane & 3);
    float v[8], u[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      v[q] = back[q];
      u[q] = back[32 + q];
    }
    const int row = first + (lane >> 2);
    if (row < nrows) {
      const int c = col0 + wn * (out_cols / 4) + 8 * (lane & 3);
      const int t = row_token[row];
      const float w = row_weight[row];
      if (c < p.n) finish8_mx4<DT>(p, tc.expert, row0 + row, t, w, c, v, u);
      if (!p.gated && c + 32 < p.n) finish8_mx4<DT>(p, tc.expert, row0 + row, t, w, c + 32, u, v);
    }
  }
}

template <int RT, int DT>
__global__ __launch_bounds__(kMtThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void mx4_tile_kernel(
    Mx4Act p, int col_blocks, int tile_grid) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  if (static_cast<int>(blockIdx.x) >= tile_grid) {
    zero_unfilled_mx4(p, blockIdx.x - tile_grid, gridDim.x - tile_grid);
    return;
  }
  constexpr int kUnits = MtLds<RT>::kUnits;
  const UnitTile tc = unit_tile<kUnits>(blockIdx.x, p.e, p.kept, p.offsets, col_blocks, kMtBand);
  if (tc.expert < 0) return;
  bool done = true;
  switch (tc.units) {
    case 1: done = mx4_tile_body<RT, DT, 1>(p, tc, lds); break;
    case 2: done = mx4_tile_body<RT, DT, 2>(p, tc, lds); break;
    case 3: done = mx4_tile_body<RT, DT, 3>(p, tc, lds); break;
    case 4: done = mx4_tile_body<RT, DT, 4>(p, tc, lds); break;
    case 5: done = mx4_tile_body<RT, DT, 5>(p, tc, lds); break;
    case 6: done = mx4_tile_body<RT, DT, 6>(p, tc, lds); break;
    case 7: done = mx4_tile_body<RT, DT, 7>(p, tc, lds); break;
    case 8: done = mx4_tile_body<RT, DT, 8>(p, tc, lds); break;
    default: done = mx4_tile_body<RT, DT, 9>(p, tc, lds); break;
  }
  if constexpr (RT == kF16)
    if (!done) mx4_tile_split<DT>(p, tc, lds);
}

int mx4_tile_rows() { return MtLds<kMx4>::kBM; }

template <int RT, int DT>
static hipError_t launch_tiles(const Mx4Act& p, int col_blocks, int64_t grid, hipStream_t stream) {
  static std::atomic<uint64_t> done{0};
  auto kern = mx4_tile_kernel<RT, DT>;
  const hipError_t err = allow_lds(reinterpret_cast<const void*>(kern), MtLds<RT>::kBytes, done);
  if (err != hipSuccess) return err;
  kern<<<static_cast<unsigned>(grid), kMtThreads, MtLds<RT>::kBytes, stream>>>(p, col_blocks,
                                                                              static_cast<int>(grid) - kZeroBlocks);
  return hipGetLastError();
}

hipError_t launch_mx4_tiles(const Mx4Act& p, int dtype, int col_blocks, int64_t grid, hipStream_t stream) {
  if (p.a_scales != nullptr)
    return dtype == kBF16 ? launch_tiles<kMx4, kBF16>(p, col_blocks, grid, stream)
                          : launch_tiles<kMx4, kF16>(p, col_blocks, grid, stream);
  return dtype == kBF16 ? launch_tiles<kBF16, kBF16>(p, col_blocks, grid, stream)
                        : launch_tiles<kF16, kF16>(p, col_blocks, grid, stream);
}

}  // namespace moe
