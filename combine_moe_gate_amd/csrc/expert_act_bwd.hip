// Backward of the expert products' epilogue on gfx950.
//
// With out[r] = w_r u(z[r]) + residual(r), u = act(z) or act(z_gate) z_up, and g = w_r
// grad_out[r], for each placed row r of expert x:
//     grad_z[r] = g act'(z)      (gated: g z_up act'(z_gate), and g act(z_gate))
//     grad_b[x] = sum_r grad_z[r],   grad_w(route at r) = <grad_out[r], u(z[r])>
// The products' own gradients are grouped GEMMs of grad_z, which is rounded to the element type
// for them, once: what the matrix cores take (grad_b sums the unrounded values). Or it goes out in
// two bf16 parts, the nearest bf16 value and the nearest to what that leaves, 16 bits of a float32
// value together: the matrix cores take those one after the other, with float32's range. z is read
// as the forward kept it, rounded to the element type or in float32 (Z32): whichever the caller
// keeps memory for.
//
// One pass over grad_out and z, bound by its traffic. A workgroup takes 64 rows (16 of few)
// of one expert by 512 output features: a wave a row at a time, a lane eight features as
// 16-byte pieces (gated: of both halves), so the bias sums of its features stay in a lane's
// registers over the rows. The waves' sums meet in LDS in order and go out as one partial
// row; a row's dot is reduced across the wave in float64 and goes out per column block. A
// second launch adds both up in a fixed order. No floating-point atomics. Four rows per wave
// are in flight, since a row's loads alone would leave memory idle while it is finished.
//
// Measured: 49152 rows of 1408 gated features (0.69 GB) 134 us, 5.2 TB/s, with float32 z (0.97
// GB) 190 us, 5.1 TB/s, and with grad_z in two parts (1.25 GB) 240 us, 5.2 TB/s; 2000 rows of 264
// gated features with bias 9.5 us and 3 us for the sums.
#include <type_traits>

#include "expert_act.h"

namespace moe {

constexpr int kBwdThreads = 256, kBwdWaves = kBwdThreads / kWave;
constexpr int kBwdRows = 64;    // most rows of a tile
// Under so many tiles of 64 rows (two per CU) tiles have 16. Microseconds with 16 and with 64,
// by tiles of 64: 16 experts, 264 gated features: 47 tiles 9.3 and 16.0, 266 18.5 and 23.8, 516
// 31.2 and 25.7, 1016 47.9 and 38.1; 128 experts, 512 features: 253 11.7 and 15.0, 628 29.2
// and 26.8; 8 experts, 4096 gated features: 312 22.5 and 25.3, 1064 76.4 and 72.8.
constexpr int64_t kBwdFewTiles = 512;
constexpr int kBwdCols = 512;   // output features per workgroup
constexpr int kBwdZero = 64;    // workgroups that clear rows no route fills

// act(z) and act'(z). The derivatives of the smooth ones are exactly 0 or 1 in float32
// at and beyond the clamps; past them their terms would meet as 0 times infinity. NaN passes.
__device__ __forceinline__ float clamp_to(float z, float c) { return z > c ? c : z < -c ? -c : z; }

template <int ACT>
__device__ __forceinline__ void act_and_slope(float z, float* f, float* d) {
  if constexpr (ACT == kActRelu) {
    *f = z > 0.0f || z != z ? z : 0.0f;
    *d = z > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == kActGelu) {
    const float y = clamp_to(z, 30.0f);
    float E;
    const float cdf = normal_cdf(y, &E);
    *f = z * cdf;
    *d = cdf + y * 0.3989422804014327f * E;
  } else if constexpr (ACT == kActGeluTanh) {
    const float y = clamp_to(z, 12.0f);
    const float s = sigmoid(kTanhB * (y + kTanhQ * y * y * y));
    *f = z * s;
    *d = s + y * s * (1.0f - s) * kTanhB * (1.0f + 3.0f * kTanhQ * y * y);
  } else if constexpr (ACT == kActSilu) {
    const float y = clamp_to(z, 120.0f);
    const float s = sigmoid(y);
    *f = z * s;
    *d = s * (1.0f + y * (1.0f - s));
  } else {
    *f = z;
    *d = 1.0f;
  }
}

// Eight values in two bf16 parts whose sum is off by at most 2^-17 of each (above bf16's subnormals).
// Past bf16's largest value a finite one's first part is that value; an infinity or NaN is all in it.
__device__ __forceinline__ void bf16_parts(const float (&v)[8], chunk_t* hi, chunk_t* lo) {
  constexpr float kMost = 3.3895313892515355e38f;  // (2 - 2^-7) 2^127
  float h[8], l[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) h[q] = __builtin_fabsf(v[q]) < INFINITY ? clamp_to(v[q], kMost) : v[q];
  *hi = pack<kBF16>(h);
  unpack<kBF16>(*hi, h);
#pragma unroll
  for (int q = 0; q < 8; ++q) l[q] = __builtin_fabsf(v[q]) < INFINITY ? v[q] - h[q] : 0.0f;
  *lo = pack<kBF16>(l);
}

template <int DT, int ACT, bool GATED, bool Z32>
__global__ __launch_bounds__(kBwdThreads) void expert_act_backward_kernel(ExpertActBackward p, int col_blocks,
                                                                          int shift, int tile_grid, float* __restrict__ bias_part,
                                                                          double* __restrict__ dot_part) {
  constexpr int H = GATED ? 2 : 1;  // halves of z
  constexpr int C = Z32 ? 2 : 1;    // 16-byte pieces of eight of its values
  __shared__ float row_w[kBwdRows];
  __shared__ float sums[kBwdWaves][kBwdCols];
  const int tid = threadIdx.x, lane = lane_id(), wv = wave_in_block();
  if (static_cast<int>(blockIdx.x) >= tile_grid) {  // rows no route fills
    const int wave = (blockIdx.x - tile_grid) * kBwdWaves + wv, waves = (gridDim.x - tile_grid) * kBwdWaves;
    const chunk_t z = {0u, 0u, 0u, 0u};
    auto clear = [&](int r) {
      if (p.grad_preact != nullptr) {
        const size_t chunks = static_cast<size_t>(p.parts) * p.nz / 8;
        chunk_t* o = static_cast<chunk_t*>(p.grad_preact) + static_cast<size_t>(r) * chunks;
        for (size_t c = lane; c < chunks; c += kWave) o[c] = z;
      }
      if (p.grad_residual != nullptr) {
        chunk_t* o = reinterpret_cast<chunk_t*>(static_cast<uint16_t*>(p.grad_residual) + static_cast<size_t>(r) * p.n);
        for (int c = lane; c < p.n / 8; c += kWave) o[c] = z;
      }
    };
    const int per = waves > p.e ? waves / p.e : 1;
    for (int64_t item = wave; item < static_cast<int64_t>(p.e) * per; item += waves) {
      const int x = static_cast<int>(item % p.e), sub = static_cast<int>(item / p.e);
      for (int r = p.offsets[x] + p.kept[x] + sub; r < p.offsets[x + 1]; r += per) clear(r);
    }
    for (int64_t r = static_cast<int64_t>(p.offsets[p.e]) + wave; r < p.rows; r += waves) clear(static_cast<int>(r));
    return;
  }
  const SegmentTile tc =
      segment_tile(blockIdx.x, p.e, p.kept, p.offsets, col_blocks, 8, [shift](int r) { return (r + (1 << shift) - 1) >> shift; });
  const int x = tc.expert;
  if (x < 0) return;
  const int row0 = tc.offset + (tc.rb << shift);
  const int rem = tc.rows - (tc.rb << shift);
  const int nrows = rem < 1 << shift ? rem : 1 << shift;
  const int c = tc.cb * kBwdCols + 8 * lane;
  const bool in = c < p.n;
  if (p.route_w != nullptr) {
    if (tid < nrows) {
      const int r = row0 + tid, t = p.src[r];
      float w = 1.0f;
      for (int j = 0; j < p.k; ++j)
        if (p.dst[static_cast<size_t>(t) * p.k + j] == r) w = p.route_w[static_cast<size_t>(t) * p.k + j];
      row_w[tid] = w;
    }
  }

  float acc[H][8];
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[h][q] = 0.0f;
  const uint16_t* gout = static_cast<const uint16_t*>(p.grad_out) + c;
  const chunk_t* zin = static_cast<const chunk_t*>(p.preact);
  // kDepth rows of a wave in flight: each is loaded that many rows before it is worked on (with
  // float32 z two measure the same)
  constexpr int kDepth = 4;
  chunk_t gv[kDepth], zv[kDepth][H][C];
  auto load = [&](int i, int b) __attribute__((always_inline)) {
    const chunk_t none = {0u, 0u, 0u, 0u};
    const size_t r = static_cast<size_t>(row0 + i);
    gv[b] = in ? *reinterpret_cast<const chunk_t*>(gout + r * p.n) : none;
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int q = 0; q < C; ++q) zv[b][h][q] = in && p.preact != nullptr ? zin[(r * p.nz + h * p.n + c) / 8 * C + q] : none;
  };
  auto work = [&](int i, int b) __attribute__((always_inline)) {
    const int r = row0 + i;
    float g[8], z[H][8], d[H][8];
    unpack<DT>(gv[b], g);
#pragma unroll
    for (int h = 0; h < H; ++h) {
      if constexpr (Z32) {
#pragma unroll
        for (int q = 0; q < 8; ++q) z[h][q] = __uint_as_float(zv[b][h][q / 4][q % 4]);
      } else {
        unpack<DT>(zv[b][h][0], z[h]);
      }
    }
    const float w = p.route_w != nullptr ? row_w[i] : 1.0f;
    float dot = 0.0f;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      float f, s;
      act_and_slope<ACT>(z[0][q], &f, &s);
      const float gw = p.route_w != nullptr ? w * g[q] : g[q];
      if constexpr (GATED) {
        dot += g[q] * (f * z[1][q]);
        d[0][q] = gw * z[1][q] * s;
        d[1][q] = gw * f;
      } else {
        dot += g[q] * f;
        d[0][q] = ACT == kActNone ? gw : gw * s;
      }
    }
    if (in) {
#pragma unroll
      for (int h = 0; h < H; ++h) {
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[h][q] += d[h][q];
        if (p.grad_preact != nullptr) {
          uint16_t* o = static_cast<uint16_t*>(p.grad_preact) + static_cast<size_t>(r) * p.nz * p.parts + h * p.n + c;
          if (p.parts == 1) *reinterpret_cast<chunk_t*>(o) = pack<DT>(d[h]);
          else bf16_parts(d[h], reinterpret_cast<chunk_t*>(o), reinterpret_cast<chunk_t*>(o + p.nz));
        }
      }
      if (p.grad_residual != nullptr)
        *reinterpret_cast<chunk_t*>(static_cast<uint16_t*>(p.grad_residual) + static_cast<size_t>(r) * p.n + c) = gv[b];
    }
    if (p.grad_w != nullptr) {  // lanes past n hold zeros
      const double total = wave_sum(static_cast<double>(dot));
      if (lane == 0) dot_part[static_cast<size_t>(r) * col_blocks + tc.cb] = total;
    }
  };
#pragma unroll
  for (int b = 0; b < kDepth; ++b)
    if (wv + b * kBwdWaves < nrows) load(wv + b * kBwdWaves, b);
  if (p.route_w != nullptr) __syncthreads();  // row_w
  for (int i = wv; i < nrows; i += kDepth * kBwdWaves) {  // uniform conditions per wave
#pragma unroll
    for (int b = 0; b < kDepth; ++b) {
      if (i + b * kBwdWaves < nrows) work(i + b * kBwdWaves, b);
      if (i + (b + kDepth) * kBwdWaves < nrows) load(i + (b + kDepth) * kBwdWaves, b);
    }
  }
  if (p.grad_bias == nullptr) return;
  // Tile rb of expert x owns partial row (offsets[x] >> shift) + x + rb: as floor(a + b) >=
  // floor(a) + ceil(b) - 1, the next expert's first is past this one's last.
  const size_t slot = static_cast<size_t>(tc.offset >> shift) + x + tc.rb;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 8; q += 4)
      *reinterpret_cast<chunk_t*>(&sums[wv][8 * lane + q]) =
          chunk_t{__float_as_uint(acc[h][q]), __float_as_uint(acc[h][q + 1]), __float_as_uint(acc[h][q + 2]),
                  __float_as_uint(acc[h][q + 3])};
    __syncthreads();
    for (int f = tid; f < kBwdCols && tc.cb * kBwdCols + f < p.n; f += kBwdThreads) {
      float sum = sums[0][f];
#pragma unroll
      for (int v = 1; v < kBwdWaves; ++v) sum += sums[v][f];
      bias_part[slot * p.nz + h * p.n + tc.cb * kBwdCols + f] = sum;
    }
  }
}

// Second launch. The first bias_grid workgroups each take 64 features of one expert: 16
// lanes of four by 16 partial rows at a time, summed in float64, then in order. The others
// take a route per thread.
template <int DT>
__global__ __launch_bounds__(kBwdThreads) void expert_act_backward_sums_kernel(ExpertActBackward p, int col_blocks, int shift,
                                                                               int bias_blocks, int64_t bias_grid,
                                                                               const float* __restrict__ bias_part,
                                                                               const double* __restrict__ dot_part) {
  __shared__ double sums[16][64];
  const int tid = threadIdx.x;
  if (static_cast<int64_t>(blockIdx.x) < bias_grid) {
    const int x = blockIdx.x / bias_blocks, c0 = blockIdx.x % bias_blocks * 64;
    const int tiles = (p.kept[x] + (1 << shift) - 1) >> shift;
    const size_t slot = static_cast<size_t>(p.offsets[x] >> shift) + x;
    const int c = c0 + 4 * (tid % 16);
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    if (c < p.nz) {  // nz is a multiple of 8
#pragma unroll 4
      for (int i = tid / 16; i < tiles; i += 16) {
        const chunk_t v = *reinterpret_cast<const chunk_t*>(bias_part + (slot + i) * p.nz + c);
#pragma unroll
        for (int q = 0; q < 4; ++q) s[q] += static_cast<double>(__uint_as_float(v[q]));
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) sums[tid / 16][4 * (tid % 16) + q] = s[q];
    __syncthreads();
    if (tid < 64 && c0 + tid < p.nz) {
      double total = 0.0;
      for (int i = 0; i < 16; ++i) total += sums[i][tid];
      const size_t at = static_cast<size_t>(x) * p.nz + c0 + tid;
      if (p.bias_f32) static_cast<float*>(p.grad_bias)[at] = static_cast<float>(total);
      else static_cast<uint16_t*>(p.grad_bias)[at] = narrow<DT>(static_cast<float>(total));
    }
    return;
  }
  const int64_t q = (static_cast<int64_t>(blockIdx.x) - bias_grid) * kBwdThreads + tid;
  if (q >= static_cast<int64_t>(p.s) * p.k) return;
  const int r = p.dst[q];
  double total = 0.0;
  if (r >= 0)
    for (int b = 0; b < col_blocks; ++b) total += dot_part[static_cast<size_t>(r) * col_blocks + b];
  p.grad_w[q] = static_cast<float>(total);
}

ExpertActBackwardPlan expert_act_backward_plan(const LayoutView& L, int n, bool gated) {
  ExpertActBackwardPlan p{};
  const int nz = gated ? 2 * n : n;
  p.col_blocks = (n + kBwdCols - 1) / kBwdCols;
  const int64_t routes = static_cast<int64_t>(L.s) * L.k;
  const int64_t placed = routes < L.rows ? routes : L.rows;
  auto tiles_of = [&](int shift) {
    return L.s == 0 ? 0 : ((placed >> shift) + (placed < L.e ? placed : L.e)) * p.col_blocks;
  };
  p.shift = tiles_of(6) < kBwdFewTiles ? 4 : 6;
  const int64_t tiles = tiles_of(p.shift);
  p.slots = (L.rows >> p.shift) + L.e + 1;
  p.grid = (tiles + kXcds - 1) / kXcds * kXcds;
  p.off_bias = 0;
  p.off_dots = (static_cast<size_t>(p.slots) * nz * 4 + 255) / 256 * 256;
  p.bytes = p.off_dots + (static_cast<size_t>(L.rows) * p.col_blocks * 8 + 255) / 256 * 256;
  return p;
}

// The second launch's workgroups: those of the bias sums, and all.
static void sums_grid(int64_t s, int k, int e, int nz, bool bias, bool weights, int64_t* bias_grid, int64_t* grid) {
  *bias_grid = bias ? static_cast<int64_t>(e) * ((nz + 63) / 64) : 0;
  *grid = *bias_grid + (weights ? (s * k + kBwdThreads - 1) / kBwdThreads : 0);
}

bool expert_act_backward_fits(const LayoutView& L, const ExpertActBackwardPlan& plan, int nz, bool bias, bool weights) {
  int64_t bias_grid = 0, grid = 0;
  sums_grid(L.s, L.k, L.e, nz, bias, weights, &bias_grid, &grid);
  return plan.grid + kBwdZero <= most_workgroups(kBwdThreads) && grid <= most_workgroups(kBwdThreads);
}

template <int DT, int ACT>
static void launch_first(const ExpertActBackward& p, const ExpertActBackwardPlan& plan, float* bias_part,
                         double* dot_part, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(plan.grid + kBwdZero);
  const int tile_grid = static_cast<int>(plan.grid);
  auto go = [&](auto gated, auto z32) {
    expert_act_backward_kernel<DT, ACT, decltype(gated)::value, decltype(z32)::value>
        <<<grid, kBwdThreads, 0, stream>>>(p, plan.col_blocks, plan.shift, tile_grid, bias_part, dot_part);
  };
  using std::true_type, std::false_type;
  if (p.gated) p.preact_f32 ? go(true_type{}, true_type{}) : go(true_type{}, false_type{});
  else p.preact_f32 ? go(false_type{}, true_type{}) : go(false_type{}, false_type{});
}

template <int DT>
static hipError_t launch_dt(const ExpertActBackward& p, const ExpertActBackwardPlan& plan, char* ws,
                            hipStream_t stream) {
  float* bias_part = reinterpret_cast<float*>(ws + plan.off_bias);
  double* dot_part = reinterpret_cast<double*>(ws + plan.off_dots);
  switch (p.act) {
    case kActRelu: launch_first<DT, kActRelu>(p, plan, bias_part, dot_part, stream); break;
    case kActGelu: launch_first<DT, kActGelu>(p, plan, bias_part, dot_part, stream); break;
    case kActGeluTanh: launch_first<DT, kActGeluTanh>(p, plan, bias_part, dot_part, stream); break;
    case kActSilu: launch_first<DT, kActSilu>(p, plan, bias_part, dot_part, stream); break;
    default: launch_first<DT, kActNone>(p, plan, bias_part, dot_part, stream); break;
  }
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || (p.grad_bias == nullptr && p.grad_w == nullptr)) return err;
  const int bias_blocks = (p.nz + 63) / 64;
  int64_t bias_grid = 0, grid = 0;
  sums_grid(p.s, p.k, p.e, p.nz, p.grad_bias != nullptr, p.grad_w != nullptr, &bias_grid, &grid);
  if (grid == 0) return hipSuccess;
  expert_act_backward_sums_kernel<DT><<<static_cast<unsigned>(grid), kBwdThreads, 0, stream>>>(
      p, plan.col_blocks, plan.shift, bias_blocks, bias_grid, bias_part, dot_part);
  return hipGetLastError();
}

hipError_t launch_expert_act_backward(const LayoutView& L, const ExpertActBackward& p,
                                      const ExpertActBackwardPlan& plan, char* ws, int dtype, hipStream_t stream) {
  return dtype == kBF16 ? launch_dt<kBF16>(p, plan, ws, stream) : launch_dt<kF16>(p, plan, ws, stream);
}

}  // namespace moe
