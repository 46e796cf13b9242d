// Activations and the epilogue shared by the kernels of the expert products.
#pragma once

#include "gemm_common.h"
#include "ops.h"

namespace moe {

// 1 / (1 + exp(-x)) through the hardware's base-2 exponential and reciprocal (each within
// an ulp or so): 0 and 1 at the ends, NaN stays NaN.
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.4426950408889634f));
}

constexpr float kTanhB = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kTanhQ = 0.044715f;

// Phi(z), the normal distribution function, with E = exp(-z^2 / 2) on the way. With x = |z| /
// sqrt 2, erfc(x) / 2 = t P(t) E, t = 1 / (1 + x / 2), in the form of Abramowitz and Stegun,
// Handbook of Mathematical Functions, 7.1.26. That formula's own coefficients bound the error of
// erfc, not its share of erfc, and far below 0 gelu would lose its digits (0.2% off at z = -5, 1%
// at -8); these are a least-maximum fit of the share for x up to 9.6: 4e-8. Evaluated in float32
// Phi(z) is within 2^-24 (22 + 1.5 z^2) of itself at z <= 0, and within 24 times 2^-24 above.
// 65536 x 4096 outputs of 256 products each take 384 us with it, 376 with 7.1.26's five
// coefficients (where erff took 1.23 times as long), 270 without an activation.
__device__ __forceinline__ float normal_cdf(float z, float* E) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.35355338f, __builtin_fabsf(z), 1.0f));
  float q = __builtin_fmaf(t, -0.029465698f, 0.14195059f);
  q = __builtin_fmaf(t, q, -0.24289933f);
  q = __builtin_fmaf(t, q, 0.13822806f);
  q = __builtin_fmaf(t, q, -0.012754773f);
  q = __builtin_fmaf(t, q, 0.10110577f);
  q = __builtin_fmaf(t, q, 0.1216124f);
  q = __builtin_fmaf(t, q, 0.14117926f);
  q = __builtin_fmaf(t, q, 0.1410437f);
  *E = __builtin_amdgcn_exp2f(z * z * -0.7213475204444817f);
  q = q * t * *E;  // erfc(x) / 2
  return z < 0.0f ? q : 1.0f - q;
}

// act(z); gelu_tanh through tanh(y) = 2 sigmoid(2 y) - 1.
__device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    case kActRelu: return z > 0.0f || z != z ? z : 0.0f;
    case kActGelu: {
      float E;
      return z * normal_cdf(z, &E);
    }
    case kActGeluTanh: return z * sigmoid(kTanhB * (z + kTanhQ * z * z * z));
    case kActSilu: return z * sigmoid(z);
    default: return z;
  }
}

// Eight elements of a bias row: float32 or the element type.
template <int DT>
__device__ __forceinline__ void load8(const void* p, size_t at, bool f32, float (&f)[8]) {
  if (f32) {
    const chunk_t* q = reinterpret_cast<const chunk_t*>(static_cast<const float*>(p) + at);
    const chunk_t a = q[0], b = q[1];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      f[u] = __uint_as_float(a[u]);
      f[4 + u] = __uint_as_float(b[u]);
    }
  } else {
    unpack<DT>(*reinterpret_cast<const chunk_t*>(static_cast<const uint16_t*>(p) + at), f);
  }
}

// Eight elements of a row of kept values: float32, or rounded to the element type. A finite value
// past f16's largest is kept as that: as an infinity it would meet a slope or an activation of 0
// in the backward, where the forward had a finite product.
template <int DT>
__device__ __forceinline__ void store8(void* p, size_t at, bool f32, const float (&f)[8]) {
  if (f32) {
    chunk_t* q = reinterpret_cast<chunk_t*>(static_cast<float*>(p) + at);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      q[h] = chunk_t{__float_as_uint(f[4 * h]), __float_as_uint(f[4 * h + 1]), __float_as_uint(f[4 * h + 2]),
                     __float_as_uint(f[4 * h + 3])};
  } else {
    float g[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      g[u] = DT == kF16 && __builtin_fabsf(f[u]) < INFINITY ? fminf(fmaxf(f[u], -65504.0f), 65504.0f) : f[u];
    *reinterpret_cast<chunk_t*>(static_cast<uint16_t*>(p) + at) = pack<DT>(g);
  }
}

// The route weight of buffer row r (token t): that of the route placed there.
__device__ __forceinline__ float route_weight(const ExpertAct& p, int r, int t) {
  float w = 1.0f;
  for (int j = 0; j < p.k; ++j)
    if (p.dst[static_cast<size_t>(t) * p.k + j] == r) w = p.route_w[static_cast<size_t>(t) * p.k + j];
  return w;
}

// Eight output features c .. c + 7 of buffer row r of expert x, from the float32 products
// v (gated: of the gate rows, u those of the up rows): bias, activation, route weight w,
// residual, one rounding, whole 16-byte stores. c + 8 <= n.
template <int DT>
__device__ __forceinline__ void finish8(const ExpertAct& p, int x, int r, int t, float w, int c, float (&v)[8],
                                        float (&u)[8]) {
  if (p.bias != nullptr) {
    float b[8];
    load8<DT>(p.bias, static_cast<size_t>(x) * p.nz + c, p.bias_f32, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
    if (p.gated) {
      load8<DT>(p.bias, static_cast<size_t>(x) * p.nz + p.n + c, p.bias_f32, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] += b[i];
    }
  }
  if (p.preact != nullptr) {
    const size_t at = static_cast<size_t>(r) * p.nz + c;
    store8<DT>(p.preact, at, p.preact_f32, v);
    if (p.gated) store8<DT>(p.preact, at + p.n, p.preact_f32, u);
  }
  switch (p.act) {  // uniform
#define MOE_ACT_CASE(A)                                         \
  case A:                                                       \
    _Pragma("unroll") for (int i = 0; i < 8; ++i) v[i] = activate(A, v[i]); \
    break;
    MOE_ACT_CASE(kActRelu)
    MOE_ACT_CASE(kActGelu)
    MOE_ACT_CASE(kActGeluTanh)
    MOE_ACT_CASE(kActSilu)
#undef MOE_ACT_CASE
    default: break;
  }
  if (p.gated) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= u[i];
  }
  if (p.route_w != nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= w;
  }
  if (p.residual != nullptr) {
    float b[8];
    unpack<DT>(*reinterpret_cast<const chunk_t*>(static_cast<const uint16_t*>(p.residual) +
                                                 static_cast<size_t>(p.residual_gather ? t : r) * p.n + c),
               b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
  }
  *reinterpret_cast<chunk_t*>(static_cast<uint16_t*>(p.out) + static_cast<size_t>(r) * p.n + c) = pack<DT>(v);
}

// Zero the rows of the output (and of the kept values) that no route fills: block b of nb,
// a row per wave at a time.
__device__ __forceinline__ void zero_unfilled(const ExpertAct& p, int b, int nb) {
  const int lane = lane_id(), wpb = blockDim.x / kWave;
  const int wave = b * wpb + wave_in_block(), waves = nb * wpb;
  const chunk_t z = {0u, 0u, 0u, 0u};
  auto clear = [&](int r) {
    chunk_t* o = reinterpret_cast<chunk_t*>(static_cast<uint16_t*>(p.out) + static_cast<size_t>(r) * p.n);
    for (int c = lane; c < p.n / 8; c += kWave) o[c] = z;
    if (p.preact != nullptr) {
      const size_t chunks = p.preact_f32 ? p.nz / 4 : p.nz / 8;
      chunk_t* q = static_cast<chunk_t*>(p.preact) + static_cast<size_t>(r) * chunks;
      for (size_t c = lane; c < chunks; c += kWave) q[c] = z;
    }
  };
  const int per = waves > p.e ? waves / p.e : 1;  // waves that share an expert's tail
  for (int64_t item = wave; item < static_cast<int64_t>(p.e) * per; item += waves) {
    const int x = static_cast<int>(item % p.e), sub = static_cast<int>(item / p.e);
    for (int r = p.offsets[x] + p.kept[x] + sub; r < p.offsets[x + 1]; r += per) clear(r);
  }
  for (int64_t r = static_cast<int64_t>(p.offsets[p.e]) + wave; r < p.rows; r += waves) clear(static_cast<int>(r));
}

// Inclusive sum over the wave's lanes, by DPP moves alone: shifts by 1, 2, 4, 8 within each
// row of 16, then each odd row takes the last lane before it, then the upper half.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15 into rows 1, 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31 into rows 2, 3
  return v;
}

struct SegmentTile {
  int expert;      // -1: this workgroup has no tile
  int rows;        // placed rows of the expert
  int offset;      // its first buffer row
  int blocks;      // its row-blocks
  int rb, cb;      // row-block and column-block
};

// This workgroup's tile. A segment of r rows has blocks(r) row-blocks. The tiles of all
// experts are numbered expert by expert, inside an expert in bands of `band` row-blocks,
// column-block by column-block, row-block fastest; workgroup b (dealt round-robin over the 8
// XCDs) takes tile (b mod 8) T8 + b / 8, T8 = ceil(tiles / 8), so that each XCD walks one
// stretch of that order and its resident workgroups share weights and rows through its L2.
// Each lane holds up to 16 neighbouring experts, so one load round and one scan find it.
template <class Blocks>
__device__ __forceinline__ SegmentTile segment_tile(int b, int e, const int32_t* __restrict__ kept,
                                                    const int32_t* __restrict__ offsets, int col_blocks, int band,
                                                    Blocks blocks) {
  const int lane = lane_id();
  const int each = (e + kWave - 1) / kWave;  // at most 16
  int rows[16], offs[16], sum = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    rows[i] = offs[i] = 0;
    if (i < each) {  // uniform
      const int x = lane * each + i;
      if (x < e) {
        rows[i] = kept[x];
        offs[i] = offsets[x];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < each) sum += blocks(rows[i]);
  const int upto = wave_scan(sum);
  const int total = __builtin_amdgcn_readlane(upto, kWave - 1);
  SegmentTile tc{-1, 0, 0, 0, 0, 0};
  const int64_t tiles = static_cast<int64_t>(total) * col_blocks;
  const int64_t per_xcd = (tiles + kXcds - 1) / kXcds;
  const int64_t slot = b / kXcds, t = (b % kXcds) * per_xcd + slot;
  if (slot >= per_xcd || t >= tiles) return tc;
  const int q = static_cast<int>(t / col_blocks);  // its ordinal among the row-blocks, less the band order
  int run = upto - sum, at = 0, at_rows = 0, at_off = 0, first = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (i < each) {
      const int nb = blocks(rows[i]);
      if (q >= run && q < run + nb) {
        at = lane * each + i;
        at_rows = rows[i];
        at_off = offs[i];
        first = run;
      }
      run += nb;
    }
  }
  const uint64_t hit = __ballot(q >= upto - sum && q < upto);  // one lane: the ranges partition [0, total)
  const int owner = static_cast<int>(__builtin_ctzll(hit));
  tc.expert = __builtin_amdgcn_readlane(at, owner);
  tc.rows = __builtin_amdgcn_readlane(at_rows, owner);
  tc.offset = __builtin_amdgcn_readlane(at_off, owner);
  first = __builtin_amdgcn_readlane(first, owner);
  tc.blocks = blocks(tc.rows);
  const int u = static_cast<int>(t - static_cast<int64_t>(first) * col_blocks);
  const int bd = u / (band * col_blocks);
  const int left = tc.blocks - bd * band;
  const int in_band = left < band ? left : band;
  const int v = u - bd * band * col_blocks;
  tc.cb = __builtin_amdgcn_readfirstlane(v / in_band);  // uniform as they are: kept in scalar registers
  tc.rb = __builtin_amdgcn_readfirstlane(bd * band + v % in_band);
  return tc;
}

}  // namespace moe
