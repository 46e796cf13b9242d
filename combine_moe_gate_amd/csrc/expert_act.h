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

// act(z); gelu_tanh through tanh(y) = 2 sigmoid(2 y) - 1.
__device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    case kActRelu: return z > 0.0f || z != z ? z : 0.0f;
    case kActGelu: return 0.5f * z * (1.0f + erff(z * 0.7071067811865476f));
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
    uint16_t* row = static_cast<uint16_t*>(p.preact) + static_cast<size_t>(r) * p.nz + c;
    *reinterpret_cast<chunk_t*>(row) = pack<DT>(v);
    if (p.gated) *reinterpret_cast<chunk_t*>(row + p.n) = pack<DT>(u);
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
      chunk_t* q = reinterpret_cast<chunk_t*>(static_cast<uint16_t*>(p.preact) + static_cast<size_t>(r) * p.nz);
      for (int c = lane; c < p.nz / 8; c += kWave) q[c] = z;
    }
  };
  const int per = waves > p.e ? waves / p.e : 1;  // waves that share an expert's tail
  for (int64_t item = wave; item < static_cast<int64_t>(p.e) * per; item += waves) {
    const int x = static_cast<int>(item % p.e), sub = static_cast<int>(item / p.e);
    for (int r = p.offsets[x] + p.kept[x] + sub; r < p.offsets[x + 1]; r += per) clear(r);
  }
  for (int64_t r = static_cast<int64_t>(p.offsets[p.e]) + wave; r < p.rows; r += waves) clear(static_cast<int>(r));
}

}  // namespace moe
