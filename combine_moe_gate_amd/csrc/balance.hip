// The router's load-balance loss, z loss and per-expert counts on gfx950, and their
// gradient with respect to the logits.
//
// For the tokens V_g of group g (a packed sequence, or the whole batch) that are not
// padding, n = |V_g|, with p_t = softmax(l_t) over all e experts and c_x the number of
// V_g's valid routes that name expert x:
//     P_x  = (1 / n) sum_t p_tx
//     loss = (e / k) sum_x (c_x / n) P_x           (1 where the load is level)
//     z    = (1 / n) sum_t logsumexp(l_t)^2
//     d/dl_ti = p_ti [ gL e / (k n^2) (c_i - sum_x p_tx c_x) + gZ (2 / n) logsumexp(l_t) ]
// The counts carry no gradient (they are whole numbers). As sum_x p_tx = 1, the bracket
// keeps its value when every c_x is shifted alike: the kernel uses c_x - k n / e, whose
// differences survive float32 where those of the counts themselves would not.
//
// Both directions stream the logits once (the backward forms the softmax again: reading
// 4 e bytes per token costs what a saved copy would) and are bound by that traffic.
//
// A token's row lies across LPT lanes (4, 16 or a whole wave, the fewest that hold e at
// four to sixteen values a lane), so a lane keeps the same experts for all its tokens and
// the column sums P stay in its registers over the tile. One softmax needs a maximum and
// a sum over the LPT lanes, DPP steps without LDS. Tiles are contiguous tokens; a tile
// adds up its waves' sums in a fixed order and writes one partial row per group it meets,
// and a second launch adds the partial rows of each group, in float64 and tile order.
// Nothing depends on an order of arrival: sums are taken in a fixed order, and the only
// atomics are integer counts.
//
// Measured: 65536 tokens, 512 experts, 10 routes: forward 43 us (35 after a pause) and 7 us for
// the partial rows, 137 MB read, 3.2 TB/s where loads alone reach 6.8; backward 46 us, 268 MB,
// 5.9 TB/s, its reads partly from the Infinity Cache. 32768 tokens, 128 experts, 8 routes: 9 + 7
// us and 10 us for 18 and 34 MB, 16381 of 60 experts in 29 groups 12 + 7 us and 7 us for 4 and 8
// MB: not bandwidth but loads that wait for each other (the group's offsets, then rows, routes
// and partial rows), with a tile or two per CU. One tile, 256 tokens, 8 experts: 5 us and 3 us.
#include <type_traits>

#include "moe_device.h"
#include "ops.h"

namespace moe {

constexpr int kBalBlock = 512;  // threads per workgroup of both directions
constexpr int kBalWaves = kBalBlock / kWave;
constexpr int kBalTiles = 512;  // most tiles: two workgroups per CU
constexpr int kBalMinTile = 32;
constexpr int kBalChunk = 16;  // experts per workgroup of the second launch
constexpr int kBalReduce = 256;  // its threads
// Batches of up to this many logits and tokens are one tile, finished by the first launch
// alone (and those of up to kBalMinTile tokens, which are one tile at any width: up to 32768
// logits). One launch against two, microseconds: 8 experts 8192 logits 8.5 to 8.7, 16384 12.2 to
// 9.3; 64 experts 16384 9.1 to 10.2, 32768 13.7 to 10.1; 256 experts 16384 8.4 to 10.8, 32768
// 12.6 to 11.0.
constexpr int64_t kBalSingle = 16384;
constexpr int kBalSingleTokens = 1024;

BalancePlan balance_plan(int32_t s, int32_t e, int32_t g) {
  BalancePlan p{};
  if (g == 1 && s <= kBalSingleTokens && static_cast<int64_t>(s) * e <= kBalSingle) {
    p.tile = s > 0 ? s : 1;
  } else {
    p.tile = (s + kBalTiles - 1) / kBalTiles;
    if (p.tile < kBalMinTile) p.tile = kBalMinTile;
  }
  p.ntiles = s > 0 ? (s - 1) / p.tile + 1 : 1;
  p.pitch = (e + 3) / 4 * 4;
  p.chunks = (e + kBalChunk - 1) / kBalChunk;
  p.slots = static_cast<int64_t>(p.ntiles) + g - 1;
  if (p.ntiles == 1 && g == 1) return p;  // finished by the first launch: no partial rows
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at = (at + n + 255) / 256 * 256;
    return here;
  };
  p.off_probs = take(static_cast<size_t>(p.slots) * p.pitch * 4);
  p.off_counts = take(static_cast<size_t>(p.slots) * p.pitch * 4);
  p.off_z = take(static_cast<size_t>(p.slots) * 8);
  p.off_tokens = take(static_cast<size_t>(p.slots) * 4);
  p.off_dots = take(static_cast<size_t>(g) * p.chunks * 8);
  p.off_arrived = take(static_cast<size_t>(g) * 4);
  p.bytes = at;
  return p;
}

// ---------------------------------------------------------------------------------
// reductions over the LPT lanes that share a token (every lane of the wave active)

template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}

template <int LPT, class Op>
__device__ __forceinline__ float lanes_reduce(float v, Op op) {
  static_assert(LPT == 4 || LPT == 16 || LPT == 64, "a quad, a row or the wave");
  v = op(v, dpp_move<0xb1>(v));  // quad_perm [1,0,3,2]
  v = op(v, dpp_move<0x4e>(v));  // quad_perm [2,3,0,1]
  if constexpr (LPT >= 16) {
    v = op(v, dpp_move<0x141>(v));  // row_half_mirror
    v = op(v, dpp_move<0x140>(v));  // row_mirror
  }
  if constexpr (LPT == 64) {
    // gfx950's swaps give every lane the values of its own and of the neighbouring row, then
    // of both halves of the wave
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(p[0]), __uint_as_float(p[1]));
    const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(q[0]), __uint_as_float(q[1]));
  }
  return v;
}

template <int LPT>
__device__ __forceinline__ float lanes_max(float v) {
  return lanes_reduce<LPT>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int LPT>
__device__ __forceinline__ float lanes_sum(float v) {
  return lanes_reduce<LPT>(v, [](float a, float b) { return a + b; });
}

// The group that holds token t: the last one that starts at or before it (-1: none does).
// Offsets that are no rising sequence give some group in range.
__device__ __forceinline__ int group_at(const int32_t* __restrict__ groups, int g, int t) {
  int lo = -1, hi = g;  // groups[lo] <= t < groups[hi], with the ends outside
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (groups[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Column i of lane r: four neighbouring experts per 16-byte load where rows allow them
// (VEC), else experts r, r + LPT, ... so that a load's lanes are neighbours.
template <int LPT, bool VEC>
__device__ __forceinline__ int column(int r, int i) {
  return VEC ? 4 * (r + LPT * (i / 4)) + i % 4 : r + LPT * i;
}

template <int LPT, int NV, bool VEC>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int e, int r, bool live, float (&v)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; i += VEC ? 4 : 1) {
    const int c = column<LPT, VEC>(r, i);
    const bool in = live && c < e;
    if constexpr (VEC) {
      const chunk_t none = {0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u};  // -inf
      chunk_t q = none;
      if (in) q = *reinterpret_cast<const chunk_t*>(row + c);
#pragma unroll
      for (int u = 0; u < 4; ++u) v[i + u] = __uint_as_float(q[u]);
    } else {
      v[i] = in ? row[c] : -INFINITY;
    }
  }
}

// exp(x) for x <= 0 through the hardware's base-2 exponential: a relative error of about
// 2^-23 + |x| 2^-24, against probabilities whose sum is kept to float32.
__device__ __forceinline__ float exp_neg(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }

// Softmax of one row in place: v becomes exp(v - top) and the row's 1 / sum and logsumexp
// come back (both 0 where every logit is -inf: such a token has no distribution and adds
// nothing). NaN and +inf logits make both NaN.
template <int LPT, int NV>
__device__ __forceinline__ void row_softmax(float (&v)[NV], float* inv, float* lse) {
  float top = v[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) top = fmaxf(top, v[i]);
  top = lanes_max<LPT>(top);
  const float base = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    v[i] = exp_neg(v[i] - base);
    sum += v[i];
  }
  sum = lanes_sum<LPT>(sum);
  const bool none = sum == 0.0f;
  *inv = none ? 0.0f : 1.0f / sum;
  *lse = none ? 0.0f : base + __logf(sum);
}

// ---------------------------------------------------------------------------------
// forward, first launch: one workgroup per tile

// Sum over the workgroup, in lane and wave order; every thread gets it. `red` holds a
// value per wave.
__device__ __forceinline__ int wave_total(int v) {
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) v += __shfl_xor(v, o, kWave);
  return v;
}
__device__ __forceinline__ double wave_total(double v) { return wave_sum(v); }
template <class T>
__device__ __forceinline__ T block_sum(T v, T* red) {
  v = wave_total(v);
  __syncthreads();
  if (lane_id() == 0) red[wave_in_block()] = v;
  __syncthreads();
  T total = red[0];
  for (int w = 1; w < static_cast<int>(blockDim.x) / kWave; ++w) total += red[w];
  return total;
}

struct BalanceOut {
  int32_t* counts;  // [g, e]
  int32_t* tokens;  // [g]
  float* probs;     // [g, e]
  float* loss;      // [g]
  float* z;         // [g]
};

struct BalancePartials {
  float* probs;     // [slots, pitch]
  int32_t* counts;  // [slots, pitch]
  double* z;        // [slots]
  int32_t* tokens;  // [slots]
  double* dots;     // [g, chunks]
  int32_t* arrived; // [g]
};

template <int LPT, int NV, bool VEC>
__global__ __launch_bounds__(kBalBlock) void balance_tile_kernel(BalanceArgs a, int tile, int pitch, bool single,
                                                                 BalancePartials part, BalanceOut out) {
  constexpr int kGroups = kBalBlock / LPT;  // tokens in work at once
  constexpr int U = NV >= 16 ? 1 : 2;       // rows in work at once per lane group
  constexpr int kCols = LPT * NV;
  __shared__ float sums[kBalWaves][kCols];
  __shared__ int32_t hist[kCols];
  __shared__ double red_z[kBalWaves];
  __shared__ int32_t red_n[kBalWaves];
  const int tid = threadIdx.x, lane = lane_id(), wv = wave_in_block();
  const int r = tid % LPT, gid = tid / LPT;
  const int t0 = blockIdx.x * tile;
  const int t1 = a.s - t0 > tile ? t0 + tile : a.s;

  if (!single)  // for the second launch
    for (int i = blockIdx.x * kBalBlock + tid; i < a.g; i += gridDim.x * kBalBlock) part.arrived[i] = 0;
  int j = 0;
  if (a.groups != nullptr) {
    j = group_at(a.groups, a.g, t0);
    if (j < 0) j = 0;
  }
  for (; j < a.g; ++j) {
    int lo = t0, hi = t1;
    if (a.groups != nullptr) {
      const int first = a.groups[j], last = a.groups[j + 1];
      if (first >= t1 && !single) break;
      lo = first > t0 ? first : t0;
      hi = last < t1 ? last : t1;
      if (hi < lo) hi = lo;
    }
    if (lo >= hi && !single) continue;  // uniform; a single tile finishes its group, empty or not

    // U rows per lane group at a time, the next ones loaded while these are worked on
    float v[2][U][NV], acc[NV];
    bool live[2][U];
    auto load = [&](int tb, int b) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = tb + u * kGroups + gid;
        live[b][u] = t < hi && (a.mask == nullptr || a.mask[t] != 0);
        load_row<LPT, NV, VEC>(a.logits + static_cast<size_t>(t < hi ? t : lo) * a.e, a.e, r, live[b][u], v[b][u]);
      }
    };
    if (lo < hi) load(lo, 0);

    // the routes meanwhile: a lane per route, 64 / k tokens to a wave; valid ones are counted,
    // one naming no expert, or the expert of an earlier route of its token, is not
    for (int c = tid; c < kCols; c += kBalBlock) hist[c] = 0;
    __syncthreads();
    const int tokens = kWave / a.k, jj = lane % a.k;
    for (int tb = lo + wv * tokens; tb < hi; tb += kBalWaves * tokens) {  // uniform per wave
      const int t = tb + lane / a.k;
      const bool mine = lane < tokens * a.k && t < hi && (a.mask == nullptr || a.mask[t] != 0);
      const int x = mine ? a.idx[static_cast<size_t>(t) * a.k + jj] : -1;
      bool ok = x >= 0 && x < a.e;
      for (int d = 1; d < a.k; ++d) {
        const int y = __shfl_up(x, d, kWave);
        ok = ok && !(d <= jj && y == x);
      }
      if (ok) atomicAdd(&hist[x], 1);
    }

#pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] = 0.0f;
    double zacc = 0.0;
    int count = 0;
    auto work = [&](int b) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float inv, lse;
        row_softmax<LPT, NV>(v[b][u], &inv, &lse);  // a row that is not live is all -inf: adds nothing
#pragma unroll
        for (int i = 0; i < NV; ++i) acc[i] = __builtin_fmaf(v[b][u][i], inv, acc[i]);
        if (r == 0) {
          zacc += static_cast<double>(lse) * static_cast<double>(lse);
          count += live[b][u];
        }
      }
    };
    constexpr int kStep = U * kGroups;
    for (int tb = lo; tb < hi; tb += 2 * kStep) {  // the same trips for every lane
      const bool more = hi - tb > kStep;           // no overflow: tb < hi
      if (more) load(tb + kStep, 1);
      work(0);
      if (!more) break;
      if (hi - tb > 2 * kStep) load(tb + 2 * kStep, 0);
      work(1);
    }
    // the wave's token groups add up column by column, then the waves in order through LDS
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int o = LPT; o < kWave; o <<= 1) acc[i] += __shfl_xor(acc[i], o, kWave);
      if (lane < LPT) sums[wv][column<LPT, VEC>(r, i)] = acc[i];
    }
    const double zsum = block_sum(zacc, red_z);  // its barriers also order sums and hist
    const int nsum = block_sum(count, red_n);
    if (!single) {
      const size_t slot = static_cast<size_t>(blockIdx.x) + j;
      for (int c = tid; c < pitch; c += kBalBlock) {
        float sum = 0.0f;
        for (int w = 0; w < kBalWaves; ++w) sum += sums[w][c];
        part.probs[slot * pitch + c] = sum;
        part.counts[slot * pitch + c] = hist[c];
      }
      if (tid == 0) {
        part.z[slot] = zsum;
        part.tokens[slot] = nsum;
      }
    } else {  // the only tile of the only group: finished here
      const double n = nsum > 0 ? static_cast<double>(nsum) : 1.0;
      double dot = 0.0;
      for (int c = tid; c < a.e; c += kBalBlock) {
        double sum = 0.0;
        for (int w = 0; w < kBalWaves; ++w) sum += static_cast<double>(sums[w][c]);
        const double p = sum / n;
        out.probs[c] = static_cast<float>(p);
        out.counts[c] = hist[c];
        dot += static_cast<double>(hist[c]) * p;
      }
      dot = block_sum(dot, red_z);
      if (tid == 0) {
        out.tokens[0] = nsum;
        out.z[0] = static_cast<float>(zsum / n);
        out.loss[0] = static_cast<float>(dot * a.e / (static_cast<double>(a.k) * n));
      }
    }
    __syncthreads();  // sums and hist are read out before the next group writes them
  }
}

// Forward, second launch: workgroup (chunk, group - group0) adds the group's partial rows over
// kBalChunk experts: 4 lanes of four experts by 64 rows at a time, in float64, then the 64 in
// order. One workgroup alone draws the partial rows, which other XCDs wrote, at some 40 GB/s:
// 512 rows of 128 experts in one workgroup took 15 us, in eight they take 7 (for 1.2 MB). The
// chunks' shares of the loss go to the group's last workgroup to arrive (counted on `arrived`,
// which the first launch clears), which adds them in chunk order.
__global__ __launch_bounds__(kBalReduce) void balance_reduce_kernel(BalanceArgs a, int group0, int tile, int pitch,
                                                                    int chunks, BalancePartials part, BalanceOut out) {
  constexpr int kRows = kBalReduce / 4;
  __shared__ double psum[kRows][kBalChunk];
  __shared__ int32_t csum[kRows][kBalChunk];
  __shared__ double red_z[kBalReduce / kWave];
  __shared__ int32_t red_n[kBalReduce / kWave];
  const int tid = threadIdx.x, chunk = blockIdx.x % chunks, j = group0 + blockIdx.x / chunks;
  int lo = 0, hi = a.s;
  if (a.groups != nullptr) {
    lo = a.groups[j] > 0 ? a.groups[j] : 0;
    hi = a.groups[j + 1] < a.s ? a.groups[j + 1] : a.s;
  }
  const int64_t s0 = lo < hi ? lo / tile + static_cast<int64_t>(j) : 0;
  const int ns = lo < hi ? (hi - 1) / tile - lo / tile + 1 : 0;

  const int c4 = chunk * kBalChunk + 4 * (tid % 4), row = tid / 4;
  double p[4] = {0.0, 0.0, 0.0, 0.0};
  int32_t q[4] = {0, 0, 0, 0};
  if (c4 < pitch) {
#pragma unroll 4
    for (int i = row; i < ns; i += kRows) {
      const size_t at = static_cast<size_t>(s0 + i) * pitch + c4;
      const chunk_t v = *reinterpret_cast<const chunk_t*>(part.probs + at);
      const chunk_t w = *reinterpret_cast<const chunk_t*>(part.counts + at);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        p[u] += static_cast<double>(__uint_as_float(v[u]));
        q[u] += static_cast<int32_t>(w[u]);
      }
    }
  }
  int count = 0;
  double zacc = 0.0;
  for (int i = tid; i < ns; i += kBalReduce) {
    count += part.tokens[s0 + i];
    zacc += part.z[s0 + i];
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    psum[row][4 * (tid % 4) + u] = p[u];
    csum[row][4 * (tid % 4) + u] = q[u];
  }
  const int nsum = block_sum(count, red_n);  // its barriers also order psum and csum
  const double zsum = block_sum(zacc, red_z);
  const double n = nsum > 0 ? static_cast<double>(nsum) : 1.0;

  double dot = 0.0;
  const int c = chunk * kBalChunk + tid;
  if (tid < kBalChunk && c < a.e) {
    double sum = 0.0;
    int32_t cnt = 0;
#pragma unroll 8
    for (int w = 0; w < kRows; ++w) {
      sum += psum[w][tid];
      cnt += csum[w][tid];
    }
    sum /= n;
    out.probs[static_cast<size_t>(j) * a.e + c] = static_cast<float>(sum);
    out.counts[static_cast<size_t>(j) * a.e + c] = cnt;
    dot = static_cast<double>(cnt) * sum;
  }
  if (tid >= kWave) return;  // the first wave holds every share
  dot = wave_sum(dot);
  if (chunk == 0 && tid == 0) {
    out.tokens[j] = nsum;
    out.z[j] = static_cast<float>(zsum / n);
  }
  const double scale = a.e / (static_cast<double>(a.k) * n);
  if (chunks == 1) {
    if (tid == 0) out.loss[j] = static_cast<float>(dot * scale);
    return;
  }
  double* dots = part.dots + static_cast<size_t>(j) * chunks;
  int before = 0;
  if (tid == 0) {
    __hip_atomic_store(dots + chunk, dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    before = __hip_atomic_fetch_add(part.arrived + j, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (__builtin_amdgcn_readfirstlane(before) != chunks - 1) return;
  // at most 1024 / kBalChunk = 64 chunks: one per lane, added in a fixed order
  static_assert(1024 / kBalChunk <= kWave, "one lane per chunk");
  const double mine = tid < chunks ? __hip_atomic_load(dots + tid, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
  const double total = wave_sum(mine);
  if (tid == 0) out.loss[j] = static_cast<float>(total * scale);
}

// ---------------------------------------------------------------------------------
// backward: the same lanes per token; a lane keeps its experts' shifted counts, scaled,
// for as long as its tokens stay in one group

template <int LPT, int NV, bool VEC>
__global__ __launch_bounds__(kBalBlock) void balance_backward_kernel(
    BalanceArgs a, int tile, const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens,
    const float* __restrict__ grad_loss, const float* __restrict__ grad_z, float* __restrict__ grad) {
  constexpr int kGroups = kBalBlock / LPT;
  constexpr int U = NV >= 16 ? 1 : 2;
  const int tid = threadIdx.x;
  const int r = tid % LPT, gid = tid / LPT;
  const int t0 = blockIdx.x * tile;
  const int t1 = a.s - t0 > tile ? t0 + tile : a.s;
  int j = -1;          // the group whose numbers are held
  float off[NV], zt = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) off[i] = 0.0f;

  for (int tb = t0; tb < t1; tb += U * kGroups) {
    float v[U][NV];
    bool live[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = tb + u * kGroups + gid;
      live[u] = t < t1 && (a.mask == nullptr || a.mask[t] != 0);
      load_row<LPT, NV, VEC>(a.logits + static_cast<size_t>(t < t1 ? t : t0) * a.e, a.e, r, live[u], v[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = tb + u * kGroups + gid;
      int here = 0;
      bool in = live[u];
      if (a.groups != nullptr) {
        here = j;
        const bool kept = j >= 0 && t >= a.groups[j] && t < a.groups[j + 1];
        if (!kept) here = group_at(a.groups, a.g, t);
        in = in && here >= 0 && t < a.groups[here + 1 > 0 ? here + 1 : 0];
      }
      if (in && here != j) {
        j = here;
        const double n = tokens[j] > 0 ? static_cast<double>(tokens[j]) : 1.0;
        const double mean = static_cast<double>(a.k) * n / a.e;
        const double scale = static_cast<double>(grad_loss != nullptr ? grad_loss[j] : 0.0f) * a.e /
                             (static_cast<double>(a.k) * n * n);
        zt = grad_z != nullptr ? static_cast<float>(static_cast<double>(grad_z[j]) * 2.0 / n) : 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = column<LPT, VEC>(r, i);
          off[i] = c < a.e ? static_cast<float>((static_cast<double>(counts[static_cast<size_t>(j) * a.e + c]) - mean) * scale)
                           : 0.0f;
        }
      }
      float inv, lse;
      row_softmax<LPT, NV>(v[u], &inv, &lse);
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        v[u][i] *= inv;
        dot += v[u][i] * off[i];
      }
      dot = lanes_sum<LPT>(dot);
      const float add = zt * lse - dot;
      if (t < t1) {
        float* row = grad + static_cast<size_t>(t) * a.e;
#pragma unroll
        for (int i = 0; i < NV; i += VEC ? 4 : 1) {
          const int c = column<LPT, VEC>(r, i);
          if constexpr (VEC) {
            chunk_t q = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int w = 0; w < 4; ++w)
              if (in) q[w] = __float_as_uint(v[u][i + w] * (off[i + w] + add));
            if (c < a.e) *reinterpret_cast<chunk_t*>(row + c) = q;
          } else {
            if (c < a.e) row[c] = in ? v[u][i] * (off[i] + add) : 0.0f;
          }
        }
      }
    }
  }
}

// Calls f with the lanes per token, values per lane and load width that e and the rows'
// alignment ask for.
template <int LPT, int NV>
struct Rows {
  static constexpr int lpt = LPT, nv = NV;
};
template <class F>
static void with_rows(int e, bool vec, F f) {
  auto go = [&](auto shape) {
    if (vec) f(shape, std::true_type{});
    else f(shape, std::false_type{});
  };
  if (e <= 16) go(Rows<4, 4>{});
  else if (e <= 64) go(Rows<16, 4>{});
  else if (e <= 128) go(Rows<16, 8>{});
  else if (e <= 256) go(Rows<64, 4>{});
  else if (e <= 512) go(Rows<64, 8>{});
  else go(Rows<64, 16>{});
}

static bool rows16(const void* p, int e) { return e % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

hipError_t launch_balance_loss(const BalanceArgs& a, const BalancePlan& p, char* ws, int32_t* counts, int32_t* tokens,
                               float* probs, float* loss, float* z, hipStream_t stream) {
  const BalanceOut out{counts, tokens, probs, loss, z};
  const BalancePartials part{reinterpret_cast<float*>(ws + p.off_probs), reinterpret_cast<int32_t*>(ws + p.off_counts),
                             reinterpret_cast<double*>(ws + p.off_z), reinterpret_cast<int32_t*>(ws + p.off_tokens),
                             reinterpret_cast<double*>(ws + p.off_dots),
                             reinterpret_cast<int32_t*>(ws + p.off_arrived)};
  const bool single = p.ntiles == 1 && a.g == 1;
  with_rows(a.e, rows16(a.logits, a.e), [&](auto shape, auto vec) {
    using S = decltype(shape);
    balance_tile_kernel<S::lpt, S::nv, decltype(vec)::value>
        <<<p.ntiles, kBalBlock, 0, stream>>>(a, p.tile, p.pitch, single, part, out);
  });
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || single) return err;
  // as many groups at a time as one launch takes: all of them, short of 262144 (at 1024 experts)
  const int most = static_cast<int>(most_workgroups(kBalReduce) / p.chunks);
  for (int64_t g0 = 0; g0 < a.g && err == hipSuccess; g0 += most) {
    const unsigned groups = static_cast<unsigned>(a.g - g0 < most ? a.g - g0 : most);
    balance_reduce_kernel<<<groups * p.chunks, kBalReduce, 0, stream>>>(a, static_cast<int>(g0), p.tile, p.pitch, p.chunks,
                                                                        part, out);
    err = hipGetLastError();
  }
  return err;
}

hipError_t launch_balance_loss_backward(const BalanceArgs& a, const int32_t* counts, const int32_t* tokens,
                                        const float* grad_loss, const float* grad_z, float* grad_logits,
                                        hipStream_t stream) {
  if (a.s == 0) return hipSuccess;
  with_rows(a.e, rows16(a.logits, a.e) && rows16(grad_logits, a.e), [&](auto shape, auto vec) {
    using S = decltype(shape);
    constexpr int kAtOnce = kBalBlock / S::lpt * (S::nv >= 16 ? 1 : 2);
    // whole rounds of tokens, up to 2048 workgroups
    int tile = (a.s + 2047) / 2048;
    tile = (tile + kAtOnce - 1) / kAtOnce * kAtOnce;
    balance_backward_kernel<S::lpt, S::nv, decltype(vec)::value>
        <<<(a.s - 1) / tile + 1, kBalBlock, 0, stream>>>(a, tile, counts, tokens, grad_loss, grad_z, grad_logits);
  });
  return hipGetLastError();
}

}  // namespace moe
