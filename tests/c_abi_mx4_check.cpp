// The 4-bit rows and products driven through the C ABI alone: no Python, no PyTorch. Checked on the
// host, by brute force, on whole numbers, so that every result is exact:
//   rows      quantised (codes and scale bytes) and read back;
//   products  4-bit weights with bf16 rows and with 4-bit rows, bias and relu, gated, gathered and not,
//             results in bf16 and in 4 bits, in every form the library has; the input gradient;
//   errors    bad arguments return their status and a message, enqueueing nothing.
// Prints "c_abi_mx4_check: ok" and exits 0, or lists the failures and exits 1.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "moe_gate.h"

static int g_failures = 0;

#define CHECK(cond, ...)                                               \
  do {                                                                 \
    if (!(cond) && ++g_failures <= 20) {                               \
      std::fprintf(stderr, "FAIL line %d: ", __LINE__);                \
      std::fprintf(stderr, __VA_ARGS__);                               \
      std::fputc('\n', stderr);                                        \
    }                                                                  \
  } while (0)

#define HIP_OK(call)                                                                        \
  do {                                                                                      \
    const hipError_t e_ = (call);                                                           \
    if (e_ != hipSuccess) {                                                                 \
      std::fprintf(stderr, "%s: %s (line %d)\n", #call, hipGetErrorString(e_), __LINE__);   \
      std::exit(2);                                                                         \
    }                                                                                       \
  } while (0)

#define MOE_OK_(call)                                                                       \
  do {                                                                                      \
    const moe_status_t s_ = (call);                                                         \
    if (s_ != MOE_OK) {                                                                     \
      std::fprintf(stderr, "%s: %s: %s (line %d)\n", #call, moe_status_string(s_),          \
                   moe_last_error(), __LINE__);                                             \
      std::exit(3);                                                                         \
    }                                                                                       \
  } while (0)

// A device array, filled from the host or with a byte that no result has.
template <class T>
struct Dev {
  T* p = nullptr;
  size_t n = 0;
  explicit Dev(size_t count) : n(count) {
    HIP_OK(hipMalloc(&p, std::max<size_t>(n, 1) * sizeof(T)));
    const std::vector<unsigned char> dirt(n * sizeof(T), 0x5b);
    if (n) HIP_OK(hipMemcpy(p, dirt.data(), dirt.size(), hipMemcpyHostToDevice));
  }
  explicit Dev(const std::vector<T>& h) : Dev(h.size()) {
    if (n) HIP_OK(hipMemcpy(p, h.data(), n * sizeof(T), hipMemcpyHostToDevice));
  }
  ~Dev() { (void)hipFree(p); }
  Dev(const Dev&) = delete;
  Dev& operator=(const Dev&) = delete;
  std::vector<T> get() const {
    std::vector<T> h(n);
    if (n) HIP_OK(hipMemcpy(h.data(), p, n * sizeof(T), hipMemcpyDeviceToHost));
    return h;
  }
};

struct Rng {  // splitmix64
  uint64_t state;
  uint64_t next() {
    uint64_t z = (state += 0x9e3779b97f4a7c15ull);
    z = (z ^ (z >> 30)) * 0xbf58476d1ce4e5b9ull;
    z = (z ^ (z >> 27)) * 0x94d049bb133111ebull;
    return z ^ (z >> 31);
  }
  int between(int lo, int hi) { return lo + static_cast<int>(next() % static_cast<uint64_t>(hi - lo + 1)); }
};

typedef uint16_t bf16;
static bf16 round_bf16(float v) {  // to nearest, ties to even
  uint32_t u;
  std::memcpy(&u, &v, sizeof(u));
  return static_cast<bf16>((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}
static float value(bf16 h) {
  const uint32_t u = static_cast<uint32_t>(h) << 16;
  float v;
  std::memcpy(&v, &u, sizeof(v));
  return v;
}

static const float kGrid[8] = {0, 0.5f, 1, 1.5f, 2, 3, 4, 6};

// One block by its definition: the code nearest to v / scale, of two equally near the even one.
static void quantize_block(const float* v, uint8_t* codes, uint8_t* scale) {
  float top = 0;
  for (int i = 0; i < 32; ++i) top = std::max(top, std::fabs(v[i]));
  int ex = 0;
  std::frexp(top, &ex);  // top = f 2^ex, f in [0.5, 1)
  const int E = top > 0 ? std::max(ex - 1 - 2 + 127, 0) : 0;
  *scale = static_cast<uint8_t>(E);
  for (int i = 0; i < 32; ++i) {
    const double a = std::fabs(static_cast<double>(v[i])) * std::ldexp(1.0, 127 - E);
    int best = 0;
    for (int c = 1; c < 8; ++c) {
      const double d = std::fabs(a - kGrid[c]), b = std::fabs(a - kGrid[best]);
      if (d < b || (d == b && c % 2 == 0)) best = c;
    }
    if (std::signbit(v[i])) best |= 8;
    codes[i / 2] = static_cast<uint8_t>(i % 2 ? (codes[i / 2] & 15) | best << 4 : best);
  }
}
static float code_value(uint8_t byte, int high, uint8_t E) {
  const int c = high ? byte >> 4 : byte & 15;
  return std::ldexp(c & 8 ? -kGrid[c & 7] : kGrid[c & 7], E - 127);
}

// Whole numbers that 4 bits hold with scale 1 in every block of 32.
static std::vector<float> whole(Rng& rng, size_t n) {
  static const float some[7] = {0, 1, 2, 3, -1, -2, -3};
  std::vector<float> v(n);
  for (size_t i = 0; i < n; ++i) v[i] = i % 32 == 5 ? 4.0f : some[rng.between(0, 6)];
  return v;
}
static std::vector<bf16> as_bf16(const std::vector<float>& v) {
  std::vector<bf16> h(v.size());
  for (size_t i = 0; i < v.size(); ++i) h[i] = round_bf16(v[i]);
  return h;
}
struct Mx4 {
  Dev<uint8_t> codes, scales;
  explicit Mx4(size_t n) : codes(n / 2), scales(n / 32) {}
};

static void rows_and_back(int rows, int m, uint64_t seed, hipStream_t st) {
  std::printf("case rows=%d m=%d\n", rows, m);
  std::fflush(stdout);
  Rng rng{seed};
  const size_t n = static_cast<size_t>(rows) * m;
  std::vector<float> x(n);
  for (size_t i = 0; i < n; ++i) x[i] = std::ldexp(static_cast<float>(rng.between(-4000, 4000)), rng.between(-3, 0) + static_cast<int>(i / 32 % 40) - 20);
  Dev<float> d_x(x), d_back(n);
  Dev<bf16> d_half(n);
  Mx4 q(n);
  MOE_OK_(moe_mx4_quantize(d_x.p, rows, m, MOE_F32, q.codes.p, q.scales.p, st));
  MOE_OK_(moe_mx4_dequantize(q.codes.p, q.scales.p, rows, m, MOE_F32, d_back.p, st));
  MOE_OK_(moe_mx4_dequantize(q.codes.p, q.scales.p, rows, m, MOE_BF16, d_half.p, st));
  HIP_OK(hipStreamSynchronize(st));
  const auto codes = q.codes.get(), scales = q.scales.get();
  const auto back = d_back.get();
  const auto half = d_half.get();
  for (size_t b = 0; b < n / 32; ++b) {
    uint8_t want[16] = {}, E = 0;
    quantize_block(&x[b * 32], want, &E);
    CHECK(scales[b] == E, "scale of block %zu: %d, not %d", b, scales[b], E);
    for (int i = 0; i < 16; ++i) CHECK(codes[b * 16 + i] == want[i], "codes of block %zu, byte %d: %02x, not %02x", b, i, codes[b * 16 + i], want[i]);
    for (int i = 0; i < 32; ++i) {
      const float v = code_value(want[i / 2], i % 2, E);
      CHECK(back[b * 32 + i] == v && value(half[b * 32 + i]) == v, "value %d of block %zu: %g, not %g", i, b, back[b * 32 + i], v);
    }
  }
}

static void products(int s, int e, int k, int m, int n, bool gated, bool gather, bool four, uint64_t seed, hipStream_t st) {
  std::printf("case product s=%d e=%d k=%d m=%d n=%d gated=%d gather=%d rows=%s\n", s, e, k, m, n, gated, gather, four ? "4-bit" : "bf16");
  std::fflush(stdout);
  Rng rng{seed};
  const int nz = gated ? 2 * n : n;
  std::vector<int32_t> idx(static_cast<size_t>(s) * k);
  for (int t = 0; t < s; ++t)
    for (int j = 0; j < k; ++j) {
      int32_t* row = &idx[static_cast<size_t>(t) * k];
      do row[j] = rng.between(0, e - 1);
      while (std::find(row, row + j, row[j]) != row + j);
    }
  Dev<int32_t> d_idx(idx);
  const moe_layout_options_t o{0, 8};  // padded segments: rows that no route fills
  const size_t wsb = moe_layout_workspace_bytes_ex(s, e, k, 0, &o);
  Dev<unsigned char> ws(wsb);
  moe_layout_t L;
  MOE_OK_(moe_dispatch_layout_ex(d_idx.p, s, e, k, 0, &o, ws.p, wsb, &L, st));
  HIP_OK(hipStreamSynchronize(st));
  const size_t rows = static_cast<size_t>(L.rows);
  std::vector<int32_t> dst(idx.size()), src(rows), expert(rows, 0);
  HIP_OK(hipMemcpy(dst.data(), L.dst, dst.size() * 4, hipMemcpyDeviceToHost));
  HIP_OK(hipMemcpy(src.data(), L.src, rows * 4, hipMemcpyDeviceToHost));
  for (size_t q = 0; q < idx.size(); ++q) expert[dst[q]] = idx[q];
  const size_t count = gather ? s : rows;
  const std::vector<float> a = whole(rng, count * m), wt = whole(rng, static_cast<size_t>(e) * nz * m);
  std::vector<float> bias(static_cast<size_t>(e) * nz), g(rows * nz);
  for (auto& v : bias) v = static_cast<float>(rng.between(-3, 3));
  for (auto& v : g) v = static_cast<float>(rng.between(-1, 1));
  Dev<float> d_wide(wt), d_bias(bias);
  Dev<bf16> d_a(as_bf16(a)), d_g(as_bf16(g)), d_out(rows * n), d_ga(rows * m);
  Mx4 w(wt.size()), aq(a.size()), oq(n % 32 == 0 ? rows * n : 0);
  MOE_OK_(moe_mx4_quantize(d_wide.p, static_cast<int64_t>(e) * nz, m, MOE_F32, w.codes.p, w.scales.p, st));
  MOE_OK_(moe_mx4_quantize(d_a.p, static_cast<int64_t>(count), m, MOE_BF16, aq.codes.p, aq.scales.p, st));
  moe_expert_epilogue_t ep{};
  ep.activation = MOE_ACT_RELU;
  ep.gated = gated;
  ep.bias = d_bias.p;
  ep.bias_dtype = MOE_F32;
  const void* rows_in = four ? static_cast<const void*>(aq.codes.p) : d_a.p;
  const uint8_t* rows_scales = four ? aq.scales.p : nullptr;
  MOE_OK_(moe_mx4_expert_gemm(&L, rows_in, rows_scales, gather, w.codes.p, w.scales.p, m, n, MOE_BF16, &ep, MOE_BF16, d_out.p, nullptr, st));
  if (n % 32 == 0)
    MOE_OK_(moe_mx4_expert_gemm(&L, rows_in, rows_scales, gather, w.codes.p, w.scales.p, m, n, MOE_BF16, &ep, MOE_BF16, oq.codes.p, oq.scales.p, st));
  MOE_OK_(moe_mx4_expert_dgrad(&L, d_g.p, w.codes.p, w.scales.p, m, nz, MOE_BF16, d_ga.p, st));
  HIP_OK(hipStreamSynchronize(st));
  const auto out = d_out.get(), ga = d_ga.get();
  const auto codes = oq.codes.get(), scales = oq.scales.get();
  std::vector<float> u(n), z(nz);
  for (size_t r = 0; r < rows; ++r) {
    const int t = src[r], x = expert[r];
    std::fill(u.begin(), u.end(), 0.0f);
    if (t >= 0) {
      const float* ar = &a[(gather ? static_cast<size_t>(t) : r) * m];
      for (int c = 0; c < nz; ++c) {
        z[c] = bias[static_cast<size_t>(x) * nz + c];
        const float* wr = &wt[(static_cast<size_t>(x) * nz + c) * m];
        for (int i = 0; i < m; ++i) z[c] += ar[i] * wr[i];
      }
      for (int c = 0; c < n; ++c) u[c] = std::max(z[c], 0.0f) * (gated ? z[n + c] : 1.0f);
    }
    for (int c = 0; c < n; ++c)
      CHECK(value(out[r * n + c]) == value(round_bf16(u[c])), "row %zu feature %d: %g, not %g", r, c, value(out[r * n + c]), u[c]);
    for (int b = 0; n % 32 == 0 && b < n / 32; ++b) {
      uint8_t want[16] = {}, E = 0;
      quantize_block(&u[b * 32], want, &E);
      const size_t at = r * (n / 32) + b;
      CHECK(scales[at] == E, "row %zu block %d: scale %d, not %d", r, b, scales[at], E);
      for (int i = 0; i < 32; ++i)  // a zero's sign follows its factors'
        CHECK(code_value(codes[at * 16 + i / 2], i % 2, E) == code_value(want[i / 2], i % 2, E), "row %zu block %d value %d", r, b, i);
    }
    for (int i = 0; i < m; ++i) {
      float want = 0.0f;
      if (t >= 0)
        for (int c = 0; c < nz; ++c) want += g[r * nz + c] * wt[(static_cast<size_t>(x) * nz + c) * m + i];
      CHECK(value(ga[r * m + i]) == value(round_bf16(want)), "gradient row %zu input %d: %g, not %g", r, i, value(ga[r * m + i]), want);
    }
  }
}

static void errors(hipStream_t st) {
  Dev<bf16> x(4 * 64), out(4 * 64);
  Mx4 q(4 * 64);
  moe_layout_t L;
  std::memset(&L, 0, sizeof(L));
  CHECK(moe_mx4_quantize(x.p, 4, 48, MOE_BF16, q.codes.p, q.scales.p, st) == MOE_ERR_MISALIGNED, "rows of a block and a half accepted");
  CHECK(moe_mx4_quantize(x.p, 4, 64, MOE_BF16, nullptr, q.scales.p, st) == MOE_ERR_INVALID_ARG, "NULL codes accepted");
  CHECK(moe_mx4_dequantize(q.codes.p, q.scales.p, -1, 64, MOE_BF16, out.p, st) == MOE_ERR_INVALID_ARG, "negative rows accepted");
  CHECK(moe_mx4_quantize(x.p, 4, 64, MOE_BF16, x.p, q.scales.p, st) == MOE_ERR_INVALID_ARG, "overlap accepted");
  CHECK(std::strlen(moe_last_error()) > 0, "no message");
  CHECK(moe_mx4_expert_gemm(&L, x.p, nullptr, 1, q.codes.p, q.scales.p, 64, 8, MOE_BF16, nullptr, MOE_BF16, out.p, nullptr, st) ==
            MOE_ERR_HANDLE_MISMATCH, "a handle of zeros accepted");
  CHECK(moe_mx4_expert_dgrad(&L, x.p, q.codes.p, q.scales.p, 64, 8, MOE_BF16, out.p, st) == MOE_ERR_HANDLE_MISMATCH,
        "a handle of zeros accepted");
  HIP_OK(hipStreamSynchronize(st));
}

int main() {
  if (moe_abi_version() != MOE_ABI_VERSION) {
    std::fprintf(stderr, "library and header ABI versions differ\n");
    return 1;
  }
  hipStream_t st;
  HIP_OK(hipStreamCreate(&st));
  rows_and_back(1, 32, 1, st);
  rows_and_back(77, 1056, 2, st);
  for (const bool four : {false, true}) {
    products(12, 8, 2, 128, 32, true, true, four, 3, st);     // a handful of rows per expert
    products(90, 4, 2, 256, 40, false, false, four, 4, st);   // more
    products(90, 4, 2, 160, 64, false, true, four, 5, st);    // rows of any length
    products(600, 2, 1, 32, 12832, false, true, four, 6, st);  // many, and wide enough for the large tiles
  }
  errors(st);
  HIP_OK(hipStreamDestroy(st));
  if (g_failures != 0) {
    std::fprintf(stderr, "c_abi_mx4_check: %d failed checks\n", g_failures);
    return 1;
  }
  std::printf("c_abi_mx4_check: ok\n");
  return 0;
}
