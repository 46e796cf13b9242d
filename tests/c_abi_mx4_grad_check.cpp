// The gradients in two parts around 4-bit experts driven through the C ABI alone: no Python, no PyTorch.
// Checked on the host, by brute force, on values whose sums are exact:
//   backward  w g in two bf16 parts, w = 1 + 2^-10: the second part is what the first leaves;
//   input     both parts times the weights, to float32, bf16 and f16, and 16-bit rows to float32;
//   errors    bad arguments return their status and a message, enqueueing nothing.
// Prints "c_abi_mx4_grad_check: ok" and exits 0, or lists the failures and exits 1.
#include <hip/hip_runtime_api.h>

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

#define HIP_OK(call)                                                                      \
  do {                                                                                    \
    const hipError_t e_ = (call);                                                         \
    if (e_ != hipSuccess) {                                                               \
      std::fprintf(stderr, "%s: %s (line %d)\n", #call, hipGetErrorString(e_), __LINE__); \
      std::exit(2);                                                                       \
    }                                                                                     \
  } while (0)

#define MOE_OK_(call)                                                                             \
  do {                                                                                            \
    const moe_status_t s_ = (call);                                                               \
    if (s_ != MOE_OK) {                                                                           \
      std::fprintf(stderr, "%s: %s: %s (line %d)\n", #call, moe_status_string(s_),                \
                   moe_last_error(), __LINE__);                                                   \
      std::exit(3);                                                                               \
    }                                                                                             \
  } while (0)

template <class T>
struct Dev {  // filled from the host, or with a byte that no result has
  T* p = nullptr;
  size_t n = 0;
  explicit Dev(size_t count) : n(count) {
    HIP_OK(hipMalloc(&p, (n ? n : 1) * sizeof(T)));
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

static uint16_t bf16_of(float v) {  // of a bf16 value
  uint32_t u;
  std::memcpy(&u, &v, sizeof(u));
  return static_cast<uint16_t>(u >> 16);
}
static float value(uint16_t h) {
  const uint32_t u = static_cast<uint32_t>(h) << 16;
  float v;
  std::memcpy(&v, &u, sizeof(v));
  return v;
}

static void gradients(int s, int e, int k, int m, int nz, hipStream_t st) {
  std::printf("case s=%d e=%d k=%d m=%d nz=%d\n", s, e, k, m, nz);
  std::fflush(stdout);
  std::vector<int32_t> idx;
  for (int t = 0; t < s; ++t)
    for (int j = 0; j < k; ++j) idx.push_back((t * 7 + j) % e);
  Dev<int32_t> d_idx(idx);
  const moe_layout_options_t o{0, 8};  // padded segments: rows that no route fills
  const size_t wsb = moe_layout_workspace_bytes_ex(s, e, k, 0, &o);
  Dev<unsigned char> ws(wsb);
  moe_layout_t L;
  MOE_OK_(moe_dispatch_layout_ex(d_idx.p, s, e, k, 0, &o, ws.p, wsb, &L, st));
  HIP_OK(hipStreamSynchronize(st));
  const size_t rows = static_cast<size_t>(L.rows);
  std::vector<int32_t> dst(idx.size()), expert(rows, -1);
  HIP_OK(hipMemcpy(dst.data(), L.dst, dst.size() * 4, hipMemcpyDeviceToHost));
  for (size_t q = 0; q < idx.size(); ++q) expert[dst[q]] = idx[q];

  // w g: g whole numbers from -3 to 3, w = 1 + 2^-10
  std::vector<uint16_t> g(rows * nz);
  for (size_t i = 0; i < g.size(); ++i) g[i] = bf16_of(static_cast<float>(static_cast<int>(i * 2654435761u % 7u) - 3));
  const std::vector<float> w(static_cast<size_t>(s) * k, 1.0f + std::ldexp(1.0f, -10));
  Dev<uint16_t> d_g(g), d_parts(rows * 2 * nz);
  Dev<float> d_w(w);
  MOE_OK_(moe_expert_act_backward_parts(&L, d_g.p, nullptr, MOE_F32, nz, MOE_BF16, MOE_ACT_NONE, 0, d_w.p, 2, d_parts.p, MOE_F32,
                                        nullptr, nullptr, nullptr, nullptr, 0, st));
  HIP_OK(hipStreamSynchronize(st));
  const auto parts = d_parts.get();
  for (size_t r = 0; r < rows; ++r)
    for (int c = 0; c < nz; ++c) {
      const float hi = expert[r] < 0 ? 0.0f : value(g[r * nz + c]);
      CHECK(value(parts[r * 2 * nz + c]) == hi, "row %zu value %d, first part", r, c);
      CHECK(value(parts[(r * 2 + 1) * nz + c]) == std::ldexp(hi, -10), "row %zu value %d, second part", r, c);
    }

  // weights of 1, 2 and -1 by place, all with scale 1
  static const float kValue[3] = {1, 2, -1};
  static const int kCode[3] = {2, 4, 10};
  std::vector<uint8_t> codes(static_cast<size_t>(e) * nz * m / 2), scales(static_cast<size_t>(e) * nz * m / 32, 127);
  auto which = [&](size_t x, size_t f, size_t i) { return static_cast<int>((x + 2 * f + i * i) % 3); };
  for (int x = 0; x < e; ++x)
    for (int f = 0; f < nz; ++f)
      for (int i = 0; i < m; i += 2)
        codes[((static_cast<size_t>(x) * nz + f) * m + i) / 2] = static_cast<uint8_t>(kCode[which(x, f, i)] | kCode[which(x, f, i + 1)] << 4);
  Dev<uint8_t> d_codes(codes), d_scales(scales);
  Dev<float> d_wide(rows * m), d_from16(rows * m);
  Dev<uint16_t> d_bf(rows * m), d_f16(rows * m);
  const struct {
    const void* g;
    int parts;
    moe_dtype_t to;
    void* out;
  } calls[4] = {{d_parts.p, 2, MOE_F32, d_wide.p}, {d_parts.p, 2, MOE_BF16, d_bf.p}, {d_parts.p, 2, MOE_F16, d_f16.p}, {d_g.p, 1, MOE_F32, d_from16.p}};
  for (const auto& c : calls)
    MOE_OK_(moe_mx4_expert_dgrad_ex(&L, c.g, c.parts, d_codes.p, d_scales.p, m, nz, MOE_BF16, c.to, c.out, st));
  HIP_OK(hipStreamSynchronize(st));
  const auto wide = d_wide.get(), from16 = d_from16.get();
  const auto bf = d_bf.get(), f16 = d_f16.get();
  for (size_t r = 0; r < rows; ++r)
    for (int i = 0; i < m; ++i) {
      double sum = 0;
      for (int c = 0; expert[r] >= 0 && c < nz; ++c) sum += value(g[r * nz + c]) * kValue[which(expert[r], c, i)];
      const double all = sum + std::ldexp(sum, -10), near = std::fabs(all);  // exact in float32
      const size_t at = r * m + i;
      _Float16 h;
      std::memcpy(&h, &f16[at], sizeof(h));
      CHECK(from16[at] == sum, "row %zu input %d: %g, not %g", r, i, from16[at], sum);
      CHECK(wide[at] == all, "row %zu input %d of parts: %.9g, not %.9g", r, i, wide[at], all);
      CHECK(std::fabs(value(bf[at]) - all) <= std::ldexp(near, -8), "row %zu input %d in bf16: %g, not %g", r, i, value(bf[at]), all);
      CHECK(std::fabs(static_cast<double>(h) - all) <= std::ldexp(near, -11), "row %zu input %d in f16", r, i);
    }

  CHECK(moe_mx4_expert_dgrad_ex(&L, d_parts.p, 3, d_codes.p, d_scales.p, m, nz, MOE_BF16, MOE_F32, d_wide.p, st) == MOE_ERR_INVALID_ARG,
        "three parts accepted");
  CHECK(moe_mx4_expert_dgrad_ex(&L, d_parts.p, 2, d_codes.p, d_scales.p, m, nz, MOE_F16, MOE_F32, d_wide.p, st) == MOE_ERR_UNSUPPORTED,
        "parts in f16 accepted");
  CHECK(moe_mx4_expert_dgrad_ex(&L, d_g.p, 1, d_codes.p, d_scales.p, m, nz, MOE_BF16, MOE_F16, d_f16.p, st) == MOE_ERR_UNSUPPORTED,
        "bf16 rows to f16 accepted");
  CHECK(moe_expert_act_backward_parts(&L, d_g.p, nullptr, MOE_F32, nz, MOE_BF16, MOE_ACT_NONE, 0, d_w.p, 0, d_parts.p, MOE_F32, nullptr,
                                      nullptr, nullptr, nullptr, 0, st) == MOE_ERR_INVALID_ARG, "no parts accepted");
  CHECK(std::strlen(moe_last_error()) > 0, "no message");
  HIP_OK(hipStreamSynchronize(st));
}

int main() {
  if (moe_abi_version() != MOE_ABI_VERSION) {
    std::fprintf(stderr, "library and header ABI versions differ\n");
    return 1;
  }
  hipStream_t st;
  HIP_OK(hipStreamCreate(&st));
  gradients(1, 3, 2, 32, 8, st);
  gradients(90, 4, 2, 288, 72, st);
  gradients(700, 2, 1, 64, 136, st);
  HIP_OK(hipStreamDestroy(st));
  if (g_failures != 0) {
    std::fprintf(stderr, "c_abi_mx4_grad_check: %d failed checks\n", g_failures);
    return 1;
  }
  std::printf("c_abi_mx4_grad_check: ok\n");
  return 0;
}
