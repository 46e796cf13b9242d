// The expert products with their epilogue and the router's losses driven through the C ABI
// alone: no Python, no PyTorch. Checked on the host, by brute force:
//   products  bias, relu (plain and gated), route weight and residual (of buffer rows and of
//             tokens), kept values in bf16 and float32, in both forms the library has for few
//             and many rows: small whole numbers, so every result is exact;
//   backward  grad_preact, grad_bias, grad_topk_w, grad_residual and the input gradient: exact
//             as well; through the kept values of either type;
//   losses    counts and tokens exact, the rest to float32, for packed groups with padded
//             tokens and for one group in one launch; the gradient against its formula;
//   errors    bad arguments return their status and a message, enqueueing nothing.
// Prints "c_abi_ops_check: ok" and exits 0, or lists the failures and exits 1.
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
static std::vector<bf16> whole(Rng& rng, size_t n, int lo, int hi) {
  std::vector<bf16> v(n);
  for (auto& q : v) q = round_bf16(static_cast<float>(rng.between(lo, hi)));
  return v;
}

static std::vector<int32_t> routes(Rng& rng, int s, int e, int k) {
  std::vector<int32_t> idx(static_cast<size_t>(s) * k);
  for (int t = 0; t < s; ++t)
    for (int j = 0; j < k; ++j) {
      int32_t* row = &idx[static_cast<size_t>(t) * k];
      do row[j] = rng.between(0, e - 1);
      while (std::find(row, row + j, row[j]) != row + j);
    }
  return idx;
}

static void products(int s, int e, int k, int m, int n, bool gated, bool gather, bool token_residual, bool wide,
                     uint64_t seed, hipStream_t st) {
  std::printf("case product s=%d e=%d k=%d m=%d n=%d gated=%d gather=%d kept=%s\n", s, e, k, m, n, gated, gather,
              wide ? "float32" : "bf16");
  std::fflush(stdout);
  Rng rng{seed};
  const int nz = gated ? 2 * n : n;
  const moe_dtype_t kept = wide ? MOE_F32 : MOE_BF16;
  const std::vector<int32_t> idx = routes(rng, s, e, k);
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
  std::vector<float> w(idx.size()), row_w(rows, 0.0f);
  for (size_t q = 0; q < idx.size(); ++q) {
    w[q] = 0.5f * static_cast<float>(1 << rng.between(0, 2));  // 0.5, 1, 2
    row_w[dst[q]] = w[q];
    expert[dst[q]] = idx[q];
  }
  const std::vector<bf16> a = whole(rng, (gather ? s : rows) * m, -1, 1), wt = whole(rng, static_cast<size_t>(e) * nz * m, -1, 1),
                          res = whole(rng, (token_residual ? s : rows) * n, -4, 4), g = whole(rng, rows * n, -2, 2);
  std::vector<float> bias(static_cast<size_t>(e) * nz);
  for (auto& v : bias) v = static_cast<float>(rng.between(-3, 3));

  Dev<bf16> d_a(a), d_wt(wt), d_res(res), d_g(g), d_out(rows * n), d_gz(rows * nz), d_gr(rows * n), d_ga(rows * m);
  Dev<float> d_w(w), d_bias(bias), d_gb(bias.size()), d_gw(w.size()), d_z32(wide ? rows * nz : 0);
  Dev<bf16> d_z16(wide ? 0 : rows * nz);
  void* d_z = wide ? static_cast<void*>(d_z32.p) : d_z16.p;
  moe_expert_epilogue_t ep{};
  ep.activation = MOE_ACT_RELU;
  ep.gated = gated;
  ep.bias = d_bias.p;
  ep.bias_dtype = MOE_F32;
  ep.topk_w = d_w.p;
  ep.residual = d_res.p;
  ep.residual_gather = token_residual;
  ep.preact = d_z;
  if (wide)
    MOE_OK_(moe_expert_gemm_act_ex(&L, d_a.p, gather, d_wt.p, m, n, MOE_BF16, &ep, kept, d_out.p, st));
  else
    MOE_OK_(moe_expert_gemm_act(&L, d_a.p, gather, d_wt.p, m, n, MOE_BF16, &ep, d_out.p, st));
  const size_t need = moe_expert_act_backward_workspace_bytes(&L, n, gated);
  Dev<unsigned char> bws(need);
  if (wide)
    MOE_OK_(moe_expert_act_backward_ex(&L, d_g.p, d_z, kept, n, MOE_BF16, MOE_ACT_RELU, gated, d_w.p, d_gz.p, MOE_F32, d_gb.p,
                                       d_gw.p, d_gr.p, bws.p, need, st));
  else
    MOE_OK_(moe_expert_act_backward(&L, d_g.p, d_z, n, MOE_BF16, MOE_ACT_RELU, gated, d_w.p, d_gz.p, MOE_F32, d_gb.p, d_gw.p,
                                    d_gr.p, bws.p, need, st));
  MOE_OK_(moe_expert_act_dgrad(&L, d_gz.p, d_wt.p, m, nz, MOE_BF16, d_ga.p, st));
  HIP_OK(hipStreamSynchronize(st));

  const auto out = d_out.get(), gz = d_gz.get(), gr = d_gr.get(), ga = d_ga.get(), z16 = d_z16.get();
  const auto gb = d_gb.get(), gw = d_gw.get(), z32 = d_z32.get();
  std::vector<double> want_gb(bias.size(), 0.0), dot(rows, 0.0);
  for (size_t r = 0; r < rows; ++r) {
    const int t = src[r], x = expert[r];
    std::vector<double> z(nz, 0.0), gzr(nz, 0.0);
    for (int c = 0; c < nz; ++c) {
      if (t >= 0) {
        const bf16* ar = &a[(gather ? static_cast<size_t>(t) : r) * m];
        const bf16* wr = &wt[(static_cast<size_t>(x) * nz + c) * m];
        for (int i = 0; i < m; ++i) z[c] += static_cast<double>(value(ar[i])) * value(wr[i]);
        z[c] += bias[static_cast<size_t>(x) * nz + c];
      }
      const double got = wide ? z32[r * nz + c] : value(z16[r * nz + c]);
      CHECK(got == z[c], "kept value row %zu feature %d: %g, not %g", r, c, got, z[c]);
    }
    for (int c = 0; c < n; ++c) {
      const double f = std::max(z[c], 0.0), up = gated ? z[n + c] : 1.0, gv = value(g[r * n + c]);
      const double rv = t < 0 ? 0.0 : value(res[(token_residual ? static_cast<size_t>(t) : r) * n + c]);
      const bf16 want = round_bf16(static_cast<float>(row_w[r] * f * up + rv));
      CHECK(out[r * n + c] == want || (value(want) == 0 && value(out[r * n + c]) == 0), "row %zu feature %d: %g, not %g", r, c,
            value(out[r * n + c]), value(want));
      if (t < 0) {
        CHECK(gr[r * n + c] == 0, "grad_residual of unfilled row %zu", r);
        continue;
      }
      gzr[c] = row_w[r] * gv * up * (z[c] > 0);
      if (gated) gzr[n + c] = row_w[r] * gv * f;
      dot[r] += gv * f * up;
      CHECK(gr[r * n + c] == g[r * n + c], "grad_residual row %zu", r);
    }
    for (int c = 0; c < nz; ++c) {
      CHECK(value(gz[r * nz + c]) == value(round_bf16(static_cast<float>(gzr[c]))), "grad_preact row %zu feature %d", r, c);
      if (t >= 0) want_gb[static_cast<size_t>(x) * nz + c] += gzr[c];
    }
    for (int i = 0; i < m; ++i) {
      double want = 0.0;
      for (int c = 0; c < nz && t >= 0; ++c)
        want += static_cast<double>(value(gz[r * nz + c])) * value(wt[(static_cast<size_t>(x) * nz + c) * m + i]);
      CHECK(value(ga[r * m + i]) == value(round_bf16(static_cast<float>(want))), "grad_a row %zu feature %d", r, i);
    }
  }
  for (size_t i = 0; i < want_gb.size(); ++i) CHECK(gb[i] == want_gb[i], "grad_bias %zu: %g, not %g", i, gb[i], want_gb[i]);
  for (size_t q = 0; q < w.size(); ++q) CHECK(gw[q] == dot[dst[q]], "grad_topk_w %zu: %g, not %g", q, gw[q], dot[dst[q]]);
}

static void losses(int s, int e, int k, const std::vector<int32_t>& groups, int masked, uint64_t seed, hipStream_t st) {
  const int g = groups.empty() ? 1 : static_cast<int>(groups.size()) - 1;
  std::printf("case losses s=%d e=%d k=%d groups=%d\n", s, e, k, g);
  std::fflush(stdout);
  Rng rng{seed};
  std::vector<float> logits(static_cast<size_t>(s) * e), gl(g), gzl(g);
  for (auto& v : logits) v = static_cast<float>(rng.between(-40, 40)) / 16.0f;
  for (auto& v : gl) v = static_cast<float>(rng.between(-8, 8)) / 4.0f;
  for (auto& v : gzl) v = static_cast<float>(rng.between(-8, 8)) / 8.0f;
  std::vector<uint8_t> mask(s, 1);
  for (auto& v : mask) v = !masked || rng.between(0, masked) != 0;
  const std::vector<int32_t> idx = routes(rng, s, e, k);
  Dev<float> d_l(logits), d_gl(gl), d_gz(gzl), d_p(static_cast<size_t>(g) * e), d_loss(g), d_z(g), d_grad(logits.size());
  Dev<int32_t> d_idx(idx), d_gr(groups), d_c(static_cast<size_t>(g) * e), d_n(g);
  Dev<uint8_t> d_m(mask);
  const size_t wsb = moe_balance_workspace_bytes(s, e, g);
  Dev<unsigned char> ws(wsb);
  const int32_t* grp = groups.empty() ? nullptr : d_gr.p;
  const uint8_t* msk = masked ? d_m.p : nullptr;
  MOE_OK_(moe_balance_loss(d_l.p, d_idx.p, msk, grp, s, e, k, g, d_c.p, d_n.p, d_p.p, d_loss.p, d_z.p, ws.p, wsb, st));
  MOE_OK_(moe_balance_loss_backward(d_l.p, msk, grp, d_c.p, d_n.p, d_gl.p, d_gz.p, s, e, k, g, d_grad.p, st));
  HIP_OK(hipStreamSynchronize(st));
  const auto c = d_c.get(), n = d_n.get();
  const auto p = d_p.get(), loss = d_loss.get(), z = d_z.get(), grad = d_grad.get();
  std::vector<char> seen(s, 0);
  // float32 sums of up to e + s terms, each off by some 2^-24 times its exponent's argument (5): 1e-5
  auto near = [](double got, double want, double size) { return std::fabs(got - want) <= 1e-5 * size + 1e-30; };
  for (int i = 0; i < g; ++i) {
    const int lo = groups.empty() ? 0 : groups[i], hi = groups.empty() ? s : groups[i + 1];
    std::vector<std::vector<double>> pt;
    std::vector<double> lse, mean(e, 0.0);
    std::vector<int> token, cnt(e, 0);
    double zz = 0.0;
    for (int t = lo; t < hi; ++t) {
      if (!mask[t]) continue;
      std::vector<double> q(e);
      double sum = 0.0;
      for (int x = 0; x < e; ++x) sum += q[x] = std::exp(static_cast<double>(logits[static_cast<size_t>(t) * e + x]));
      for (int x = 0; x < e; ++x) mean[x] += q[x] /= sum;
      for (int j = 0; j < k; ++j) ++cnt[idx[static_cast<size_t>(t) * k + j]];
      zz += std::log(sum) * std::log(sum);
      pt.push_back(q);
      lse.push_back(std::log(sum));
      token.push_back(t);
      seen[t] = 1;
    }
    const double m = std::max<double>(1.0, static_cast<double>(token.size()));
    double want = 0.0;
    CHECK(n[i] == static_cast<int>(token.size()), "tokens of group %d", i);
    for (int x = 0; x < e; ++x) {
      const size_t at = static_cast<size_t>(i) * e + x;
      CHECK(c[at] == cnt[x], "counts of group %d expert %d", i, x);
      CHECK(near(p[at], mean[x] / m, mean[x] / m), "probs of group %d expert %d", i, x);
      want += cnt[x] / m * mean[x] / m * e / k;
    }
    CHECK(near(loss[i], want, want), "loss of group %d: %g, not %g", i, loss[i], want);
    CHECK(near(z[i], zz / m, zz / m + 1), "z of group %d: %g, not %g", i, z[i], zz / m);
    for (size_t q = 0; q < token.size(); ++q) {
      double dot = 0.0, size = 0.0;
      for (int x = 0; x < e; ++x) {
        dot += pt[q][x] * cnt[x];
        size = std::max(size, std::fabs(cnt[x] - k * m / e));
      }
      const double scale = gl[i] * static_cast<double>(e) / (k * m * m), zs = gzl[i] * 2.0 / m;
      for (int x = 0; x < e; ++x)
        CHECK(near(grad[static_cast<size_t>(token[q]) * e + x], pt[q][x] * (scale * (cnt[x] - dot) + zs * lse[q]),
                   pt[q][x] * (2 * std::fabs(scale) * size + std::fabs(zs) * (std::fabs(lse[q]) + 1))),
              "gradient of token %d expert %d", token[q], x);
    }
  }
  for (int t = 0; t < s; ++t)
    if (!seen[t])
      for (int x = 0; x < e; ++x) CHECK(grad[static_cast<size_t>(t) * e + x] == 0.0f, "gradient of padded token %d", t);
}

static void errors(hipStream_t st) {
  std::printf("case argument errors\n");
  std::fflush(stdout);
  Rng rng{9};
  Dev<int32_t> d_idx(routes(rng, 16, 4, 2));
  const size_t wsb = moe_layout_workspace_bytes(16, 4, 2, 0);
  Dev<unsigned char> ws(wsb);
  moe_layout_t L;
  MOE_OK_(moe_dispatch_layout(d_idx.p, 16, 4, 2, 0, ws.p, wsb, &L, st));
  Dev<bf16> x(16 * 8), wt(4 * 8 * 8), out(32 * 8);
  moe_expert_epilogue_t ep{};
  ep.activation = 9;
  CHECK(moe_expert_gemm_act(&L, x.p, 1, wt.p, 8, 8, MOE_BF16, &ep, out.p, st) == MOE_ERR_INVALID_ARG, "activation 9 accepted");
  CHECK(std::strlen(moe_last_error()) > 0, "no message for activation 9");
  ep = moe_expert_epilogue_t{};
  ep.preact = out.p;
  CHECK(moe_expert_gemm_act(&L, x.p, 1, wt.p, 8, 8, MOE_BF16, &ep, out.p, st) == MOE_ERR_INVALID_ARG, "preact over out accepted");
  Dev<float> z(32 * 8);
  ep.preact = z.p;
  CHECK(moe_expert_gemm_act_ex(&L, x.p, 1, wt.p, 8, 8, MOE_BF16, &ep, MOE_F16, out.p, st) == MOE_ERR_UNSUPPORTED,
        "f16 kept values of bf16 rows accepted");
  CHECK(moe_expert_act_backward(&L, out.p, nullptr, 8, MOE_BF16, MOE_ACT_SILU, 0, nullptr, wt.p, MOE_F32, nullptr, nullptr, nullptr,
                                nullptr, 0, st) == MOE_ERR_INVALID_ARG, "silu's backward without kept values accepted");
  CHECK(moe_expert_act_dgrad(&L, out.p, wt.p, 8, 4, MOE_BF16, z.p, st) == MOE_ERR_MISALIGNED, "8-byte rows accepted");
  Dev<float> l(16 * 4);
  CHECK(moe_balance_loss(l.p, d_idx.p, nullptr, nullptr, 16, 4, 2, 3, d_idx.p, d_idx.p, l.p, l.p, l.p, nullptr, 0, st) ==
            MOE_ERR_INVALID_ARG, "three groups without offsets accepted");
  CHECK(moe_balance_loss_backward(l.p, nullptr, nullptr, d_idx.p, d_idx.p, l.p, nullptr, 16, 4, 2, 1, l.p, st) ==
            MOE_ERR_INVALID_ARG, "a gradient over its logits accepted");
  HIP_OK(hipStreamSynchronize(st));
}

int main() {
  if (moe_abi_version() != MOE_ABI_VERSION) {
    std::fprintf(stderr, "library and header ABI versions differ\n");
    return 1;
  }
  hipStream_t st;
  HIP_OK(hipStreamCreate(&st));
  products(12, 8, 2, 72, 40, true, true, true, false, 1, st);    // a handful of rows per expert
  products(12, 8, 2, 72, 40, false, false, false, true, 2, st);
  products(300, 6, 3, 64, 72, true, true, false, true, 3, st);   // many
  products(300, 6, 3, 40, 200, false, false, true, false, 4, st);
  products(260, 2, 1, 24, 4000, true, true, true, true, 5, st);  // and wide enough for the large tiles
  losses(96, 10, 3, {}, 0, 6, st);                               // one launch
  losses(2000, 24, 4, {}, 5, 7, st);
  losses(500, 130, 6, {3, 3, 40, 41, 260, 490}, 4, 8, st);
  errors(st);
  HIP_OK(hipStreamDestroy(st));
  if (g_failures != 0) {
    std::fprintf(stderr, "c_abi_ops_check: %d failed checks\n", g_failures);
    return 1;
  }
  std::printf("c_abi_ops_check: ok\n");
  return 0;
}
