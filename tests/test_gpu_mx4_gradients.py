"""Gradients around 4-bit experts kept in more than the element type's bits: dz in two bf16 parts, the rows'
gradient in float32 until a token's rows are summed.

Tolerances as at the top of test_gpu_kept_values.py and test_gpu_mx4.py, u = 2^-24. Two parts hold a float32
value to 2^-17 of itself (the first is off by at most 2^-8 of its leading power of two, the second by at most
2^-9 of that), above 2^-116 at least, where the second is no bf16 subnormal. A product of a part and a 4-bit value
is exact; the float32 sum of 2 n of them is off by at most (2 n + 3) 2u of the sum of their magnitudes, 16-bit
rows as in test_gpu_mx4.py. A token's k rows are then summed in float32: k u of their magnitudes.
"""
import numpy as np
import pytest
import torch

import combine_moe_gate_amd as M
import combine_moe_gate_amd.autograd as A
import oracle
import workloads as W
from oracle import epilogue as E
from oracle import mx4
from tests.gpu_util import TORCH_DTYPE, assert_bits_equal, to_dev, to_host
from tests.test_gpu_expert_act import U, announce, rand, real, within
from tests.test_gpu_kept_values import gradients
from tests.test_gpu_mx4 import HEIGHTS, four_bits, pair

pytestmark = pytest.mark.gpu


def bf16_value(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32)


def in_parts(v):
    """[rows, 2, n] bf16 bits of float32 v [rows, n], and the two parts' values."""
    hi = oracle.from_f32(v, "bf16")
    lo = oracle.from_f32((v - bf16_value(hi)).astype(np.float32), "bf16")
    return np.stack([hi, lo], 1), bf16_value(hi), bf16_value(lo)


CASES = [
    # s, m, n, e, k, capacity, pad, route_major, dtype, act, gated, bias, weighted, gather
    (1, 32, 8, 3, 2, 0, 1, False, "bf16", "silu", True, None, False, True),         # smallest rows
    (1, 544, 72, 16, 8, 0, 1, False, "f16", "gelu", False, "f32", True, True),      # one token
    (40, 288, 200, 2, 2, 0, 1, False, "bf16", "gelu_tanh", True, "own", True, False),
    (200, 96, 64, 16, 2, 0, 16, False, "bf16", "none", False, "own", True, True),   # padded segments
    (1000, 160, 264, 8, 3, 200, 1, True, "f16", "silu", True, "f32", True, True),   # drops, ragged columns
    (2000, 64, 40, 4, 2, 0, 1, False, "bf16", "none", True, "f32", False, True),
    (600, 288, 520, 3, 1, 0, 64, False, "f16", "silu", False, None, True, False),
    (300, 96, 136, 700, 8, 6, 1, False, "bf16", "silu", True, "own", False, True),  # rows of many experts, mostly empty
    (500, 512, 128, 4, 2, 0, 1, False, "bf16", "none", False, None, False, True),   # neither bent nor weighted
]
IDS = [f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-{c[9]}" for c in CASES]


def made(case):
    s, m, n, e, k, cap, pad, rm, dtype, name, gated, bias, weighted, gather = case
    rng = np.random.default_rng(s + m + n)
    idx = W.random_idx(rng, s, e, k)
    L = oracle.dispatch_layout(idx, e, cap, route_major=rm, pad_multiple=pad)
    Lg = M.moe_dispatch_layout(to_dev(idx), e, cap, route_major=rm, pad_multiple=pad)
    nz = 2 * n if gated else n
    wc, ws, w_val = four_bits(rng, (e, nz, m), zero_blocks=True)
    b = None if bias is None else rng.standard_normal((e, nz)).astype(np.float32) if bias == "f32" else rand(rng, (e, nz), dtype)
    return rng, L, Lg, (wc, ws), w_val, b, W.random_weights(rng, s, k) if weighted else None


def dev(t, dtype):
    return None if t is None else to_dev(t, dtype if t.dtype != np.float32 else None)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward_in_parts(case):
    announce("dz in parts", *case)
    s, m, n, e, k, cap, pad, rm, dtype, name, gated, bias, weighted, gather = case
    rng, L, Lg, _, _, _, w = made(case)
    nz = 2 * n if gated else n
    placed = (L.src >= 0)[:, None]
    g = rand(rng, (L.rows, n), dtype)
    g64 = np.where(placed, oracle.to_f32(g, dtype).astype(np.float64), 0)
    z = np.where(placed, rng.standard_normal((L.rows, nz)).astype(np.float32), np.float32(np.nan))  # not read where not placed
    z64 = np.where(placed, z, 0).astype(np.float64)
    kw = dict(act=name, gated=gated, w=dev(w, dtype), need_w=weighted, bias_dtype=torch.float32, need_residual=True)
    got = M.moe_expert_act_backward(Lg, to_dev(g, dtype), to_dev(z), parts=2, **kw)
    one = M.moe_expert_act_backward(Lg, to_dev(g, dtype), to_dev(z), **kw)
    assert got[0].shape == (L.rows, 2, nz) and got[0].dtype == torch.bfloat16
    for a, b in zip(got[1:], one[1:]):
        assert (a is None and b is None) or torch.equal(a, b), "the other gradients do not depend on it"
    parts = to_host(got[0])
    if dtype == "bf16":
        assert_bits_equal(parts[:, 0].copy(), to_host(one[0]), "the first part is the rounded gradient")
    assert not parts[~placed[:, 0]].any(), "unfilled rows not +0"
    want, tol = gradients(L, g64, z64, np.zeros_like(z64), name, gated, w)
    total = bf16_value(parts[:, 0]).astype(np.float64) + bf16_value(parts[:, 1])
    bound = np.where(placed, tol[0], 0) + 2.0 ** -17 * (np.abs(want[0]) + np.where(placed, tol[0], 0)) + 2.0 ** -134
    assert (np.abs(total - want[0]) <= bound).all()


def test_parts_at_the_ends_of_the_range():
    """Without an activation dz is w g: float32 values of every size, infinities and NaN."""
    announce("dz in parts, range")
    vals = np.array([0, -0.0, 1, 1 + 2.0 ** -8, 1 + 2.0 ** -8 + 2.0 ** -9, 3.0e38, 3.39e38, 3.4028234e38, -3.4028234e38, 65504 * 3,
                     2.0 ** -30, 2.0 ** -126, np.inf, -np.inf, np.nan, 1 / 3], np.float32)
    s = len(vals)
    L = M.moe_dispatch_layout(torch.zeros((s, 1), dtype=torch.int32, device="cuda"), 1, 0)
    g = torch.ones((s, 8), dtype=torch.float16, device="cuda")
    parts = M.moe_expert_act_backward(L, g, w=to_dev(vals[:, None].copy()), parts=2)[0]
    hi, lo = (bf16_value(to_host(parts)[:, i]).astype(np.float64) for i in (0, 1))
    v = vals.astype(np.float64)[:, None]
    fine = np.isfinite(v[:, 0])
    assert np.isfinite(hi[fine]).all() and (np.abs(hi[fine] + lo[fine] - v[fine]) <= 2.0 ** -17 * np.abs(v[fine]) + 2.0 ** -134).all()
    assert np.array_equal(hi[~fine], np.repeat(v[~fine], 8, 1), equal_nan=True) and not lo[~fine].any()


def check_dgrad(rng, L, Lg, w_dev, w_val, m, nz, what):
    """Rows in parts to every type, 16-bit rows to float32."""
    unfilled = L.src < 0
    v = rng.standard_normal((L.rows, nz)).astype(np.float32)
    planes, hi, lo = in_parts(v)
    planes[unfilled] = 0x7FC0  # not read
    exact = np.where(unfilled[:, None], 0, hi.astype(np.float64) + lo).astype(np.float32)
    _, want = oracle.expert_gemm_dgrad(L, exact, w_val, "f32")
    _, mag = oracle.expert_gemm_dgrad(L, np.where(unfilled[:, None], 0, np.abs(hi) + np.abs(lo)).astype(np.float32), np.abs(w_val), "f32")
    for to in ("f32", "bf16", "f16"):
        ga = torch.full((L.rows + 2, m), 3.0, dtype=TORCH_DTYPE[to], device="cuda")
        M.moe_mx4_expert_dgrad(Lg, to_dev(planes, "bf16"), w_dev, out=ga[1:-1])
        assert (ga[0] == 3).all() and (ga[-1] == 3).all(), "rows beside the input gradient were written"
        within(to_host(ga[1:-1]), want, (2 * nz + 3) * 2 * U * mag, to, f"{what}, parts to {to}")
        assert not oracle.to_f32(to_host(ga[1:-1])[unfilled], to).view(np.uint32).any(), "unfilled rows not +0"
    for dtype in ("bf16", "f16"):
        g = rand(rng, (L.rows, nz), dtype)
        g[unfilled] = np.uint16(0x7FC0) if dtype == "bf16" else np.float16(np.nan)
        gv = np.where(unfilled[:, None], 0, oracle.to_f32(g, dtype)).astype(np.float32)
        _, want = oracle.expert_gemm_dgrad(L, gv, w_val, "f32")
        _, mag = oracle.expert_gemm_dgrad(L, np.abs(gv), np.abs(w_val), "f32")
        ga = torch.full((L.rows + 2, m), 3.0, device="cuda")
        M.moe_mx4_expert_dgrad(Lg, to_dev(g, dtype), w_dev, out=ga[1:-1])
        assert (ga[0] == 3).all() and (ga[-1] == 3).all(), "rows beside the input gradient were written"
        terms = 2 * nz + 6 if dtype == "f16" else nz + 3
        within(to_host(ga[1:-1]), want, terms * 2 * U * mag, "f32", f"{what}, {dtype} to f32")
        assert not to_host(ga[1:-1])[unfilled].view(np.uint32).any()
        rounded = M.moe_mx4_expert_dgrad(Lg, to_dev(g, dtype), w_dev)
        assert_bits_equal(to_host(rounded), to_host(ga[1:-1].to(TORCH_DTYPE[dtype])), "the rounded gradient is this one, rounded")


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_input_gradient(case):
    announce("4-bit input gradient in parts", *case)
    s, m, n, e, k, cap, pad, rm, dtype, name, gated, bias, weighted, gather = case
    rng, L, Lg, w, w_val, _, _ = made(case)
    check_dgrad(rng, L, Lg, pair(*w), w_val, m, 2 * n if gated else n, "case")


@pytest.mark.parametrize("nz", [8, 64, 72, 128, 200])
@pytest.mark.parametrize("m", [32, 288])
def test_input_gradient_at_every_tile_height(m, nz):
    announce("4-bit input gradient in parts, heights", m, nz)
    rng = np.random.default_rng(m + nz)
    e = len(HEIGHTS) + 1
    idx = np.repeat(np.arange(e), [1, *HEIGHTS]).astype(np.int32)
    idx = idx[rng.permutation(len(idx))][:, None]
    L, Lg = oracle.dispatch_layout(idx, e, 0), M.moe_dispatch_layout(to_dev(idx), e, 0)
    wc, ws, w_val = four_bits(rng, (e, nz, m))
    check_dgrad(rng, L, Lg, pair(wc, ws), w_val, m, nz, "heights")


def test_infinities_stay_in_their_rows():
    announce("4-bit input gradient in parts, infinities")
    rng = np.random.default_rng(3)
    s, e, m, nz = 300, 3, 96, 72
    idx = W.random_idx(rng, s, e, 1)
    L = M.moe_dispatch_layout(to_dev(idx), e, 0)
    codes = np.full((e, nz, m // 2), 0x22, np.uint8)  # ones
    w = pair(codes, np.full((e, nz, m // 32), 127, np.uint8))
    g = torch.zeros((s, 2, nz), dtype=torch.bfloat16, device="cuda")
    g[:, 0], g[:, 1] = 1, 2.0 ** -9
    g[5, 0, 71], g[17, 0, 3], g[200, 0, 64], g[200, 0, 0] = float("inf"), float("nan"), float("inf"), float("-inf")
    for r, i in ((5, 71), (17, 3), (200, 64), (200, 0)):
        g[r, 1, i] = 0
    ga = M.moe_mx4_expert_dgrad(L, g, w, out_dtype=torch.float32)
    want = torch.full((s, m), 72 * (1 + 2.0 ** -9), device="cuda")
    want[5], want[17], want[200] = float("inf"), float("nan"), float("nan")
    assert torch.equal(ga.nan_to_num(-1.0, posinf=-2.0, neginf=-3.0), want.nan_to_num(-1.0, posinf=-2.0, neginf=-3.0))


def test_more_bytes_than_32_bits_count():
    """9.2 GB of parts, and 4.9 GB of float32 gradients: whole numbers at both ends."""
    announce("4-bit gradients past 4 GiB")
    e, k = 8, 8
    for s, m, nz in ((70000, 64, 4096), (40000, 4096, 32)):
        idx = torch.arange(e, device="cuda").repeat(s, 1).int()
        L = M.moe_dispatch_layout(idx, e, 0)
        codes = torch.full((e, nz, m // 2), 0x22, dtype=torch.uint8, device="cuda")
        w = (codes, torch.full((e, nz, m // 32), 127, dtype=torch.uint8, device="cuda"))
        parts = torch.zeros((L.rows, 2, nz), dtype=torch.bfloat16, device="cuda")
        parts[0, 0, 0], parts[0, 1, -1], parts[-1, 0, -1], parts[-1, 1, 0] = 3, 2, 5, 4
        ga = M.moe_mx4_expert_dgrad(L, parts, w, out_dtype=torch.float32)
        assert (ga[0] == 5).all() and (ga[-1] == 9).all() and not ga[1:-1].any()
        del parts, ga
        g = torch.zeros((L.rows, nz), dtype=torch.bfloat16, device="cuda")
        g[0, 0], g[-1, -1] = 3, 5
        back = M.moe_expert_act_backward(L, g, w=torch.ones((s, k), device="cuda") * (1 + 2.0 ** -10), parts=2)[0]
        assert back[0, 0, 0] == 3 and back[0, 1, 0] == 3 * 2.0 ** -10 and back[-1, 0, -1] == 5 and back[-1, 1, -1] == 5 * 2.0 ** -10
        assert not back[1:-1].any()
        del back, g
        torch.cuda.empty_cache()


@pytest.mark.parametrize("quantize", [False, True])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_one_rounding_of_the_gradient(case, quantize):
    """x's gradient of one projection, element by element: one rounding to the element type besides the float32
    bounds, where without grad_dtype dz and each route's row are rounded too."""
    announce("4-bit gradient, one rounding", quantize, *case)
    s, m, n, e, k, cap, pad, rm, dtype, name, gated, bias, weighted, gather = case
    rng, L, Lg, w4, w_val, b, w = made(case)
    nz = 2 * n if gated else n
    count = s if gather else L.rows
    a = rand(rng, (count, m), dtype)
    a_val = mx4.values(*mx4.quantize(oracle.to_f32(a, dtype).astype(np.float64))).astype(np.float32) if quantize else oracle.to_f32(a, dtype)
    g = rand(rng, (L.rows, n), dtype)
    placed = (L.src >= 0)[:, None]
    rb = None if b is None else real(b, dtype)
    _, z = oracle.expert_gemm_act(L, a_val, w_val, "f32", gather, rb, name, gated, w)
    _, mag = oracle.expert_gemm_act(L, np.abs(a_val), np.abs(w_val), "f32", gather, None if rb is None else np.abs(rb))
    terms = 2 * m + 6 if dtype == "f16" and not quantize else m + 3
    g64 = np.where(placed, oracle.to_f32(g, dtype).astype(np.float64), 0)
    want, tol = gradients(L, g64, z, terms * 2 * U * mag, name, gated, w)
    tol_z = np.where(placed, tol[0], 0) + 2.0 ** -17 * (np.abs(want[0]) + np.where(placed, tol[0], 0)) + 2.0 ** -134
    aw = np.abs(w_val.astype(np.float64))
    ga, ta = np.zeros((L.rows, m)), np.zeros((L.rows, m))
    for x, r in E.segments(L):
        ga[r] = want[0][r] @ w_val[x].astype(np.float64)
        most = np.abs(want[0][r]) + tol_z[r]
        ta[r] = tol_z[r] @ aw[x] + (2 * nz + 3) * 2 * U * ((1 + 2.0 ** -7) * most @ aw[x])
    if gather:
        gx, tx, sums = np.zeros((s, m)), np.zeros((s, m)), np.zeros((s, m))
        for r in range(L.rows):
            if L.src[r] >= 0:
                gx[L.src[r]] += ga[r]
                tx[L.src[r]] += ta[r]
                sums[L.src[r]] += np.abs(ga[r]) + ta[r]
        ga, ta = gx, tx + k * U * sums
    x = to_dev(a, dtype).requires_grad_()
    y = A.expert_linear_mx4(x, pair(*w4), Lg, bias=dev(b, dtype), act=name, gated=gated, w=dev(w, dtype), gather=gather,
                            quantize_rows=quantize, preact_dtype=torch.float32, grad_dtype=torch.float32)
    (got,) = torch.autograd.grad(y, x, to_dev(g, dtype))
    assert got.dtype == x.dtype
    if name != "relu":
        within(to_host(got), ga, ta, dtype, "gradient of x")


def test_gradients_past_f16():
    """dz of 2^17 and of 2^-30 on weights that bring them back into f16's range: both reach x whole."""
    announce("4-bit gradient past f16")
    s, n, m = 70, 64, 64
    L = M.moe_dispatch_layout(torch.zeros((s, 1), dtype=torch.int32, device="cuda"), 1, 0)
    codes = torch.full((1, 2 * n, m // 2), 0x22, dtype=torch.uint8, device="cuda")
    for up, grad, scale in ((512.0, 256.0, 127 - 9), (2.0 ** -14, 2.0 ** -16, 127 + 9)):
        # z = bias: the gate's half 1 (slope 1), the up half `up`; dz of the gate's half is grad times up
        scales = torch.full((1, 2 * n, m // 32), scale, dtype=torch.uint8, device="cuda")
        x = torch.zeros((s, m), dtype=torch.float16, device="cuda", requires_grad=True)
        bias = torch.cat([torch.ones(n), torch.full((n,), up)])[None].cuda()
        y = A.expert_linear_mx4(x, (codes, scales), L, bias=bias, act="relu", gated=True, preact_dtype=torch.float32,
                                grad_dtype=torch.float32)
        (got,) = torch.autograd.grad(y, x, torch.full_like(y, grad))
        want = n * 2.0 ** (scale - 127) * (grad * up + grad)
        assert (got.double() - want).abs().max() <= 2.0 ** -11 * want, (up, got[0, 0], want)


def step(t, L, leaves):
    h = A.expert_linear_mx4(leaves["x"], t["up"], L, bias=leaves["up_bias"], act="silu", gated=True, quantize_rows=True,
                            preact_dtype=torch.float32, grad_dtype=torch.float32)
    o = A.expert_linear_mx4(h, t["down"], L, bias=leaves["down_bias"], gather=False, quantize_rows=True)
    y = A.combine(o, leaves["w"], L)
    return (y.detach(), *torch.autograd.grad(y, list(leaves.values()), t["grad"]))


def test_captured_and_replayed_with_new_inputs():
    announce("4-bit gradient in parts, graph")
    rng = np.random.default_rng(31)
    s, m, n, e, k = 700, 128, 96, 4, 2
    t = {"grad": to_dev(rand(rng, (s, m), "bf16"), "bf16")}
    for name, f, d in (("up", 2 * n, m), ("down", m, n)):
        t[name] = pair(*four_bits(rng, (e, f, d))[:2])
    static = {"x": to_dev(rand(rng, (s, m), "bf16"), "bf16"), "up_bias": to_dev(rand(rng, (e, 2 * n), "bf16"), "bf16"),
              "down_bias": to_dev(rand(rng, (e, m), "bf16"), "bf16"), "w": to_dev(W.random_weights(rng, s, k))}
    L = M.moe_dispatch_layout(to_dev(W.random_idx(rng, s, e, k)), e, 0)
    fresh = lambda: {v: q.detach().requires_grad_() for v, q in static.items()}  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(t, L, fresh())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(t, L, fresh())
    for rep in range(4):
        static["x"].copy_(to_dev(rand(rng, (s, m), "bf16"), "bf16"))
        want = [v.clone() for v in step(t, L, {v: q.clone().requires_grad_() for v, q in static.items()})]
        torch.cuda.synchronize()
        for v in outs:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs, want)), f"replay {rep}"


def test_no_tokens():
    announce("4-bit gradient in parts, empty")
    for cap in (0, 3):
        L = M.moe_dispatch_layout(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 4, cap)
        w = pair(np.full((4, 16, 32), 0x22, np.uint8), np.full((4, 16, 2), 127, np.uint8))
        z = torch.full((L.rows, 16), 9.0, device="cuda")
        gz = M.moe_expert_act_backward(L, torch.ones((L.rows, 8), dtype=torch.float16, device="cuda"), z, act="silu", gated=True, parts=2)[0]
        assert gz.shape == (L.rows, 2, 16) and not gz.any()
        ga = M.moe_mx4_expert_dgrad(L, gz, w, out=torch.full((L.rows, 64), 5.0, device="cuda"))
        assert ga.shape == (L.rows, 64) and not ga.any()
