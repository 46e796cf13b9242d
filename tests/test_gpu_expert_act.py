"""The expert products with an epilogue, and its backward, on the GPU against the float64
oracle.

Tolerances, with u = 2^-24 and half(v) half the element type's step at v. The float32 sum of
m products is off by at most (m + 3) 2u of the sum of their magnitudes (any order, bias
included): dz. An activation moves that by at most its steepest slope, 1.13, and adds its own
float32 error: sigmoid(y) is off by eps = u (16 + 8 |y| (1 - sigmoid)) of itself (exponent
argument 2 |y| u for the constant and product, four more roundings for the cubic of the tanh
form, exponential and reciprocal within 4 u each), the error function by 24 u. Each further
product or sum rounds by u; the result by half(result).
"""
import ctypes

import numpy as np
import pytest
import torch

import combine_moe_gate_amd as M
import combine_moe_gate_amd.autograd as A
import oracle
import workloads as W
from oracle import epilogue as E
from tests.gpu_util import assert_bits_equal, to_dev, to_host

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def announce(*what):
    print("CASE", *what, flush=True)


def half(v, dtype):
    """Half the spacing of dtype's values at |v|."""
    p, emin = (8, -126) if dtype == "bf16" else (11, -14) if dtype == "f16" else (24, -126)
    ex = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** emin)))
    return 2.0 ** (ex - p)


def act_err(name, z):
    """Float32 error of act(z) and act'(z) at an exact z."""
    a = np.abs(z)
    if name in ("none", "relu"):
        return np.zeros_like(z), np.zeros_like(z)
    if name == "gelu":
        return 0.5 * a * 28 * U, 28 * U + a * np.exp(-0.5 * z * z) * 0.4 * (8 + 2 * z * z) * U
    b = 2 * np.sqrt(2 / np.pi)
    y = z if name == "silu" else b * (z + 0.044715 * z ** 3)
    inner = np.ones_like(z) if name == "silu" else b * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + np.exp(-np.clip(y, -700, 700)))
    eps = U * (16 + 8 * np.abs(y) * (1 - s))
    # slope: s + z inner s (1 - s); s enters three times, eight roundings besides; below the
    # clamps (12 for the tanh form) it is constant to 1e-30
    return a * s * eps + 1e-30, s * eps * (1 + 2 * a * inner) + 8 * U * s * (1 + a * inner * (1 - s)) + 1e-30


def within(got, want, tol, dtype, what):
    g = oracle.to_f32(got, dtype).astype(np.float64) if dtype != "f32" else got.astype(np.float64)
    tol = tol + half(np.maximum(np.abs(g), np.abs(want)), dtype)
    bad = np.argwhere(~(np.abs(g - want) <= tol))
    assert len(bad) == 0, (f"{what}: {len(bad)} outside the bound, first {tuple(bad[0])}: got {g[tuple(bad[0])]!r} "
                           f"want {want[tuple(bad[0])]!r} tol {tol[tuple(bad[0])]!r}")


def absolute(a, dtype):
    return (a & np.uint16(0x7FFF)) if dtype == "bf16" else np.abs(a)


def check_forward(got, pre, L, a, wts, dtype, gather, bias, name, gated, w, res, res_gather, what):
    out, z = oracle.expert_gemm_act(L, a, wts, dtype, gather, bias, name, gated, w, res, res_gather)
    _, mag = oracle.expert_gemm_act(L, absolute(a, dtype), absolute(wts, dtype), dtype, gather,
                                    None if bias is None else np.abs(bias))
    m, n = a.shape[1], out.shape[1]
    dz = (m + 3) * 2 * U * mag
    zg = z[:, :n]
    f = E.act(name, zg)[0]
    df = 1.13 * dz[:, :n] + act_err(name, zg)[0]
    if gated:
        up, dup = z[:, n:], dz[:, n:]
        du = np.abs(f) * dup + np.abs(up) * df + df * dup + U * np.abs(f * up)
    else:
        du = df
    rw = np.abs(E.row_weights(L, w))[:, None]
    tol = rw * du * (1 + U) + 2 * U * (np.abs(out) + rw * np.abs(E.finish(z, name, gated)))
    tol[L.src < 0] = 0
    within(to_host(got), out, tol, dtype, what)
    unfilled = L.src < 0
    assert not oracle.to_f32(to_host(got)[unfilled], dtype).view(np.uint32).any(), f"{what}: unfilled rows not +0"
    if pre is not None:
        within(to_host(pre), z, dz, dtype, what + ", kept values")
        assert not oracle.to_f32(to_host(pre)[unfilled], dtype).view(np.uint32).any(), f"{what}: unfilled kept rows not +0"


def check_backward(got, L, g, zk, dtype, name, gated, w, bias_dt, what):
    """got = (grad_preact, grad_bias, grad_w, grad_residual), zk the kept values (exact inputs)."""
    g64, z64 = oracle.to_f32(g, dtype).astype(np.float64), oracle.to_f32(zk, dtype).astype(np.float64)
    n = g64.shape[1]
    placed = L.src >= 0
    g64, z64 = np.where(placed[:, None], g64, 0), np.where(placed[:, None], z64, 0)  # garbage elsewhere is not read
    gz, gb, gw, gr = oracle.expert_act_backward(L, g64, z64, name, gated, w)
    rw = np.abs(E.row_weights(L, w))[:, None]
    f, d = E.act(name, z64[:, :n])
    ef, ed = act_err(name, z64[:, :n])
    ag = rw * np.abs(g64)
    if gated:
        up = np.abs(z64[:, n:])
        tol = np.concatenate([ag * up * (ed + 4 * U * np.abs(d)), ag * (ef + 4 * U * np.abs(f))], 1)
        tol_u = up * ef + 4 * U * np.abs(f) * up
    else:
        tol, tol_u = ag * (ed + 4 * U * np.abs(d)), ef + 4 * U * np.abs(f)
    tol[~placed] = 0
    if got[0] is not None:
        within(to_host(got[0]), gz, tol, dtype, what + ", grad_preact")
        assert not oracle.to_f32(to_host(got[0])[~placed], dtype).view(np.uint32).any()
    if got[1] is not None:
        tol_b = np.zeros_like(gb)
        for x, rows in E.segments(L):
            tol_b[x] = (tol[rows] + 24 * U * np.abs(gz[rows])).sum(0)
        within(to_host(got[1]), gb, tol_b + U * np.abs(gb), bias_dt, what + ", grad_bias")
    if got[2] is not None:
        row = (np.abs(g64) * (tol_u + 16 * U * np.abs(E.finish(z64, name, gated)))).sum(1)
        tol_w = np.where(L.dst >= 0, row[np.where(L.dst >= 0, L.dst, 0)], 0)
        within(to_host(got[2]), gw, tol_w, "f32", what + ", grad_w")
    if got[3] is not None:
        want = np.where(placed[:, None], g, np.zeros((), g.dtype))
        assert_bits_equal(to_host(got[3]), want, what + ", grad_residual")


def rand(rng, shape, dtype, scale=1.0):
    return W.cast_input((rng.standard_normal(shape) * scale).astype(np.float32), dtype)


def real(a, dtype):
    return a.astype(np.float64) if a.dtype == np.float32 else oracle.to_f32(a, dtype).astype(np.float64)


def run_case(idx, m, n, e, cap, pad, rm, dtype, name, gated, bias, weighted, residual, gather, seed):
    rng = np.random.default_rng(seed)
    s, k = idx.shape
    L = oracle.dispatch_layout(idx, e, cap, route_major=rm, pad_multiple=pad)
    Lg = M.moe_dispatch_layout(to_dev(idx), e, cap, route_major=rm, pad_multiple=pad)
    nz = 2 * n if gated else n
    a = rand(rng, (s if gather else L.rows, m), dtype)
    wts = W.expert_weights(seed, e, nz, m, dtype)
    b = None if bias is None else rng.standard_normal((e, nz)).astype(np.float32) if bias == "f32" else rand(rng, (e, nz), dtype)
    w = W.random_weights(rng, s, k) if weighted else None
    res = None if residual is None else rand(rng, (s if residual == "tokens" else L.rows, n), dtype)
    dev = lambda t: None if t is None else to_dev(t, dtype if t.dtype != np.float32 else None)  # noqa: E731
    kw = dict(gather=gather, bias=dev(b), act=name, gated=gated, w=dev(w), residual=dev(res),
              residual_gather=residual == "tokens")
    # the outputs between rows that nothing may touch
    big = [torch.full((L.rows + 2, c), 3.0, dtype=torch.bfloat16 if dtype == "bf16" else torch.float16, device="cuda")
           for c in (n, nz)]
    out, pre = M.moe_expert_gemm_act(Lg, dev(a), dev(wts), out=big[0][1:-1], preact=big[1][1:-1], **kw)
    for t in big:
        assert (t[0] == 3).all() and (t[-1] == 3).all(), "rows beside the output were written"
    what = f"s{s} m{m} n{n} e{e} {name} gated={gated}"
    rb = None if b is None else real(b, dtype)
    check_forward(out, pre, L, a, wts, dtype, gather, rb, name, gated, w, res, residual == "tokens", what)
    alone = M.moe_expert_gemm_act(Lg, dev(a), dev(wts), **kw)  # without keeping z: the same bits
    assert_bits_equal(to_host(alone), to_host(out), "without the kept values")

    g, zk = rand(rng, (L.rows, n), dtype), to_host(pre).copy()
    if (L.src < 0).any():  # what lies in rows no route fills is not read
        nan = np.uint16(0x7FC0) if dtype == "bf16" else np.float16(np.nan)
        g[L.src < 0], zk[L.src < 0] = nan, nan
    bias_dt = "f32" if bias in (None, "f32") else dtype
    got = M.moe_expert_act_backward(Lg, dev(g), dev(zk), act=name, gated=gated, w=dev(w), need_w=weighted,
                                    bias_dtype=torch.float32 if bias_dt == "f32" else big[0].dtype, need_residual=True)
    check_backward(got, L, g, zk, dtype, name, gated, w, bias_dt, what)
    gz = to_host(got[0])
    ga = torch.full((L.rows + 2, m), 3.0, dtype=big[0].dtype, device="cuda")
    M.moe_expert_act_dgrad(Lg, got[0], dev(wts), out=ga[1:-1])
    assert (ga[0] == 3).all() and (ga[-1] == 3).all(), "rows beside the input gradient were written"
    _, want = oracle.expert_gemm_dgrad(L, gz, wts, dtype)
    _, mag = oracle.expert_gemm_dgrad(L, absolute(gz, dtype), absolute(wts, dtype), dtype)
    within(to_host(ga[1:-1].contiguous()), want, (nz + 3) * 2 * U * mag, dtype, what + ", grad_a")
    if gated or name != "none":
        less = M.moe_expert_act_backward(Lg, dev(g), dev(zk), act=name, gated=gated, w=dev(w))
        assert_bits_equal(to_host(less[0]), to_host(got[0]), "grad_preact alone")
        assert less[1] is None and less[2] is None and less[3] is None


CASES = [
    # s, m, n, e, k, capacity, pad, route_major, dtype, act, gated, bias, weighted, residual, gather
    (1, 8, 8, 3, 2, 0, 1, False, "bf16", "silu", True, None, False, None, True),        # smallest rows
    (1, 520, 72, 16, 8, 0, 1, False, "f16", "gelu", False, "f32", True, "tokens", True), # one token
    (16, 264, 200, 8, 2, 0, 1, False, "bf16", "relu", True, "own", True, "rows", True),
    (17, 1024, 96, 4, 4, 0, 1, False, "bf16", "gelu_tanh", False, None, False, None, False),
    (60, 136, 40, 2, 2, 0, 1, False, "f16", "silu", True, "f32", False, "tokens", True),
    (200, 72, 64, 16, 2, 0, 16, False, "bf16", "none", False, "own", True, None, True),  # padded segments
    (300, 64, 128, 4, 2, 0, 1, False, "bf16", "gelu", True, "own", False, "rows", False),
    (1000, 264, 200, 8, 2, 0, 1, False, "bf16", "silu", True, "f32", True, "tokens", True),  # ragged everywhere
    (1000, 136, 264, 8, 3, 200, 1, True, "f16", "gelu_tanh", False, "own", True, "rows", True),  # drops, route-major
    (2000, 512, 328, 16, 4, 0, 128, False, "f16", "relu", False, "f32", False, None, True),
    (777, 64, 64, 1024, 16, 0, 1, True, "bf16", "silu", True, None, False, None, True),  # most experts empty
    (4000, 72, 136, 4, 2, 600, 1, False, "bf16", "none", True, "own", True, "tokens", False),
    (700, 8, 520, 2, 1, 0, 1, False, "bf16", "gelu", False, None, True, None, True),     # one K chunk
    (900, 128, 8, 3, 3, 0, 1, False, "f16", "silu", True, "own", False, "rows", True),   # one column chunk
    (20, 136, 72, 1024, 4, 0, 1, False, "bf16", "silu", True, "own", True, "tokens", True),  # few of many experts
    (20, 72, 264, 700, 8, 3, 1, False, "f16", "gelu", False, "f32", True, "rows", False),    # capacity, mostly empty
]


@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-{c[9]}" for c in CASES])
def test_matches_the_oracle(case):
    announce("expert act", *case)
    s, m, n, e, k, cap, pad, rm, dtype, name, gated, bias, weighted, residual, gather = case
    idx = W.random_idx(np.random.default_rng(s + m + n), s, e, k)
    run_case(idx, m, n, e, cap, pad, rm, dtype, name, gated, bias, weighted, residual, gather, s + n)


# rows of one expert: every tile height (32 to 288), the last row and the first of the next
ROWS = [66, 96, 97, 128, 160, 192, 193, 224, 256, 257, 288, 289, 320, 577, 865]


@pytest.mark.parametrize("rows", ROWS)
def test_every_tile_height(rows):
    announce("expert act height", rows)
    run_case(np.zeros((rows, 1), np.int32), 136, 144, 1, 0, 1, False, "bf16", "silu", True, "own", True, "tokens", True, rows)


def test_uneven_segments():
    """Segments of 1, 30, 33, 0, 700 and 64 rows beside each other."""
    announce("expert act uneven")
    idx = np.repeat(np.arange(6), [1, 30, 33, 0, 700, 64]).astype(np.int32)
    idx = idx[np.random.default_rng(1).permutation(len(idx))][:, None]
    for gated in (False, True):
        run_case(idx, 200, 272, 6, 0, 1, False, "f16", "gelu_tanh", gated, "own", True, "rows", True, 5)


WIDE = [  # products wide enough for the large tiles, columns as above
    (1000, 264, 1000, 8, 2, 0, 1, False, "bf16", "silu", True, "f32", True, "tokens", True),
    (1000, 136, 1096, 8, 3, 200, 1, True, "f16", "gelu_tanh", False, "own", True, "rows", True),
    (300, 64, 2056, 4, 2, 0, 64, False, "bf16", "gelu", True, "own", False, "rows", False),
    (700, 8, 2600, 2, 1, 0, 1, False, "bf16", "none", False, None, True, None, True),
    (60, 136, 5000, 2, 2, 0, 1, False, "f16", "silu", True, "f32", False, "tokens", True),
    (40, 72, 4096, 64, 8, 0, 1, False, "bf16", "relu", False, "own", True, "tokens", True),  # five rows an expert
]


@pytest.mark.parametrize("case", WIDE, ids=[f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-{c[9]}" for c in WIDE])
def test_wide_products_match_the_oracle(case):
    test_matches_the_oracle(case)


@pytest.mark.parametrize("rows", ROWS)
def test_every_tile_height_of_wide_products(rows):
    """As many columns as make 64-row pieces too many for the form of short segments."""
    announce("expert act wide height", rows)
    n = 32 * -(-449 // (rows // 64 + 1)) + 8
    run_case(np.zeros((rows, 1), np.int32), 72, n, 1, 0, 1, False, "bf16", "silu", True, "own", True, "tokens", True, rows)


def test_uneven_segments_of_wide_products():
    announce("expert act wide uneven")
    idx = np.repeat(np.arange(6), [1, 30, 33, 0, 700, 64]).astype(np.int32)
    idx = idx[np.random.default_rng(1).permutation(len(idx))][:, None]
    for gated in (False, True):
        run_case(idx, 200, 1608, 6, 0, 1, False, "f16", "gelu_tanh", gated, "own", True, "rows", True, 5)


@pytest.mark.parametrize("n", [72, 1512])
@pytest.mark.parametrize("s,e,k", [(40, 8, 4), (300, 64, 4), (1500, 3, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_whole_numbers_are_exact(s, e, k, n, dtype):
    """Products of small whole numbers have exact sums in any order: all forms agree bit for bit."""
    announce("expert act integers", s, e, k, n, dtype)
    rng = np.random.default_rng(s)
    m = 120
    idx = W.random_idx(rng, s, e, k)
    L = oracle.dispatch_layout(idx, e, 0)
    Lg = M.moe_dispatch_layout(to_dev(idx), e, 0)
    x = W.cast_input(rng.integers(-2, 3, (s, m)).astype(np.float32), dtype)
    wts = W.cast_input(rng.integers(-2, 3, (e, n, m)).astype(np.float32), dtype)
    b = rng.integers(-3, 4, (e, n)).astype(np.float32)
    xd, wd = to_dev(x, dtype), to_dev(wts, dtype)
    want, _ = oracle.expert_gemm_act(L, x, wts, dtype, True, b, "relu")
    got = M.moe_expert_gemm_act(Lg, xd, wd, bias=to_dev(b), act="relu")
    assert_bits_equal(to_host(got), oracle.from_f32(want.astype(np.float32), dtype), "relu")
    plain = M.moe_expert_gemm_act(Lg, xd, wd)
    assert_bits_equal(to_host(plain), to_host(M.moe_expert_gemm(Lg, xd, wd)), "no epilogue: the plain product")
    rows = M.moe_expert_gemm_act(Lg, M.moe_dispatch(Lg, xd), wd, gather=False)
    assert_bits_equal(to_host(rows), to_host(plain), "from the dispatched buffer")


def test_routes_that_name_no_expert():
    announce("expert act bad routes")
    rng = np.random.default_rng(2)
    idx = W.random_idx(rng, 500, 6, 3)
    idx[::5, 1], idx[7], idx[9, 2] = -1, 6, idx[9, 0]
    run_case(idx, 72, 136, 6, 0, 1, False, "bf16", "silu", True, "own", True, "tokens", True, 3)
    run_case(np.full((90, 2), -1, np.int32), 72, 136, 6, 0, 1, False, "bf16", "silu", True, "own", True, "rows", False, 3)


def test_nan_and_inf_stay_where_they_are():
    """A token's or an expert's NaN and infinities reach their own rows and features alone,
    also through the K tail and the rows a tile repeats."""
    announce("expert act nan")
    rng = np.random.default_rng(4)
    m = 72
    for s, e, k, n in ((12, 8, 2, 136), (700, 3, 2, 136), (700, 3, 2, 1608)):
        idx = W.random_idx(rng, s, e, k)
        idx[0], idx[1] = [0, 1], [1, 2]
        Lg = M.moe_dispatch_layout(to_dev(idx), e, 0)
        L = oracle.dispatch_layout(idx, e, 0)
        x = rng.standard_normal((s, m)).astype(np.float32)
        wts = rng.standard_normal((e, 2 * n, m)).astype(np.float32)
        x[0, 3], x[1, 0] = np.nan, np.inf
        wts[2, 5, 1], wts[0, n + 7, 0] = np.inf, np.nan
        with np.errstate(all="ignore"):
            out, _ = oracle.expert_gemm_act(L, W.cast_input(x, "bf16"), W.cast_input(wts, "bf16"), "bf16", True, None,
                                            "gelu", True)
        got = to_host(M.moe_expert_gemm_act(Lg, to_dev(W.cast_input(x, "bf16"), "bf16"),
                                            to_dev(W.cast_input(wts, "bf16"), "bf16"), act="gelu", gated=True))
        f = oracle.to_f32(got, "bf16")
        assert np.array_equal(np.isfinite(f), np.isfinite(out))


def test_input_gradient_of_whole_numbers_is_exact():
    """K tails of every length, and infinities in weights past which nothing may reach."""
    announce("expert act dgrad integers")
    rng = np.random.default_rng(11)
    for s, e, k, nz, m, dtype in ((700, 3, 2, 8, 264, "bf16"), (90, 1, 1, 72, 8, "f16"), (300, 4, 1, 200, 520, "bf16"),
                                  (2000, 4, 2, 64, 136, "f16"), (20, 8, 2, 136, 72, "bf16")):
        idx = W.random_idx(rng, s, e, k)
        L, Lg = oracle.dispatch_layout(idx, e, 0), M.moe_dispatch_layout(to_dev(idx), e, 0)
        g = W.cast_input(rng.integers(-2, 3, (L.rows, nz)).astype(np.float32), dtype)
        wts = W.cast_input(rng.integers(-2, 3, (e, nz, m)).astype(np.float32), dtype)
        want, _ = oracle.expert_gemm_dgrad(L, g, wts, dtype)
        got = M.moe_expert_act_dgrad(Lg, to_dev(g, dtype), to_dev(wts, dtype))
        assert_bits_equal(to_host(got), want, f"{s} {nz} {m}")
        assert torch.equal(got, M.moe_expert_gemm_dgrad(Lg, to_dev(g, dtype), to_dev(wts, dtype)))
        w32 = oracle.to_f32(wts, dtype).copy()
        w32[0, nz - 1, 3], g32 = np.inf, np.abs(oracle.to_f32(g, dtype)) + 1  # positive rows: sums of one sign at inf
        got = M.moe_expert_act_dgrad(Lg, to_dev(W.cast_input(g32, dtype), dtype), to_dev(W.cast_input(w32, dtype), dtype))
        f = oracle.to_f32(to_host(got), dtype)
        rows = slice(int(L.offsets[0]), int(L.offsets[0]) + int(L.kept[0]))
        assert np.isposinf(f[rows, 3]).all()
        f[rows, 3] = 0
        assert np.isfinite(f).all()


@pytest.mark.parametrize("name", E.ACTS)
def test_activations_over_their_range(name):
    """One product per output sets z to any element value: every finite bf16 from 1e-3 to 1e5,
    both signs and zeros, forward and slope."""
    announce("expert act range", name)
    bits = np.arange(0x3A83, 0x47C4, dtype=np.uint16)
    bits = np.concatenate([bits, bits | np.uint16(0x8000), np.array([0, 0x8000], np.uint16)])
    n = (len(bits) + 7) // 8 * 8
    vals = np.zeros(n, np.uint16)
    vals[:len(bits)] = bits
    wts = np.zeros((1, n, 8), np.uint16)
    wts[0, :, 0] = vals
    x = np.zeros((1, 8), np.uint16)
    x[0, 0] = 0x3F80
    idx = np.zeros((1, 1), np.int32)
    L, Lg = oracle.dispatch_layout(idx, 1, 0), M.moe_dispatch_layout(to_dev(idx), 1, 0)
    out, pre = M.moe_expert_gemm_act(Lg, to_dev(x, "bf16"), to_dev(wts, "bf16"), act=name, save_preact=True)
    check_forward(out, pre, L, x, wts, "bf16", True, None, name, False, None, None, False, name)
    g = np.full((1, n), 0x3F80, np.uint16)
    got = M.moe_expert_act_backward(Lg, to_dev(g, "bf16"), pre, act=name, bias_dtype=torch.float32)
    check_backward(got, L, g, to_host(pre), "bf16", name, False, None, "f32", name)
    for inf in (0x7F80, 0xFF80):  # slopes at the infinities are 0 or 1, not NaN
        z = torch.full((1, 8), float(np.uint32(inf << 16).view(np.float32)), dtype=torch.bfloat16, device="cuda")
        d = M.moe_expert_act_backward(Lg, torch.ones((1, 8), dtype=torch.bfloat16, device="cuda"), z, act=name)[0] \
            if name != "none" else torch.ones(1, device="cuda")
        assert torch.equal(d.float().unique(), torch.tensor([1.0 if inf == 0x7F80 or name == "none" else 0.0], device="cuda"))


def test_empty_batches():
    announce("expert act empty")
    idx = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    w = torch.randn((4, 16, 8), device="cuda").to(torch.bfloat16)
    for cap, pad in ((0, 1), (3, 1), (0, 8)):
        L = M.moe_dispatch_layout(idx, 4, cap, pad_multiple=pad)
        x = torch.empty((0, 8), dtype=torch.bfloat16, device="cuda")
        out, pre = M.moe_expert_gemm_act(L, x, w, act="silu", gated=True, save_preact=True,
                                         out=torch.full((L.rows, 8), 9.0, dtype=torch.bfloat16, device="cuda"))
        assert out.shape == (L.rows, 8) and pre.shape == (L.rows, 16) and not out.any() and not pre.any()
        got = M.moe_expert_act_backward(L, out, pre, act="silu", gated=True, w=torch.empty((0, 2), device="cuda"),
                                        need_w=True, bias_dtype=torch.float32, need_residual=True)
        assert got[0].shape == pre.shape and not got[0].any() and not got[1].any() and got[2].shape == (0, 2) and not got[3].any()


@pytest.mark.parametrize("s,n", [(24, 104), (900, 104), (900, 1000)])
def test_replays_from_a_graph_and_runs_beside_another_stream(s, n):
    announce("expert act graph", s, n)
    rng = np.random.default_rng(6)
    m, e, k = 136, 8, 2
    idx = to_dev(W.random_idx(rng, s, e, k))
    x, wts = to_dev(rand(rng, (s, m), "bf16"), "bf16"), to_dev(W.expert_weights(2, e, 2 * n, m, "bf16"), "bf16")
    bias, w = to_dev(rand(rng, (e, 2 * n), "bf16"), "bf16"), to_dev(W.random_weights(rng, s, k))
    g = to_dev(rand(rng, (s * k, n), "bf16"), "bf16")

    def step():
        L = M.moe_dispatch_layout(idx, e, 0)
        out, pre = M.moe_expert_gemm_act(L, x, wts, bias=bias, act="silu", gated=True, w=w, save_preact=True)
        gz, gb, gw, _ = M.moe_expert_act_backward(L, g, pre, act="silu", gated=True, w=w, need_w=True, bias_dtype=torch.bfloat16)
        return out, pre, gz, gb, gw, M.moe_expert_act_dgrad(L, gz, wts), M.moe_expert_gemm_wgrad(L, x, gz)

    first = [t.clone() for t in step()]
    torch.cuda.synchronize()
    streams, runs = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(3):
        for st in streams:
            with torch.cuda.stream(st):
                runs.append(step())
    torch.cuda.synchronize()
    for r in runs:
        assert all(torch.equal(p, q) for p, q in zip(r, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for rep in range(3):
        x.copy_(to_dev(rand(rng, (s, m), "bf16"), "bf16"))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs, want)), f"replay {rep}"


def test_more_values_than_32_bits_count():
    """560000 rows of 4096 outputs: offsets past 2^31 elements, checked at both ends."""
    announce("expert act 2.3e9 outputs")
    s, m, n, e, k = 70000, 64, 4096, 8, 8
    gen = torch.Generator("cuda").manual_seed(3)
    idx = torch.rand((s, e), generator=gen, device="cuda").argsort(1).int()
    x = torch.randn((s, m), generator=gen, device="cuda").to(torch.bfloat16)
    wts = (torch.randn((e, n, m), generator=gen, device="cuda") / 8).to(torch.bfloat16)
    L = M.moe_dispatch_layout(idx, e, 0)
    out, pre = M.moe_expert_gemm_act(L, x, wts, act="silu", save_preact=True)
    for rows in (slice(0, 50), slice(L.rows - 50, L.rows)):
        r = torch.arange(L.rows, device="cuda")[rows]
        ex = torch.searchsorted(L.offsets[1:].long(), r, right=True)
        z = (x[L.src[rows].long()].double()[:, None, :] * wts[ex].double()).sum(2)
        want = z / (1 + torch.exp(-z))
        err = (out[rows].double() - want).abs()
        assert (err <= 2.0 ** -8 * want.abs() + (m + 3) * 2 * U * 8).all()
        assert ((pre[rows].double() - z).abs() <= 2.0 ** -8 * z.abs() + (m + 3) * 2 * U * 8).all()
    gz, _, gw, _ = M.moe_expert_act_backward(L, out, pre, act="silu", w=torch.ones((s, k), device="cuda"), need_w=True)
    tail = slice(L.rows - 50, L.rows)
    z, g = pre[tail].double(), out[tail].double()
    sg = torch.sigmoid(z)
    want = g * sg * (1 + z * (1 - sg))
    assert ((gz[tail].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5 * g.abs()).all()
    dots = (g * z * sg).sum(1)
    last = (L.dst.flatten()[:, None] == torch.arange(L.rows - 50, L.rows, device="cuda")).int().argmax(0)
    assert ((gw.flatten()[last].double() - dots).abs() <= 1e-5 * (g * z * sg).abs().sum(1)).all()


@pytest.mark.parametrize("s", [4, 300])
def test_weights_past_4_gib(s):
    """Both ends of 4.8 GB of weights, forward and input gradient."""
    announce("expert act weights past 4 GiB", s)
    e, n, m = 36, 8192, 8192
    wts = torch.zeros((e, n, m), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator("cuda").manual_seed(8)
    for x in (0, e - 1):
        wts[x] = (torch.randn((n, m), generator=gen, device="cuda") / 8).to(torch.bfloat16)
    idx = torch.where(torch.arange(s, device="cuda") % 2 == 0, 0, e - 1).int()[:, None].contiguous()
    L = M.moe_dispatch_layout(idx, e, 0)
    a = torch.randn((s, m), generator=gen, device="cuda").to(torch.bfloat16)
    out = M.moe_expert_gemm_act(L, a, wts, act="relu")
    g = torch.randn((s, n), generator=gen, device="cuda").to(torch.bfloat16)
    ga = M.moe_expert_act_dgrad(L, g, wts)
    for x, rows in ((0, slice(0, (s + 1) // 2)), (e - 1, slice((s + 1) // 2, s))):
        w64, a64, g64 = wts[x].double(), a[L.src[rows].long()].double(), g[rows].double()
        want, mag = (a64 @ w64.t()).clamp(min=0), a64.abs() @ w64.t().abs()
        assert ((out[rows].double() - want).abs() <= 2.0 ** -8 * want.abs() + (m + 3) * 2 * U * mag).all()
        want, mag = g64 @ w64, g64.abs() @ w64.abs()
        assert ((ga[rows].double() - want).abs() <= 2.0 ** -8 * want.abs() + (n + 3) * 2 * U * mag).all()


GRADS = [("silu", True, True, False, "own", None, "bf16"), ("gelu", False, False, True, "f32", "rows", "bf16"),
         ("none", False, True, True, "own", "tokens", "f16"), ("relu", True, False, False, None, "tokens", "bf16"),
         ("none", False, False, False, "own", None, "f16")]


@pytest.mark.parametrize("name,gated,gather,weighted,bias,residual,dtype", GRADS)
def test_autograd_matches_the_oracle_chain(name, gated, gather, weighted, bias, residual, dtype):
    """expert_linear's gradients: the epilogue's backward, then the products' on it."""
    announce("expert act autograd", name, gated, gather)
    rng = np.random.default_rng(7)
    s, m, n, e, k, cap = 200, 72, 40, 6, 2, 50
    td = torch.bfloat16 if dtype == "bf16" else torch.float16
    idx = W.random_idx(rng, s, e, k)
    L, Lg = oracle.dispatch_layout(idx, e, cap), M.moe_dispatch_layout(to_dev(idx), e, cap)
    nz = 2 * n if gated else n
    leaf = lambda a, d=dtype: to_dev(a, d).requires_grad_()  # noqa: E731
    x = leaf(rand(rng, (s if gather else L.rows, m), dtype))
    wts = leaf(W.expert_weights(8, e, nz, m, dtype))
    b = None if bias is None else leaf(rand(rng, (e, nz), dtype)) if bias == "own" else leaf(rng.standard_normal((e, nz)).astype(np.float32), None)
    w = leaf(W.random_weights(rng, s, k), None) if weighted else None
    res = None if residual is None else leaf(rand(rng, (s if residual == "tokens" else L.rows, n), dtype))
    out = A.expert_linear(x, wts, Lg, bias=b, act=name, gated=gated, w=w, residual=res,
                          residual_gather=residual == "tokens", gather=gather)
    g = rand(rng, (L.rows, n), dtype)
    leaves = [t for t in (x, wts, b, w, res) if t is not None]
    grads = dict(zip([q for q, t in zip(("x", "wts", "b", "w", "res"), (x, wts, b, w, res)) if t is not None],
                     torch.autograd.grad(out, leaves, to_dev(g, dtype), retain_graph=True)))
    kw = dict(gather=gather, bias=b.detach() if b is not None else None, act=name, gated=gated,
              w=w.detach() if w is not None else None)
    _, pre = M.moe_expert_gemm_act(Lg, x.detach(), wts.detach(), save_preact=True, **kw)
    gz, gb, gw, gr = M.moe_expert_act_backward(Lg, to_dev(g, dtype), pre, act=name, gated=gated, w=kw["w"],
                                               bias_dtype=None if b is None else b.dtype, need_w=weighted, need_residual=True)
    check_backward((gz, gb, gw, gr), L, g, to_host(pre), dtype, name, gated, None if w is None else to_host(w),
                   "f32" if bias == "f32" else dtype, "chain")
    ga = M.moe_expert_act_dgrad(Lg, gz, wts.detach())
    assert torch.equal(grads["x"], M.moe_dispatch_backward(Lg, ga) if gather else ga)
    assert torch.equal(grads["wts"], M.moe_expert_gemm_wgrad(Lg, x.detach(), gz, gather=gather, out_dtype=td))
    if b is not None:
        assert torch.equal(grads["b"], gb)
    if w is not None:
        assert torch.equal(grads["w"], gw)
    if res is not None:
        assert torch.equal(grads["res"], M.moe_dispatch_backward(Lg, to_dev(g, dtype)) if residual == "tokens" else gr)
    # one leaf at a time gives the same
    for q, t in zip(grads, leaves):
        (one,) = torch.autograd.grad(out, t, to_dev(g, dtype), retain_graph=True)
        assert torch.equal(one, grads[q]), q


def test_plain_expert_linear_is_unchanged():
    announce("expert act plain linear")
    rng = np.random.default_rng(9)
    idx = W.random_idx(rng, 300, 8, 2)
    Lg = M.moe_dispatch_layout(to_dev(idx), 8, 0)
    x, wts = to_dev(rand(rng, (300, 72), "bf16"), "bf16"), to_dev(W.expert_weights(3, 8, 40, 72, "bf16"), "bf16")
    assert torch.equal(A.expert_linear(x, wts, Lg), M.moe_expert_gemm(Lg, x, wts))


def test_a_layer_of_all_the_pieces():
    """Router losses, gated up projection, down projection with bias, combine: one backward
    through everything; the gradient against differences along a direction, in float64 on the
    oracle's chain at the same routing."""
    announce("whole layer")
    rng = np.random.default_rng(12)
    s, m, n, e, k, dtype = 96, 64, 48, 8, 2, "f16"
    logits = (rng.standard_normal((s, e)) * 2).astype(np.float32)
    x, up, down = rand(rng, (s, m), dtype), W.expert_weights(1, e, 2 * n, m, dtype), W.expert_weights(2, e, m, n, dtype)
    b1, b2, gy = rand(rng, (e, 2 * n), dtype, 0.1), rand(rng, (e, m), dtype, 0.1), rand(rng, (s, m), dtype)
    leaves = [to_dev(t, dtype if t.dtype != np.float32 else None).requires_grad_() for t in (logits, x, up, down, b1, b2)]
    tl, tx, tup, tdown, tb1, tb2 = leaves
    idx, w = A.route(tl, k)
    loss, z, _ = A.balance_loss(tl, idx)
    L, _ = A.layout(idx, e)
    h = A.expert_linear(tx, tup, L, bias=tb1, act="silu", gated=True)
    y = A.combine(A.expert_linear(h, tdown, L, bias=tb2, gather=False, residual=tx, residual_gather=True), w, L)
    grads = torch.autograd.grad([y, loss, z], leaves, [to_dev(gy, dtype), torch.full((1,), 5.0, device="cuda"), torch.full((1,), 2.0, device="cuda")])
    ids = idx.cpu().numpy()
    Lo = oracle.dispatch_layout(ids, e, 0)

    def value(l, x_, up_, down_, b1_, b2_):
        """The scalar whose gradient the grads are, in float64."""
        sel = np.take_along_axis(l, ids, 1)
        wt = np.exp(sel - sel.max(1, keepdims=True))
        wt /= wt.sum(1, keepdims=True)
        bl = oracle.balance_loss(l, ids)
        rows = np.zeros((Lo.rows, m))
        for ex, r in E.segments(Lo):
            zz = x_[Lo.src[r]] @ up_[ex].T + b1_[ex]
            rows[r] = E.finish(zz, "silu", True) @ down_[ex].T + b2_[ex] + x_[Lo.src[r]]
        yy = (wt[:, :, None] * rows[Lo.dst]).sum(1)
        return float((yy * real(gy, dtype)).sum() + 5.0 * bl.loss[0] + 2.0 * bl.z[0])

    at = [real(t, dtype) for t in (logits, x, up, down, b1, b2)]
    for i, g in enumerate(grads):
        d = rng.standard_normal(at[i].shape)
        step = 1e-4
        ends = [value(*[t + (c * d if j == i else 0) for j, t in enumerate(at)]) for c in (step, -step)]
        want = (ends[0] - ends[1]) / (2 * step)
        got = float((g.double().cpu().numpy() * d).sum())
        # a chain of five f16 roundings (2^-11 each, independent per element) against the size of the terms
        size = np.sqrt((g.double().cpu().numpy() ** 2).sum())
        assert abs(got - want) <= 5 * 2.0 ** -11 * 8 * size + 1e-4, (i, got, want, size)


def test_a_captured_training_step_replays():
    """Router, both losses, a gated and a weighted projection and their backward in one graph:
    each replay gives the eager step's bits, also between eager steps on other leaves."""
    announce("captured step")
    rng = np.random.default_rng(31)
    s, m, n, e, k = 300, 72, 136, 8, 2
    data = [to_dev(t, "bf16" if t.dtype != np.float32 else None) for t in (
        rng.standard_normal((s, e)).astype(np.float32), rand(rng, (s, m), "bf16"), W.expert_weights(1, e, 2 * n, m, "bf16"),
        W.expert_weights(2, e, m, n, "bf16"), rand(rng, (e, m), "bf16"))]
    gy = to_dev(rand(rng, (s, m), "bf16"), "bf16")

    def step(values):
        leaves = [t.detach().requires_grad_() for t in values]  # new leaves: none is shared with another graph
        logits, x, up, down, bias = leaves
        idx, w = A.route(logits, k)
        loss, z, _ = A.balance_loss(logits, idx)
        L, _ = A.layout(idx, e)
        h = A.expert_linear(x, up, L, act="silu", gated=True)
        y = A.combine(A.expert_linear(h, down, L, bias=bias, w=w, gather=False), None, L)
        return (y.detach(), *torch.autograd.grad([y, loss.sum() + 0.5 * z.sum()], leaves, [gy, torch.ones((), device="cuda")]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(data)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(data)
    for rep in range(3):
        data[0].copy_(torch.from_numpy(rng.standard_normal((s, e)).astype(np.float32)))
        data[1].copy_(to_dev(rand(rng, (s, m), "bf16"), "bf16"))
        want = [t.clone() for t in step(data)]
        torch.cuda.synchronize()
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), f"replay {rep}, output {i}"


def test_refusals():
    announce("expert act refusals")
    idx = to_dev(W.random_idx(np.random.default_rng(1), 20, 4, 2))
    L = M.moe_dispatch_layout(idx, 4, 0)
    x, w = torch.zeros((20, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((4, 64, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(M.MoeError, match="overlap"):
        buf = torch.zeros((40, 64), dtype=torch.bfloat16, device="cuda")
        M.moe_expert_gemm_act(L, buf, w, gather=False, out=buf)
    with pytest.raises(M.MoeError, match="overlap"):
        buf = torch.zeros((40, 64), dtype=torch.bfloat16, device="cuda")
        M.moe_expert_gemm_act(L, x, w, residual=buf, out=buf)
    with pytest.raises(M.MoeError, match="overlap"):
        M.moe_expert_gemm_act(L, x, w, out=w.view(-1, 64)[:40])
    with pytest.raises(M.MoeError, match="MISALIGNED"):
        M.moe_expert_gemm_act(L, x, torch.zeros((4, 60, 64), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(M.MoeError, match="MISALIGNED"):
        M.moe_expert_gemm_act(L, x, w, bias=torch.zeros(257, device="cuda")[1:].view(4, 64))
    with pytest.raises(M.MoeError, match="WORKSPACE"):
        M.moe_expert_act_backward(L, torch.zeros((40, 64), dtype=torch.bfloat16, device="cuda"), bias_dtype=torch.float32,
                                  workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        M.moe_expert_gemm_act(L, torch.zeros((64, 20), dtype=torch.bfloat16, device="cuda").t(), w)
