"""Experts in microscaled 4-bit floating point on the GPU against float64 oracles.

Quantising and reading back are exact definitions: equal bit for bit. Products: each product of two
values is exact (a 4-bit value has 2 significant bits, a bf16 value 8; an f16 value meets the weight
whole, or split in two parts of the same sum). With u = 2^-24 the float32 sum of m of them is off by at
most (m + 3) 2u of the sum of their magnitudes in any order (2 m of them where split, whose magnitudes
are at most 1 + 2^-7 times the whole's, hence (2 m + 6) 2u for f16 rows). What follows a sum, and the
roundings at the end, are bounded as at the top of test_gpu_expert_act.py. A result rounded to 4 bits
lies between what the two ends of its bound round to (rounding is monotone), on a scale between those
of the two ends.
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
from tests.test_gpu_expert_act import U, act_err, announce, half, rand, real, within

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------------
# rows to 4 bits and back


def patterns(rng, dtype, rows, m):
    """Rows whose blocks mix magnitudes, borders between codes, zeros of both signs and, here and there,
    subnormals, the largest values, infinities and NaN."""
    x = rng.standard_normal((rows, m)) * np.exp2(rng.integers(-12, 12, (rows, m // 32)).repeat(32, 1))
    scale = np.exp2(rng.integers(-6, 6, (rows, m // 32))).repeat(32, 1)
    border = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.75, 0.0, 4.0], (rows, m)) * rng.choice([-1, 1], (rows, m))
    x = np.where(rng.random((rows, m)) < 0.5, x, border * scale)
    x = np.where(rng.random((rows, m // 32)).repeat(32, 1) < 0.05, border * 0, x)
    with np.errstate(over="ignore"):
        x = W.cast_input(x.astype(np.float32), dtype)
    it = {"f32": np.uint32, "bf16": np.uint16, "f16": np.uint16}[dtype]
    bits = x.view(it).copy()
    any_bits = rng.integers(0, 2 ** (32 if dtype == "f32" else 16), (rows, m), dtype=np.uint64).astype(it)
    some = rng.random((rows, m // 32)).repeat(32, 1) < 0.2
    bits = np.where(some, any_bits, bits)
    mant = {"f32": 23, "bf16": 7, "f16": 10}[dtype]
    tiny = rng.random((rows, m // 32)).repeat(32, 1) < 0.05
    bits = np.where(tiny, bits & it((1 << mant) - 1), bits).astype(it)  # blocks of subnormals
    return bits.view(x.dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,m", [(1, 32), (1, 2848), (3, 96), (7, 32), (129, 160), (333, 1056), (4097, 64), (70001, 128)])
def test_rows_to_four_bits_and_back(rows, m, dtype):
    announce("mx4 rows", rows, m, dtype)
    x = patterns(np.random.default_rng(rows + m), dtype, rows, m)
    with np.errstate(invalid="ignore"):
        want_c, want_s = mx4.quantize(oracle.to_f32(x, dtype).astype(np.float64))
    codes = torch.full((rows + 2, m // 2), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows * (m // 32) + 2,), 0xA5, dtype=torch.uint8, device="cuda")
    c, s = M.moe_mx4_quantize(to_dev(x, dtype), codes=codes[1:-1], scales=scales[1:-1].view(rows, m // 32))
    assert (codes[[0, -1]] == 0xA5).all() and (scales[[0, -1]] == 0xA5).all(), "bytes beside the outputs were written"
    assert np.array_equal(to_host(s), want_s) and np.array_equal(to_host(c), want_c)
    for to in ("bf16", "f16", "f32"):
        with np.errstate(invalid="ignore", over="ignore"):
            want = mx4.values(want_c, want_s).astype(np.float32)
            want = oracle.from_f32(want, to)
        out = torch.full((rows + 2, m), 7.0, dtype=TORCH_DTYPE[to], device="cuda")
        got = to_host(M.moe_mx4_dequantize(c, s, out=out[1:-1]))
        assert (out[[0, -1]] == 7).all(), "rows beside the output were written"
        nan = np.repeat(want_s == 255, 32, -1)
        assert np.isnan(oracle.to_f32(got, to)[nan]).all()
        assert_bits_equal(np.where(nan, 0, got).astype(got.dtype), np.where(nan, 0, want).astype(want.dtype), f"read back as {to}")


def test_every_scale_and_code():
    announce("mx4 every scale and code")
    c = np.arange(256, dtype=np.uint8)[None].repeat(256, 0)  # 16 blocks a row
    s = np.arange(256, dtype=np.uint8)[:, None].repeat(16, 1)
    for to in ("bf16", "f16", "f32"):
        with np.errstate(over="ignore", invalid="ignore"):
            want = oracle.from_f32(mx4.values(c, s).astype(np.float32), to)
        got = to_host(M.moe_mx4_dequantize(to_dev(c), to_dev(s), TORCH_DTYPE[to]))
        assert_bits_equal(got[:255], want[:255], to)
        assert np.isnan(oracle.to_f32(got[255], to)).all()


def test_every_bf16_value():
    """Every finite bf16 value as the largest of a block, with its halves and borders beside it."""
    announce("mx4 every bf16 value")
    top = np.arange(0x7F80, dtype=np.uint32) << 16
    f = top.view(np.float32)
    x = np.zeros((len(f), 32), np.float32)
    for i in range(32):
        x[:, i] = f * np.float32((i + 1) / 32) * np.float32(1 if i % 3 else -1)
    x[:, 31] = f
    x = W.cast_input(x, "bf16")
    want_c, want_s = mx4.quantize(oracle.to_f32(x, "bf16").astype(np.float64))
    c, s = M.moe_mx4_quantize(to_dev(x, "bf16"))
    assert np.array_equal(to_host(s), want_s) and np.array_equal(to_host(c), want_c)


def test_leading_dimensions_and_no_rows():
    announce("mx4 shapes")
    x = torch.randn(3, 5, 64, device="cuda")
    c, s = M.moe_mx4_quantize(x)
    assert c.shape == (3, 5, 32) and s.shape == (3, 5, 2)
    c1, s1 = M.moe_mx4_quantize(x.view(-1))
    assert torch.equal(c1, c.view(-1)) and torch.equal(s1, s.view(-1))
    back = M.moe_mx4_dequantize(c, s, torch.float32)
    assert back.shape == x.shape and torch.equal(M.moe_mx4_dequantize(c1, s1, torch.float32), back.view(-1))
    c, s = M.moe_mx4_quantize(torch.empty(0, 64, device="cuda"))
    assert c.shape == (0, 32) and s.shape == (0, 2) and M.moe_mx4_dequantize(c, s).shape == (0, 64)


def test_past_four_gib():
    """Values, and codes, at offsets past 32 bits."""
    announce("mx4 past 4 GiB")
    rows, m = (1 << 33) // 4096 + 3, 4096  # codes of 4 GiB and a little
    x = torch.zeros((rows, m), dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.arange(m, device="cuda").remainder(13) - 6
    x[0] = 3.0
    c, s = M.moe_mx4_quantize(x)
    want_c, want_s = mx4.quantize(oracle.to_f32(to_host(x[-1:]), "bf16").astype(np.float64))
    assert np.array_equal(to_host(c[-1:]), want_c) and np.array_equal(to_host(s[-1:]), want_s)
    x.fill_(9.0)
    M.moe_mx4_dequantize(c, s, out=x)
    want = torch.from_numpy(mx4.values(want_c, want_s)).cuda().bfloat16()
    assert torch.equal(x[-1:], want) and (x[0] == 3).all() and not x[1:-1].any()


# ---------------------------------------------------------------------------------
# products


def four_bits(rng, shape, zero_blocks=False):
    """(codes, scales, float32 values) of normal draws of another magnitude each row."""
    x = rng.standard_normal(shape) * shape[-1] ** -0.5 * np.exp2(rng.integers(-3, 4, (*shape[:-1], 1)))
    if zero_blocks:
        x[..., ::3, :32] = 0
    c, s = mx4.quantize(x)
    return c, s, mx4.values(c, s).astype(np.float32)


def pair(c, s):
    return to_dev(c), to_dev(s)


def product_bounds(L, a_val, w_val, m, rows16, dtype, gather, bias, name, gated, w, res, res_gather):
    """(out, z, tolerance of out before its rounding, tolerance of z)"""
    out, z = oracle.expert_gemm_act(L, a_val, w_val, "f32", gather, bias, name, gated, w, res, res_gather)
    _, mag = oracle.expert_gemm_act(L, np.abs(a_val), np.abs(w_val), "f32", gather, None if bias is None else np.abs(bias))
    n = out.shape[1]
    terms = 2 * m + 6 if rows16 and dtype == "f16" else m + 3
    dz = terms * 2 * U * mag
    f = E.act(name, z[:, :n])[0]
    df = 1.13 * dz[:, :n] + act_err(name, z[:, :n])[0]
    if gated:
        up, dup = z[:, n:], dz[:, n:]
        du = np.abs(f) * dup + np.abs(up) * df + df * dup + U * np.abs(f * up)
    else:
        du = df
    rw = np.abs(E.row_weights(L, w))[:, None]
    tol = rw * du * (1 + U) + 2 * U * (np.abs(out) + rw * np.abs(E.finish(z, name, gated)))
    tol[L.src < 0] = 0
    return out, z, tol, dz


def check_quantized(codes, scales, out, tol, what):
    """4-bit results against exact values and their bound."""
    ab = np.abs(out).reshape(len(out), -1, 32)
    tb = tol.reshape(ab.shape)
    lo_E = mx4.scale_bytes(np.maximum(ab - tb, 0).reshape(out.shape))
    hi_E = mx4.scale_bytes((ab + tb).reshape(out.shape))
    assert ((scales >= lo_E) & (scales <= hi_E)).all(), f"{what}: a scale is outside its bound"
    got = mx4.values(codes, scales).reshape(ab.shape)
    s = np.ldexp(1.0, scales.astype(np.int64) - 127)[..., None]
    ob = out.reshape(ab.shape)

    def rounded(v):
        c = mx4.round_codes(v / s)
        return np.where(c & 8, -1.0, 1.0) * mx4.GRID[c & 7] * s

    bad = np.argwhere(~((got >= rounded(ob - tb)) & (got <= rounded(ob + tb))))
    assert len(bad) == 0, f"{what}: {len(bad)} outside the bound, first {tuple(bad[0])}"


def run_case(idx, m, n, e, cap, pad, rm, dtype, rows, name, gated, bias, weighted, residual, gather, seed, keep="own"):
    """rows: "16" (16-bit rows) or "4" (4-bit rows). Forward in both result types, kept values, input gradient."""
    rng = np.random.default_rng(seed)
    s, k = idx.shape
    L = oracle.dispatch_layout(idx, e, cap, route_major=rm, pad_multiple=pad)
    Lg = M.moe_dispatch_layout(to_dev(idx), e, cap, route_major=rm, pad_multiple=pad)
    nz = 2 * n if gated else n
    count = s if gather else L.rows
    tdt = TORCH_DTYPE[dtype]
    if rows == "16":
        a16 = rand(rng, (count, m), dtype)
        a_val, a_dev = oracle.to_f32(a16, dtype), to_dev(a16, dtype)
    else:
        ac, as_, a_val = four_bits(rng, (count, m))
        a_dev = pair(ac, as_)
    wc, ws, w_val = four_bits(rng, (e, nz, m), zero_blocks=True)
    w_dev = pair(wc, ws)
    b = None if bias is None else rng.standard_normal((e, nz)).astype(np.float32) if bias == "f32" else rand(rng, (e, nz), dtype)
    w = W.random_weights(rng, s, k) if weighted else None
    res = None if residual is None else rand(rng, (s if residual == "tokens" else L.rows, n), dtype)
    dev = lambda t: None if t is None else to_dev(t, dtype if t.dtype != np.float32 else None)  # noqa: E731
    kw = dict(gather=gather, bias=dev(b), act=name, gated=gated, w=dev(w), residual=dev(res),
              residual_gather=residual == "tokens", dtype=tdt)
    keep_dt = torch.float32 if keep == "f32" else tdt
    out = torch.full((L.rows + 2, n), 3.0, dtype=tdt, device="cuda")
    pre = torch.full((L.rows + 2, nz), 3.0, dtype=keep_dt, device="cuda")
    M.moe_mx4_expert_gemm(Lg, a_dev, w_dev, out=out[1:-1], preact=pre[1:-1], **kw)
    for t in (out, pre):
        assert (t[0] == 3).all() and (t[-1] == 3).all(), "rows beside the output were written"
    what = f"s{s} m{m} n{n} e{e} {name} gated={gated} rows {rows} {dtype}"
    want, z, tol, dz = product_bounds(L, a_val, w_val, m, rows == "16", dtype, gather, None if b is None else real(b, dtype), name,
                                      gated, w, None if res is None else oracle.to_f32(res, dtype), residual == "tokens")
    unfilled = L.src < 0
    got = to_host(out[1:-1].contiguous())
    within(got, want, tol, dtype, what)
    kept = to_host(pre[1:-1].contiguous())
    within(kept, z, dz, "f32" if keep == "f32" else dtype, what + ", kept values")
    for t, d in ((got, dtype), (kept, "f32" if keep == "f32" else dtype)):
        assert not oracle.to_f32(t[unfilled], d).view(np.uint32).any(), f"{what}: unfilled rows not +0"
    alone = M.moe_mx4_expert_gemm(Lg, a_dev, w_dev, **kw)  # without keeping z: the same bits
    assert_bits_equal(to_host(alone), got, "without the kept values")

    if n % 32 == 0:  # the same results, rounded to 4 bits instead
        qc = torch.full((L.rows + 2, n // 2), 0xA5, dtype=torch.uint8, device="cuda")
        qs = torch.full((L.rows * (n // 32) + 2,), 0xA5, dtype=torch.uint8, device="cuda")
        M.moe_mx4_expert_gemm(Lg, a_dev, w_dev, quantize_out=True, out=(qc[1:-1], qs[1:-1].view(L.rows, n // 32)), **kw)
        assert (qc[[0, -1]] == 0xA5).all() and (qs[[0, -1]] == 0xA5).all(), "bytes beside the outputs were written"
        codes, scales = to_host(qc[1:-1].contiguous()), to_host(qs[1:-1].contiguous()).reshape(L.rows, n // 32)
        check_quantized(codes, scales, want, tol, what + ", 4-bit results")
        assert not codes[unfilled].any() and not scales[unfilled].any(), "unfilled 4-bit rows not zero"

    gz = rand(rng, (L.rows, nz), dtype)
    if unfilled.any():  # what lies in rows no route fills is not read
        gz[unfilled] = np.uint16(0x7FC0) if dtype == "bf16" else np.float16(np.nan)
    ga = torch.full((L.rows + 2, m), 3.0, dtype=tdt, device="cuda")
    M.moe_mx4_expert_dgrad(Lg, to_dev(gz, dtype), w_dev, out=ga[1:-1])
    assert (ga[0] == 3).all() and (ga[-1] == 3).all(), "rows beside the input gradient were written"
    gv = np.where(unfilled[:, None], 0, oracle.to_f32(gz, dtype)).astype(np.float32)
    _, want = oracle.expert_gemm_dgrad(L, gv, w_val, "f32")
    _, mag = oracle.expert_gemm_dgrad(L, np.abs(gv), np.abs(w_val), "f32")
    terms = 2 * nz + 6 if dtype == "f16" else nz + 3
    within(to_host(ga[1:-1].contiguous()), want, terms * 2 * U * mag, dtype, what + ", grad_a")
    assert not oracle.to_f32(to_host(ga[1:-1])[unfilled], dtype).view(np.uint32).any()


CASES = [
    # s, m, n, e, k, capacity, pad, route_major, dtype, act, gated, bias, weighted, residual, gather
    (1, 32, 8, 3, 2, 0, 1, False, "bf16", "silu", True, None, False, None, True),         # smallest rows
    (1, 544, 96, 16, 8, 0, 1, False, "f16", "gelu", False, "f32", True, "tokens", True),  # one token
    (16, 288, 200, 8, 2, 0, 1, False, "bf16", "relu", True, "own", True, "rows", True),
    (17, 1024, 96, 4, 4, 0, 1, False, "bf16", "gelu_tanh", False, None, False, None, False),
    (60, 160, 64, 2, 2, 0, 1, False, "f16", "silu", True, "f32", False, "tokens", True),
    (200, 96, 64, 16, 2, 0, 16, False, "bf16", "none", False, "own", True, None, True),   # padded segments
    (300, 64, 128, 4, 2, 0, 1, False, "bf16", "gelu", True, "own", False, "rows", False),
    (1000, 288, 200, 8, 2, 0, 1, False, "bf16", "silu", True, "f32", True, "tokens", True),  # ragged everywhere
    (1000, 160, 288, 8, 3, 200, 1, True, "f16", "gelu_tanh", False, "own", True, "rows", True),  # drops, route-major
    (2000, 512, 352, 16, 4, 0, 128, False, "f16", "relu", False, "f32", False, None, True),
    (777, 64, 64, 1024, 16, 0, 1, True, "bf16", "silu", True, None, False, None, True),   # most experts empty
    (4000, 96, 160, 4, 2, 600, 1, False, "bf16", "none", True, "own", True, "tokens", False),
    (700, 32, 544, 2, 1, 0, 1, False, "bf16", "gelu", False, None, True, None, True),     # one block long
    (900, 128, 8, 3, 3, 0, 1, False, "f16", "silu", True, "own", False, "rows", True),    # one column chunk
    (20, 160, 96, 1024, 4, 0, 1, False, "bf16", "silu", True, "own", True, "tokens", True),  # few of many experts
    (20, 96, 288, 700, 8, 3, 1, False, "f16", "gelu", False, "f32", True, "rows", False),    # capacity, mostly empty
    (40, 2848, 136, 4, 2, 0, 1, False, "bf16", "silu", True, None, False, None, True),    # long rows, an odd number of blocks
]


@pytest.mark.parametrize("rows", ["16", "4"])
@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-{c[9]}" for c in CASES])
def test_matches_the_oracle(case, rows):
    announce("mx4 product", rows, *case)
    s, m, n, e, k, cap, pad, rm, dtype, name, gated, bias, weighted, residual, gather = case
    idx = W.random_idx(np.random.default_rng(s + m + n), s, e, k)
    run_case(idx, m, n, e, cap, pad, rm, dtype, rows, name, gated, bias, weighted, residual, gather, s + n,
             "f32" if s % 2 else "own")


# rows of one expert: every tile height (32 to 288), the last row and the first of the next
HEIGHTS = [15, 33, 66, 96, 97, 128, 160, 192, 193, 224, 256, 257, 288, 289, 320, 577, 865]


@pytest.mark.parametrize("rows", ["16", "4"])
@pytest.mark.parametrize("height", HEIGHTS)
def test_every_tile_height(height, rows):
    """As wide as makes the large tiles worth while, and narrow."""
    announce("mx4 product height", height, rows)
    for n, dtype in ((160, "bf16"), (32 * -(-449 // (height // 64 + 1)) + 32, "f16")):
        run_case(np.zeros((height, 1), np.int32), 96, n, 1, 0, 1, False, dtype, rows, "silu", True, "own", True, "tokens", True, height)


@pytest.mark.parametrize("rows", ["16", "4"])
@pytest.mark.parametrize("m,dtype", [(96, "bf16"), (544, "f16"), (768, "bf16"), (32, "f16")])
def test_large_tiles_at_every_height(m, dtype, rows):
    """Experts with as many rows as make every tile height, enough of them for the large tiles of either
    row type, gated and not, with a last column tile that is partly there."""
    announce("mx4 large tiles", m, dtype, rows)
    idx = np.repeat(np.arange(len(HEIGHTS) + 1), [1, *HEIGHTS]).astype(np.int32)
    idx = idx[np.random.default_rng(1).permutation(len(idx))][:, None]
    run_case(idx, m, 864, len(HEIGHTS) + 1, 0, 1, False, dtype, rows, "silu", True, "own", True, "tokens", True, 7)
    run_case(idx, m, 1672, len(HEIGHTS) + 1, 0, 1, False, dtype, rows, "gelu", False, "f32", False, None, False, 8)


# rows an expert that ask for each height of the streams
@pytest.mark.parametrize("rows", ["16", "4"])
@pytest.mark.parametrize("m,dtype", [(128, "bf16"), (1408, "f16"), (2688, "bf16")])
@pytest.mark.parametrize("s,n,gated", [(1, 64, True), (11, 136, False), (50, 200, False), (160, 96, True), (200, 160, False)])
def test_streams(s, n, gated, m, dtype, rows):
    announce("mx4 streams", s, n, gated, m, dtype, rows)
    idx = W.random_idx(np.random.default_rng(m + s), s, 8, 3)
    run_case(idx, m, n, 8, 0, 1, False, dtype, rows, "gelu_tanh", gated, "own", True, "rows", True, s)
    run_case(idx, m, n, 8, 4 * s // 8 + 1, 1, True, dtype, rows, "relu", gated, "f32", False, "tokens", False, s)


@pytest.mark.parametrize("rows", ["16", "4"])
@pytest.mark.parametrize("n", [288, 1632])
def test_uneven_segments(rows, n):
    """Segments of 1, 30, 33, 0, 700 and 64 rows beside each other."""
    announce("mx4 product uneven", rows, n)
    idx = np.repeat(np.arange(6), [1, 30, 33, 0, 700, 64]).astype(np.int32)
    idx = idx[np.random.default_rng(1).permutation(len(idx))][:, None]
    for gated in (False, True):
        run_case(idx, 224, n, 6, 0, 1, False, "f16" if gated else "bf16", rows, "gelu_tanh", gated, "own", True, "rows", True, 5)


@pytest.mark.parametrize("rows", ["16", "4"])
@pytest.mark.parametrize("m", [32, 64, 96, 128, 160, 256, 288, 480, 512, 544, 1024, 1056])
def test_every_k_tail(m, rows):
    announce("mx4 product K tail", m, rows)
    for s, n in ((5, 40), (600, 1064)):
        idx = W.random_idx(np.random.default_rng(m), s, 3, 2)
        run_case(idx, m, n, 3, 0, 1, False, "f16" if m % 64 else "bf16", rows, "none", False, None, False, None, True, m)


@pytest.mark.parametrize("rows", ["16", "4"])
@pytest.mark.parametrize("n,m", [(96, 160), (1536, 160), (96, 384), (4160, 160)])
@pytest.mark.parametrize("s,e,k", [(1, 8, 4), (40, 8, 4), (300, 64, 4), (1500, 3, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_whole_numbers_are_exact(s, e, k, n, m, dtype, rows):
    """Products of small whole numbers have exact sums in any order: all forms agree bit for bit. Results
    rounded to 4 bits are then those of the rounded results, whole numbers below 2^8 being bf16 values."""
    announce("mx4 product integers", s, e, k, n, m, dtype, rows)
    rng = np.random.default_rng(s)
    idx = W.random_idx(rng, s, e, k)
    L, Lg = oracle.dispatch_layout(idx, e, 0), M.moe_dispatch_layout(to_dev(idx), e, 0)
    x = rng.integers(-2, 3, (s, m)).astype(np.float32)
    x[:, ::32] = 4  # a scale of 1 in every block
    wts = rng.integers(-2, 3, (e, n, m)).astype(np.float32)
    wts[:, :, 5::32] = -6
    xq, wq = mx4.quantize(x), mx4.quantize(wts)
    assert np.array_equal(mx4.values(*xq), x) and np.array_equal(mx4.values(*wq), wts)
    b = rng.integers(-3, 4, (e, n)).astype(np.float32)
    xd = to_dev(W.cast_input(x, dtype), dtype) if rows == "16" else pair(*xq)
    kw = dict(bias=to_dev(b), act="relu", dtype=TORCH_DTYPE[dtype])
    want, _ = oracle.expert_gemm_act(L, x, wts, "f32", True, b, "relu")
    got = M.moe_mx4_expert_gemm(Lg, xd, pair(*wq), **kw)
    assert_bits_equal(to_host(got), oracle.from_f32(want.astype(np.float32), dtype), "relu")
    codes, scales = M.moe_mx4_expert_gemm(Lg, xd, pair(*wq), quantize_out=True, **kw)
    c, sc = mx4.quantize(want)
    assert np.array_equal(to_host(codes), c) and np.array_equal(to_host(scales), sc)
    if rows == "16":
        buf = M.moe_dispatch(Lg, xd)
    else:  # the buffer's 4-bit rows, gathered on the host
        buf = pair(xq[0][L.src], xq[1][L.src])
    assert_bits_equal(to_host(M.moe_mx4_expert_gemm(Lg, buf, pair(*wq), gather=False, **kw)), to_host(got), "from the buffer")
    g = rng.integers(-2, 3, (L.rows, n)).astype(np.float32)
    _, ga = oracle.expert_gemm_dgrad(L, g, wts, "f32")
    got = M.moe_mx4_expert_dgrad(Lg, to_dev(W.cast_input(g, dtype), dtype), pair(*wq))
    assert_bits_equal(to_host(got), oracle.from_f32(ga.astype(np.float32), dtype), "input gradient")


@pytest.mark.parametrize("m", [1920, 2048, 2176, 2304, 4224])
@pytest.mark.parametrize("s", [1, 9, 40, 130])
def test_long_rows_of_few_tokens(s, m):
    """Rows on both sides of what the streams take for short, with whole and partial last stages; 1, 3, 14
    and 44 routes an expert. Whole numbers: exact in any order."""
    announce("mx4 product long rows", s, m)
    rng = np.random.default_rng(s + m)
    e, k, n = 3, 1, 160
    idx = W.random_idx(rng, s, e, k)
    L, Lg = oracle.dispatch_layout(idx, e, 0), M.moe_dispatch_layout(to_dev(idx), e, 0)
    x = rng.integers(-2, 3, (s, m)).astype(np.float32)
    wts = rng.integers(-2, 3, (e, n, m)).astype(np.float32)
    x[:, ::32], wts[:, :, 5::32] = 4, -6  # a scale of 1 in every block
    xq, wq = mx4.quantize(x), mx4.quantize(wts)
    want, _ = oracle.expert_gemm_act(L, x, wts, "f32", True)
    for dtype in ("bf16", "f16"):
        rounded = oracle.from_f32(want.astype(np.float32), dtype)
        for rows in (to_dev(W.cast_input(x, dtype), dtype), pair(*xq)):
            got = M.moe_mx4_expert_gemm(Lg, rows, pair(*wq), dtype=TORCH_DTYPE[dtype])
            assert_bits_equal(to_host(got), rounded, dtype)


@pytest.mark.parametrize("m", [128, 640, 1152])
@pytest.mark.parametrize("s", [40, 600, 1600])
def test_short_rows_of_many_workgroups(s, m):
    """Few routes an expert (1, 15, 40) and more workgroups than CUs. Products are multiples of 1/4 whose sums
    stay below 2^16: exact in any order."""
    announce("mx4 product short rows", s, m)
    rng = np.random.default_rng(s + m)
    e, k, n = 40, 1, 1024
    idx = W.random_idx(rng, s, e, k)
    L, Lg = oracle.dispatch_layout(idx, e, 0), M.moe_dispatch_layout(to_dev(idx), e, 0)
    xq = rng.integers(0, 256, (s, m // 2)).astype(np.uint8), np.full((s, m // 32), 127, np.uint8)
    wq = rng.integers(0, 256, (e, n, m // 2)).astype(np.uint8), np.full((e, n, m // 32), 127, np.uint8)
    x = mx4.values(*xq).astype(np.float32)
    want, _ = oracle.expert_gemm_act(L, x, mx4.values(*wq).astype(np.float32), "f32", True)
    for dtype in ("bf16", "f16"):
        rounded = oracle.from_f32(want.astype(np.float32), dtype)
        for rows in (to_dev(W.cast_input(x, dtype), dtype), pair(*xq)):
            got = M.moe_mx4_expert_gemm(Lg, rows, pair(*wq), dtype=TORCH_DTYPE[dtype])
            assert_bits_equal(to_host(got), rounded, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scales_of_every_size(dtype):
    """Weights whose blocks lie far apart, f16's range and its subnormals included: rows and gradients are
    powers of two times small whole numbers that bring every product back to the same size, and one block
    of each row carries all of it, so that the results are exact."""
    announce("mx4 product scales", dtype)
    rng = np.random.default_rng(8)
    e, k = 3, 1
    lo, hi = (-24, 15) if dtype == "f16" else (-120, 120)
    draw = (lambda shape: 127 + rng.integers(-30, 25, shape)) if dtype == "f16" else lambda shape: 127 + rng.integers(-120, 121, shape)
    for s, n, m in ((6, 32, 512), (700, 1504, 512), (6, 32, 544), (200, 96, 544), (1400, 7456, 512), (1400, 7456, 160)):  # streams, few rows, tiles
        idx = W.random_idx(rng, s, e, k)
        L, Lg = oracle.dispatch_layout(idx, e, 0), M.moe_dispatch_layout(to_dev(idx), e, 0)
        E_ = draw((e, 1, m // 32)).repeat(n, 1).astype(np.uint8)
        codes = rng.integers(0, 256, (e, n, m // 2)).astype(np.uint8)
        x = np.zeros((s, m), np.float32)
        for t in range(s):  # one block of a row, of the size that its expert's scales ask for
            blk = rng.integers(0, m // 32)
            x[t, 32 * blk:32 * blk + 32] = rng.integers(-3, 4, 32) * 2.0 ** np.clip(127 - int(E_[idx[t, 0], 0, blk]), lo, hi - 2)
        w_val = mx4.values(codes, E_).astype(np.float32)
        want, _ = oracle.expert_gemm_act(L, x, w_val, "f32", True)
        with np.errstate(over="ignore"):
            want = oracle.from_f32(want.astype(np.float32), dtype)
        got = M.moe_mx4_expert_gemm(Lg, to_dev(W.cast_input(x, dtype), dtype), pair(codes, E_))
        assert_bits_equal(to_host(got), want, f"s {s}")
        Eg = draw((e, n, 1)).repeat(m // 32, 2).astype(np.uint8)
        g = np.zeros((L.rows, n), np.float32)
        for r in range(L.rows):
            x_of = int(idx[L.src[r], 0])
            f = rng.integers(0, n)
            g[r, f] = rng.integers(-3, 4) * 2.0 ** np.clip(127 - int(Eg[x_of, f, 0]), lo, hi - 2)
        _, want = oracle.expert_gemm_dgrad(L, g, mx4.values(codes, Eg).astype(np.float32), "f32")
        got = M.moe_mx4_expert_dgrad(Lg, to_dev(W.cast_input(g, dtype), dtype), pair(codes, Eg))
        assert_bits_equal(to_host(got), oracle.from_f32(want.astype(np.float32), dtype), f"input gradient, s {s}")


def test_subnormal_weights_and_rows():
    """Values below bf16's normal range on one side and large ones on the other: their products are
    ordinary, and whole numbers times one power of two."""
    announce("mx4 product subnormals")
    rng = np.random.default_rng(21)
    e, k = 2, 1
    for s, n, m in ((5, 64, 256), (40, 64, 160), (700, 4160, 256)):  # streams, few rows, tiles
        idx = W.random_idx(rng, s, e, k)
        L, Lg = oracle.dispatch_layout(idx, e, 0), M.moe_dispatch_layout(to_dev(idx), e, 0)
        codes = rng.integers(0, 256, (e, n, m // 2)).astype(np.uint8)
        x = rng.integers(-3, 4, (s, m)).astype(np.float32)
        x[:, ::32] = 3
        g = rng.integers(-3, 4, (L.rows, n)).astype(np.float32)
        for E_, power in ((0, 120), (1, 119), (3, 110), (240, -130), (245, -133)):
            scales = np.full((e, n, m // 32), E_, np.uint8)
            scaled = (x * np.float32(2.0) ** power).astype(np.float32)
            wide = mx4.values(codes, scales).astype(np.float64)
            want, _ = oracle.expert_gemm_act(L, x, (wide * 2.0 ** power).astype(np.float32), "f32", True)
            want = oracle.from_f32(want.astype(np.float32), "bf16")
            got = M.moe_mx4_expert_gemm(Lg, to_dev(W.cast_input(scaled, "bf16"), "bf16"), pair(codes, scales))
            assert_bits_equal(to_host(got), want, f"s {s}, scale {E_}")
            if power > -128:  # 4-bit rows of halves: their scale is 2^(power - 1)
                got = M.moe_mx4_expert_gemm(Lg, pair(*mx4.quantize(scaled)), pair(codes, scales))
                assert_bits_equal(to_host(got), want, f"4-bit rows, s {s}, scale {E_}")
            _, want = oracle.expert_gemm_dgrad(L, g, (wide * 2.0 ** power).astype(np.float32), "f32")
            got = M.moe_mx4_expert_dgrad(Lg, to_dev(W.cast_input((g * np.float32(2.0) ** power).astype(np.float32), "bf16"), "bf16"),
                                         pair(codes, scales))
            assert_bits_equal(to_host(got), oracle.from_f32(want.astype(np.float32), "bf16"), f"input gradient, s {s}, scale {E_}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_large_scales_before_a_tail(dtype):
    """Rows whose last K stage is not whole, the largest scales in their first blocks but small codes under
    them, and large codes under small scales: nothing of that may meet past the rows' end. One block alone
    carries each sum, whole numbers times a power of two."""
    announce("mx4 product large scales before a tail", dtype)
    rng = np.random.default_rng(12)
    e, k = 2, 1
    for s, n, m in ((5, 64, 128), (40, 64, 384), (40, 64, 160), (1100, 4160, 384), (1100, 4160, 160)):
        idx = W.random_idx(rng, s, e, k)
        L, Lg = oracle.dispatch_layout(idx, e, 0), M.moe_dispatch_layout(to_dev(idx), e, 0)
        codes = np.full((e, n, m // 2), 0x77, np.uint8)  # sixes
        scales = np.full((e, n, m // 32), 127, np.uint8)
        codes[:, :, 16:64] = 0x11  # blocks 1 to 3: halves
        scales[:, :, 1:4] = 254
        x = np.zeros((s, m), np.float32)
        x[:, m - 32:] = rng.integers(-3, 4, (s, 32)) if m > 128 else 0
        x[:, :32] = rng.integers(-3, 4, (s, 32))
        want, _ = oracle.expert_gemm_act(L, x, mx4.values(codes, scales).astype(np.float32), "f32", True)
        want = oracle.from_f32(want.astype(np.float32), dtype)
        got = M.moe_mx4_expert_gemm(Lg, to_dev(W.cast_input(x, dtype), dtype), pair(codes, scales))
        assert_bits_equal(to_host(got), want, f"s {s}, m {m}")
        got = M.moe_mx4_expert_gemm(Lg, pair(*mx4.quantize(x)), pair(codes, scales), dtype=TORCH_DTYPE[dtype])
        assert_bits_equal(to_host(got), want, f"4-bit rows, s {s}, m {m}")


def test_blocks_that_are_not_numbers_stay_where_they_are():
    """A token's or a weight row's NaN block (scale 255) reaches its own rows and features alone, also
    through the K tail and the rows a tile repeats; infinities of 16-bit rows likewise."""
    announce("mx4 product nan")
    rng = np.random.default_rng(4)
    for m in (96, 288, 384):
        for s, e, k, n in ((12, 8, 2, 160), (700, 3, 2, 160), (1500, 3, 2, 2080)):
            idx = W.random_idx(rng, s, e, k)
            idx[0], idx[1] = [0, 1], [1, 2]
            L, Lg = oracle.dispatch_layout(idx, e, 0), M.moe_dispatch_layout(to_dev(idx), e, 0)
            xc, xs, _ = four_bits(rng, (s, m))
            wc, ws, _ = four_bits(rng, (e, 2 * n, m))
            xs[0, -1], xs[1, 0] = 255, 255
            ws[2, 5, 1], ws[0, n + 7, -1], ws[1, 2 * n - 1, 0] = 255, 255, 255
            x_val, w_val = mx4.values(xc, xs), mx4.values(wc, ws)
            bad = np.zeros((L.rows, 2 * n), bool)
            for x, r in E.segments(L):
                bad[r] = np.isnan(x_val[L.src[r]]).any(1)[:, None] | np.isnan(w_val[x]).any(1)[None]
            want = bad[:, :n] | bad[:, n:]
            out = to_host(M.moe_mx4_expert_gemm(Lg, pair(xc, xs), pair(wc, ws), act="gelu", gated=True))
            assert np.array_equal(np.isnan(oracle.to_f32(out, "bf16")), want)
            codes, scales = M.moe_mx4_expert_gemm(Lg, pair(xc, xs), pair(wc, ws), act="gelu", gated=True, quantize_out=True)
            assert np.array_equal(to_host(scales) == 255, want.reshape(L.rows, -1, 32).any(2))
            for dtype in ("bf16", "f16"):
                x16 = rand(rng, (s, m), dtype)
                big = oracle.to_f32(x16, dtype)
                big[0, m - 1], big[1, 0] = np.nan, np.inf
                x16 = W.cast_input(big, dtype)
                rows_bad = np.isin(L.src, [0, 1])
                want16 = rows_bad[:, None] | np.concatenate([np.isnan(w_val).any(2)[x][None].repeat(len(r), 0) for x, r in E.segments(L)])
                got = oracle.to_f32(to_host(M.moe_mx4_expert_gemm(Lg, to_dev(x16, dtype), pair(wc, ws))), dtype)
                with np.errstate(all="ignore"):
                    exact, _ = oracle.expert_gemm_act(L, oracle.to_f32(x16, dtype), w_val.astype(np.float32), "f32", True)
                assert np.array_equal(~np.isfinite(got), want16)
                assert np.array_equal(np.isnan(got), np.isnan(exact)) and np.array_equal(got[np.isinf(got)], exact[np.isinf(got)])


def test_routes_that_name_no_expert_and_no_tokens():
    announce("mx4 product bad routes")
    rng = np.random.default_rng(2)
    idx = W.random_idx(rng, 500, 6, 3)
    idx[::5, 1], idx[7], idx[9, 2] = -1, 6, idx[9, 0]
    for rows in ("16", "4"):
        run_case(idx, 96, 160, 6, 0, 1, False, "bf16", rows, "silu", True, "own", True, "tokens", True, 3)
        run_case(np.full((90, 2), -1, np.int32), 96, 160, 6, 0, 1, False, "bf16", rows, "silu", True, "own", True, "rows", False, 3)
    L = M.moe_dispatch_layout(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 4, 3)  # 12 rows, none filled
    wc, ws, _ = four_bits(rng, (4, 64, 96))
    out = torch.full((12, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    M.moe_mx4_expert_gemm(L, torch.empty((0, 96), dtype=torch.bfloat16, device="cuda"), pair(wc, ws), out=out)
    assert not out.any()
    codes, scales = M.moe_mx4_expert_gemm(L, torch.empty((0, 96), dtype=torch.bfloat16, device="cuda"), pair(wc, ws), quantize_out=True)
    assert not codes.any() and not scales.any()
    L = M.moe_dispatch_layout(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 4, 0)
    assert M.moe_mx4_expert_gemm(L, torch.empty((0, 96), dtype=torch.bfloat16, device="cuda"), pair(wc, ws)).shape == (0, 64)
    assert M.moe_mx4_expert_dgrad(L, torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), pair(wc, ws)).shape == (0, 96)


def test_unaligned_scales():
    """Scale bytes at any address, of rows, weights and results. The products are multiples of 2^-4 whose
    sums stay below 2^20 and so are exact in any order: all forms agree bit for bit."""
    announce("mx4 unaligned scales")
    rng = np.random.default_rng(9)

    def halves(shape):
        return (rng.integers(0, 256, (*shape[:-1], shape[-1] // 2)).astype(np.uint8),
                rng.integers(126, 129, (*shape[:-1], shape[-1] // 32)).astype(np.uint8))

    for s, n, m in ((9, 64, 544), (9, 64, 512), (600, 1536, 512), (1500, 4160, 544)):
        e, k = 3, 2
        idx = W.random_idx(rng, s, e, k)
        Lg = M.moe_dispatch_layout(to_dev(idx), e, 0)
        xc, xs = halves((s, m))
        wc, ws = halves((e, n, m))
        want = M.moe_mx4_expert_gemm(Lg, pair(xc, xs), pair(wc, ws), quantize_out=True)
        grad = to_dev(rand(rng, (Lg.rows, n), "bf16"), "bf16")
        want_g = M.moe_mx4_expert_dgrad(Lg, grad, pair(wc, ws))

        def moved(t, by):
            flat = torch.zeros(t.numel() + 8, dtype=torch.uint8, device="cuda")
            view = flat[by:by + t.numel()].view(t.shape)
            view.copy_(t)
            return view

        for by in (1, 2, 3):
            out = (torch.empty_like(want[0]), moved(torch.zeros_like(want[1]), by))
            w_pair = (to_dev(wc), moved(to_dev(ws), 4 - by))
            got = M.moe_mx4_expert_gemm(Lg, (to_dev(xc), moved(to_dev(xs), by)), w_pair, quantize_out=True, out=out)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert torch.equal(M.moe_mx4_expert_dgrad(Lg, grad, w_pair), want_g)


def test_weights_past_four_gib():
    """The last of many experts, its codes past 4 GiB."""
    announce("mx4 weights past 4 GiB")
    e, n, m = 130, 8192, 8192  # 4.06 GiB of codes
    codes = torch.zeros((e, n, m // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((e, n, m // 32), 127, dtype=torch.uint8, device="cuda")
    codes[-1, :, :] = 0x22  # ones
    codes[-1, -1, 0] = 0x27
    for s in (1, 400):
        idx = torch.full((s, 1), e - 1, dtype=torch.int32, device="cuda")
        L = M.moe_dispatch_layout(idx, e, 0)
        x = torch.zeros((s, m), dtype=torch.bfloat16, device="cuda")
        x[:, 0], x[:, -1] = 2, 1
        for rows in (x, M.moe_mx4_quantize(x)):
            out = M.moe_mx4_expert_gemm(L, rows, (codes, scales))
            assert (out[:, :-1] == 3).all() and (out[:, -1] == 13).all()
        g = torch.zeros((s, n), dtype=torch.bfloat16, device="cuda")
        g[:, -1] = 1
        ga = M.moe_mx4_expert_dgrad(L, g, (codes, scales))
        assert (ga[:, 0] == 6).all() and (ga[:, 1:] == 1).all()


# ---------------------------------------------------------------------------------
# layers, gradients, streams and graphs


def layer_inputs(rng, s, m, n, e, k, dtype, bias=True):
    t = {"x": to_dev(rand(rng, (s, m), dtype), dtype), "logits": to_dev(rng.standard_normal((s, e)).astype(np.float32)),
         "grad": to_dev(rand(rng, (s, m), dtype), dtype)}
    for name, f, d in (("up", 2 * n, m), ("down", m, n)):
        c, sc, v = four_bits(rng, (e, f, d))
        t[name], t[name + "_values"] = pair(c, sc), to_dev(v)
        t[name + "_bias"] = to_dev(rand(rng, (e, f), dtype, 0.3), dtype) if bias else None
    return t


def test_a_layer_in_four_bits():
    """Rows quantised, gated projection with 4-bit hidden rows, down projection, combine: each step against
    the values that the step before it handed on."""
    announce("mx4 layer")
    rng = np.random.default_rng(12)
    for s, m, n, e, k, dtype in ((1, 96, 64, 8, 4, "bf16"), (37, 352, 96, 8, 2, "f16"), (900, 256, 1056, 4, 2, "bf16")):
        t = layer_inputs(rng, s, m, n, e, k, dtype)
        idx, w = M.moe_gate_topk(t["logits"], k)
        L = M.moe_dispatch_layout(idx, e, 0)
        Lo = oracle.dispatch_layout(to_host(idx), e, 0)
        xq = M.moe_mx4_quantize(t["x"])
        h = M.moe_mx4_expert_gemm(L, xq, t["up"], bias=t["up_bias"], act="silu", gated=True, dtype=t["x"].dtype, quantize_out=True)
        o = M.moe_mx4_expert_gemm(L, h, t["down"], gather=False, bias=t["down_bias"], dtype=t["x"].dtype)
        y = M.moe_combine(L, o, w)
        xv = mx4.values(*map(to_host, xq)).astype(np.float32)
        want, _, tol, _ = product_bounds(Lo, xv, to_host(t["up_values"]), m, False, dtype, True, real(to_host(t["up_bias"]), dtype),
                                         "silu", True, None, None, False)
        check_quantized(to_host(h[0]), to_host(h[1]), want, tol, "hidden rows")
        hv = mx4.values(*map(to_host, h)).astype(np.float32)
        want, _, tol, _ = product_bounds(Lo, hv, to_host(t["down_values"]), n, False, dtype, False, real(to_host(t["down_bias"]), dtype),
                                         "none", False, None, None, False)
        within(to_host(o), want, tol, dtype, "down projection")
        assert_bits_equal(to_host(y), oracle.combine(Lo, to_host(o), to_host(w), dtype), "combine")


def plain_step(t, L, k, dtype, quantize, act):
    """The step's outputs and gradients in float64 with torch on the CPU, the rounding of rows passed
    through; h and o rounded to the element type as the operators' outputs are."""
    cpu = lambda v: None if v is None else v.detach().double().cpu()  # noqa: E731
    tdt = TORCH_DTYPE[dtype]

    class Rounded(torch.autograd.Function):
        @staticmethod
        def forward(ctx, v):
            return torch.from_numpy(mx4.values(*mx4.quantize(v.numpy())))

        @staticmethod
        def backward(ctx, g):
            return g

    class Stored(torch.autograd.Function):
        @staticmethod
        def forward(ctx, v):
            return v.to(tdt).double()

        @staticmethod
        def backward(ctx, g):
            return g

    leaves = {v: cpu(t[v]).requires_grad_() for v in ("x", "up_bias", "down_bias", "w")}
    src = torch.from_numpy(L.src.astype(np.int64))
    expert = torch.zeros(L.rows, dtype=torch.long)
    for x, r in E.segments(L):
        expert[torch.from_numpy(r)] = x
    xr = Rounded.apply(leaves["x"]) if quantize else leaves["x"]
    z = torch.bmm(cpu(t["up_values"])[expert], xr[src][:, :, None])[:, :, 0] + leaves["up_bias"][expert]
    n = z.shape[1] // 2
    f = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[act]
    h = Stored.apply(f(z[:, :n]) * z[:, n:])
    hr = Rounded.apply(h) if quantize else h
    o = Stored.apply(torch.bmm(cpu(t["down_values"])[expert], hr[:, :, None])[:, :, 0] + leaves["down_bias"][expert])
    y = (o[torch.from_numpy(L.dst.astype(np.int64))] * leaves["w"][:, :, None]).sum(1)
    grads = torch.autograd.grad(y, list(leaves.values()), cpu(t["grad"]))
    return y.detach(), dict(zip(leaves, grads))


def own_step(t, L, quantize, act, leaves):
    h = A.expert_linear_mx4(leaves["x"], t["up"], L, bias=leaves["up_bias"], act=act, gated=True, quantize_rows=quantize,
                            preact_dtype=torch.float32)
    o = A.expert_linear_mx4(h, t["down"], L, bias=leaves["down_bias"], gather=False, quantize_rows=quantize)
    y = A.combine(o, leaves["w"], L)
    return y, torch.autograd.grad(y, list(leaves.values()), t["grad"])


@pytest.mark.parametrize("quantize", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_tuning_step_against_float64(dtype, quantize):
    """Gradients of rows, biases and route weights around frozen 4-bit experts, in the 2-norm. Between the
    operators values are rounded to the element type (h, o, dz, each row's gradient): at most half a step,
    eps / 2, each relative to its own value, four in a chain; a hidden value next to a border between two
    codes may round to the other one, a share of at most 2^-9 of the values by up to a third of themselves:
    sqrt(2^-9) / 3 in the 2-norm at most."""
    announce("mx4 tuning step", dtype, quantize)
    rng = np.random.default_rng(21)
    for s, m, n, e, k, act in ((3, 32, 32, 2, 2, "gelu"), (60, 96, 64, 4, 2, "silu"), (300, 64, 160, 3, 1, "gelu")):
        t = layer_inputs(rng, s, m, n, e, k, dtype)
        idx, w = M.moe_gate_topk(t["logits"], k)
        t["w"] = w
        L, Lo = M.moe_dispatch_layout(idx, e, 0), oracle.dispatch_layout(to_host(idx), e, 0)
        leaves = {v: t[v].clone().requires_grad_() for v in ("x", "up_bias", "down_bias", "w")}
        y, grads = own_step(t, L, quantize, act, leaves)
        want_y, want = plain_step(t, Lo, k, dtype, quantize, act)
        tol = 8 * torch.finfo(TORCH_DTYPE[dtype]).eps / 2 + (2 ** -4.5 / 3 if quantize else 0)
        for name, got, ref in [("y", y, want_y)] + [(v, g, want[v]) for v, g in zip(leaves, grads)]:
            assert got.dtype == (torch.float32 if name == "w" else TORCH_DTYPE[dtype])
            off = (got.detach().double().cpu() - ref).norm() / ref.norm()
            assert off <= tol, (name, float(off), tol)


def test_gradient_of_whole_numbers_against_differences():
    """Without an activation the projection is linear in its rows: with whole numbers the difference of
    two forwards is the gradient, exactly; also through the rounding of rows where they are 4-bit values."""
    announce("mx4 gradient differences")
    rng = np.random.default_rng(5)
    s, m, n, e, k = 40, 64, 32, 4, 2
    idx = W.random_idx(rng, s, e, k)
    L = M.moe_dispatch_layout(to_dev(idx), e, 0)
    x = rng.integers(-2, 3, (s, m)).astype(np.float32)
    x[:, ::32] = 4
    d = np.zeros_like(x)
    d[:, 1::32] = rng.integers(-1, 2, (s, 2))
    x[:, 1::32] = 0
    wts = rng.integers(-2, 3, (e, n, m)).astype(np.float32)
    wts[:, :, 5::32] = -6
    wq = pair(*mx4.quantize(wts))
    g = torch.from_numpy(rng.integers(-2, 3, (L.rows, n)).astype(np.float32)).cuda()
    for quantize in (False, True):
        for dtype in (torch.bfloat16, torch.float16):
            xt, dt = (torch.from_numpy(v).cuda().to(dtype) for v in (x, d))
            xt.requires_grad_()
            f = lambda v: A.expert_linear_mx4(v, wq, L, quantize_rows=quantize)  # noqa: E731
            (gx,) = torch.autograd.grad(f(xt), xt, g.to(dtype))
            with torch.no_grad():
                diff = ((f(xt + dt) - f(xt)).double() * g.double()).sum()
            assert float((gx.double() * dt.double()).sum()) == float(diff)


def test_expert_linear_mx4_keeps_only_what_a_backward_needs():
    announce("mx4 kept values")
    rng = np.random.default_rng(6)
    t = layer_inputs(rng, 20, 64, 32, 4, 2, "bf16")
    idx, w = M.moe_gate_topk(t["logits"], 2)
    L = M.moe_dispatch_layout(idx, 4, 0)
    x = t["x"].clone().requires_grad_()
    with torch.no_grad():
        y0 = A.expert_linear_mx4(x, t["up"], L, act="silu", gated=True)
    y1 = A.expert_linear_mx4(x, t["up"], L, act="silu", gated=True)
    assert torch.equal(y0, y1) and y1.requires_grad and not y0.requires_grad
    torch.cuda.synchronize()
    res = torch.randn(20, 32, device="cuda").bfloat16().requires_grad_()
    bias = torch.randn(4, 64, device="cuda").requires_grad_()
    wt = w.clone().requires_grad_()
    y = A.expert_linear_mx4(x, t["up"], L, bias=bias, act="gelu", gated=True, w=wt, residual=res, residual_gather=True)
    ref = A.expert_linear(x, t["up_values"].bfloat16(), L, bias=bias, act="gelu", gated=True, w=wt, residual=res, residual_gather=True)
    gy = torch.randn_like(y)
    got, want = (torch.autograd.grad(o, (x, bias, wt, res), gy) for o in (y, ref))
    # the weights are bf16 values too: the same formulas on the same numbers, sums in another order
    for a, b in zip((y, *got), (ref, *want)):
        assert (a.double() - b.double()).norm() <= 2 ** -8 * b.double().norm()


def test_captured_and_replayed_with_new_inputs():
    """A layer and a tuning step captured in a HIP graph: replays on new inputs, eager work between them,
    equal the eager results bit for bit."""
    announce("mx4 graph")
    rng = np.random.default_rng(31)
    for s, m, n, e, k in ((3, 96, 64, 8, 2), (500, 128, 1056, 4, 2), (3000, 256, 2048, 4, 2)):
        t = layer_inputs(rng, s, m, n, e, k, "bf16")
        idx, w = M.moe_gate_topk(t["logits"], k)
        t["w"] = w
        L = M.moe_dispatch_layout(idx, e, 0)
        names = ("x", "up_bias", "down_bias", "w")

        def forward(x):
            h = M.moe_mx4_expert_gemm(L, M.moe_mx4_quantize(x), t["up"], bias=t["up_bias"], act="silu", gated=True, quantize_out=True)
            return M.moe_combine(L, M.moe_mx4_expert_gemm(L, h, t["down"], gather=False, bias=t["down_bias"]), w)

        def step(v):
            return own_step(t, L, True, "silu", v)

        static = {v: t[v].clone() for v in names}
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            forward(static["x"])
            step({v: static[v].detach().requires_grad_() for v in names})
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = forward(static["x"])
            ys, grads = step({v: static[v].detach().requires_grad_() for v in names})
        for i in range(4):
            fresh = {v: (t[v] * (1 + i) + 0.125 * i).to(t[v].dtype) for v in names}
            fresh["w"] = t["w"]
            for v in names:
                static[v].copy_(fresh[v])
            graph.replay()
            torch.cuda.synchronize()
            want = forward(fresh["x"])
            want_ys, want_grads = step({v: fresh[v].clone().requires_grad_() for v in names})
            torch.cuda.synchronize()
            assert torch.equal(y, want), i
            assert torch.equal(ys, want_ys) and all(torch.equal(a, b) for a, b in zip(grads, want_grads)), i


def test_two_streams_at_once():
    announce("mx4 streams")
    rng = np.random.default_rng(41)
    ts = [layer_inputs(rng, 400, 128, 1056, 4, 2, "bf16") for _ in range(2)]
    made = []
    for t in ts:
        idx, w = M.moe_gate_topk(t["logits"], 2)
        made.append((M.moe_dispatch_layout(idx, 4, 0), w))

    def forward(t, L, w):
        h = M.moe_mx4_expert_gemm(L, M.moe_mx4_quantize(t["x"]), t["up"], bias=t["up_bias"], act="silu", gated=True, quantize_out=True)
        return M.moe_combine(L, M.moe_mx4_expert_gemm(L, h, t["down"], gather=False), w)

    want = [forward(t, *p) for t, p in zip(ts, made)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    got = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(forward(ts[i], *made[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])
