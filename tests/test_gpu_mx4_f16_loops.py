"""f16 rows and gradients on 4-bit weights, in both loops of the tiles and in the other forms: weights that f16
holds are multiplied as f16, others in two bf16 parts of each row value. The scale bytes say on the host
which of the two a case is for: every block fits (or is all zeros), or each 32 weight rows of each block column,
and so any tile, hold one that does not.

Tolerances as at the top of test_gpu_mx4.py: m + 3 roundings of the float32 sum where products are whole, 2 m + 6
where split. Values are compared in float32 as well, which shows what a rounding to f16 would hide."""
import numpy as np
import pytest
import torch

import combine_moe_gate_amd as M
import oracle
import workloads as W
from oracle import mx4
from tests.gpu_util import to_dev, to_host
from tests.test_gpu_expert_act import U, announce, rand, real, within
from tests.test_gpu_mx4 import HEIGHTS, check_quantized, four_bits, pair, product_bounds

pytestmark = pytest.mark.gpu


def weights(rng, shape, loop):
    c, s, _ = four_bits(rng, shape)
    if loop == "split":
        s[:, ::2] -= 25  # 2^-25 of what they were: below f16's smallest value
        assert (s[:, ::2] < 104).all()
    if loop == "zeros":
        c[:, ::3, :16], s[:, ::3, 0] = 0, 0
    fits = (s >= 104) & (s <= 140) | (c.reshape(*s.shape, 16) & 0x77 == 0).all(-1)
    assert fits.all() if loop != "split" else not fits[:, ::2].any()
    return c, s, mx4.values(c, s).astype(np.float32)


def run(idx, m, n, e, loop, name, gated, bias, weighted, residual, gather, seed, pad=1):
    rng = np.random.default_rng(seed)
    s, k = idx.shape
    L, Lg = oracle.dispatch_layout(idx, e, 0, pad_multiple=pad), M.moe_dispatch_layout(to_dev(idx), e, 0, pad_multiple=pad)
    nz = 2 * n if gated else n
    c, sc, w_val = weights(rng, (e, nz, m), loop)
    a = rand(rng, (s if gather else L.rows, m), "f16")
    b = None if bias is None else rng.standard_normal((e, nz)).astype(np.float32) if bias == "f32" else rand(rng, (e, nz), "f16")
    w = W.random_weights(rng, s, k) if weighted else None
    res = None if residual is None else rand(rng, (s if residual == "tokens" else L.rows, n), "f16")
    dev = lambda t: None if t is None else to_dev(t)  # noqa: E731
    kw = dict(gather=gather, bias=dev(b), act=name, gated=gated, w=dev(w), residual=dev(res), residual_gather=residual == "tokens")
    out, pre = M.moe_mx4_expert_gemm(Lg, to_dev(a), pair(c, sc), save_preact=True, preact_dtype=torch.float32, **kw)
    want, z, tol, dz = product_bounds(L, oracle.to_f32(a, "f16"), w_val, m, loop == "split", "f16", gather,
                                      None if b is None else real(b, "f16"), name, gated, w, None if res is None else oracle.to_f32(res, "f16"),
                                      residual == "tokens")
    what = f"{loop} s{s} m{m} n{n} e{e}"
    within(to_host(pre), z, dz, "f32", what + ", kept values")
    within(to_host(out), want, tol, "f16", what)
    unfilled = L.src < 0
    assert not to_host(out)[unfilled].any() and not to_host(pre)[unfilled].any()
    if n % 32 == 0:
        codes, scales = M.moe_mx4_expert_gemm(Lg, to_dev(a), pair(c, sc), quantize_out=True, **kw)
        check_quantized(to_host(codes), to_host(scales), want, tol, what + ", 4-bit results")
    g = rand(rng, (L.rows, nz), "f16")
    gv = np.where(unfilled[:, None], 0, oracle.to_f32(g, "f16")).astype(np.float32)
    _, want = oracle.expert_gemm_dgrad(L, gv, w_val, "f32")
    _, mag = oracle.expert_gemm_dgrad(L, np.abs(gv), np.abs(w_val), "f32")
    ga = M.moe_mx4_expert_dgrad(Lg, to_dev(g), pair(c, sc), out_dtype=torch.float32)
    within(to_host(ga), want, (2 * nz + 6 if loop == "split" else nz + 3) * 2 * U * mag, "f32", what + ", grad_a")


LOOPS = ["whole", "zeros", "split"]


@pytest.mark.parametrize("loop", LOOPS)
@pytest.mark.parametrize("m", [32, 96, 544, 768])
def test_large_tiles_at_every_height(m, loop):
    announce("f16 loops, heights", m, loop)
    e = len(HEIGHTS) + 1
    idx = np.repeat(np.arange(e), [1, *HEIGHTS]).astype(np.int32)
    idx = idx[np.random.default_rng(1).permutation(len(idx))][:, None]
    run(idx, m, 864, e, loop, "silu", True, "own", True, "tokens", True, 7)
    run(idx, m, 1672, e, loop, "gelu", False, "f32", False, None, False, 8)


@pytest.mark.parametrize("loop", LOOPS)
@pytest.mark.parametrize("m", [32, 64, 96, 128, 160, 256, 288, 480, 512, 1024, 1056])
def test_every_k_tail(m, loop):
    announce("f16 loops, K tail", m, loop)
    for s, e, n in ((5, 3, 40), (60, 3, 96), (600, 3, 4136)):  # few rows (streams where m allows), more, tiles
        idx = W.random_idx(np.random.default_rng(m), s, e, 2)
        run(idx, m, n, e, loop, "none", False, None, False, None, True, m)


@pytest.mark.parametrize("loop", LOOPS)
@pytest.mark.parametrize("s,m,n,e,k,name,gated,bias,weighted,residual,gather,pad", [
    (1, 544, 96, 16, 8, "gelu", False, "f32", True, "tokens", True, 1),      # one token
    (60, 160, 64, 2, 2, "silu", True, "f32", False, "tokens", True, 1),
    (200, 384, 200, 8, 3, "gelu_tanh", True, "own", True, "rows", True, 16),  # streams, padded segments
    (300, 64, 128, 4, 2, "gelu", True, "own", False, "rows", False, 1),
    (2000, 512, 2080, 4, 2, "relu", False, "f32", False, None, True, 128),   # tiles, padded segments
    (3000, 640, 1064, 6, 2, "silu", True, "own", True, "tokens", True, 1),   # tiles, a column tile partly there
])
def test_forms_and_epilogues(s, m, n, e, k, name, gated, bias, weighted, residual, gather, pad, loop):
    announce("f16 loops, forms", s, m, n, e, k, name, gated, loop)
    run(W.random_idx(np.random.default_rng(s + m), s, e, k), m, n, e, loop, name, gated, bias, weighted, residual, gather, s, pad)
