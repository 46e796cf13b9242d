"""f16 rows and gradients meet weights with blocks of zeros: the quantiser gives those scale 0, far below what
f16 holds, but zeros are f16 values under any scale. They must be multiplied as f16 like the rest: the results
are, bit for bit, those of the same values with a scale of 1 (sums in two parts would be ordered otherwise), so
that padded features, pruned rows and unused experts cost nothing."""
import numpy as np
import pytest
import torch

import combine_moe_gate_amd as M
import oracle
import workloads as W
from oracle import epilogue as E
from oracle import mx4
from tests.gpu_util import to_dev, to_host
from tests.test_gpu_expert_act import U, announce, rand, within
from tests.test_gpu_mx4 import pair

pytestmark = pytest.mark.gpu

FORMS = [  # s, e, k, m, n: streams of 16 and 32 rows, rows of any length, tiles
    (5, 8, 2, 384, 160), (90, 8, 2, 256, 160), (40, 8, 2, 160, 96), (1500, 3, 2, 160, 2112), (2500, 3, 1, 640, 2112),
]


def weights(rng, shape):
    """4-bit weights that f16 holds, with zeros in a fifth of the blocks: (codes, scales, where the zeros are)."""
    c, s = mx4.quantize(rng.standard_normal(shape) * shape[-1] ** -0.5)
    zero = rng.random(s.shape) < 0.2
    zero[0, :8] = True  # whole rows
    signs = rng.choice(np.array([0x00, 0x08, 0x80, 0x88], np.uint8), c.shape)  # zeros of both signs
    c = np.where(zero.repeat(16, -1), signs, c)
    return c, s, zero


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("s,e,k,m,n", FORMS)
def test_scales_of_zeros_do_not_matter(s, e, k, m, n, gated):
    announce("4-bit zero blocks", s, e, k, m, n, gated)
    rng = np.random.default_rng(s + m)
    idx = W.random_idx(rng, s, e, k)
    L, Lg = oracle.dispatch_layout(idx, e, 0), M.moe_dispatch_layout(to_dev(idx), e, 0)
    nz = 2 * n if gated else n
    codes, scales, zero = weights(rng, (e, nz, m))
    x = rand(rng, (s, m), "f16")
    g = rand(rng, (L.rows, nz), "f16")
    w_val = mx4.values(codes, np.where(zero, 127, scales).astype(np.uint8)).astype(np.float32)
    results = []
    for byte in (127, 0, 1, 103, 141, 254):
        w = pair(codes, np.where(zero, byte, scales).astype(np.uint8))
        out, pre = M.moe_mx4_expert_gemm(Lg, to_dev(x, "f16"), w, act="silu", gated=gated, save_preact=True, preact_dtype=torch.float32)
        ga = M.moe_mx4_expert_dgrad(Lg, to_dev(g, "f16"), w, out_dtype=torch.float32)
        results.append((out, pre, ga))
    for byte, got in zip((0, 1, 103, 141, 254), results[1:]):
        for name, a, b in zip(("out", "preact", "grad_a"), got, results[0]):
            assert torch.equal(a, b), f"{name} with scale {byte} under zeros"
    # and they are right: an f16 value times a 4-bit one is exact, sums of m (nz) of them in float32
    _, z = oracle.expert_gemm_act(L, oracle.to_f32(x, "f16"), w_val, "f32", True)
    _, mag = oracle.expert_gemm_act(L, np.abs(oracle.to_f32(x, "f16")), np.abs(w_val), "f32", True)
    within(to_host(results[0][1]), z, (m + 3) * 2 * U * mag, "f32", "kept values")
    _, want = oracle.expert_gemm_dgrad(L, oracle.to_f32(g, "f16"), w_val, "f32")
    _, mag = oracle.expert_gemm_dgrad(L, np.abs(oracle.to_f32(g, "f16")), np.abs(w_val), "f32")
    within(to_host(results[0][2]), want, (nz + 3) * 2 * U * mag, "f32", "input gradient")


@pytest.mark.parametrize("s,e,k,m,n", FORMS)
def test_zeros_under_scale_255_are_not_numbers(s, e, k, m, n):
    announce("4-bit zero blocks, not numbers", s, e, k, m, n)
    rng = np.random.default_rng(s)
    idx = W.random_idx(rng, s, e, k)
    L, Lg = oracle.dispatch_layout(idx, e, 0), M.moe_dispatch_layout(to_dev(idx), e, 0)
    codes, scales, zero = weights(rng, (e, n, m))
    zero[0, 9, 2] = zero[2, n - 1, -1] = True
    codes = np.where(zero.repeat(16, -1), 0, codes).astype(np.uint8)
    scales[0, 9, 2] = scales[2, n - 1, -1] = 255
    w = pair(codes, scales)
    out = to_host(M.moe_mx4_expert_gemm(Lg, to_dev(rand(rng, (s, m), "f16"), "f16"), w))
    ga = to_host(M.moe_mx4_expert_dgrad(Lg, to_dev(rand(rng, (L.rows, n), "f16"), "f16"), w))
    bad = np.isnan(mx4.values(codes, scales))
    want_out, want_ga = np.zeros((L.rows, n), bool), np.zeros((L.rows, m), bool)
    for x, r in E.segments(L):
        want_out[r], want_ga[r] = bad[x].any(1), bad[x].any(0)
    assert np.array_equal(np.isnan(out), want_out) and np.array_equal(np.isnan(ga), want_ga)
