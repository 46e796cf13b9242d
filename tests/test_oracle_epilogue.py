"""Pins of the epilogue oracle: activations at closed values, slopes and the whole backward
against central differences."""
import numpy as np
import pytest

import oracle
import workloads as W
from oracle import epilogue as E


def test_activations_at_closed_values():
    z = np.array([0.0, 1.0, -1.0, 40.0, -40.0])
    assert E.act("relu", z)[0].tolist() == [0, 1, 0, 40, 0] and E.act("relu", z)[1].tolist() == [0, 1, 0, 1, 0]
    phi1 = 0.8413447460685429  # normal distribution function at 1
    np.testing.assert_allclose(E.act("gelu", z)[0], [0, phi1, phi1 - 1, 40, 0], atol=1e-14)
    sg = 1 / (1 + np.exp(-1.0))
    np.testing.assert_allclose(E.act("silu", z)[0], [0, sg, sg - 1, 40, 0], atol=1e-15)
    t = np.tanh(np.sqrt(2 / np.pi) * 1.044715)
    np.testing.assert_allclose(E.act("gelu_tanh", z)[0], [0, 0.5 * (1 + t), -0.5 * (1 - t), 40, 0], atol=1e-15)


@pytest.mark.parametrize("name", E.ACTS)
def test_slopes_against_differences(name):
    z, h = np.linspace(-6, 6, 241) + 0.0123, 1e-5
    want = (E.act(name, z + h)[0] - E.act(name, z - h)[0]) / (2 * h)
    np.testing.assert_allclose(E.act(name, z)[1], want, atol=1e-9)


@pytest.mark.parametrize("name,gated", [("silu", True), ("gelu", False), ("none", True), ("relu", True)])
def test_backward_against_differences(name, gated):
    rng = np.random.default_rng(3)
    s, m, n, e, k = 5, 8, 3, 4, 2
    idx = W.random_idx(rng, s, e, k)
    L = oracle.dispatch_layout(idx, e, 2)  # capacity 2: some routes dropped, some rows unfilled
    nz = 2 * n if gated else n
    a, wts = rng.standard_normal((s, m)).astype(np.float32), rng.standard_normal((e, nz, m)).astype(np.float32)
    bias, w, g = rng.standard_normal((e, nz)), rng.uniform(0.2, 1, (s, k)), rng.standard_normal((L.rows, n))

    def total(bias, w, shift):
        out, z = oracle.expert_gemm_act(L, a, wts, "f32", True, bias, name, gated)
        z = z + shift
        u = E.finish(z, name, gated) * (L.src >= 0)[:, None]
        return float((g * E.row_weights(L, w)[:, None] * u).sum())

    _, z = oracle.expert_gemm_act(L, a, wts, "f32", True, bias, name, gated)
    gz, gb, gw, gr = oracle.expert_act_backward(L, g, z, name, gated, w)
    assert not gz[L.src < 0].any() and np.array_equal(gr[L.src >= 0], g[L.src >= 0]) and not gr[L.src < 0].any()
    h, zero = 1e-6, np.zeros(z.shape)

    def slope(at):
        return (total(*at(h)) - total(*at(-h))) / (2 * h)

    for i in np.ndindex(gb.shape):
        assert abs(slope(lambda d: (bias + d * (np.arange(gb.size).reshape(gb.shape) == np.ravel_multi_index(i, gb.shape)), w, zero)) - gb[i]) < 1e-7
    for i in np.ndindex(gw.shape):
        assert abs(slope(lambda d: (bias, w + d * (np.arange(gw.size).reshape(gw.shape) == np.ravel_multi_index(i, gw.shape)), zero)) - gw[i]) < 1e-7
    for i in np.ndindex(gz.shape):
        d1 = zero.copy()
        d1[i] = 1
        assert abs(slope(lambda d: (bias, w, d * d1)) - gz[i]) < 1e-7


def test_forward_equals_the_plain_product():
    rng = np.random.default_rng(4)
    idx = W.random_idx(rng, 30, 6, 2)
    L = oracle.dispatch_layout(idx, 6, 0, pad_multiple=4)
    x = W.cast_input(rng.standard_normal((30, 16)).astype(np.float32), "bf16")
    wts = W.expert_weights(1, 6, 8, 16, "bf16")
    out, z = oracle.expert_gemm_act(L, x, wts, "bf16", True)
    np.testing.assert_allclose(out, oracle.expert_gemm(L, x, wts, "bf16", True)[1], rtol=1e-14)
    assert np.array_equal(out, z)
    res = W.cast_input(rng.standard_normal((30, 8)).astype(np.float32), "bf16")
    more, _ = oracle.expert_gemm_act(L, x, wts, "bf16", True, residual=res, residual_gather=True)
    placed = L.src >= 0
    np.testing.assert_allclose(more[placed], out[placed] + oracle.to_f32(res, "bf16")[L.src[placed]], rtol=1e-14)
    assert not more[~placed].any()
