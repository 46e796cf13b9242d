"""Pins of the 4-bit oracle: hand-worked blocks, the nearest code by search, round trips, and the input
gradient of a product against differences."""
import numpy as np
import pytest

import oracle
import workloads as W
from oracle import mx4


def block(*v):
    x = np.zeros((1, 32))
    x[0, :len(v)] = v
    return x


def codes_of(x):
    c, E = mx4.quantize(x)
    return np.stack([c & 15, c >> 4], -1).reshape(-1), E


def test_hand_worked_blocks():
    # top 6.5 has floor(log2) = 2, so scale 2^0: ties go to the even code, past 6 to 6
    c, E = codes_of(block(6.5, 2.5, 5.0, 0.25, 0.75, 1.25, 1.75, 3.5, -0.25, -0.0, -3.4, 0.2500001))
    assert E.tolist() == [[127]]
    assert c[:12].tolist() == [7, 4, 6, 0, 2, 2, 4, 6, 8, 8, 13, 1]
    c, E = codes_of(block(0.5, 0.125))  # floor(log2 0.5) - 2 = -3: 0.5 = 4 / 8, 0.125 = 1 / 8
    assert E.tolist() == [[124]] and c[:2].tolist() == [6, 2]
    c, E = codes_of(block(2.0 ** -149, -(2.0 ** -149)))  # scale 2^-127 is the least
    assert E.tolist() == [[0]] and c[:2].tolist() == [0, 8]
    c, E = codes_of(block(2.0 ** -126, 2.0 ** -127))
    assert E.tolist() == [[0]] and c[:2].tolist() == [4, 2]
    c, E = codes_of(block(3.0e38))  # floor(log2) = 127
    assert E.tolist() == [[252]] and c[0] == 7
    for bad in (np.inf, -np.inf, np.nan):
        c, E = codes_of(block(1.0, bad))
        assert E.tolist() == [[255]] and not c.any()
        assert np.isnan(mx4.values(*mx4.quantize(block(1.0, bad)))).all()
    c, E = codes_of(block())
    assert E.tolist() == [[0]] and not c.any()


def test_low_half_holds_the_first_value():
    c, _ = mx4.quantize(block(4.0, 6.0))  # scale 1
    assert c[0, 0] == 6 | (7 << 4)


def test_nearest_by_search():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((400, 64)) * np.exp2(rng.integers(-20, 20, (400, 1)))
    got = mx4.values(*mx4.quantize(x))
    b, g = x.reshape(400, 2, 32), got.reshape(400, 2, 32)
    for r in range(400):
        for j in range(2):
            s = 2.0 ** (np.floor(np.log2(np.abs(b[r, j]).max())) - 2)
            grid = np.concatenate([mx4.GRID, -mx4.GRID]) * s
            best = np.abs(b[r, j][:, None] - grid).min(1)
            assert np.array_equal(np.abs(b[r, j] - g[r, j]), best)


def test_values_of_the_format_come_back():
    for E in (0, 1, 100, 127, 200, 250):
        c = np.arange(256, dtype=np.uint8).reshape(16, 16).copy()
        c[:, 15] = 0x77  # a 6 in each block keeps its scale
        s = np.full((16, 1), E, np.uint8)
        c2, s2 = mx4.quantize(mx4.values(c, s))
        assert np.array_equal(c2, c) and np.array_equal(s2, s)


@pytest.mark.parametrize("plant", ["ceil", "truncate", "odd", "high_first"])
def test_planted_mistakes_fail_a_pin(plant, monkeypatch):
    if plant == "ceil":
        real = mx4.scale_bytes
        monkeypatch.setattr(mx4, "scale_bytes", lambda x: np.minimum(real(x) + 1, 254).astype(np.uint8))
    elif plant == "truncate":
        monkeypatch.setattr(mx4, "round_codes", lambda q: (np.searchsorted(mx4.GRID, np.abs(q), side="right") - 1 + 8 * np.signbit(q)).astype(np.uint8))
    elif plant == "odd":
        monkeypatch.setattr(mx4, "round_codes", lambda q: (np.searchsorted(mx4.MIDDLE, np.abs(q), side="left") + 8 * np.signbit(q)).astype(np.uint8))
    else:
        real_q = mx4.quantize
        monkeypatch.setattr(mx4, "quantize", lambda x: ((lambda c, s: ((c >> 4) | (c << 4), s))(*real_q(x))))
    failed = 0
    for pin in (test_hand_worked_blocks, test_low_half_holds_the_first_value, test_nearest_by_search):
        try:
            pin()
        except AssertionError:
            failed += 1
    assert failed


def test_input_gradient_against_differences():
    """The frozen product's gradient of its rows, and the chain through the dispatch, by differences of
    the forward (rows as they are: the rounding of rows is passed through by definition)."""
    rng = np.random.default_rng(2)
    s, m, n, e, k = 6, 32, 8, 3, 2
    idx = W.random_idx(rng, s, e, k)
    L = oracle.dispatch_layout(idx, e, 3)
    wts = mx4.values(*mx4.quantize(rng.standard_normal((e, n, m)))).astype(np.float32)
    x = rng.integers(-3, 4, (s, m)).astype(np.float32)
    g = rng.standard_normal((L.rows, n)).astype(np.float32) * (L.src >= 0)[:, None]
    _, ga = oracle.expert_gemm_dgrad(L, g, wts, "f32")
    gx = np.zeros((s, m))
    for r in range(L.rows):
        if L.src[r] >= 0:
            gx[L.src[r]] += ga[r]

    def total(x):
        return float((g * oracle.expert_gemm_act(L, x, wts, "f32", True)[0]).sum())

    for t in range(s):
        for i in range(0, m, 5):
            d = np.zeros_like(x)
            d[t, i] = 1
            assert abs((total(x + d) - total(x - d)) / 2 - gx[t, i]) < 1e-9 * max(1, abs(gx[t, i]))
