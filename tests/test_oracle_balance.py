"""Pins of the balance-loss oracle: a case worked by hand, and the gradient against central
differences of the losses."""
import numpy as np

import oracle


def test_two_tokens_by_hand():
    # token 0: logits ln 3, 0 -> p = 3/4, 1/4; token 1: 0, 0 -> p = 1/2, 1/2; both choose expert 0
    logits = np.array([[np.log(3.0), 0.0], [0.0, 0.0]])
    b = oracle.balance_loss(logits, np.array([[0], [0]]))
    assert b.counts.tolist() == [[2, 0]] and b.tokens.tolist() == [2]
    np.testing.assert_allclose(b.probs, [[0.625, 0.375]], rtol=1e-15)
    np.testing.assert_allclose(b.loss, [2 * 1.0 * 0.625], rtol=1e-15)
    np.testing.assert_allclose(b.z, [(np.log(4.0) ** 2 + np.log(2.0) ** 2) / 2], rtol=1e-15)


def test_a_level_load_costs_one():
    e, s = 8, 16
    idx = np.stack([np.arange(s) % e, (np.arange(s) + 3) % e], 1)
    np.testing.assert_allclose(oracle.balance_loss(np.zeros((s, e)), idx).loss, [1.0], rtol=1e-14)


def test_groups_padding_and_bad_routes():
    rng = np.random.default_rng(1)
    logits = rng.standard_normal((9, 5))
    logits[3] = np.nan  # padded
    logits[4] = -np.inf  # no distribution: counted among the tokens and routes, nothing else
    idx = np.array([[0, 1], [1, 1], [-1, 5], [0, 0], [2, 3], [4, 0], [0, 1], [2, 3], [3, 4]])
    mask = np.ones(9, bool)
    mask[3] = False
    b = oracle.balance_loss(logits, idx, mask, [1, 4, 4, 8])  # tokens 0 and 8 in no group
    assert b.tokens.tolist() == [2, 0, 4]
    assert b.counts.tolist() == [[0, 1, 0, 0, 0], [0] * 5, [2, 1, 2, 2, 1]]
    assert np.isfinite(b.loss).all() and b.loss[1] == 0 and b.z[1] == 0
    np.testing.assert_allclose(b.probs[2].sum(), 3 / 4, rtol=1e-14)
    g = oracle.balance_loss_backward(logits, b, 2, np.ones(3), np.ones(3), mask, [1, 4, 4, 8])
    assert not g[[0, 3, 4, 8]].any() and g[[1, 2, 5, 6, 7]].any(1).all()


def test_gradient_against_differences():
    rng = np.random.default_rng(2)
    logits = rng.standard_normal((7, 6))
    idx = np.stack([rng.permutation(6)[:2] for _ in range(7)])
    mask, groups = np.array([1, 1, 0, 1, 1, 1, 1], bool), [0, 3, 7]
    gl, gz = np.array([0.7, -1.3]), np.array([0.2, 0.4])

    def total(l):
        b = oracle.balance_loss(l, idx, mask, groups)
        return float((gl * b.loss + gz * b.z).sum())

    got = oracle.balance_loss_backward(logits, oracle.balance_loss(logits, idx, mask, groups), 2, gl, gz, mask, groups)
    h = 1e-5  # differences good to h^2 and 2^-53 / h: about 1e-10
    for t in range(7):
        for x in range(6):
            up, down = logits.copy(), logits.copy()
            up[t, x] += h
            down[t, x] -= h
            assert abs((total(up) - total(down)) / (2 * h) - got[t, x]) < 1e-8
