"""CPU oracle of the router's balance loss: counts, mean probabilities, load-balance loss
and z loss per group of tokens, and their gradient with respect to the logits, in float64,
token by token.

Parity: a hand-worked two-token case, and the gradient against central differences of the
losses (tests/test_oracle_balance.py).
"""
from __future__ import annotations

import dataclasses

import numpy as np


@dataclasses.dataclass
class Balance:
    counts: np.ndarray  # [g, e] int64
    tokens: np.ndarray  # [g] int64
    probs: np.ndarray   # [g, e] float64
    loss: np.ndarray    # [g] float64
    z: np.ndarray       # [g] float64


def softmax_row(row: np.ndarray) -> tuple[np.ndarray, float]:
    """(probabilities, logsumexp) of one token's logits; zeros where all are -inf."""
    row = np.asarray(row, np.float64)
    if np.all(row == -np.inf):
        return np.zeros_like(row), 0.0
    if np.isnan(row).any() or np.any(row == np.inf):
        return np.full_like(row, np.nan), np.nan
    top = row.max()
    ex = np.exp(row - top)
    return ex / ex.sum(), float(top + np.log(ex.sum()))


def group_tokens(s: int, mask, groups) -> list[list[int]]:
    """The unpadded tokens of each group."""
    bounds = [0, s] if groups is None else [int(v) for v in groups]
    return [[t for t in range(bounds[i], bounds[i + 1]) if mask is None or mask[t]]
            for i in range(len(bounds) - 1)]


def balance_loss(logits: np.ndarray, idx: np.ndarray, mask=None, groups=None) -> Balance:
    s, e = logits.shape
    k = idx.shape[1]
    members = group_tokens(s, mask, groups)
    g = len(members)
    out = Balance(np.zeros((g, e), np.int64), np.zeros(g, np.int64), np.zeros((g, e)), np.zeros(g), np.zeros(g))
    for i, tokens in enumerate(members):
        n = out.tokens[i] = len(tokens)
        if n == 0:
            continue
        for t in tokens:
            p, lse = softmax_row(logits[t])
            out.probs[i] += p / n
            out.z[i] += lse * lse / n
            named = []
            for x in idx[t]:
                if 0 <= x < e and x not in named:
                    out.counts[i, x] += 1
                named.append(x)
        out.loss[i] = e / k * float((out.counts[i] / n * out.probs[i]).sum())
    return out


def balance_loss_backward(logits: np.ndarray, fwd: Balance, k: int, grad_loss, grad_z, mask=None, groups=None) -> np.ndarray:
    s, e = logits.shape
    grad = np.zeros((s, e))
    for i, tokens in enumerate(group_tokens(s, mask, groups)):
        n = len(tokens)
        for t in tokens:
            p, lse = softmax_row(logits[t])
            d_p = grad_loss[i] * e / k * fwd.counts[i] / (n * n)  # d loss / d p_tx
            grad[t] = p * (d_p - (p * d_p).sum()) + grad_z[i] * 2.0 * lse / n * p
    return grad
