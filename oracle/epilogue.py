"""CPU oracle of the expert products with an epilogue and of that epilogue's backward, in
float64, expert by expert.

Definitions: z[r] = A(r) @ W[x]^T + b[x] for each placed row r of expert x; u = act(z), or
act(z[:n]) * z[n:] if gated; out[r] = w_r u + residual(r); unfilled rows 0. Nothing is
rounded on the way: the results are the exact values a float32 kernel comes close to.

Parity: activations against their closed values and slopes against central differences;
the whole backward against differences of the forward (tests/test_oracle_epilogue.py).
"""
from __future__ import annotations

import numpy as np
from scipy.special import erfc

from .moe import Layout, to_f32

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def logistic(y: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """s(y) = 1 / (1 + exp(-y)) and 1 - s(y) = s(-y), each to full relative precision."""
    y = np.clip(y, -700, 700)
    return 1 / (1 + np.exp(-y)), 1 / (1 + np.exp(y))


def act(name: str, z: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """(act(z), act'(z)); relu' is 0 at 0."""
    z = np.asarray(z, np.float64)
    if name == "none":
        return z, np.ones_like(z)
    if name == "relu":
        return np.where(z > 0, z, 0.0), (z > 0).astype(np.float64)
    if name == "gelu":
        cdf = 0.5 * erfc(-z / np.sqrt(2.0))
        return z * cdf, cdf + z * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
    if name == "gelu_tanh":
        # (1 + tanh y) / 2 = s(2 y) and (1 - tanh^2 y) / 4 = s(2 y) s(-2 y) with the logistic
        # function s: 1 + tanh loses every digit where tanh is near -1
        b, q = np.sqrt(2 / np.pi), 0.044715
        s, rest = logistic(2 * b * (z + q * z ** 3))
        return z * s, s + 2 * z * s * rest * b * (1 + 3 * q * z * z)
    if name == "silu":
        s, rest = logistic(z)
        return z * s, s * (1 + z * rest)
    raise ValueError(f"unknown activation {name!r}")


def row_weights(layout: Layout, w: np.ndarray | None) -> np.ndarray:
    """[rows] the weight of the route placed at each row (1 without weights)."""
    out = np.ones(layout.rows)
    if w is not None:
        placed = layout.dst >= 0
        out[layout.dst[placed]] = np.asarray(w, np.float64)[placed]
    return out


def segments(layout: Layout):
    """(expert, its placed rows) for every expert with rows."""
    for x in range(layout.e):
        r0 = int(layout.offsets[x])
        if layout.kept[x]:
            yield x, np.arange(r0, r0 + int(layout.kept[x]))


def finish(z: np.ndarray, name: str, gated: bool) -> np.ndarray:
    """u(z)"""
    if not gated:
        return act(name, z)[0]
    n = z.shape[-1] // 2
    return act(name, z[..., :n])[0] * z[..., n:]


def expert_gemm_act(layout: Layout, a, weights, dtype: str, gather: bool, bias=None, name: str = "none",
                    gated: bool = False, w=None, residual=None, residual_gather: bool = False):
    """(out, z) in float64; a, weights and residual in dtype's storage, bias real-valued."""
    a64 = to_f32(a, dtype).astype(np.float64)
    nz = weights.shape[1]
    z = np.zeros((layout.rows, nz))
    out = np.zeros((layout.rows, nz // 2 if gated else nz))
    rw = row_weights(layout, w)
    for x, rows in segments(layout):
        z[rows] = a64[layout.src[rows] if gather else rows] @ to_f32(weights[x], dtype).astype(np.float64).T
        if bias is not None:
            z[rows] += np.asarray(bias[x], np.float64)
        out[rows] = rw[rows, None] * finish(z[rows], name, gated)
        if residual is not None:
            out[rows] += to_f32(residual, dtype).astype(np.float64)[layout.src[rows] if residual_gather else rows]
    return out, z


def expert_act_backward(layout: Layout, grad_out, z, name: str, gated: bool, w=None):
    """(grad_z [rows, nz], grad_bias [e, nz], grad_w [s, k], grad_residual [rows, n]) in
    float64, for real-valued grad_out [rows, n] and z [rows, nz]."""
    g64, z64 = np.asarray(grad_out, np.float64), np.asarray(z, np.float64)
    n = g64.shape[1]
    gz, gb = np.zeros(z64.shape), np.zeros((layout.e, z64.shape[1]))
    gr, dots = np.zeros(g64.shape), np.zeros(layout.rows)
    rw = row_weights(layout, w)
    for x, rows in segments(layout):
        g = rw[rows, None] * g64[rows]
        f, d = act(name, z64[rows, :n])
        if gated:
            gz[rows] = np.concatenate([g * z64[rows, n:] * d, g * f], 1)
        else:
            gz[rows] = g * d
        gb[x] = gz[rows].sum(0)
        gr[rows] = g64[rows]
        dots[rows] = (g64[rows] * finish(z64[rows], name, gated)).sum(1)
    placed = layout.dst >= 0
    gw = np.where(placed, dots[np.where(placed, layout.dst, 0)], 0.0)
    return gz, gb, gw, gr
