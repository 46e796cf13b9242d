"""CPU oracle of microscaled 4-bit floating point: rows to 4 bits and back, in float64.

Definitions: a block of 32 values has a scale byte E, 2^(E - 127) (255: not a number); a value four
bits, a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6. E = floor(log2 top) - 2 + 127 of the block's largest
magnitude, at least 0 (0 in a block of zeros, 255 with codes 0 in one that holds an infinity or NaN);
values over the scale go to the nearest of the eight, half-way cases to the even code, past 6 to 6.

Parity: hand-worked blocks, an exhaustive search for the nearest code, and the round trip of every value
the format holds (tests/test_oracle_mx4.py). The products are those of oracle.epilogue on the values.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MIDDLE = (GRID[:-1] + GRID[1:]) / 2


def scale_bytes(x: np.ndarray) -> np.ndarray:
    """[..., m / 32] of real x [..., m]."""
    top = np.abs(np.asarray(x, np.float64)).reshape(*x.shape[:-1], -1, BLOCK).max(-1)  # NaN wins
    fine = np.isfinite(top)
    _, ex = np.frexp(np.where(fine & (top > 0), top, 1.0))  # top = f 2^ex, f in [0.5, 1)
    E = np.maximum(ex - 1 - 2 + 127, 0)
    return np.where(fine, np.where(top > 0, E, 0), 255).astype(np.uint8)


def round_codes(q: np.ndarray) -> np.ndarray:
    """Codes (with sign) of q, already over the scale."""
    a = np.abs(q)
    low = np.searchsorted(MIDDLE, a, side="left")  # midpoints below a
    tie = (low < 7) & (a == MIDDLE[np.minimum(low, 6)]) & (low % 2 == 1)
    return (low + tie + 8 * np.signbit(q)).astype(np.uint8)


def quantize(x: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """(codes [..., m / 2], scales [..., m / 32]) of real x [..., m]."""
    x = np.asarray(x, np.float64)
    E = scale_bytes(x)
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    bad = (E == 255)[..., None]
    q = np.where(bad, 0.0, b) * np.ldexp(1.0, 127 - E.astype(np.int64))[..., None]
    c = np.where(bad, 0, round_codes(q)).astype(np.uint8).reshape(x.shape)
    return c[..., 0::2] | (c[..., 1::2] << 4), E


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """[..., m] float64 values of codes [..., m / 2] and scales [..., m / 32]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = np.where(c & 8, -GRID[c & 7], GRID[c & 7])
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, BLOCK, -1)
