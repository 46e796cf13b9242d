"""Which values of the 4-bit format float32 holds, and what include/moe_gate.h says about it."""
import os

import numpy as np

from oracle import mx4

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_gate.h")


def test_values_past_float32():
    codes = np.arange(8, dtype=np.uint8)[None, :].repeat(16, 0).reshape(1, -1)[:, :16] & 7  # 0 .. 7 in low halves
    past = {}
    for E in (252, 253, 254):
        with np.errstate(over="ignore"):
            v = mx4.values(codes, np.full((1, 1), E, np.uint8)).astype(np.float32)[0, 0:16:2]
        past[E] = [float(g) for g, x in zip(mx4.GRID, v) if np.isinf(x)]
    assert past == {252: [], 253: [4.0, 6.0], 254: [2.0, 3.0, 4.0, 6.0]}


def test_the_header_says_so():
    text = " ".join(line.strip(" *\n") for line in open(HEADER))
    assert "is infinite: 4 and 6 under E = 253, 2 to 6 under E = 254" in text
    assert "E = 254 with codes above 1" not in text
