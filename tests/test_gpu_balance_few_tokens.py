"""The balance loss on both sides of its one-launch form's borders, wide rows among them, on
the GPU against the float64 oracle (tolerances in tests/test_gpu_balance.py)."""
import numpy as np
import pytest

import workloads as W
from tests.test_gpu_balance import announce, run_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("s,e,k,groups,masked", [
    (31, 1024, 16, None, 0.0),
    (32, 1024, 16, None, 0.2),       # 32768 logits in one launch
    (33, 1024, 16, None, 0.2),       # two
    (32, 1021, 5, [3, 30], 0.0),     # one group of part of the batch, rows no 16-byte load fits
    (32, 1024, 8, [0, 16, 32], 0.0), # two groups: two launches
    (1024, 16, 4, None, 0.1),        # 16384 logits in one launch
    (1025, 15, 4, None, 0.1),        # more tokens than one launch takes
    (64, 257, 2, None, 0.0),         # more logits
])
def test_both_sides_of_one_launch(s, e, k, groups, masked):
    announce("balance borders", s, e, k, groups, masked)
    rng = np.random.default_rng(s * e)
    logits = (rng.standard_normal((s, e)) * 2).astype(np.float32)
    run_case(logits, W.random_idx(rng, s, e, k), rng.random(s) >= masked if masked else None, groups)
