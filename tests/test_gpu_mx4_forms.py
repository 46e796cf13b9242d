"""4-bit products on rows that no stream takes, on both sides of where the tiles take over: whole numbers, so that
every form gives the same bits. Scales at another address ask for the same forms."""
import numpy as np
import pytest
import torch

import combine_moe_gate_amd as M
import oracle
import workloads as W
from oracle import mx4
from tests.gpu_util import TORCH_DTYPE, assert_bits_equal, to_dev, to_host
from tests.test_gpu_expert_act import announce
from tests.test_gpu_mx4 import pair

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m", [992, 1056])
@pytest.mark.parametrize("mean", [15, 16, 17, 20, 21, 24, 25, 32, 33, 72])
def test_rows_of_any_length(mean, m, dtype):
    announce("4-bit forms", mean, m, dtype)
    rng = np.random.default_rng(mean + m)
    e, k, n = 30, 1, 1800  # 30 segments or more by eight column tiles
    s = mean * e
    idx = W.random_idx(rng, s, e, k)
    L, Lg = oracle.dispatch_layout(idx, e, 0), M.moe_dispatch_layout(to_dev(idx), e, 0)
    x = rng.integers(-2, 3, (s, m)).astype(np.float32)
    wts = rng.integers(-2, 3, (e, n, m)).astype(np.float32)
    x[:, ::32], wts[:, :, 5::32] = 4, -6  # a scale of 1 in every block
    xq, wq = mx4.quantize(x), mx4.quantize(wts)
    want, _ = oracle.expert_gemm_act(L, x, wts, "f32", True)
    want = oracle.from_f32(want.astype(np.float32), dtype)
    for rows in (to_dev(W.cast_input(x, dtype), dtype), pair(*xq)):
        got = M.moe_mx4_expert_gemm(Lg, rows, pair(*wq), dtype=TORCH_DTYPE[dtype])
        assert_bits_equal(to_host(got), want, f"mean {mean}")


@pytest.mark.parametrize("mean", [8, 20, 24, 40])
def test_scales_at_any_address(mean):
    announce("4-bit forms, addresses", mean)
    rng = np.random.default_rng(mean)
    e, k, n, m = 30, 1, 1800, 1024
    s = mean * e
    idx = W.random_idx(rng, s, e, k)
    L = M.moe_dispatch_layout(to_dev(idx), e, 0)
    x = to_dev(W.cast_input(rng.integers(-3, 4, (s, m)).astype(np.float32), "bf16"), "bf16")
    c = to_dev(rng.integers(0, 256, (e, n, m // 2)).astype(np.uint8))
    sc = torch.full((e * n * (m // 32) + 1,), 127, dtype=torch.uint8, device="cuda")
    # sums of multiples of 1/2 below 2^15: exact in any order
    want = M.moe_mx4_expert_gemm(L, x, (c, sc[:-1].view(e, n, -1)))
    assert torch.equal(M.moe_mx4_expert_gemm(L, x, (c, sc[1:].view(e, n, -1))), want)
