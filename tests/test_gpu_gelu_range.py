"""gelu and its slope at every finite value of the element types, on the GPU against float64:
each result within its own rounding, also where it is far smaller than its argument.

With u = 2^-24: for z <= 0 the kernels form Phi(z) = P(t) t E, t = 1 / (1 + p |z|), E =
exp2(-z^2 log2(e) / 2). Off by, relative to itself: E 1.5 u z^2 (its argument's three
roundings) and 4 u (the hardware's exponential); t 4 u (constant, sum and hardware reciprocal),
which P(t) t amplifies by at most 2.3 (erfcx'(0) / p); P's nine coefficients and eight steps
6 u, its fit u, two products 2 u: 22 u + 1.5 u z^2 in all. For z > 0 it is 1 - Phi(-z), off by
no larger a share of a larger value (z^2 Phi(-z) < Phi(z) / 4), and u: 24 u. The product with z
rounds once more. A slope is Phi(z) + z phi(z), the second as far off as E, its constant and
two products: 8 u + 1.5 u z^2. E below 2^-126 may be 0: 2^-126 times |z| or 1, z up to 20.
"""
import numpy as np
import pytest
import torch

import combine_moe_gate_amd as M
import oracle
from oracle import epilogue as E
from tests.gpu_util import to_dev, to_host
from tests.test_gpu_expert_act import U, announce, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gelu_at_every_value(dtype):
    announce("gelu range", dtype)
    bits = np.arange(0x7F80 if dtype == "bf16" else 0x7C00, dtype=np.uint16)
    vals = np.concatenate([bits, bits | np.uint16(0x8000)])
    if dtype == "f16":
        vals = vals.view(np.float16)
    n = len(vals)
    wts, x = np.zeros((1, n, 8), vals.dtype), np.zeros((1, 8), vals.dtype)
    wts[0, :, 0], x[0, 0] = vals, oracle.from_f32(np.ones(1, np.float32), dtype)[0]
    z = oracle.to_f32(vals, dtype).astype(np.float64)[None]
    L = M.moe_dispatch_layout(torch.zeros((1, 1), dtype=torch.int32, device="cuda"), 1, 0)
    out, pre = M.moe_expert_gemm_act(L, to_dev(x, dtype), to_dev(wts, dtype), act="gelu", save_preact=True)
    assert np.array_equal(oracle.to_f32(to_host(pre), dtype), z.astype(np.float32)), "z is the value itself"
    # far below 0 float32 holds nothing of phi: no tolerance is more than the value
    eps = np.where(z > 0, 26 * U, np.minimum(1.0, U * (24 + 2 * z * z)))
    with np.errstate(over="ignore", under="ignore"):
        f, d = E.act("gelu", z)
        phi = np.exp(-0.5 * np.minimum(z * z, 1400.0)) / np.sqrt(2 * np.pi)
    within(to_host(out), f, eps * np.abs(f) + 2.0 ** -126 * np.abs(z).clip(max=20), dtype, "gelu")
    cdf = np.abs(f) / np.maximum(np.abs(z), 1e-300)
    cdf[z == 0] = 0.5
    one = torch.ones((1, n), dtype=pre.dtype, device="cuda")
    got = M.moe_expert_act_backward(L, one, pre, act="gelu")[0]
    within(to_host(got), d, eps * cdf + U * (10 + 2 * z * z) * np.abs(z) * phi + 2.0 ** -126 * np.abs(z).clip(1, 20), dtype, "slope")
