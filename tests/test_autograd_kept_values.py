"""When expert_linear has its product keep the values before the activation: only where a
backward can follow (the product itself replaced, so that no GPU is needed)."""
import pytest
import torch

import combine_moe_gate_amd.autograd as A
from tests.test_abi import fake_layout


@pytest.fixture
def asked(monkeypatch):
    calls = []

    def product(layout, a, weights, act="none", gated=False, save_preact=False, preact_dtype=None, **kw):
        calls.append((save_preact, preact_dtype))
        nz = weights.shape[1]
        out = torch.zeros((layout.rows, nz // 2 if gated else nz), dtype=a.dtype)
        return (out, torch.zeros((layout.rows, nz), dtype=preact_dtype or a.dtype)) if save_preact else out

    monkeypatch.setattr(A, "moe_expert_gemm_act", product)
    return calls


def test_kept_for_a_backward_only(asked):
    L = fake_layout()  # s=6, e=4, k=2, rows=12
    x, w = torch.zeros((6, 8), dtype=torch.bfloat16), torch.zeros((4, 16, 8), dtype=torch.bfloat16)
    param, bias, route = torch.nn.Parameter(w), torch.nn.Parameter(torch.zeros(4, 16)), torch.ones((6, 2), requires_grad=True)
    run = lambda **kw: A.expert_linear(x, kw.pop("weights", param), L, **kw)  # noqa: E731
    run(act="silu", gated=True)
    run(act="silu", preact_dtype=torch.float32)
    run(bias=bias, w=route)          # the route weights' gradient needs them
    assert asked == [(True, None), (True, torch.float32), (True, None)]
    asked.clear()
    run(bias=bias)                   # nothing needs them
    run(weights=w, act="silu")       # no input has a gradient
    for off in (torch.no_grad, torch.inference_mode):
        with off():                  # no backward follows, whatever the parameters ask for
            run(act="silu", gated=True)
            run(bias=bias, w=route, act="gelu", preact_dtype=torch.float32)
    assert [keep for keep, _ in asked] == [False] * 6
