"""The balance loss over more groups than one launch of its second kernel takes, on the GPU
against the formulas in float64 (tolerances as in tests/test_gpu_balance.py)."""
import pytest
import torch

import combine_moe_gate_amd as M

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def test_more_groups_than_a_launch_takes():
    """262143 groups of 1024 experts are the most of one launch: 262200 single tokens, those
    past the border and the first ones checked."""
    print("CASE balance 262200 groups", flush=True)
    e, k, s = 1024, 4, 262200
    gen = torch.Generator("cuda").manual_seed(2)
    logits = torch.randn((s, e), generator=gen, device="cuda")
    idx = torch.randint(0, e // k, (s, k), generator=gen, device="cuda").int() + torch.arange(k, device="cuda").int() * (e // k)
    groups = torch.arange(s + 1, device="cuda").int()
    counts, tokens, probs, loss, z = M.moe_balance_loss(logits, idx, groups=groups)
    assert (tokens == 1).all()
    assert torch.equal(counts.sum(1), torch.full((s,), k, device="cuda"))
    grad = M.moe_balance_loss_backward(logits, counts, tokens, k, torch.ones(s, device="cuda"), groups=groups)
    for part in (slice(0, 100), slice(262043, s)):  # 262143 is the first group of the second launch
        l64 = logits[part].double()
        p, lse = torch.softmax(l64, 1), torch.logsumexp(l64, 1)
        c = torch.zeros_like(p).scatter_(1, idx[part].long(), 1.0)
        assert torch.equal(counts[part].double(), c)
        D = l64.amax(1, keepdim=True) - l64
        rel = U * (4 * D + 4 * (p * D).sum(1, keepdim=True) + 32)
        # one token: its row is the tile's sum, rounded to float32 at the end
        assert ((probs[part].double() - p).abs() <= p * (rel + 2 * U)).all()
        want = e / k * (c * p).sum(1)
        assert ((loss[part].double() - want).abs() <= e / k * (c * p * (rel + 2 * U)).sum(1) + U * want).all()
        err = U * (4 * (p * D).sum(1) + 26 + 4 * 7 + lse.abs())
        assert ((z[part].double() - lse ** 2).abs() <= 2 * lse.abs() * err + err ** 2 + U * lse ** 2).all()
        off = (c - k / e).abs() * e / k
        dot = (p * off).sum(1, keepdim=True)
        want = p * (e / k * c - (p * e / k * c).sum(1, keepdim=True))
        tol = p * (rel * (off + dot) + (p * off * (rel + 24 * U)).sum(1, keepdim=True) + 4 * U * (off + dot)) + 1e-44
        assert ((grad[part].double() - want).abs() <= tol + U * want.abs()).all()
