"""Refusals of the balance loss's C entries and of its binding, before anything reaches a
GPU (fake addresses: only where there is none)."""
import ctypes
import os

import pytest
import torch

import combine_moe_gate_amd as M

no_gpu_only = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                 reason="fake-pointer validation tests run only without a GPU")
P = [ctypes.c_void_p(1 << (20 + i)) for i in range(12)]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(M.LIB_PATH):
        from combine_moe_gate_amd import _build
        _build.build()
    return M.lib()


def test_workspace_bytes(lib):
    f = lib.moe_balance_workspace_bytes
    assert f(0, 8, 1) == 0 and f(256, 8, 1) == 0  # one launch, no partial rows
    assert f(0, 8, 2) > 0 and f(256, 8, 2) % 256 == 0
    # a partial row of 2 x 4 bytes per expert for each of up to 512 tiles
    assert f(100000, 128, 1) >= 512 * 128 * 8 > f(100000, 128, 1) - (1 << 15)
    assert f(100000, 128, 100) > f(100000, 128, 1)
    assert f(-1, 8, 1) == 0 and f(5, 0, 1) == 0 and f(5, 2000, 1) == 0 and f(5, 8, 0) == 0


@no_gpu_only
def test_balance_argument_checks(lib):
    need = lib.moe_balance_workspace_bytes(10000, 8, 1)

    def fwd(logits=P[0], idx=P[1], mask=None, groups=None, s=10000, e=8, k=2, g=1, counts=P[2], tokens=P[3], probs=P[4],
            loss=P[5], z=P[6], ws=P[7], n=need):
        return lib.moe_balance_loss(logits, idx, mask, groups, s, e, k, g, counts, tokens, probs, loss, z, ws, n, None)

    assert fwd(k=9) == 1 and fwd(e=2000) == 2 and fwd(k=17, e=64) == 2 and fwd(s=-1) == 1
    assert fwd(g=0) == 1 and fwd(g=2) == 1  # groups without offsets
    assert "groups" in lib.moe_last_error().decode()
    assert fwd(groups=P[8], g=2 ** 31 - 1) == 2
    for name in ("logits", "idx", "counts", "tokens", "probs", "loss", "z", "ws"):
        assert fwd(**{name: None}) == 1, name
    assert fwd(ws=ctypes.c_void_p((1 << 27) + 16)) == 5
    assert fwd(n=need - 1) == 3

    def bwd(logits=P[0], counts=P[2], tokens=P[3], gl=P[4], gz=None, s=100, e=8, k=2, g=1, groups=None, out=P[9]):
        return lib.moe_balance_loss_backward(logits, None, groups, counts, tokens, gl, gz, s, e, k, g, out, None)

    for name in ("logits", "counts", "tokens", "out"):
        assert bwd(**{name: None}) == 1, name
    assert bwd(out=ctypes.c_void_p((1 << 20) + 64)) == 1
    assert "overlap" in lib.moe_last_error().decode()
    assert bwd(g=3) == 1 and bwd(e=0) == 1


def test_binding_refuses_mismatched_tensors(monkeypatch):
    def refuse():
        raise AssertionError("the library was called with arguments the binding should have refused")
    monkeypatch.setattr(M, "lib", refuse)
    x, i = torch.zeros(6, 8), torch.zeros((6, 2), dtype=torch.int32)
    c, n, g = torch.zeros((1, 8), dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(1)
    for call, text in [
        (lambda: M.moe_balance_loss(x.half(), i), "logits must be"),
        (lambda: M.moe_balance_loss(x, i.long()), "idx must be"),
        (lambda: M.moe_balance_loss(x, i[:5]), r"idx must have shape [6, *]"),
        (lambda: M.moe_balance_loss(x, i, mask=torch.zeros(6)), "mask must be"),
        (lambda: M.moe_balance_loss(x, i, mask=torch.zeros(5, dtype=torch.bool)), "mask must have shape [6]"),
        (lambda: M.moe_balance_loss(x, i, groups=torch.zeros(3)), "groups must be"),
        (lambda: M.moe_balance_loss(x, i, out=(c, n)), "out must be"),
        (lambda: M.moe_balance_loss(x, i, out=(c, n, torch.zeros(1, 7), g, g)), "probs must have shape [1, 8]"),
        (lambda: M.moe_balance_loss(x, i, out=(c, n, torch.zeros(1, 8), g, None)), "z is None"),
        (lambda: M.moe_balance_loss_backward(x, c[:, :7], n, 2, g), "counts must have shape [1, 8]"),
        (lambda: M.moe_balance_loss_backward(x, c, n, 2, g.double()), "grad_loss must be"),
        (lambda: M.moe_balance_loss_backward(x, c, n, 2, g, torch.zeros(2)), "grad_z must have shape [1]"),
        (lambda: M.moe_balance_loss_backward(x, c, n, 2, g, out=torch.zeros(5, 8)), "out must have shape [6, 8]"),
        (lambda: M.moe_balance_loss(x, i), "on the GPU"),
    ]:
        with pytest.raises(ValueError) as err:
            call()
        assert text in str(err.value), (text, str(err.value))
