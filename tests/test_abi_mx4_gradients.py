"""Refusals of the gradients in two parts and in float32 around 4-bit experts, before anything reaches a GPU
(fake addresses: only where there is none)."""
import ctypes
import os

import pytest
import torch

import combine_moe_gate_amd as M
import combine_moe_gate_amd.autograd as A
from tests.test_abi import _fake_handle, fake_layout
from tests.test_abi_mx4 import at, no_gpu_only

F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(M.LIB_PATH):
        from combine_moe_gate_amd import _build
        _build.build()
    return M.lib()


@no_gpu_only
def test_input_gradient_argument_checks(lib):
    st = _fake_handle(40, 8, 2, 0, 1 << 24, M.workspace_bytes(40, 8, 2, 0))  # 80 rows

    def call(g=at(0), parts=2, w=at(1), w_s=at(2, 1), m=64, nz=64, dtype=BF16, to=F32, out=at(3), layout=st):
        return lib.moe_mx4_expert_dgrad_ex(ctypes.byref(layout), g, parts, w, w_s, m, nz, dtype, to, out, None)

    assert call(parts=0) == 1 and call(parts=3) == 1 and "parts must be 1 or 2" in lib.moe_last_error().decode()
    assert call(dtype=F16) == 2 and "bf16" in lib.moe_last_error().decode()
    assert call(to=3) == 2 and call(to=-1) == 2 and call(parts=1, to=F16) == 2 and call(parts=1, dtype=F16, to=BF16) == 2
    assert call(dtype=F32) == 2 and call(nz=4) == 5 and call(m=40) == 5 and call(layout=M.LayoutStruct()) == 4
    assert call(g=None) == 1 and call(w=None) == 1 and call(w_s=None) == 1 and call(out=None) == 1 and call(g=at(0, 8)) == 5
    # gradients of 80 rows of 64: 10240 bytes a part; results 20480 in float32: what only those sizes reach
    for clash in (dict(out=at(0, 10240)), dict(g=at(3, 10240)), dict(out=at(1, 16368)), dict(out=at(2, 1008)),
                  dict(parts=1, g=at(3, 20464))):
        assert call(**clash) == 1, clash
        assert "overlap" in lib.moe_last_error().decode()


@no_gpu_only
def test_backward_argument_checks(lib):
    st = _fake_handle(40, 8, 2, 0, 1 << 24, M.workspace_bytes(40, 8, 2, 0))

    def call(parts=2, z=at(1), gz=at(3), gr=at(6), dtype=F16, kept=F32):
        return lib.moe_expert_act_backward_parts(ctypes.byref(st), at(0), z, kept, 64, dtype, 4, 0, None, parts, gz, 0, None, None,
                                                 gr, None, 0, None)

    assert call(parts=0) == 1 and call(parts=3) == 1 and "parts must be 1 or 2" in lib.moe_last_error().decode()
    assert call(dtype=F32) == 2 and call(kept=BF16) == 2 and call(gz=at(3, 8)) == 5
    for clash in (dict(gr=at(3, 10240)), dict(z=at(3, 20464))):
        assert call(**clash) == 1, clash
        assert "overlap" in lib.moe_last_error().decode()


def test_binding_refuses_mismatched_tensors(monkeypatch):
    monkeypatch.setattr(M, "lib", lambda: pytest.fail("the library was called"))
    L = fake_layout()  # s=6, e=4, k=2, rows=12
    bf, f32 = torch.bfloat16, torch.float32
    w = torch.zeros((4, 48, 32), dtype=torch.uint8), torch.zeros((4, 48, 2), dtype=torch.uint8)
    g, parts = torch.zeros(12, 48, dtype=bf), torch.zeros(12, 2, 48, dtype=bf)
    x = torch.zeros(6, 64, dtype=bf)
    for call, text in [
        (lambda: M.moe_mx4_expert_dgrad(L, torch.zeros(12, 3, 48, dtype=bf), w), "grad_preact must have shape [12, 2, *]"),
        (lambda: M.moe_mx4_expert_dgrad(L, parts[:6], w), "grad_preact must have shape [12, 2, *]"),
        (lambda: M.moe_mx4_expert_dgrad(L, parts.half(), w), "grad_preact must be"),
        (lambda: M.moe_mx4_expert_dgrad(L, g.float(), w), "grad_preact must be"),
        (lambda: M.moe_mx4_expert_dgrad(L, g, w, out_dtype=torch.float16), "out_dtype must be"),
        (lambda: M.moe_mx4_expert_dgrad(L, g, w, out=torch.zeros(12, 64).half()), "out must be"),
        (lambda: M.moe_mx4_expert_dgrad(L, g, w, out=torch.zeros(12, 64), out_dtype=bf), "out must be"),
        (lambda: M.moe_mx4_expert_dgrad(L, parts, w, out=torch.zeros(12, 64).double()), "out must be"),
        (lambda: M.moe_mx4_expert_dgrad(L, parts, w, out=torch.zeros(12, 32)), "out must have shape [12, 64]"),
        (lambda: M.moe_mx4_expert_dgrad(L, parts, w, out_dtype=f32), "on the GPU"),
        (lambda: M.moe_expert_act_backward(L, g, parts=3), "parts must be"),
        (lambda: M.moe_expert_act_backward(L, g, parts=2), "on the GPU"),
        (lambda: A.expert_linear_mx4(x, w, L, grad_dtype=torch.float16), "grad_dtype must be"),
    ]:
        with pytest.raises(ValueError) as err:
            call()
        assert text in str(err.value), (text, str(err.value))
