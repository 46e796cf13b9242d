"""Refusals of the entries that take the kept values' type, and of their binding, before
anything reaches a GPU (fake addresses: only where there is none)."""
import ctypes
import os

import pytest
import torch

import combine_moe_gate_amd as M
import combine_moe_gate_amd.autograd as A
from tests.test_abi import _fake_handle, fake_layout
from tests.test_abi_expert_act import at, no_gpu_only

F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(M.LIB_PATH):
        from combine_moe_gate_amd import _build
        _build.build()
    return M.lib()


@no_gpu_only
def test_forward_argument_checks(lib):
    s, e, k, m, n = 40, 8, 2, 64, 64  # 80 rows: kept values of 10240 bytes in bf16, 20480 in float32
    st = _fake_handle(s, e, k, 0, 1 << 24, M.workspace_bytes(s, e, k, 0))

    def call(kept=F32, dtype=BF16, preact=at(5), residual=None, out=at(2), a=at(0)):
        q = M.Epilogue(0, 0, None, 0, 0, None, residual, preact)
        return lib.moe_expert_gemm_act_ex(ctypes.byref(st), a, 1, at(1), m, n, dtype, ctypes.byref(q), kept, out, None)

    assert call(kept=F16) == 2 and "preact_dtype" in lib.moe_last_error().decode()
    assert call(kept=7) == 2 and call(kept=BF16, dtype=F16) == 2 and call(dtype=F32) == 2
    assert call(preact=at(5, 8)) == 5 and call(a=None) == 1
    # what only the float32 rows reach
    near = ctypes.c_void_p(at(5).value + 10240)
    for clash in (dict(out=near), dict(a=near), dict(residual=near)):
        assert call(**clash) == 1, clash
        assert "overlap" in lib.moe_last_error().decode()


@no_gpu_only
def test_backward_argument_checks(lib):
    s, e, k, n = 40, 8, 2, 64
    st = _fake_handle(s, e, k, 0, 1 << 24, M.workspace_bytes(s, e, k, 0))

    def call(kept=F32, z=at(1), act=4, gz=at(3), gr=at(6), dtype=BF16):
        return lib.moe_expert_act_backward_ex(ctypes.byref(st), at(0), z, kept, n, dtype, act, 0, None, gz, 0, None, None,
                                              gr, None, 0, None)

    assert call(kept=F16) == 2 and "preact_dtype" in lib.moe_last_error().decode()
    assert call(kept=-1) == 2 and call(dtype=F32) == 2 and call(z=None) == 1 and call(z=at(1, 4)) == 5
    near = ctypes.c_void_p(at(1).value + 10240)
    for clash in (dict(gz=near), dict(gr=near)):
        assert call(**clash) == 1, clash
        assert "overlap" in lib.moe_last_error().decode()


def test_binding_refuses_mismatched_tensors(monkeypatch):
    def refuse():
        raise AssertionError("the library was called with arguments the binding should have refused")
    monkeypatch.setattr(M, "lib", refuse)
    L = fake_layout()  # s=6, e=4, k=2, rows=12
    bf, f32 = torch.bfloat16, torch.float32
    x, w, g, z = (torch.zeros(q, dtype=bf) for q in ((6, 8), (4, 16, 8), (12, 8), (12, 16)))
    for call, text in [
        (lambda: M.moe_expert_gemm_act(L, x, w, save_preact=True, preact_dtype=torch.float16), "preact_dtype must be"),
        (lambda: M.moe_expert_gemm_act(L, x, w, preact=z, preact_dtype=f32), "preact must be"),
        (lambda: M.moe_expert_gemm_act(L, x, w, preact=z.float(), preact_dtype=bf), "preact must be"),
        (lambda: M.moe_expert_gemm_act(L, x, w, preact=z.half()), "preact must be"),
        (lambda: M.moe_expert_gemm_act(L, x, w, preact=z.float()[:, :8]), "preact must have shape [12, 16]"),
        (lambda: M.moe_expert_act_backward(L, g, z.half(), gated=True), "preact must be"),
        (lambda: M.moe_expert_act_backward(L, g, z.double(), gated=True), "preact must be"),
        (lambda: A.expert_linear(x, w, L, act="silu", preact_dtype=torch.float64), "preact_dtype must be"),
        (lambda: M.moe_expert_gemm_act(L, x, w, preact=z.float()), "on the GPU"),
    ]:
        with pytest.raises(ValueError) as err:
            call()
        assert text in str(err.value), (text, str(err.value))
