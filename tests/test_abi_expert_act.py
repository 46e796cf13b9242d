"""Refusals of the expert products' epilogue entries and of their binding, before anything
reaches a GPU (fake addresses: only where there is none)."""
import ctypes
import os

import pytest
import torch

import combine_moe_gate_amd as M
from tests.test_abi import _fake_handle, fake_layout

no_gpu_only = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                 reason="fake-pointer validation tests run only without a GPU")


def at(i, off=0):
    return ctypes.c_void_p((1 << 30) + (i << 24) + off)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(M.LIB_PATH):
        from combine_moe_gate_amd import _build
        _build.build()
    return M.lib()


def test_struct_matches_the_header():
    assert ctypes.sizeof(M.Epilogue) == 4 + 4 + 8 + 4 + 4 + 8 + 8 + 8
    text = open(os.path.join(os.path.dirname(__file__), "..", "include", "moe_gate.h")).read()
    for name, code in M.ACTIVATIONS.items():
        assert f"MOE_ACT_{name.upper()} = {code}" in text


@no_gpu_only
def test_forward_argument_checks(lib):
    s, e, k = 40, 8, 2
    st = _fake_handle(s, e, k, 0, 1 << 24, M.workspace_bytes(s, e, k, 0))

    def call(a=at(0), gather=1, w=at(1), m=64, n=64, dtype=1, out=at(2), layout=st, **ep):
        q = M.Epilogue(ep.get("act", 0), ep.get("gated", 0), ep.get("bias"), ep.get("bias_dtype", 0),
                       ep.get("residual_gather", 0), ep.get("topk_w"), ep.get("residual"), ep.get("preact"))
        return lib.moe_expert_gemm_act(ctypes.byref(layout), a, gather, w, m, n, dtype, ctypes.byref(q), out, None)

    assert call(dtype=0) == 2 and call(dtype=7) == 2
    assert call(gather=2) == 1 and call(act=5) == 1 and call(act=-1) == 1 and call(gated=2) == 1
    assert call(residual_gather=3) == 1
    assert call(m=60) == 5 and call(n=4) == 5 and call(m=0) == 1
    assert call(a=None) == 1 and call(w=None) == 1 and call(out=None) == 1
    assert call(a=at(0, 8)) == 5 and call(out=at(2, 2)) == 5
    assert call(bias=at(3).value, bias_dtype=2) == 2  # f16 bias of bf16 weights
    assert call(bias=at(3, 4).value) == 5 and call(residual=at(4, 8).value) == 5 and call(preact=at(5, 8).value) == 5
    for clash in (dict(out=at(0, 256)), dict(residual=at(2, 64).value), dict(preact=at(2, 1024).value),
                  dict(out=at(1, 64)), dict(preact=at(1, 65520).value),  # the last of the weights' 65536 bytes
                  dict(preact=at(0, 16).value), dict(preact=at(6).value, residual=at(6, 32).value)):
        assert call(**clash) == 1, clash
        assert "overlap" in lib.moe_last_error().decode()
    assert call(layout=M.LayoutStruct()) == 4


@no_gpu_only
def test_backward_argument_checks(lib):
    s, e, k, n = 40, 8, 2, 64
    st = _fake_handle(s, e, k, 0, 1 << 24, M.workspace_bytes(s, e, k, 0))
    need = lib.moe_expert_act_backward_workspace_bytes(ctypes.byref(st), n, 1)
    assert need > lib.moe_expert_act_backward_workspace_bytes(ctypes.byref(st), n, 0) > 0
    assert lib.moe_expert_act_backward_workspace_bytes(ctypes.byref(M.LayoutStruct()), n, 1) == 0
    assert lib.moe_expert_act_backward_workspace_bytes(ctypes.byref(st), 0, 0) == 0
    assert lib.moe_expert_act_backward_workspace_bytes(ctypes.byref(st), n, 2) == 0

    def call(g=at(0), z=at(1), n=n, dtype=1, act=4, gated=1, w=at(2), gz=at(3), bt=0, gb=at(4), gw=at(5), gr=at(6),
             ws=at(7), nb=need):
        return lib.moe_expert_act_backward(ctypes.byref(st), g, z, n, dtype, act, gated, w, gz, bt, gb, gw, gr, ws, nb, None)

    assert call(dtype=0) == 2 and call(act=9) == 1 and call(gated=-1) == 1 and call(n=12) == 5
    assert call(bt=2) == 2 and call(g=None) == 1 and call(z=None) == 1
    assert call(w=None) == 1 and "needs topk_w" in lib.moe_last_error().decode()
    assert call(z=None, act=0, gated=0) == 1  # the route weights' gradient needs the kept values
    assert call(ws=None) == 1 and call(nb=need - 1) == 3 and call(ws=at(7, 8)) == 5
    assert call(gz=at(3, 4)) == 5 and call(gr=at(6, 4)) == 5
    for clash in (dict(gz=at(0, 64)), dict(gz=at(1, 64)), dict(gr=at(0, 64)), dict(gr=at(3, 64))):
        assert call(**clash) == 1, clash
        assert "overlap" in lib.moe_last_error().decode()


@no_gpu_only
def test_input_gradient_argument_checks(lib):
    st = _fake_handle(40, 8, 2, 0, 1 << 24, M.workspace_bytes(40, 8, 2, 0))

    def call(g=at(0), w=at(1), m=64, nz=64, dtype=1, out=at(2), layout=st):
        return lib.moe_expert_act_dgrad(ctypes.byref(layout), g, w, m, nz, dtype, out, None)

    assert call(dtype=0) == 2 and call(nz=4) == 5 and call(m=12) == 5 and call(m=0) == 1
    assert call(g=None) == 1 and call(w=None) == 1 and call(out=None) == 1
    assert call(out=at(2, 8)) == 5 and call(layout=M.LayoutStruct()) == 4
    for out in (at(0, 512), at(1, 65520)):
        assert call(out=out) == 1 and "overlap" in lib.moe_last_error().decode()


def test_binding_refuses_mismatched_tensors(monkeypatch):
    def refuse():
        raise AssertionError("the library was called with arguments the binding should have refused")
    monkeypatch.setattr(M, "lib", refuse)
    L = fake_layout()  # s=6, e=4, k=2, rows=12
    bf = torch.bfloat16
    x, w, g, z = (torch.zeros(q, dtype=bf) for q in ((6, 8), (4, 16, 8), (12, 8), (12, 16)))
    for call, text in [
        (lambda: M.moe_expert_gemm_act(L, x.float(), w), "a must be"),
        (lambda: M.moe_expert_gemm_act(L, x, w, gather=False), "a must have shape [12, *]"),
        (lambda: M.moe_expert_gemm_act(L, x, w.half()), "weights must be"),
        (lambda: M.moe_expert_gemm_act(L, x, w[:, :15], gated=True), "even number of rows"),
        (lambda: M.moe_expert_gemm_act(L, x, w, bias=torch.zeros(4, 15)), "bias must have shape [4, 16]"),
        (lambda: M.moe_expert_gemm_act(L, x, w, bias=torch.zeros(4, 16).half()), "bias must be"),
        (lambda: M.moe_expert_gemm_act(L, x, w, act="tanh"), "act must be one of"),
        (lambda: M.moe_expert_gemm_act(L, x, w, act=None), "act must be one of"),
        (lambda: M.moe_expert_gemm_act(L, x, w, w=torch.zeros(6, 3)), "w must have shape [6, 2]"),
        (lambda: M.moe_expert_gemm_act(L, x, w, residual=g), "residual must have shape [12, 16]"),
        (lambda: M.moe_expert_gemm_act(L, x, w, gated=True, residual=g, residual_gather=True), "residual must have shape [6, 8]"),
        (lambda: M.moe_expert_gemm_act(L, x, w, gated=True, out=z), "out must have shape [12, 8]"),
        (lambda: M.moe_expert_gemm_act(L, x, w, gated=True, preact=g), "preact must have shape [12, 16]"),
        (lambda: M.moe_expert_act_backward(L, g.float(), z), "grad_out must be"),
        (lambda: M.moe_expert_act_backward(L, g, z, act="silu"), "preact must have shape [12, 8]"),
        (lambda: M.moe_expert_act_backward(L, g, act="silu"), "preact is required"),
        (lambda: M.moe_expert_act_backward(L, g, z, gated=True, need_w=True), "w is required"),
        (lambda: M.moe_expert_act_backward(L, g, z, gated=True, bias_dtype=torch.float16), "bias_dtype must be"),
        (lambda: M.moe_expert_act_dgrad(L, z, w[:, :15]), "weights must have shape [4, 16, *]"),
        (lambda: M.moe_expert_act_dgrad(L, z, w, out=g[:11]), "out must have shape [12, 8]"),
        (lambda: M.moe_expert_gemm_act(L, x, w), "on the GPU"),
    ]:
        with pytest.raises(ValueError) as err:
            call()
        assert text in str(err.value), (text, str(err.value))
