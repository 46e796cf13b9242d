"""Refusals of the 4-bit entries and of their binding, before anything reaches a GPU (fake addresses:
only where there is none)."""
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


@no_gpu_only
def test_row_argument_checks(lib):
    def quant(x=at(0), rows=4, m=64, dtype=1, c=at(1), s=at(2, 3)):
        return lib.moe_mx4_quantize(x, rows, m, dtype, c, s, None)

    def back(x=at(0), rows=4, m=64, dtype=1, c=at(1), s=at(2, 3)):
        return lib.moe_mx4_dequantize(c, s, rows, m, dtype, x, None)

    for call in (quant, back):
        assert call(dtype=3) == 1 and call(dtype=-1) == 1
        assert call(rows=-1) == 1 and call(m=0) == 1 and call(m=-32) == 1
        assert call(m=48) == 5 and "multiple of 32" in lib.moe_last_error().decode()
        assert call(rows=1 << 60, m=32) == 2
        assert call(x=None) == 1 and call(c=None) == 1 and call(s=None) == 1
        assert call(x=at(0, 8)) == 5 and call(c=at(1, 4)) == 5
        for clash in (dict(c=at(0, 496)), dict(s=at(0, 511)), dict(s=at(1, 127)), dict(x=at(1, 112)), dict(x=at(2, 0))):
            assert call(**clash) == 1, clash
            assert "overlap" in lib.moe_last_error().decode()
        assert call(rows=0, x=None, c=None, s=None) == 0  # nothing to do


@no_gpu_only
def test_product_argument_checks(lib):
    s, e, k = 40, 8, 2
    st = _fake_handle(s, e, k, 0, 1 << 24, M.workspace_bytes(s, e, k, 0))

    def call(a=at(0), a_s=None, gather=1, w=at(1), w_s=at(2, 1), m=64, n=64, dtype=1, pdt=1, out=at(3), out_s=None, layout=st, **ep):
        q = M.Epilogue(ep.get("act", 0), ep.get("gated", 0), ep.get("bias"), ep.get("bias_dtype", 0),
                       ep.get("residual_gather", 0), ep.get("topk_w"), ep.get("residual"), ep.get("preact"))
        return lib.moe_mx4_expert_gemm(ctypes.byref(layout), a, a_s, gather, w, w_s, m, n, dtype, ctypes.byref(q), pdt,
                                       out, out_s, None)

    assert call(dtype=0) == 2 and call(dtype=7) == 2
    assert call(gather=2) == 1 and call(act=5) == 1 and call(gated=2) == 1 and call(residual_gather=3) == 1
    assert call(m=48) == 5 and call(m=0) == 1 and call(n=4) == 5
    assert call(n=40, out_s=at(4)) == 5 and "multiple of 32" in lib.moe_last_error().decode()
    assert call(a=None) == 1 and call(w=None) == 1 and call(w_s=None) == 1 and call(out=None) == 1
    assert call(a=at(0, 8)) == 5 and call(w=at(1, 8)) == 5 and call(out=at(3, 2)) == 5
    assert call(bias=at(5).value, bias_dtype=2) == 2 and call(bias=at(5, 4).value) == 5
    assert call(preact=at(6).value, pdt=2) == 2 and call(preact=at(6, 8).value) == 5 and call(residual=at(7, 8).value) == 5
    # 40 rows of 64: 5120 bytes (4-bit: 1280 and 80); the buffer's 80 rows: 10240 (2560, 160); weights 16384 and 1024
    clashes = [dict(out=at(0, 5104)), dict(out=at(1, 16368)), dict(out=at(2, 1008)), dict(out_s=at(3, 2559)),
               dict(preact=at(3, 10224).value), dict(residual=at(3, 64).value), dict(out_s=at(0, 5119)),
               dict(a_s=at(3, 10239)), dict(a_s=at(3, 2559), out_s=at(4)), dict(a_s=at(4, 150), out_s=at(4)),
               dict(preact=at(2, 1008).value), dict(preact=at(4).value, out_s=at(4, 100))]
    # the bias' 8 times 64 float32 values: 2048 bytes, 1024 in bf16; the 80 weights: 320
    clashes += [dict(bias=at(4).value, out=at(4, 2032)), dict(bias=at(4).value, bias_dtype=1, out_s=at(4, 1023)),
                dict(topk_w=at(4).value, out=at(4, 304)), dict(topk_w=at(4).value, preact=at(4, 304).value)]
    for clash in clashes:
        assert call(**clash) == 1, clash
        assert "overlap" in lib.moe_last_error().decode()
    assert call(layout=M.LayoutStruct()) == 4


@no_gpu_only
def test_input_gradient_argument_checks(lib):
    st = _fake_handle(40, 8, 2, 0, 1 << 24, M.workspace_bytes(40, 8, 2, 0))

    def call(g=at(0), w=at(1), w_s=at(2, 1), m=64, nz=64, dtype=1, out=at(3), layout=st):
        return lib.moe_mx4_expert_dgrad(ctypes.byref(layout), g, w, w_s, m, nz, dtype, out, None)

    assert call(dtype=0) == 2 and call(nz=4) == 5 and call(m=40) == 5 and call(m=0) == 1
    assert call(g=None) == 1 and call(w=None) == 1 and call(w_s=None) == 1 and call(out=None) == 1
    assert call(out=at(3, 8)) == 5 and call(w=at(1, 8)) == 5 and call(layout=M.LayoutStruct()) == 4
    for out in (at(0, 512), at(1, 16368), at(2, 1008)):
        assert call(out=out) == 1 and "overlap" in lib.moe_last_error().decode()


@no_gpu_only
def test_launch_limits(lib):
    """Grids of more than 2^32 work items are refused by name."""
    s = 1 << 24
    st = _fake_handle(s, 8, 8, 0, 1 << 40, M.workspace_bytes(s, 8, 8, 0))
    ep = M.Epilogue()
    assert lib.moe_mx4_expert_gemm(ctypes.byref(st), at(0), None, 1, at(1), at(2), 32, 1 << 24, 1, ctypes.byref(ep), 1, at(3), None, None) == 2
    assert lib.moe_mx4_expert_dgrad(ctypes.byref(st), at(0), at(1), at(2), 1 << 24, 32, 1, at(3), None) == 2
    assert "too large" in lib.moe_last_error().decode()


def test_binding_refuses_mismatched_tensors(monkeypatch):
    def refuse():
        raise AssertionError("the library was called with arguments the binding should have refused")
    monkeypatch.setattr(M, "lib", refuse)
    L = fake_layout()  # s=6, e=4, k=2, rows=12
    u8, bf = torch.uint8, torch.bfloat16

    def mx(*shape):
        return torch.zeros((*shape[:-1], shape[-1] // 2), dtype=u8), torch.zeros((*shape[:-1], shape[-1] // 32), dtype=u8)

    x, w, g = torch.zeros(6, 64, dtype=bf), mx(4, 48, 64), torch.zeros(12, 48, dtype=bf)
    for call, text in [
        (lambda: M.moe_mx4_quantize(torch.zeros(3, 40)), "whole blocks"),
        (lambda: M.moe_mx4_quantize(torch.zeros(3, 0)), "whole blocks"),
        (lambda: M.moe_mx4_quantize(torch.zeros(())), "whole blocks"),
        (lambda: M.moe_mx4_quantize(torch.zeros(3, 64, dtype=torch.float64)), "x must be"),
        (lambda: M.moe_mx4_quantize(torch.zeros(3, 64), codes=torch.zeros(3, 31, dtype=u8)), "codes must have shape [3, 32]"),
        (lambda: M.moe_mx4_quantize(torch.zeros(3, 64), scales=torch.zeros(3, 2)), "scales must be"),
        (lambda: M.moe_mx4_dequantize(torch.zeros(3, 24, dtype=u8), torch.zeros(3, 1, dtype=u8)), "whole blocks"),
        (lambda: M.moe_mx4_dequantize(torch.zeros(3, 32, dtype=u8), torch.zeros(3, 1, dtype=u8)), "scales must have shape [3, 2]"),
        (lambda: M.moe_mx4_dequantize(torch.zeros(3, 32), torch.zeros(3, 2, dtype=u8)), "codes must be"),
        (lambda: M.moe_mx4_dequantize(*mx(3, 64), dtype=torch.float64), "unsupported element type"),
        (lambda: M.moe_mx4_dequantize(*mx(3, 64), out=torch.zeros(3, 32)), "out must have shape [3, 64]"),
        (lambda: M.moe_mx4_expert_gemm(L, x.float(), w), "a must be"),
        (lambda: M.moe_mx4_expert_gemm(L, x, w, gather=False), "a must have shape [12, *]"),
        (lambda: M.moe_mx4_expert_gemm(L, torch.zeros(6, 40, dtype=bf), w), "whole blocks"),
        (lambda: M.moe_mx4_expert_gemm(L, x, mx(4, 48, 96)), "codes must have shape [4, *, 32]"),
        (lambda: M.moe_mx4_expert_gemm(L, x, (w[0], w[1][:, :, :1])), "scales must have shape [4, 48, 2]"),
        (lambda: M.moe_mx4_expert_gemm(L, mx(5, 64), w), "codes must have shape [6, *]"),
        (lambda: M.moe_mx4_expert_gemm(L, mx(12, 64), w, gather=False, dtype=torch.float32), "dtype must be"),
        (lambda: M.moe_mx4_expert_gemm(L, x, w, dtype=torch.float16), "dtype must be that of the rows"),
        (lambda: M.moe_mx4_expert_gemm(L, x, mx(4, 15, 64), gated=True), "even number of rows"),
        (lambda: M.moe_mx4_expert_gemm(L, x, w, gated=True, quantize_out=True), "whole blocks"),
        (lambda: M.moe_mx4_expert_gemm(L, x, mx(4, 64, 64), quantize_out=True, out=mx(12, 32)), "out: codes must have shape [12, 32]"),
        (lambda: M.moe_mx4_expert_gemm(L, x, w, bias=torch.zeros(4, 48).half()), "bias must be"),
        (lambda: M.moe_mx4_expert_gemm(L, x, w, act="tanh"), "act must be one of"),
        (lambda: M.moe_mx4_expert_gemm(L, x, w, w=torch.zeros(6, 3)), "w must have shape [6, 2]"),
        (lambda: M.moe_mx4_expert_gemm(L, x, w, residual=torch.zeros(12, 64, dtype=bf)), "residual must have shape [12, 48]"),
        (lambda: M.moe_mx4_expert_gemm(L, x, w, out=torch.zeros(12, 48)), "out must be"),
        (lambda: M.moe_mx4_expert_gemm(L, x, w, save_preact=True, preact_dtype=torch.float16), "preact_dtype must be"),
        (lambda: M.moe_mx4_expert_gemm(L, x, w, preact=torch.zeros(12, 24, dtype=bf)), "preact must have shape [12, 48]"),
        (lambda: M.moe_mx4_expert_dgrad(L, g.float(), w), "grad_preact must be"),
        (lambda: M.moe_mx4_expert_dgrad(L, g, mx(4, 40, 64)), "codes must have shape [4, 48, *]"),
        (lambda: M.moe_mx4_expert_dgrad(L, g, w, out=torch.zeros(12, 32, dtype=bf)), "out must have shape [12, 64]"),
        (lambda: M.moe_mx4_quantize(x), "on the GPU"),
        (lambda: M.moe_mx4_dequantize(*mx(3, 64)), "on the GPU"),
        (lambda: M.moe_mx4_expert_gemm(L, x, w), "on the GPU"),
        (lambda: M.moe_mx4_expert_dgrad(L, g, w), "on the GPU"),
    ]:
        with pytest.raises(ValueError) as err:
            call()
        assert text in str(err.value), (text, str(err.value))
    for call in (lambda: M.moe_mx4_quantize([1.0]), lambda: M.moe_mx4_dequantize(None, None), lambda: M.moe_mx4_expert_gemm(L, x, w[0]),
                 lambda: M.moe_mx4_expert_gemm(L, x, (w[0], None)), lambda: M.moe_mx4_expert_gemm(L, None, w),
                 lambda: M.moe_mx4_expert_dgrad(L, g, w[0]), lambda: M.moe_mx4_dequantize(w[0], None)):
        with pytest.raises(TypeError):
            call()


def test_binding_refuses_strided_and_other_devices(monkeypatch):
    monkeypatch.setattr(M, "lib", lambda: pytest.fail("the library was called"))
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="on the GPU"):
        M.moe_mx4_quantize(x)
