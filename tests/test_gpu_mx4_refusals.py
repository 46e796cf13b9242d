"""Strided tensors, and tensors of another device than the layout's, are refused by the 4-bit operators before the
library is called."""
import pytest
import torch

import combine_moe_gate_amd as M
from tests.test_gpu_expert_act import announce

pytestmark = pytest.mark.gpu


@pytest.fixture
def made(monkeypatch):
    L = M.moe_dispatch_layout(torch.zeros((6, 2), dtype=torch.int32, device="cuda"), 4, 3)  # 12 rows
    x = torch.zeros((6, 64), dtype=torch.bfloat16, device="cuda")
    w = M.moe_mx4_quantize(torch.zeros((4, 32, 64), device="cuda"))
    torch.cuda.synchronize()
    monkeypatch.setattr(M, "lib", lambda: pytest.fail("the library was called"))
    return L, x, w


def strided(t):
    """The same values in a tensor whose rows do not follow each other."""
    big = torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=t.dtype, device=t.device)
    big[..., ::2] = t
    return big[..., ::2]


def test_strided_tensors(made):
    announce("4-bit refusals, strided")
    L, x, (c, s) = made
    xq = torch.zeros((6, 32), dtype=torch.uint8, device="cuda"), torch.zeros((6, 2), dtype=torch.uint8, device="cuda")
    out = torch.zeros((12, 16), dtype=torch.uint8, device="cuda"), torch.zeros((12, 1), dtype=torch.uint8, device="cuda")
    g = torch.zeros((12, 32), dtype=torch.bfloat16, device="cuda")
    parts = torch.zeros((12, 2, 32), dtype=torch.bfloat16, device="cuda")
    wide_scale = torch.zeros((12, 2), dtype=torch.uint8, device="cuda")[:, :1]
    for call in (
        lambda: M.moe_mx4_quantize(strided(x)),
        lambda: M.moe_mx4_quantize(x.t().contiguous().t()),
        lambda: M.moe_mx4_quantize(x, codes=strided(xq[0])),
        lambda: M.moe_mx4_quantize(x, scales=strided(xq[1])),
        lambda: M.moe_mx4_dequantize(strided(xq[0]), xq[1]),
        lambda: M.moe_mx4_dequantize(xq[0], strided(xq[1])),
        lambda: M.moe_mx4_dequantize(*xq, out=strided(x)),
        lambda: M.moe_mx4_expert_gemm(L, strided(x), (c, s)),
        lambda: M.moe_mx4_expert_gemm(L, (strided(xq[0]), xq[1]), (c, s)),
        lambda: M.moe_mx4_expert_gemm(L, (xq[0], strided(xq[1])), (c, s)),
        lambda: M.moe_mx4_expert_gemm(L, x, (strided(c), s)),
        lambda: M.moe_mx4_expert_gemm(L, x, (c, strided(s))),
        lambda: M.moe_mx4_expert_gemm(L, x, (c.transpose(0, 1).contiguous().transpose(0, 1), s)),
        lambda: M.moe_mx4_expert_gemm(L, x, (c, s), quantize_out=True, out=(strided(out[0]), out[1])),
        lambda: M.moe_mx4_expert_gemm(L, x, (c, s), quantize_out=True, out=(out[0], wide_scale)),
        lambda: M.moe_mx4_expert_gemm(L, x, (c, s), out=strided(g)),
        lambda: M.moe_mx4_expert_gemm(L, x, (c, s), preact=strided(g)),
        lambda: M.moe_mx4_expert_gemm(L, x, (c, s), residual=strided(g)),
        lambda: M.moe_mx4_expert_gemm(L, x, (c, s), bias=strided(torch.zeros((4, 32), device="cuda"))),
        lambda: M.moe_mx4_expert_gemm(L, x, (c, s), w=strided(torch.zeros((6, 2), device="cuda"))),
        lambda: M.moe_mx4_expert_dgrad(L, strided(g), (c, s)),
        lambda: M.moe_mx4_expert_dgrad(L, strided(parts), (c, s)),
        lambda: M.moe_mx4_expert_dgrad(L, parts.transpose(0, 1).contiguous().transpose(0, 1), (c, s)),
        lambda: M.moe_mx4_expert_dgrad(L, g, (strided(c), s)),
        lambda: M.moe_mx4_expert_dgrad(L, g, (c, strided(s))),
        lambda: M.moe_mx4_expert_dgrad(L, g, (c, s), out=strided(torch.zeros((12, 64), device="cuda"))),
    ):
        with pytest.raises(ValueError, match="contiguous"):
            call()


def test_other_devices(made):
    announce("4-bit refusals, devices")
    L, x, (c, s) = made
    g = torch.zeros((12, 32), dtype=torch.bfloat16, device="cuda")
    for call in (
        lambda: M.moe_mx4_quantize(x, codes=torch.zeros((6, 32), dtype=torch.uint8)),
        lambda: M.moe_mx4_dequantize(c, s.cpu()),
        lambda: M.moe_mx4_expert_gemm(L, x.cpu(), (c, s)),
        lambda: M.moe_mx4_expert_gemm(L, x, (c, s.cpu())),
        lambda: M.moe_mx4_expert_dgrad(L, g, (c.cpu(), s)),
        lambda: M.moe_mx4_expert_dgrad(L, g, (c, s), out=torch.zeros((12, 64), dtype=torch.bfloat16)),
    ):
        with pytest.raises(ValueError, match="on the GPU"):
            call()
