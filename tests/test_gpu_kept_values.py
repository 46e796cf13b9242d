"""Values kept in float32 between an expert product's forward and backward, on the GPU
against the float64 oracle.

Tolerances as in tests/test_gpu_expert_act.py, with u = 2^-24: z, a float32 sum of m products
and a bias, is off by at most dz = (m + 3) 2u of the sum of their magnitudes. Kept in float32
nothing else happens to it, so a gradient is off by what the activation's own float32 error
(act_err) and dz make of it: act' moves by at most 0.8 dz (gelu'' peaks at 2 phi(0) = 0.798,
silu'' at 1/2, the tanh form's below 0.9: 0.9 for all), act by at most 1.13 dz. Rounding z to
the element type first would put half a step of it, 2^-9 |z| for bf16, in the place of dz.
"""
import numpy as np
import pytest
import torch

import combine_moe_gate_amd as M
import combine_moe_gate_amd.autograd as A
import oracle
import workloads as W
from oracle import epilogue as E
from tests.gpu_util import assert_bits_equal, to_dev, to_host
from tests.test_gpu_expert_act import U, absolute, act_err, announce, rand, real, within

pytestmark = pytest.mark.gpu

CASES = [
    # s, m, n, e, k, capacity, pad, dtype, act, gated, bias, weighted, gather
    (1, 8, 8, 3, 2, 0, 1, "bf16", "silu", True, None, True, True),          # smallest rows
    (1, 520, 72, 16, 8, 0, 1, "f16", "gelu", False, "f32", True, True),     # one token
    (40, 264, 200, 2, 2, 0, 1, "bf16", "gelu_tanh", True, "own", True, False),
    (200, 72, 64, 16, 2, 0, 16, "bf16", "relu", False, "own", True, True),  # padded segments
    (1000, 136, 264, 8, 3, 200, 1, "f16", "silu", True, "f32", True, True), # drops, ragged columns
    (2000, 64, 40, 4, 2, 0, 1, "bf16", "none", True, "f32", True, True),
    (1000, 72, 1096, 8, 3, 200, 1, "bf16", "gelu", True, "f32", True, True),  # the large tiles
    (600, 136, 2056, 3, 1, 0, 64, "f16", "silu", False, None, True, False),
    (300, 72, 520, 700, 8, 6, 1, "bf16", "silu", True, "own", True, True),    # rows of many experts, mostly empty
]


def inputs(case):
    s, m, n, e, k, cap, pad, dtype, name, gated, bias, weighted, gather = case
    rng = np.random.default_rng(s + m + n)
    idx = W.random_idx(rng, s, e, k)
    L = oracle.dispatch_layout(idx, e, cap, pad_multiple=pad)
    Lg = M.moe_dispatch_layout(to_dev(idx), e, cap, pad_multiple=pad)
    nz = 2 * n if gated else n
    a, wts = rand(rng, (s if gather else L.rows, m), dtype), W.expert_weights(s + n, e, nz, m, dtype)
    b = None if bias is None else rng.standard_normal((e, nz)).astype(np.float32) if bias == "f32" else rand(rng, (e, nz), dtype)
    return L, Lg, a, wts, b, W.random_weights(rng, s, k) if weighted else None, rand(rng, (L.rows, n), dtype)


def dev(t, dtype):
    return None if t is None else to_dev(t, dtype if t.dtype != np.float32 else None)


def gradients(L, g64, z, dz, name, gated, w):
    """The oracle's gradients from z, and how far a float32 backward from a z off by dz may be:
    of grad_preact before its rounding, of grad_bias and of grad_w."""
    n = g64.shape[1]
    want = oracle.expert_act_backward(L, g64, z, name, gated, w)
    rw = np.abs(E.row_weights(L, w))[:, None]
    f, d = E.act(name, z[:, :n])
    ef, ed = act_err(name, z[:, :n])
    ef, ed = ef + 1.13 * dz[:, :n], ed + (0 if name in ("none", "relu") else 0.9) * dz[:, :n]
    ag = rw * np.abs(g64)
    if gated:
        up, dup = np.abs(z[:, n:]), dz[:, n:]
        tol = np.concatenate([ag * ((up + dup) * (ed + 4 * U * np.abs(d)) + dup * np.abs(d)), ag * (ef + 4 * U * np.abs(f))], 1)
        tol_u = (up + dup) * ef + np.abs(f) * dup + 4 * U * np.abs(f) * up
    else:
        tol, tol_u = ag * (ed + 4 * U * np.abs(d)), ef + 4 * U * np.abs(f)
    tol_b = np.zeros_like(want[1])
    for x, rows in E.segments(L):
        tol_b[x] = (tol[rows] + 24 * U * np.abs(want[0][rows])).sum(0)
    row = (np.abs(g64) * (tol_u + 16 * U * np.abs(E.finish(z, name, gated)))).sum(1)
    return want, (tol, tol_b + U * np.abs(want[1]), np.where(L.dst >= 0, row[np.where(L.dst >= 0, L.dst, 0)], 0))


@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-{c[8]}" for c in CASES])
def test_gradients_start_from_the_forward_s_values(case):
    announce("kept float32", *case)
    s, m, n, e, k, cap, pad, dtype, name, gated, bias, weighted, gather = case
    L, Lg, a, wts, b, w, g = inputs(case)
    placed = L.src >= 0
    nz = wts.shape[1]
    kw = dict(gather=gather, bias=dev(b, dtype), act=name, gated=gated, w=dev(w, dtype))
    ad, wd, gd = dev(a, dtype), dev(wts, dtype), dev(g, dtype)
    out, pre = M.moe_expert_gemm_act(Lg, ad, wd, save_preact=True, preact_dtype=torch.float32, **kw)
    big = torch.full((L.rows + 2, nz), 3.0, device="cuda")  # rows beside it that nothing may touch
    again = M.moe_expert_gemm_act(Lg, ad, wd, preact=big[1:-1], **kw)
    assert again[1].dtype == torch.float32 and torch.equal(again[1], pre) and (big[0] == 3).all() and (big[-1] == 3).all()
    narrow = M.moe_expert_gemm_act(Lg, ad, wd, save_preact=True, **kw)
    assert torch.equal(narrow[0], out) and torch.equal(again[0], out), "the output does not depend on what is kept"
    assert_bits_equal(to_host(narrow[1]), to_host(pre.to(narrow[1].dtype)), "and the narrow values are these, rounded")

    rb = None if b is None else real(b, dtype)
    _, z = oracle.expert_gemm_act(L, a, wts, dtype, gather, rb, name, gated, w)
    _, mag = oracle.expert_gemm_act(L, absolute(a, dtype), absolute(wts, dtype), dtype, gather, None if rb is None else np.abs(rb))
    dz = (m + 3) * 2 * U * mag
    within(to_host(pre), z, dz, "f32", "kept values")
    assert not to_host(pre)[~placed].view(np.uint32).any(), "unfilled rows not +0"

    # the backward at the kept values themselves, whatever lies in rows no route fills
    zk = pre.clone()
    zk[torch.from_numpy(~placed).cuda()] = float("nan")
    z32 = np.where(placed[:, None], to_host(pre).astype(np.float64), 0)
    g64 = np.where(placed[:, None], oracle.to_f32(g, dtype).astype(np.float64), 0)
    got = M.moe_expert_act_backward(Lg, gd, zk, act=name, gated=gated, w=kw["w"], need_w=weighted, bias_dtype=torch.float32,
                                    need_residual=True)
    want, tol = gradients(L, g64, z32, np.zeros_like(z32), name, gated, w)
    within(to_host(got[0]), want[0], np.where(placed[:, None], tol[0], 0), dtype, "grad_preact")
    assert not oracle.to_f32(to_host(got[0])[~placed], dtype).view(np.uint32).any()
    within(to_host(got[1]), want[1], tol[1], "f32", "grad_bias")
    within(to_host(got[2]), want[2], tol[2], "f32", "grad_w")
    assert_bits_equal(to_host(got[3]), np.where(placed[:, None], g, np.zeros((), g.dtype)), "grad_residual")

    # and through autograd, against the exact z: float32 all the way to a float32 bias and w
    b32 = torch.zeros((e, nz), device="cuda") if b is None else to_dev(rb.astype(np.float32))
    leaves = [t.detach().requires_grad_() for t in (ad, wd, b32, kw["w"])]
    y = A.expert_linear(leaves[0], leaves[1], Lg, bias=leaves[2], act=name, gated=gated, w=leaves[3], gather=gather,
                        preact_dtype=torch.float32)
    assert torch.equal(y, out)
    grads = torch.autograd.grad(y, leaves, gd)
    want, tol = gradients(L, g64, z, dz, name, gated, w)
    if name != "relu":  # whose slope jumps: a z near 0 may lie on either side
        within(to_host(grads[2]), want[1], tol[1], "f32", "bias gradient")
    within(to_host(grads[3]), want[2], tol[2], "f32", "weight gradient")
    gz = M.moe_expert_act_backward(Lg, gd, pre, act=name, gated=gated, w=kw["w"])[0]
    ga = M.moe_expert_act_dgrad(Lg, gz, wd)
    assert torch.equal(grads[0], M.moe_dispatch_backward(Lg, ga) if gather else ga)
    assert torch.equal(grads[1], M.moe_expert_gemm_wgrad(Lg, ad, gz, gather=gather, out_dtype=wd.dtype))


def test_replays_from_a_graph():
    """A training step with float32 kept values in a graph, eager steps between the replays."""
    announce("kept float32 graph")
    rng = np.random.default_rng(5)
    s, m, n, e, k = 300, 72, 136, 8, 2
    idx = to_dev(W.random_idx(rng, s, e, k))
    x, up = to_dev(rand(rng, (s, m), "bf16"), "bf16"), to_dev(W.expert_weights(1, e, 2 * n, m, "bf16"), "bf16")
    g = to_dev(rand(rng, (s * k, n), "bf16"), "bf16")
    L = M.moe_dispatch_layout(idx, e, 0)

    def step():
        leaves = [t.detach().requires_grad_() for t in (x, up)]
        y = A.expert_linear(*leaves, L, act="silu", gated=True, preact_dtype=torch.float32)
        return (y.detach(), *torch.autograd.grad(y, leaves, g))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for rep in range(3):
        x.copy_(to_dev(rand(rng, (s, m), "bf16"), "bf16"))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs, want)), f"replay {rep}"


@pytest.mark.parametrize("n", [8, 4104])
@pytest.mark.parametrize("name", E.ACTS)
def test_values_past_f16_stay_finite(name, n):
    """z = -70000 and -200 in the gate, 70000 in the up half: every activation but none makes 0 of
    them, so the output, the gradients and the route weight's are 0 and not NaN. An infinite z
    stays infinite."""
    announce("kept values past f16", name, n)
    s = 300
    L = M.moe_dispatch_layout(torch.zeros((s, 1), dtype=torch.int32, device="cuda"), 1, 0)
    x = torch.zeros((s, 8), dtype=torch.float16, device="cuda")
    x[:, 0], x[:, 1] = 200, 1
    wts = torch.zeros((1, 2 * n, 8), dtype=torch.float16, device="cuda")
    wts[0, :n:2, 0], wts[0, 1:n:2, 1], wts[0, n:, 0] = -350, -200, 350
    w = torch.ones((s, 1), device="cuda")
    kw = dict(act=name, gated=True, w=w)
    out, pre = M.moe_expert_gemm_act(L, x, wts, save_preact=True, **kw)
    want = torch.full((n,), -65504.0)
    want[1::2] = -200
    assert torch.equal(pre.cpu().float(), torch.cat([want, torch.full((n,), 65504.0)]).expand(s, -1))
    gz, gb, gw, _ = M.moe_expert_act_backward(L, torch.ones_like(out), pre, need_w=True, bias_dtype=torch.float32, **kw)
    if name != "none":
        assert not out.any() and not gz.any() and not gb.any() and not gw.any()
    x[:, 0] = float("inf")
    _, pre = M.moe_expert_gemm_act(L, x, wts, save_preact=True, **kw)
    assert torch.isneginf(pre[:, :n:2]).all() and torch.isposinf(pre[:, n:]).all()


def test_empty_batch_and_capacity_rows():
    announce("kept float32 empty")
    idx = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    w = torch.randn((4, 16, 8), device="cuda").to(torch.bfloat16)
    for cap in (0, 3):
        L = M.moe_dispatch_layout(idx, 4, cap)
        out, pre = M.moe_expert_gemm_act(L, torch.empty((0, 8), dtype=torch.bfloat16, device="cuda"), w, act="silu", gated=True,
                                         preact=torch.full((L.rows, 16), 9.0, device="cuda"))
        assert pre.dtype == torch.float32 and not pre.any() and not out.any()
        gz, gb, _, _ = M.moe_expert_act_backward(L, out, pre, act="silu", gated=True, bias_dtype=torch.float32)
        assert gz.shape == pre.shape and gz.dtype == torch.bfloat16 and not gz.any() and not gb.any()


def test_more_bytes_than_32_bits_count():
    """9.2 GB of kept values, 2.3e9 of them: both ends, forward and backward."""
    announce("kept float32 9.2 GB")
    s, m, n, e, k = 70000, 64, 4096, 8, 8
    gen = torch.Generator("cuda").manual_seed(3)
    idx = torch.rand((s, e), generator=gen, device="cuda").argsort(1).int()
    x = torch.randn((s, m), generator=gen, device="cuda").to(torch.bfloat16)
    wts = (torch.randn((e, n, m), generator=gen, device="cuda") / 8).to(torch.bfloat16)
    L = M.moe_dispatch_layout(idx, e, 0)
    out, pre = M.moe_expert_gemm_act(L, x, wts, act="silu", save_preact=True, preact_dtype=torch.float32)
    gz, gb, _, _ = M.moe_expert_act_backward(L, out, pre, act="silu", bias_dtype=torch.float32)
    for rows in (slice(0, 50), slice(L.rows - 50, L.rows)):
        r = torch.arange(L.rows, device="cuda")[rows]
        ex = torch.searchsorted(L.offsets[1:].long(), r, right=True)
        p = x[L.src[rows].long()].double()[:, None, :] * wts[ex].double()
        assert ((pre[rows].double() - p.sum(2)).abs() <= (m + 3) * 2 * U * p.abs().sum(2)).all()
        z, g = pre[rows].double(), out[rows].double()
        sg = torch.sigmoid(z)
        want = g * sg * (1 + z * (1 - sg))
        # act_err's slope error, and half a step of bf16
        eps = U * (16 + 8 * z.abs() * (1 - sg)) * (1 + 2 * z.abs()) + 8 * U * (1 + z.abs())
        assert ((gz[rows].double() - want).abs() <= 2.0 ** -8 * want.abs() + g.abs() * sg * eps + 1e-30).all()
    assert torch.isfinite(gb).all()
