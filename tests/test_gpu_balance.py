"""The router's balance loss, its counts and its gradient on the GPU against the float64
oracle.

Tolerances, with u = 2^-24 (half a float32 step). A probability is exp2((l - top) log2 e) /
sum: the subtraction, the constant and the product each put at most u D (D = top - l) on the
exponent's argument, at most 4 u D and 4 u for the hardware exponential on the value; the sum
of up to 1024 such terms adds their mean error, 4 u E (E = sum_x p_x D_x), and 22 u for its
16 steps in a lane and 6 across lanes; the reciprocal and the product 3 u. So a probability
is off by at most rel = u (4 D + 4 E + 32) of itself. logsumexp = top + ln(sum): off by at
most lse_err = u (4 E + 26 + 4 ln(1024) + |lse|). Sums over a tile's tokens add at most 64 + 8
steps of u each of the sum; the rest is float64.
"""
import ctypes

import numpy as np
import pytest
import torch

import combine_moe_gate_amd as M
import combine_moe_gate_amd.autograd as A
import oracle
import workloads as W
from oracle.router import group_tokens, softmax_row

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def announce(*what):
    print("CASE", *what, flush=True)


def bounds(logits, idx, mask, groups, gl, gz):
    """The oracle's results and how far each may be off."""
    s, e = logits.shape
    k = idx.shape[1]
    b = oracle.balance_loss(logits, idx, mask, groups)
    grad = oracle.balance_loss_backward(logits, b, k, gl, gz, mask, groups)
    t_probs, t_loss, t_z, t_grad = np.zeros(b.probs.shape), np.zeros(len(b.z)), np.zeros(len(b.z)), np.zeros((s, e))
    for i, tokens in enumerate(group_tokens(s, mask, groups)):
        n = max(1, len(tokens))
        c = b.counts[i]
        for t in tokens:
            p, lse = softmax_row(logits[t])
            l64 = logits[t].astype(np.float64)
            D = np.where(p > 0, l64.max() - np.where(np.isfinite(l64), l64, l64.max()), 0.0)
            E = float((p * D).sum())
            rel = U * (4 * D + 4 * E + 32)
            lse_err = U * (4 * E + 26 + 4 * np.log(1024) + abs(lse))
            t_probs[i] += p * rel / n
            t_z[i] += 2 * abs(lse) * lse_err / n
            off = np.abs(gl[i]) * e / (k * n * n) * np.abs(c - k * n / e)
            zt = abs(gz[i]) * 2 / n
            # the shifted counts and their scale are rounded once; the dot's 22 steps; three operations
            dot, dot_err = (p * off).sum(), (p * off * (rel + 24 * U)).sum()
            t_grad[t] = p * (rel * (off + dot + zt * abs(lse)) + dot_err + zt * lse_err
                             + 4 * U * (off + dot + zt * abs(lse)))
        t_probs[i] += 73 * U * b.probs[i]
        t_loss[i] = e / (k * n) * (c * t_probs[i]).sum() + U * b.loss[i]
        t_z[i] += U * b.z[i]
    return b, grad, (t_probs, t_loss, t_z, t_grad + 1e-44)


def check(got, want, tol, what):
    got = got.detach().cpu().numpy().astype(np.float64)
    # what float32 cannot hold (2^128 - 2^103 and up) rounds to infinity: (3e38)^2 in a mean of squares
    huge = np.abs(want) >= 2.0 ** 128 - 2.0 ** 103
    assert np.array_equal(got[huge], np.copysign(np.inf, want[huge])), what
    got, want, tol = got[~huge], want[~huge], tol[~huge]
    bad = np.argwhere(~(np.abs(got - want) <= tol))
    assert len(bad) == 0, (f"{what}: {len(bad)} outside the bound, first {tuple(bad[0])}: got {got[tuple(bad[0])]!r} "
                           f"want {want[tuple(bad[0])]!r} tol {tol[tuple(bad[0])]!r}")


def run_case(logits, idx, mask, groups, seed=0):
    g = 1 if groups is None else len(groups) - 1
    rng = np.random.default_rng(seed)
    gl, gz = rng.uniform(-2, 2, g).astype(np.float32), rng.uniform(-1, 1, g).astype(np.float32)
    dev = [None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (logits, idx, mask, gl, gz)]
    gd = None if groups is None else torch.tensor(groups, dtype=torch.int32, device="cuda")
    ld, idd, md, gld, gzd = dev
    out = M.moe_balance_loss(ld, idd, md, gd)
    grad = M.moe_balance_loss_backward(ld, out[0], out[1], idx.shape[1], gld, gzd, md, gd)
    b, want_grad, (t_probs, t_loss, t_z, t_grad) = bounds(logits, idx, mask, groups, gl.astype(np.float64),
                                                           gz.astype(np.float64))
    assert np.array_equal(out[0].cpu().numpy(), b.counts), "counts"
    assert np.array_equal(out[1].cpu().numpy(), b.tokens), "tokens"
    check(out[2], b.probs, t_probs, "probs")
    check(out[3], b.loss, t_loss, "loss")
    check(out[4], b.z, t_z, "z")
    check(grad, want_grad, t_grad, "grad")
    return out, grad


CASES = [
    # s, e, k, groups, masked share
    (0, 8, 2, None, 0.0),
    (0, 8, 2, [0, 0, 0], 0.0),
    (1, 1, 1, None, 0.0),
    (1, 8, 2, None, 0.0),
    (1, 1024, 16, None, 0.0),
    (256, 8, 2, None, 0.0),             # one launch
    (128, 128, 8, None, 0.0),           # the largest batch of one launch
    (129, 128, 8, None, 0.0),           # and one token more: two
    (1000, 16, 4, None, 0.3),
    (1000, 7, 3, None, 0.0),            # rows no 16-byte load fits
    (700, 60, 4, None, 0.1),
    (700, 61, 4, [0, 1, 350, 700], 0.1),
    (515, 129, 5, None, 0.0),           # three launches
    (300, 256, 8, [0, 300], 0.0),
    (130, 500, 8, None, 0.5),
    (97, 1024, 16, [0, 0, 50, 50, 97], 0.2),
    (90, 1023, 16, None, 0.0),
    (3000, 64, 4, list(range(0, 3001, 3)), 0.2),            # a thousand groups
    (3000, 32, 2, [5, 5, 31, 32, 33, 96, 1500, 2990], 0.1), # tokens before and after every group
    (200, 32, 2, None, 1.0),            # nothing but padding
    (200, 32, 2, [50, 170], 0.2),       # one group of part of the batch, in one launch
    (200, 32, 2, [200, 200], 0.0),      # and of none of it
]


@pytest.mark.parametrize("s,e,k,groups,masked", CASES)
def test_balance_loss_matches_the_oracle(s, e, k, groups, masked):
    announce("balance", s, e, k, None if groups is None else len(groups) - 1, masked)
    rng = np.random.default_rng(s + e + k)
    logits = (rng.standard_normal((s, e)) * 2).astype(np.float32)
    idx = W.random_idx(rng, s, e, k)
    mask = rng.random(s) >= masked if masked else None
    run_case(logits, idx, mask, groups)


def test_infinities_nan_and_bad_routes():
    announce("balance infinities")
    rng = np.random.default_rng(5)
    s, e, k = 400, 40, 3
    logits = rng.standard_normal((s, e)).astype(np.float32)
    idx = W.random_idx(rng, s, e, k)
    mask = np.ones(s, bool)
    logits[::7, :20] = -np.inf                              # experts a token may not choose
    logits[5] = -np.inf                                     # a token that may choose none
    logits[6] = np.finfo(np.float32).min                    # the type's lowest value everywhere
    logits[8, 1:] = np.finfo(np.float32).min
    logits[10] = rng.standard_normal(e) * 1e4               # one expert takes all
    logits[11] = 3e38
    idx[20], idx[21], idx[22] = (1, 1, 2), (-1, 40, 3), (2 ** 31 - 1, -2 ** 31, 0)
    for t, v in ((30, np.nan), (31, np.inf), (399, np.nan)):  # padding may hold anything
        logits[t], mask[t], idx[t] = v, False, -7
    run_case(logits, idx, mask, [0, 100, 400])
    run_case(logits, idx, mask, None)


def test_nan_stays_in_its_group():
    announce("balance nan")
    rng = np.random.default_rng(6)
    logits = rng.standard_normal((100, 24)).astype(np.float32)
    logits[40, 3] = np.nan
    logits[70, 3] = np.inf
    idx = W.random_idx(rng, 100, 24, 2)
    ld, idd = torch.from_numpy(logits).cuda(), torch.from_numpy(idx).cuda()
    groups = torch.tensor([0, 30, 60, 100], dtype=torch.int32, device="cuda")
    counts, tokens, probs, loss, z = M.moe_balance_loss(ld, idd, groups=groups)
    assert torch.isfinite(loss).tolist() == [True, False, False] == torch.isfinite(z).tolist()
    assert torch.isfinite(probs[0]).all() and counts.sum(1).tolist() == [60, 60, 80]
    ones = torch.ones(3, device="cuda")
    grad = M.moe_balance_loss_backward(ld, counts, tokens, 2, ones, ones, groups=groups)
    bad = (~torch.isfinite(grad)).any(1).nonzero().flatten().tolist()
    assert bad == [40, 70]


def test_rows_off_16_bytes_and_uint8_masks():
    """Logits that start 4 bytes past a 16-byte boundary take the other loads: equal bits."""
    announce("balance misaligned")
    rng = np.random.default_rng(7)
    for s, e in ((300, 64), (200, 256)):
        flat = torch.from_numpy(rng.standard_normal(s * e + 1).astype(np.float32)).cuda()
        ld = flat[1:].view(s, e)
        idx = torch.from_numpy(W.random_idx(rng, s, e, 2)).cuda()
        mask = torch.from_numpy(rng.random(s) < 0.8).cuda()
        run_case(ld.cpu().numpy(), idx.cpu().numpy(), mask.cpu().numpy(), None)
        got = M.moe_balance_loss(ld, idx, mask)
        run_case(ld.cpu().numpy(), idx.cpu().numpy(), mask.cpu().numpy(), [0, s])
        assert all(torch.equal(a, b) for a, b in zip(got, M.moe_balance_loss(ld, idx, mask.to(torch.uint8))))
        want, _, tol = bounds(ld.cpu().numpy(), idx.cpu().numpy(), mask.cpu().numpy(), None, np.zeros(1), np.zeros(1))
        check(got[2], want.probs, tol[0], "probs")
        # the gradient of misaligned rows into misaligned rows
        out = torch.empty(s * e + 1, device="cuda")[1:].view(s, e)
        one = torch.ones(1, device="cuda")
        M.moe_balance_loss_backward(ld, got[0], got[1], 2, one, one, mask, out=out)
        _, g, t = bounds(ld.cpu().numpy(), idx.cpu().numpy(), mask.cpu().numpy(), None, np.ones(1), np.ones(1))
        check(out, g, t[3], "grad")


def test_same_results_every_time_and_beside_another_stream():
    announce("balance determinism")
    rng = np.random.default_rng(8)
    logits = torch.from_numpy(rng.standard_normal((20000, 128)).astype(np.float32)).cuda()
    idx = torch.from_numpy(W.random_idx(rng, 20000, 128, 8)).cuda()
    one = torch.ones(1, device="cuda")
    first = M.moe_balance_loss(logits, idx)
    grad = M.moe_balance_loss_backward(logits, first[0], first[1], 8, one, one)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for st in streams:
            with torch.cuda.stream(st):
                o = M.moe_balance_loss(logits, idx)
                got.append((*o, M.moe_balance_loss_backward(logits, o[0], o[1], 8, one, one)))
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(a, b) for a, b in zip(o, (*first, grad)))


@pytest.mark.parametrize("s,e,groups", [(64, 8, None), (5000, 200, [0, 17, 4000, 5000])])
def test_replays_from_a_graph(s, e, groups):
    announce("balance graph", s, e)
    rng = np.random.default_rng(9)
    logits = torch.from_numpy(rng.standard_normal((s, e)).astype(np.float32)).cuda()
    idx = torch.from_numpy(W.random_idx(rng, s, e, 2)).cuda()
    gd = None if groups is None else torch.tensor(groups, dtype=torch.int32, device="cuda")
    w = torch.rand(1 if groups is None else len(groups) - 1, device="cuda")

    def step():
        o = M.moe_balance_loss(logits, idx, groups=gd)
        return (*o, M.moe_balance_loss_backward(logits, o[0], o[1], 2, w, w, groups=gd))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for rep in range(3):
        logits.copy_(torch.from_numpy(rng.standard_normal((s, e)).astype(np.float32)))
        want = step()
        torch.cuda.synchronize()
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), f"replay {rep}"


def test_two_graphs_share_a_workspace():
    """Replayed in turn on one stream, as two captured parts of one program are."""
    announce("balance two graphs")
    rng = np.random.default_rng(21)
    parts, workspace = [], None
    for s, e, groups in ((6000, 40, None), (3000, 72, [0, 100, 100, 3000])):
        logits = torch.from_numpy(rng.standard_normal((s, e)).astype(np.float32)).cuda()
        idx = torch.from_numpy(W.random_idx(rng, s, e, 3)).cuda()
        gd = None if groups is None else torch.tensor(groups, dtype=torch.int32, device="cuda")
        parts.append((logits, idx, gd))
    need = [M.lib().moe_balance_workspace_bytes(p[0].shape[0], p[0].shape[1], 1 if p[2] is None else len(p[2]) - 1) for p in parts]
    assert min(need) > 0
    workspace = torch.full((max(need),), 0xA5, dtype=torch.uint8, device="cuda")
    run = lambda p, ws: M.moe_balance_loss(p[0], p[1], groups=p[2], workspace=ws)  # noqa: E731
    graphs, outs = [], []
    for p in parts:
        run(p, workspace)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(run(p, workspace))
    for rep in range(3):
        for p in parts:
            p[0].copy_(torch.from_numpy(rng.standard_normal(tuple(p[0].shape)).astype(np.float32)))
        want = [run(p, None) for p in parts]
        for g in (graphs if rep % 2 == 0 else graphs[::-1]):
            g.replay()
        torch.cuda.synchronize()
        for o, v in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, v)), f"replay {rep}"


def test_autograd_gives_the_gradient():
    announce("balance autograd")
    rng = np.random.default_rng(10)
    logits = rng.standard_normal((200, 32)).astype(np.float32)
    ld = torch.from_numpy(logits).cuda().requires_grad_()
    idx, w = A.route(ld, 4)
    groups = torch.tensor([0, 90, 200], dtype=torch.int32, device="cuda")
    loss, z, counts = A.balance_loss(ld, idx, groups=groups)
    assert not counts.requires_grad and counts.sum().item() == 800
    (0.5 * loss.sum() + 0.25 * z.sum()).backward()
    gl, gz = np.full(2, 0.5), np.full(2, 0.25)
    _, want, tol = bounds(logits, idx.cpu().numpy(), None, [0, 90, 200], gl, gz)
    check(ld.grad, want, tol[3], "both losses")
    (grad,) = torch.autograd.grad(A.balance_loss(ld, idx, groups=groups)[0].sum(), ld)  # z unused
    _, want, tol = bounds(logits, idx.cpu().numpy(), None, [0, 90, 200], np.ones(2), np.zeros(2))
    check(grad, want, tol[3], "load balance alone")
    (grad,) = torch.autograd.grad(A.balance_loss(ld.t().contiguous().t(), idx)[1].sum(), ld)  # strided logits
    _, want, tol = bounds(logits, idx.cpu().numpy(), None, None, np.zeros(1), np.ones(1))
    check(grad, want, tol[3], "z alone")
    with pytest.raises(RuntimeError):
        g = torch.autograd.grad(A.balance_loss(ld, idx)[0].sum(), ld, create_graph=True)[0]
        g.sum().backward()


def test_counts_are_the_layouts():
    announce("balance counts")
    rng = np.random.default_rng(11)
    idx = torch.from_numpy(W.skewed_idx(rng, 3000, 40, 3, 7)).cuda()
    idx[5], idx[6, 1] = -1, idx[6, 0]
    counts = M.moe_balance_loss(torch.randn((3000, 40), device="cuda"), idx)[0]
    assert torch.equal(counts[0], M.moe_dispatch_layout(idx, 40, 100).counts)


def test_falling_offsets_stay_in_bounds():
    """Offsets that are no rising sequence give no particular numbers, and write only the
    outputs: every tile and group index the kernels form lies within its array."""
    announce("balance falling offsets")
    logits, idx = torch.randn((500, 16), device="cuda"), torch.zeros((500, 1), dtype=torch.int32, device="cuda")
    for offs in ([0, 400, 100, 500], [500, 0, -5, 700], [-9, 2 ** 31 - 1]):
        groups = torch.tensor(offs, dtype=torch.int32, device="cuda")
        g = len(offs) - 1
        guard = [torch.full((n + 64,), 7, dtype=torch.int32, device="cuda") for n in (g * 16, g, g * 16, g, g)]
        outs = [guard[0][32:32 + g * 16].view(g, 16), guard[1][32:32 + g],
                guard[2][32:32 + g * 16].view(torch.float32).view(g, 16), guard[3][32:32 + g].view(torch.float32),
                guard[4][32:32 + g].view(torch.float32)]
        M.moe_balance_loss(logits, idx, groups=groups, out=outs)
        grad = torch.full((502, 16), 7.0, device="cuda")
        M.moe_balance_loss_backward(logits, outs[0], outs[1], 1, torch.ones(g, device="cuda"), None, groups=groups,
                                    out=grad[1:501])
        torch.cuda.synchronize()
        for t in guard:
            assert (t[:32] == 7).all() and (t[-32:] == 7).all()
        assert (grad[0] == 7).all() and (grad[-1] == 7).all()


@pytest.mark.slow
def test_more_logits_than_32_bits_count():
    announce("balance 2.3e9 logits")
    s, e, k = 2_250_000, 1024, 2
    logits = torch.empty((s, e), device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    idx = torch.stack([torch.arange(s, device="cuda") % e, (torch.arange(s, device="cuda") + 5) % e], 1).int()
    one = torch.ones(1, device="cuda")
    counts, tokens, probs, loss, z = M.moe_balance_loss(logits, idx)
    grad = M.moe_balance_loss_backward(logits, counts, tokens, k, one, one)
    assert tokens.item() == s and torch.equal(counts[0].long(), torch.bincount(idx.flatten().long(), minlength=e))
    total = torch.zeros(e, dtype=torch.float64, device="cuda")
    for t in range(0, s, 50000):
        total += torch.softmax(logits[t:t + 50000].double(), 1).sum(0)
    # a tile holds 4395 tokens, 275 to each of a lane's 8 waves
    tol = U * (4 * 12 + 4 * 3 + 32 + 600) * (total / s)
    assert (torch.abs(probs[0].double() - total / s) <= tol).all()
    tail = logits[-300:].double()
    p, lse = torch.softmax(tail, 1), torch.logsumexp(tail, 1)
    dp = counts[0].double() * e / (k * float(s) ** 2)
    want = p * (dp - (p * dp).sum(1, keepdim=True) + 2 * lse[:, None] / s)
    assert (torch.abs(grad[-300:].double() - want) <= 1e-5 * p * (2 * lse[:, None] / s) + 1e-5 * want.abs()).all()


def test_refusals():
    announce("balance refusals")
    logits, idx = torch.randn((10, 8), device="cuda"), torch.zeros((10, 2), dtype=torch.int32, device="cuda")
    ok = M.moe_balance_loss(logits, idx)
    with pytest.raises(ValueError, match="contiguous"):
        M.moe_balance_loss(torch.randn((8, 10), device="cuda").t(), idx)
    groups = torch.tensor([0, 5, 10], dtype=torch.int32, device="cuda")
    with pytest.raises(M.MoeError, match="MOE_ERR_WORKSPACE"):
        M.moe_balance_loss(logits, idx, groups=groups, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(M.MoeError, match="k must be"):
        M.moe_balance_loss(logits, torch.zeros((10, 9), dtype=torch.int32, device="cuda"))
    with pytest.raises(M.MoeError, match="overlap"):
        M.moe_balance_loss_backward(logits, ok[0], ok[1], 2, torch.ones(1, device="cuda"), out=logits)
    with pytest.raises(ValueError, match="on the GPU"):
        M.moe_balance_loss(logits, idx.cpu())
    with pytest.raises(ValueError, match="at least two"):
        M.moe_balance_loss(logits, idx, groups=torch.zeros(1, dtype=torch.int32, device="cuda"))
