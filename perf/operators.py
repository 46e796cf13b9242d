"""Cases that measure the router's balance loss and the experts' products with their epilogue.

Three kinds of pass:

  balance   the load-balance and z losses of a router with the per-expert counts, and their gradient
            with respect to the logits (a training step's share of the router)
  gemm      one projection of every placed row by its expert, with bias, activation (plain or gated),
            route weight and residual applied before the one rounding (a forward pass; with few tokens,
            a decoding step)
  ffn_step  up projection (gated), down projection, combine, and the gradients of all inputs: a training
            step of the expert layer
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------------------------
# cases


def _balance(name, s, e, k, groups=1, masked=False):
    return {"name": name, "kind": "balance", "s": s, "e": e, "k": k, "groups": groups, "masked": masked}


def _gemm(name, s, m, n, e, k, dtype, act="none", gated=False, bias="none", weighted=False, residual="none",
          gather=True, capacity=0, pad=1, save=False, hot=False):
    """n: output features (a gated projection's weights have 2 n rows). bias: none, f32 or own (the element
    type). residual: none, rows (one for each buffer row) or tokens (gathered). save: the values before the
    activation are kept for a backward pass. hot: a tenth of the tokens prefer expert 0."""
    return {"name": name, "kind": "gemm", "s": s, "m": m, "n": n, "e": e, "k": k, "dtype": dtype, "act": act,
            "gated": gated, "bias": bias, "weighted": weighted, "residual": residual, "gather": gather,
            "capacity": capacity, "pad": pad, "save": save, "hot": hot}


def _ffn(name, s, m, n, e, k, dtype, act="silu", bias=True):
    return {"name": name, "kind": "ffn_step", "s": s, "m": m, "n": n, "e": e, "k": k, "dtype": dtype, "act": act,
            "bias": bias}


def listed():
    return [
        # a small router's training step, where launches and host time are the cost
        _balance("balance 256 tokens", 256, 8, 2),
        # the router of a large training batch
        _balance("balance 32768 tokens", 32768, 128, 8),
        # packed sequences of different lengths with padded tokens, a loss for each sequence
        _balance("balance packed and masked", 16381, 60, 4, groups=29, masked=True),
        # many small experts
        _balance("balance 512 experts", 65536, 512, 10),
        # decoding: one token's up projection, where the weights of its 8 experts are what is read
        _gemm("decode one token", 1, 4096, 1536, 128, 8, "bf16", act="silu", gated=True),
        # decoding a batch: the down projection, weighted, over rows that the up projection left
        _gemm("decode 24 tokens down", 24, 1408, 2816, 64, 6, "f16", bias="own", weighted=True, gather=False),
        # prompts: up projection of 4096 tokens
        _gemm("prompt 4096 tokens", 4096, 2816, 1408, 128, 8, "bf16", act="silu", gated=True),
        # the largest: a training batch's up projection with the values before the activation kept
        _gemm("training batch gated", 8192, 4096, 2048, 128, 8, "bf16", act="silu", gated=True, bias="own", save=True),
        # capacity-bounded routing with drops, bias, exact gelu and the tokens' own rows added
        _gemm("capacity gelu residual", 16384, 1024, 1024, 64, 4, "f16", act="gelu", bias="f32",
              residual="tokens", capacity=1024, hot=True),
        # odd sizes: ragged row and column tiles, padded segments, more experts than a power of two
        _gemm("ragged relu", 777, 264, 200, 129, 5, "bf16", act="relu", bias="f32", weighted=True,
              residual="rows", pad=16),
        # training steps of the whole expert layer: a small one and an ordinary one
        _ffn("layer step 1000 tokens", 1000, 520, 264, 16, 2, "bf16", act="gelu_tanh"),
        _ffn("layer step 8192 tokens", 8192, 2048, 1408, 64, 6, "bf16", bias=False),
    ]


def _log(rng, lo, hi, multiple=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(multiple, int(round(v / multiple)) * multiple)


def draw(rng):
    kind = rng.choice(["balance", "gemm", "gemm", "ffn_step"])
    e = rng.choice([8, 16, 60, 64, 128, 129, 160])
    k = rng.choice([1, 2, 3, 4, 6, 8])
    if kind == "balance":
        e = rng.choice([e, 384, 512])
        s = _log(rng, 1, 65536)
        c = _balance("", s, e, k, groups=_log(rng, 1, min(s, 64)), masked=rng.random() < 0.5)
    elif kind == "gemm":
        s = _log(rng, 1, 8192)
        m, n = _log(rng, 64, 4096, 8), _log(rng, 64, 2048, 8)
        capacity = 0 if rng.random() < 0.7 or s < 64 else -(-s * k // e)
        c = _gemm("", s, m, n, e, k, rng.choice(["bf16", "f16"]), act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                  gated=rng.random() < 0.5, bias=rng.choice(["none", "f32", "own"]), weighted=rng.random() < 0.5,
                  residual=rng.choice(["none", "rows", "tokens"]), gather=rng.random() < 0.6, capacity=capacity,
                  pad=1 if capacity or rng.random() < 0.7 else 16, save=rng.random() < 0.4, hot=rng.random() < 0.3)
    else:
        e = min(e, 64)
        s = _log(rng, 16, 8192)
        c = _ffn("", s, _log(rng, 64, 2048, 8), _log(rng, 64, 1408, 8), e, min(k, 6), rng.choice(["bf16", "f16"]),
                 act=rng.choice(["gelu", "gelu_tanh", "silu"]), bias=rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------
# inputs


def _routing(c, gen, hot=False):
    """Router logits, the k best experts of each token and their renormalised weights."""
    logits = torch.randn((c["s"], c["e"]), generator=gen, device="cuda")
    if hot:
        logits[torch.rand(c["s"], generator=gen, device="cuda") < 0.1, 0] += 3.0
    top, idx = torch.topk(logits, c["k"], dim=1)
    return logits, idx.to(torch.int32), torch.softmax(top, 1)


def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _weights(gen, e, rows, cols, dtype):
    """[e, rows, cols], drawn expert by expert: a float32 draw of all would take several times their room."""
    w = torch.empty((e, rows, cols), device="cuda", dtype=dtype)
    for x in range(e):
        w[x].normal_(0.0, cols ** -0.5, generator=gen)
    return w


def _plan(idx, e, capacity, pad):
    """Where each route's row goes: expert by expert, in token order within an expert; an expert's rows start
    at a multiple of `pad` (or of the capacity, past which routes are dropped). Also the rows as a table
    [experts with rows, most rows of one] for batched products, with `rows` where an expert has fewer."""
    s, k = idx.shape
    order = torch.sort(idx.reshape(-1).long(), stable=True)
    counts = torch.bincount(order.values, minlength=e)
    first = torch.cumsum(counts, 0) - counts
    slot = torch.arange(s * k, device="cuda") - first[order.values]
    size = torch.full_like(counts, capacity) if capacity else (counts + pad - 1) // pad * pad
    base = torch.cumsum(size, 0) - size
    rows = e * capacity if capacity else s * k + e * (pad - 1)
    keep = slot < capacity if capacity else slot >= 0
    route, where = order.indices[keep], (base[order.values] + slot)[keep]
    src = torch.full((rows,), -1, device="cuda", dtype=torch.long)
    src[where] = torch.div(route, k, rounding_mode="floor")
    dst = torch.full((s * k,), -1, device="cuda", dtype=torch.long)
    dst[route] = where
    kept = counts.clamp(max=capacity) if capacity else counts
    active = torch.nonzero(kept).reshape(-1)
    most = int(kept.max())
    at = base[active, None] + torch.arange(most, device="cuda")
    at = torch.where(torch.arange(most, device="cuda") < kept[active, None], at, rows)
    return {"rows": rows, "src": src, "dst": dst.view(s, k), "active": active, "at": at, "base": base, "kept": kept}


def _rows_of(c):
    if c.get("capacity", 0):
        return c["e"] * c["capacity"]
    return c["s"] * c["k"] + c["e"] * (c.get("pad", 1) - 1)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": c}
    if c["kind"] == "balance":
        logits, idx, _ = _routing(c, gen)
        st |= {"logits": logits, "idx": idx, "mask": None, "groups": None}
        if c["masked"]:
            st["mask"] = torch.rand(c["s"], generator=gen, device="cuda") < 0.9
        g = c["groups"]
        if g > 1:
            cuts = torch.sort(torch.randint(0, c["s"] + 1, (g - 1,), generator=gen, device="cuda")).values
            ends = torch.tensor([0, c["s"]], device="cuda")
            st["groups"] = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)
        st["grad_loss"] = torch.rand(g, generator=gen, device="cuda") + 0.5
        st["grad_z"] = torch.rand(g, generator=gen, device="cuda") * 0.1
        return st
    s, m, n, e, dt = c["s"], c["m"], c["n"], c["e"], DTYPES[c["dtype"]]
    _, idx, w = _routing(c, gen, hot=c.get("hot", False))
    rows = _rows_of(c)
    if own:  # the handle a program keeps for a batch's routing
        import combine_moe_gate_amd as M
        st["layout"] = M.moe_dispatch_layout(idx, e, c.get("capacity", 0), pad_multiple=c.get("pad", 1))
    else:
        st["plan"] = _plan(idx, e, c.get("capacity", 0), c.get("pad", 1))
    st["w"] = w if c["kind"] == "gemm" else w.to(dt)
    if c["kind"] == "gemm":
        nz = 2 * n if c["gated"] else n
        st["a"] = _normal(gen, (s if c["gather"] else rows, m), dt)
        st["weights"] = _weights(gen, e, nz, m, dt)
        st["bias"] = None if c["bias"] == "none" else _normal(gen, (e, nz), dt if c["bias"] == "own" else torch.float32, 0.1)
        st["residual"] = None if c["residual"] == "none" else _normal(gen, (rows if c["residual"] == "rows" else s, n), dt)
        return st
    st["x"] = _normal(gen, (s, m), dt)
    st["up"] = _weights(gen, e, 2 * n, m, dt)
    st["down"] = _weights(gen, e, m, n, dt)
    st["up_bias"] = _normal(gen, (e, 2 * n), dt, 0.1) if c["bias"] else None
    st["down_bias"] = _normal(gen, (e, m), dt, 0.1) if c["bias"] else None
    st["grad_y"] = _normal(gen, (s, m), dt)
    for v in ("x", "up", "down", "up_bias", "down_bias", "w"):
        if st[v] is not None:
            st[v].requires_grad_()
    return st


# ---------------------------------------------------------------------------------------------
# plain forms, in 32 bits


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _group_sums(st, x):
    """[g, columns] of [s, columns]: the sums of each group's unpadded tokens, in 64 bits as they run over up
    to all tokens (a running sum over the tokens where there are several groups, exact for whole numbers)."""
    if st["mask"] is not None:
        x = torch.where(st["mask"][:, None], x, 0.0)
    if st["groups"] is None:
        return x.sum(0, keepdim=True, dtype=torch.float64)
    run = torch.cumsum(x.t().contiguous(), 1, dtype=torch.float64)
    run = torch.cat([run.new_zeros((run.shape[0], 1)), run], 1)[:, st["groups"].long()]
    return (run[:, 1:] - run[:, :-1]).t()


def _plain_balance(st):
    c, logits, idx = st["case"], st["logits"], st["idx"]
    s, e, k = c["s"], c["e"], c["k"]
    tokens = _group_sums(st, torch.ones((s, 1), device="cuda"))[:, 0]
    counts = _group_sums(st, torch.zeros_like(logits).scatter_(1, idx.long(), 1.0))
    top = logits.max(1, keepdim=True).values
    ex = torch.exp(logits - top)
    total = ex.sum(1, keepdim=True)
    p, lse = ex / total, top + torch.log(total)
    n = tokens.clamp(min=1)
    probs = _group_sums(st, p) / n[:, None]
    z = _group_sums(st, lse * lse)[:, 0] / n
    loss = (counts * probs).sum(1) * e / (k * n)
    # the gradient, with the counts' distance from their mean (their differences are what matters)
    off = (counts - k * n[:, None] / e) * (st["grad_loss"].double() * e / (k * n * n))[:, None]
    zt = (st["grad_z"].double() * 2 / n)[:, None]
    off, zt = off.float(), zt.float()
    if st["groups"] is not None:  # each token takes its group's row
        of = torch.bucketize(torch.arange(s, device="cuda"), st["groups"][1:].long(), right=True)
        off, zt = off[of], zt[of]
    grad = p * (off - (p * off).sum(1, keepdim=True) + zt * lse)
    if st["mask"] is not None:
        grad = torch.where(st["mask"][:, None], grad, 0.0)
    return {"counts": counts.int().contiguous(), "tokens": tokens.int(), "probs": probs.float().contiguous(), "loss": loss.float(), "z": z.float(),
            "grad": grad}


def _project(plan, a, weights, bias):
    """[rows, features] in 32 bits: each placed row times its expert's weights, plus its bias; other rows 0."""
    active, at, rows = plan["active"], plan["at"], plan["rows"]
    padded = torch.cat([a, a.new_zeros((1, a.shape[1]))])
    z = torch.matmul(padded[at], weights[active].float().transpose(1, 2).contiguous())
    if bias is not None:
        z = z + bias[active].float()[:, None, :]
    return z.new_zeros((rows + 1, z.shape[2])).index_copy(0, at.reshape(-1), z.reshape(-1, z.shape[2]))[:rows]


def _tokens_to_rows(plan, x):
    """[rows, m]: each row's token, 0 where a row has none."""
    padded = torch.cat([x, x.new_zeros((1, x.shape[1]))])
    return padded[torch.where(plan["src"] >= 0, plan["src"], x.shape[0])]


def _row_weights(plan, w):
    rows = w.new_zeros(plan["rows"] + 1)
    return rows.index_copy(0, torch.where(plan["dst"] >= 0, plan["dst"], plan["rows"]).reshape(-1), w.reshape(-1))[:-1]


def _gate_up(z, act, gated):
    if not gated:
        return _act(z, act)
    n = z.shape[1] // 2
    return _act(z[:, :n], act) * z[:, n:]


def _plain_gemm(st):
    c, plan = st["case"], st["plan"]
    dt = st["a"].dtype
    a = st["a"].float()
    z = _project(plan, _tokens_to_rows(plan, a) if c["gather"] else a, st["weights"], st["bias"])
    u = _gate_up(z, c["act"], c["gated"])
    if c["weighted"]:
        u = u * _row_weights(plan, st["w"])[:, None]
    if st["residual"] is not None:
        r = st["residual"].float()
        u = u + (_tokens_to_rows(plan, r) if c["residual"] == "tokens" else r)
    out = {"out": torch.where(plan["src"][:, None] >= 0, u, 0.0).to(dt)}
    if c["save"]:
        out["preact"] = z.to(dt)
    return out


def _plain_ffn(st):
    """What passes from one operator to the next is in the element type, its gradient too."""
    c, plan = st["case"], st["plan"]
    x, dt = st["x"], st["x"].dtype
    h = _gate_up(_project(plan, _tokens_to_rows(plan, x.float()), st["up"], st["up_bias"]), c["act"], True).to(dt)
    o = _project(plan, h.float(), st["down"], st["down_bias"]).to(dt).float()
    o = torch.cat([o, o.new_zeros((1, o.shape[1]))])
    y = (o[torch.where(plan["dst"] >= 0, plan["dst"], plan["rows"])] * st["w"].float()[:, :, None]).sum(1)
    return _with_grads(st, y.to(dt))


def _with_grads(st, y):
    names = [v for v in ("x", "up", "down", "up_bias", "down_bias", "w") if st[v] is not None]
    grads = torch.autograd.grad(y, [st[v] for v in names], st["grad_y"])
    return {"y": y.detach()} | {"grad_" + v: g for v, g in zip(names, grads)}


# ---------------------------------------------------------------------------------------------
# the framework's operators


def _own_balance(st):
    import combine_moe_gate_amd as M
    counts, tokens, probs, loss, z = M.moe_balance_loss(st["logits"], st["idx"], mask=st["mask"], groups=st["groups"])
    grad = M.moe_balance_loss_backward(st["logits"], counts, tokens, st["case"]["k"], st["grad_loss"], st["grad_z"],
                                       mask=st["mask"], groups=st["groups"])
    return {"counts": counts, "tokens": tokens, "probs": probs, "loss": loss, "z": z, "grad": grad}


def _own_gemm(st):
    import combine_moe_gate_amd as M
    c = st["case"]
    got = M.moe_expert_gemm_act(st["layout"], st["a"], st["weights"], gather=c["gather"], bias=st["bias"], act=c["act"],
                                gated=c["gated"], w=st["w"] if c["weighted"] else None, residual=st["residual"],
                                residual_gather=c["residual"] == "tokens", save_preact=c["save"])
    return {"out": got[0], "preact": got[1]} if c["save"] else {"out": got}


def _own_ffn(st):
    import combine_moe_gate_amd.autograd as A
    c, L = st["case"], st["layout"]
    # the gradient of the z that the forward used, in 32 bits as inside any operator here
    h = A.expert_linear(st["x"], st["up"], L, bias=st["up_bias"], act=c["act"], gated=True, preact_dtype=torch.float32)
    o = A.expert_linear(h, st["down"], L, bias=st["down_bias"], gather=False)
    return _with_grads(st, A.combine(o, st["w"].float(), L))


def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"balance": _own_balance, "gemm": _own_gemm, "ffn_step": _own_ffn}[kind](state)
    return {"balance": _plain_balance, "gemm": _plain_gemm, "ffn_step": _plain_ffn}[kind](state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    c = case
    s, e, k = c["s"], c["e"], c["k"]
    if c["kind"] == "balance":
        g = c["groups"]
        # the logits once for the loss and once for the gradient, which is written
        return {"bytes": 12 * s * e + 4 * s * k + s * c["masked"] + 8 * g * e + 20 * g, "flops": 16 * s * e}
    m, n, routes = c["m"], c["n"], s * k
    used = e * (1 - (1 - k / e) ** s)  # experts that some token chose (its mean under level routing)
    if c.get("capacity", 0):
        routes = min(routes, e * c["capacity"])
    if c["kind"] == "gemm":
        nz = 2 * n if c["gated"] else n
        rows = _rows_of(c)
        b = 2 * ((s if c["gather"] else routes) * m + used * nz * m + rows * n + (rows * nz if c["save"] else 0))
        b += 0 if c["residual"] == "none" else 2 * n * (routes if c["residual"] == "rows" else s)
        b += 0 if c["bias"] == "none" else used * nz * (2 if c["bias"] == "own" else 4)
        b += 4 * s * k if c["weighted"] else 0
        return {"bytes": b, "flops": 2 * routes * m * nz}
    # x, grad_y and the weights read; y, the gradient of x and of all experts' weights written
    return {"bytes": 2 * (4 * s * m + (used + e) * 3 * n * m) + 4 * s * k, "flops": 3 * 2 * routes * 3 * n * m}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits, expert by expert


def _exact_plan(idx, e, capacity, pad):
    """Per expert with rows: (expert, its tokens in order, their route number, its first row)."""
    ids = idx.long().cpu()
    rows, plan = 0, []
    for x in range(e):
        t, j = torch.nonzero(ids == x, as_tuple=True)  # tokens ascending
        size = capacity if capacity else -(-len(t) // pad) * pad
        if capacity:
            t, j = t[:capacity], j[:capacity]
        if len(t):
            plan.append((x, t.cuda(), j.cuda(), rows))
        rows += size
    return plan


def _act64(z, act):
    """(value, derivative)"""
    if act == "relu":
        return torch.where(z > 0, z, 0.0), (z > 0).double()
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        b, q = math.sqrt(2 / math.pi), 0.044715
        t = torch.tanh(b * (z + q * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * b * (1 + 3 * q * z * z)
    if act == "silu":
        sg = torch.sigmoid(z)
        return z * sg, sg * (1 + z * (1 - sg))
    return z, torch.ones_like(z)


def _exact_balance(st):
    c = st["case"]
    s, e, k, g = c["s"], c["e"], c["k"], c["groups"]
    l64 = st["logits"].double()
    bounds = [0, s] if st["groups"] is None else st["groups"].tolist()
    out = {"counts": None, "tokens": None, "probs": torch.zeros((g, e), device="cuda", dtype=torch.float64),
           "loss": torch.zeros(g, device="cuda", dtype=torch.float64), "z": torch.zeros(g, device="cuda", dtype=torch.float64),
           "grad": torch.zeros((s, e), device="cuda", dtype=torch.float64)}
    for i in range(g):
        t = torch.arange(bounds[i], bounds[i + 1], device="cuda")
        if st["mask"] is not None:
            t = t[st["mask"][t]]
        n = len(t)
        if n == 0:
            continue
        p, lse = torch.softmax(l64[t], 1), torch.logsumexp(l64[t], 1)
        f = torch.bincount(st["idx"][t].reshape(-1).long(), minlength=e).double() / (n * k)
        out["probs"][i] = p.mean(0)
        out["loss"][i] = e * (f * p.mean(0)).sum()
        out["z"][i] = (lse ** 2).mean()
        dp = st["grad_loss"][i].double() * e * f / n
        out["grad"][t] = p * (dp - (p * dp).sum(1, keepdim=True)) + st["grad_z"][i].double() * 2 / n * lse[:, None] * p
    return out


def exact(case, seed):
    global own
    asked, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = asked
    c = case
    if c["kind"] == "balance":
        return _exact_balance(st)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    _, idx, _ = _routing(c, gen, hot=c.get("hot", False))  # the first thing that prepare() draws
    plan = _exact_plan(idx, c["e"], c.get("capacity", 0), c.get("pad", 1))
    rows, n, act = _rows_of(c), c["n"], c["act"]
    f64 = {"device": "cuda", "dtype": torch.float64}
    if c["kind"] == "gemm":
        nz = 2 * n if c["gated"] else n
        out = torch.zeros((rows, n), **f64)
        pre = torch.zeros((rows, nz), **f64) if c["save"] else None
        for x, t, j, r0 in plan:
            r = torch.arange(r0, r0 + len(t), device="cuda")
            z = st["a"][t if c["gather"] else r].double() @ st["weights"][x].double().T
            if st["bias"] is not None:
                z = z + st["bias"][x].double()
            u = _act64(z[:, :n], act)[0] * (z[:, n:] if c["gated"] else 1.0)
            if c["weighted"]:
                u = u * st["w"][t, j].double()[:, None]
            if st["residual"] is not None:
                u = u + st["residual"][r if c["residual"] == "rows" else t].double()
            out[r] = u
            if pre is not None:
                pre[r] = z
        return {"out": out, "preact": pre} if c["save"] else {"out": out}
    with torch.no_grad():
        s, m = c["s"], c["m"]
        y, gx, gw = torch.zeros((s, m), **f64), torch.zeros((s, m), **f64), torch.zeros((s, c["k"]), **f64)
        gup, gdown = torch.zeros(st["up"].shape, **f64), torch.zeros(st["down"].shape, **f64)
        gub, gdb = torch.zeros((c["e"], 2 * n), **f64), torch.zeros((c["e"], m), **f64)
        for x, t, j, _ in plan:
            up, down = st["up"][x].double(), st["down"][x].double()
            xt, wt, gy = st["x"][t].double(), st["w"][t, j].double()[:, None], st["grad_y"][t].double()
            z = xt @ up.T + (st["up_bias"][x].double() if c["bias"] else 0.0)
            v, d = _act64(z[:, :n], act)
            h = v * z[:, n:]
            o = h @ down.T + (st["down_bias"][x].double() if c["bias"] else 0.0)
            y[t] += wt * o  # a token names an expert once
            gw[t, j] = (gy * o).sum(1)
            go = wt * gy
            gdb[x], gdown[x] = go.sum(0), go.T @ h
            gh = go @ down
            gz = torch.cat([gh * z[:, n:] * d, gh * v], 1)
            gub[x], gup[x] = gz.sum(0), gz.T @ xt
            gx[t] += gz @ up
        out = {"y": y, "grad_x": gx, "grad_up": gup, "grad_down": gdown, "grad_w": gw}
        return out | ({"grad_up_bias": gub, "grad_down_bias": gdb} if c["bias"] else {})
