"""Cases that measure experts held in microscaled 4-bit floating point.

A row is cut into blocks of 32 values; a block has one scale, a power of two in a byte E (2^(E - 127), 255: not a number),
and each value one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 times it, with a sign, in four bits. Four kinds of pass:

  round  rows quantised, and read back
  gemm   one projection of every placed row by its expert's 4-bit weights, with bias, activation (plain or gated), route
         weight and residual before the one rounding; rows in 16 bits, or quantised in the pass as well
  block  a layer's forward in 4 bits: rows quantised, gated up projection whose hidden rows are quantised in turn, down
         projection, weighted combine
  step   fine-tuning around frozen 4-bit experts: gated up and down projections, combine, and the gradients of rows, biases
         and route weights (through a rounding of rows to 4 bits the gradient passes as it is)
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------
# cases


def _round(name, rows, m, dtype):
    return {"name": name, "kind": "round", "rows": rows, "m": m, "dtype": dtype}


def _gemm(name, s, m, n, e, k, dtype, quantized=False, act="none", gated=False, bias="none", weighted=False, residual="none",
          gather=True, capacity=0, pad=1, save=False, hot=False):
    """n: output features (a gated projection's weights have 2 n rows). quantized: the rows go to 4 bits as well. bias: none,
    f32 or own (the element type). residual: none, rows (one for each buffer row) or tokens (gathered). save: the values
    before the activation are kept. hot: a tenth of the tokens prefer expert 0."""
    return {"name": name, "kind": "gemm", "s": s, "m": m, "n": n, "e": e, "k": k, "dtype": dtype, "quantized": quantized,
            "act": act, "gated": gated, "bias": bias, "weighted": weighted, "residual": residual, "gather": gather,
            "capacity": capacity, "pad": pad, "save": save, "hot": hot}


def _layer(name, kind, s, m, n, e, k, dtype, quantized=True, act="silu", bias=False):
    return {"name": name, "kind": kind, "s": s, "m": m, "n": n, "e": e, "k": k, "dtype": dtype, "quantized": quantized,
            "act": act, "bias": bias}


def listed():
    return [
        # a decoding batch's rows, an odd number of blocks each: latency
        _round("rows of 24 tokens", 24, 2848, "bf16"),
        # 64 experts' weights taken from 16 bits to 4, and checked by reading them back
        _round("weights of 64 experts", 64 * 2816, 1408, "bf16"),
        # decoding: one token's up projection, where the weights of its 8 experts are what is read
        _gemm("decode one token", 1, 4096, 2048, 128, 8, "bf16", act="silu", gated=True),
        # decoding a batch: the down projection, weighted, over rows that the up projection left
        _gemm("decode 24 tokens down", 24, 1408, 2816, 64, 6, "f16", bias="own", weighted=True, gather=False),
        # prompts, rows in 4 bits too: up projection of 4096 tokens
        _gemm("prompt 4096 tokens", 4096, 2816, 1408, 128, 8, "bf16", quantized=True, act="silu", gated=True),
        # a large batch with rows in 16 bits, the values before the activation kept
        _gemm("batch gated 16-bit rows", 8192, 4096, 2048, 128, 8, "bf16", act="silu", gated=True, bias="own", save=True),
        # capacity-bounded routing with drops, bias, exact gelu and the tokens' own rows added
        _gemm("capacity gelu residual", 16384, 1024, 1024, 64, 4, "f16", quantized=True, act="gelu", bias="f32",
              residual="tokens", capacity=1024, hot=True),
        # odd sizes: ragged row and column tiles, padded segments, more experts than a power of two
        _gemm("ragged relu", 777, 288, 200, 129, 5, "bf16", act="relu", bias="f32", weighted=True, residual="rows", pad=16),
        # a decoding batch through the whole layer in 4 bits
        _layer("layer 32 tokens", "block", 32, 2816, 1408, 128, 8, "bf16"),
        # the largest: a prompt batch through the whole layer in 4 bits
        _layer("layer 8192 tokens", "block", 8192, 4096, 2048, 128, 8, "bf16"),
        # fine-tuning around frozen experts: a small step with rows in 16 bits and an ordinary one with rows in 4
        _layer("tuning step 1000 tokens", "step", 1000, 544, 288, 16, 2, "bf16", quantized=False, act="gelu_tanh", bias=True),
        _layer("tuning step 8192 tokens", "step", 8192, 2048, 1408, 64, 6, "bf16", bias=True),
    ]


def _log(rng, lo, hi, multiple=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(multiple, int(round(v / multiple)) * multiple)


def draw(rng):
    kind = rng.choice(["round", "gemm", "gemm", "block", "step"])
    e = rng.choice([8, 16, 60, 64, 128, 129, 160])
    k = rng.choice([1, 2, 3, 4, 6, 8])
    if kind == "round":
        m = _log(rng, 32, 4096, 32)
        c = _round("", _log(rng, 1, 250_000_000 // m), m, rng.choice(["bf16", "f16", "f32"]))
    elif kind == "gemm":
        s = _log(rng, 1, 8192)
        m, n = _log(rng, 64, 4096, 32), _log(rng, 64, 2048, 8)
        capacity = 0 if rng.random() < 0.7 or s < 64 else -(-s * k // e)
        c = _gemm("", s, m, n, e, k, rng.choice(["bf16", "f16"]), quantized=rng.random() < 0.5,
                  act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), gated=rng.random() < 0.5,
                  bias=rng.choice(["none", "f32", "own"]), weighted=rng.random() < 0.5,
                  residual=rng.choice(["none", "rows", "tokens"]), gather=rng.random() < 0.6, capacity=capacity,
                  pad=1 if capacity or rng.random() < 0.7 else 16, save=rng.random() < 0.4, hot=rng.random() < 0.3)
    elif kind == "block":
        s = _log(rng, 1, 8192)
        c = _layer("", "block", s, _log(rng, 64, 4096, 32), _log(rng, 64, 2048, 32), min(e, 128), k, rng.choice(["bf16", "f16"]),
                   act=rng.choice(["gelu", "gelu_tanh", "silu"]), bias=rng.random() < 0.5)
    else:
        s = _log(rng, 16, 8192)
        c = _layer("", "step", s, _log(rng, 64, 2048, 32), _log(rng, 64, 1408, 32), min(e, 64), min(k, 6),
                   rng.choice(["bf16", "f16"]), quantized=rng.random() < 0.5, act=rng.choice(["gelu", "gelu_tanh", "silu"]),
                   bias=rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------
# 4-bit values, in 32 bits


def _quantize(x):
    """(codes [..., m / 2], scales [..., m / 32]), two values to a byte, the first in its low half."""
    b = x.float().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    exponent = torch.frexp(top).exponent  # top = f 2^exponent, f in [0.5, 1): floor(log2 top) = exponent - 1
    scale = torch.where(top > 0, (exponent - 3 + 127).clamp(min=0), 0)
    fine = torch.isfinite(top)
    scale = torch.where(fine, scale, 255)
    a = b.abs() * torch.exp2((127 - scale).float())[..., None]
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6)  # half-way cases to the even code
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, 0.5 * a + 4)) + 8 * torch.signbit(b)
    code = torch.where(fine[..., None], code, 0.0).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.to(torch.uint8)


def _values(codes, scales):
    """What the codes and scales stand for, in 32 bits."""
    table = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2).unflatten(-1, (-1, 32))
    scale = torch.where(scales == 255, math.nan, torch.exp2(scales.float() - 127))
    return (v * scale[..., None]).flatten(-2)


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
    return {"rows": rows, "src": src, "dst": dst.view(s, k), "active": active, "at": at}


def _rows_of(c):
    if c.get("capacity", 0):
        return c["e"] * c["capacity"]
    return c["s"] * c["k"] + c["e"] * (c.get("pad", 1) - 1)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": c}
    if c["kind"] == "round":
        # magnitudes that differ from row to row, as activations' and weights' do
        x = torch.randn((c["rows"], c["m"]), generator=gen, device="cuda")
        x *= torch.exp2(torch.randint(-6, 7, (c["rows"], 1), generator=gen, device="cuda").float())
        st["x"] = x.to(DTYPES[c["dtype"]])
        return st
    s, m, n, e, dt = c["s"], c["m"], c["n"], c["e"], DTYPES[c["dtype"]]
    _, idx, w = _routing(c, gen, hot=c.get("hot", False))
    rows = _rows_of(c)
    if own:  # the handle a program keeps for a batch's routing
        import combine_moe_gate_amd as M
        st["layout"] = M.moe_dispatch_layout(idx, e, c.get("capacity", 0), pad_multiple=c.get("pad", 1))
    else:
        st["plan"] = _plan(idx, e, c.get("capacity", 0), c.get("pad", 1))
    st["w"] = w.to(dt) if c["kind"] == "step" else w
    gated = c.get("gated", True)
    nz = 2 * n if gated else n
    # the experts' 4-bit weights, expert by expert: a float32 draw of all would take several times their room
    for name, f, d in (("up", nz, m), ("down", m, n)):
        if name == "down" and c["kind"] == "gemm":
            break
        codes = torch.empty((e, f, d // 2), device="cuda", dtype=torch.uint8)
        scales = torch.empty((e, f, d // 32), device="cuda", dtype=torch.uint8)
        for x in range(e):
            codes[x], scales[x] = _quantize(_normal(gen, (f, d), torch.bfloat16, d ** -0.5))
        st[name] = (codes, scales)
    if c["kind"] == "gemm":
        st["x"] = _normal(gen, (s if c["gather"] else rows, m), dt)
        st["bias"] = None if c["bias"] == "none" else _normal(gen, (e, nz), dt if c["bias"] == "own" else torch.float32, 0.1)
        st["residual"] = None if c["residual"] == "none" else _normal(gen, (rows if c["residual"] == "rows" else s, n), dt)
        return st
    st["x"] = _normal(gen, (s, m), dt)
    st["up_bias"] = _normal(gen, (e, 2 * n), dt, 0.1) if c["bias"] else None
    st["down_bias"] = _normal(gen, (e, m), dt, 0.1) if c["bias"] else None
    if c["kind"] == "step":
        st["grad_y"] = _normal(gen, (s, m), dt)
        for v in ("x", "up_bias", "down_bias", "w"):
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


def _gate_up(z, act, gated):
    if not gated:
        return _act(z, act)
    n = z.shape[1] // 2
    return _act(z[:, :n], act) * z[:, n:]


class _Rounded(torch.autograd.Function):
    """Rows rounded to 4 bits; the gradient passes as it is."""

    @staticmethod
    def forward(ctx, x):
        return _values(*_quantize(x))

    @staticmethod
    def backward(ctx, g):
        return g


def _plain_round(st):
    codes, scales = _quantize(st["x"])
    return {"scales": scales, "values": _values(codes, scales).to(st["x"].dtype)}


def _project(plan, a, weights, bias):
    """[rows, features] in 32 bits: each placed row times its expert's weights, plus its bias; other rows 0."""
    active, at, rows = plan["active"], plan["at"], plan["rows"]
    padded = torch.cat([a, a.new_zeros((1, a.shape[1]))])
    w = _values(weights[0][active], weights[1][active])
    z = torch.matmul(padded[at], w.transpose(1, 2).contiguous())
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


def _combine(plan, o, w):
    o = torch.cat([o, o.new_zeros((1, o.shape[1]))])
    return (o[torch.where(plan["dst"] >= 0, plan["dst"], plan["rows"])] * w[:, :, None]).sum(1)


def _plain_gemm(st):
    c, plan = st["case"], st["plan"]
    dt = st["x"].dtype
    a = _Rounded.apply(st["x"]) if c["quantized"] else st["x"].float()
    z = _project(plan, _tokens_to_rows(plan, a) if c["gather"] else a, st["up"], st["bias"])
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


def _plain_layer(st):
    """Rows that pass from one operator to the next are in 4 bits; in a step whose gradient needs them, in the element
    type first. What the combine takes is in the element type."""
    c, plan = st["case"], st["plan"]
    x, dt = st["x"], st["x"].dtype
    rows = _tokens_to_rows(plan, _Rounded.apply(x.float()) if c["quantized"] else x.float())
    h = _gate_up(_project(plan, rows, st["up"], st["up_bias"]), c["act"], True)
    if c["kind"] == "step":
        h = h.to(dt).float()
    o = _project(plan, _Rounded.apply(h) if c["quantized"] else h, st["down"], st["down_bias"]).to(dt).float()
    y = _combine(plan, o, st["w"].float()).to(dt)
    return _with_grads(st, y) if c["kind"] == "step" else {"y": y}


def _with_grads(st, y):
    names = [v for v in ("x", "up_bias", "down_bias", "w") if st[v] is not None]
    grads = torch.autograd.grad(y, [st[v] for v in names], st["grad_y"])
    return {"y": y.detach()} | {"grad_" + v: g for v, g in zip(names, grads)}


# ---------------------------------------------------------------------------------------------
# the framework's operators


def _own_round(st):
    import combine_moe_gate_amd as M
    codes, scales = M.moe_mx4_quantize(st["x"])
    return {"scales": scales, "values": M.moe_mx4_dequantize(codes, scales, st["x"].dtype)}


def _own_gemm(st):
    import combine_moe_gate_amd as M
    c, x = st["case"], st["x"]
    rows = M.moe_mx4_quantize(x) if c["quantized"] else x
    got = M.moe_mx4_expert_gemm(st["layout"], rows, st["up"], gather=c["gather"], bias=st["bias"], act=c["act"], gated=c["gated"],
                                w=st["w"] if c["weighted"] else None, residual=st["residual"],
                                residual_gather=c["residual"] == "tokens", save_preact=c["save"], dtype=x.dtype)
    return {"out": got[0], "preact": got[1]} if c["save"] else {"out": got}


def _own_block(st):
    import combine_moe_gate_amd as M
    c, x, L = st["case"], st["x"], st["layout"]
    h = M.moe_mx4_expert_gemm(L, M.moe_mx4_quantize(x), st["up"], bias=st["up_bias"], act=c["act"], gated=True, dtype=x.dtype,
                              quantize_out=True)
    o = M.moe_mx4_expert_gemm(L, h, st["down"], gather=False, bias=st["down_bias"], dtype=x.dtype)
    return {"y": M.moe_combine(L, o, st["w"])}


def _own_step(st):
    import combine_moe_gate_amd.autograd as A
    c, L = st["case"], st["layout"]
    # the gradient of the z that the forward used, and no rounding on its way to x: as inside any operator here
    h = A.expert_linear_mx4(st["x"], st["up"], L, bias=st["up_bias"], act=c["act"], gated=True, quantize_rows=c["quantized"],
                            preact_dtype=torch.float32, grad_dtype=torch.float32)
    o = A.expert_linear_mx4(h, st["down"], L, bias=st["down_bias"], gather=False, quantize_rows=c["quantized"])
    return _with_grads(st, A.combine(o, st["w"].float(), L))


def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"round": _own_round, "gemm": _own_gemm, "block": _own_block, "step": _own_step}[kind](state)
    return {"round": _plain_round, "gemm": _plain_gemm, "block": _plain_layer, "step": _plain_layer}[kind](state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    c = case
    m, q = c["m"], 0.5 + 1 / 32  # bytes of a 4-bit value and its share of a scale
    if c["kind"] == "round":
        size = 4 if c["dtype"] == "f32" else 2
        # the rows read, the 4-bit values written and read, the rows written; a maximum, a scaling and a rounding each
        return {"bytes": c["rows"] * m * (2 * size + 2 * q), "flops": 4 * c["rows"] * m}
    s, n, e, k = c["s"], c["n"], c["e"], c["k"]
    routes = s * k
    used = e * (1 - (1 - k / e) ** s)  # experts that some token chose (its mean under level routing)
    if c.get("capacity", 0):
        routes = min(routes, e * c["capacity"])
    if c["kind"] == "gemm":
        nz = 2 * n if c["gated"] else n
        rows = _rows_of(c)
        b = 2 * ((s if c["gather"] else routes) * m + rows * n + (rows * nz if c["save"] else 0)) + q * used * nz * m
        b += 0 if c["residual"] == "none" else 2 * n * (routes if c["residual"] == "rows" else s)
        b += 0 if c["bias"] == "none" else used * nz * (2 if c["bias"] == "own" else 4)
        b += 4 * s * k if c["weighted"] else 0
        return {"bytes": b, "flops": 2 * routes * m * nz}
    # x and the weights read, y written; in a step the weights again, grad_y and the gradient of x
    step = c["kind"] == "step"
    b = 2 * (4 if step else 2) * s * m + (2 if step else 1) * used * 3 * n * m * q + 4 * s * k
    return {"bytes": b, "flops": (2 if step else 1) * 2 * routes * 3 * n * m}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits, expert by expert


def _nearest(x):
    """(what x rounds to in 4 bits, scale bytes) in 64 bits, by distance: of two equally near, the one with the even code."""
    grid = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6], device=x.device, dtype=torch.float64)
    blocks = x.double().reshape(*x.shape[:-1], -1, 32)
    top = blocks.abs().amax(-1, keepdim=True)
    # the largest power of two that is not above top, by comparison with its neighbours
    p = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    p = p + (torch.exp2(p + 1) <= top).double() - (torch.exp2(p) > top).double() * (top > 0)
    byte = torch.where(top > 0, p - 2 + 127, 0.0).clamp(0, 254)
    scale = torch.exp2(byte - 127)
    a = blocks.abs() / scale
    mid = (grid[:-1] + grid[1:]) / 2
    low = torch.bucketize(a, mid)  # the number of midpoints below a
    tie = (a == mid[low.clamp(max=6)]) & (low % 2 == 1) & (low < 7)
    v = torch.copysign(grid[low + tie.long()], blocks) * scale
    return v.reshape(x.shape), byte[..., 0].to(torch.uint8)


def _read64(codes, scales):
    c = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1).long()
    exponent, mantissa = (c >> 1) & 3, (c & 1).double()
    v = torch.where(exponent == 0, 0.5 * mantissa, (1 + 0.5 * mantissa) * torch.exp2(exponent.double() - 1))
    v = torch.where(c >= 8, -v, v) * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)
    return v


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


def exact(case, seed):
    global own
    asked, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = asked
    c = case
    if c["kind"] == "round":
        if c["rows"] * c["m"] > 100_000_000:  # slice by slice: 64-bit blocks take room
            parts = [_nearest(x)[0].to(st["x"].dtype).double() for x in st["x"].split(max(1, 30_000_000 // c["m"]))]
            return {"scales": None, "values": torch.cat(parts)}
        return {"scales": None, "values": _nearest(st["x"])[0]}
    gen = torch.Generator(device="cuda").manual_seed(seed)
    _, idx, _ = _routing(c, gen, hot=c.get("hot", False))  # the first thing that prepare() draws
    plan = _exact_plan(idx, c["e"], c.get("capacity", 0), c.get("pad", 1))
    rows, n, act = _rows_of(c), c["n"], c["act"]
    f64 = {"device": "cuda", "dtype": torch.float64}
    weights = lambda name, x: _read64(st[name][0][x], st[name][1][x])  # noqa: E731
    with torch.no_grad():
        a = _nearest(st["x"])[0] if c["quantized"] else st["x"].double()
        if c["kind"] == "gemm":
            nz = 2 * n if c["gated"] else n
            out = torch.zeros((rows, n), **f64)
            pre = torch.zeros((rows, nz), **f64) if c["save"] else None
            for x, t, j, r0 in plan:
                r = torch.arange(r0, r0 + len(t), device="cuda")
                z = a[t if c["gather"] else r] @ weights("up", x).T
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
        s, m, step = c["s"], c["m"], c["kind"] == "step"
        y, gx, gw = torch.zeros((s, m), **f64), torch.zeros((s, m), **f64), torch.zeros((s, c["k"]), **f64)
        gub, gdb = torch.zeros((c["e"], 2 * n), **f64), torch.zeros((c["e"], m), **f64)
        for x, t, j, _ in plan:
            up, down = weights("up", x), weights("down", x)
            wt = st["w"][t, j].double()[:, None]
            z = a[t] @ up.T + (st["up_bias"][x].double() if c["bias"] else 0.0)
            v, d = _act64(z[:, :n], act)
            h = v * z[:, n:]
            if step:  # h is an output of its operator, in the element type
                h = h.to(st["x"].dtype).double()
            o = (_nearest(h)[0] if c["quantized"] else h) @ down.T + (st["down_bias"][x].double() if c["bias"] else 0.0)
            y[t] += wt * o  # a token names an expert once
            if not step:
                continue
            gy = st["grad_y"][t].double()
            gw[t, j] = (gy * o).sum(1)
            go = wt * gy
            gdb[x] = go.sum(0)
            gh = go @ down
            gz = torch.cat([gh * z[:, n:] * d, gh * v], 1)
            gub[x] = gz.sum(0)
            gx[t] += gz @ up
        if not step:
            return {"y": y}
        out = {"y": y, "grad_x": gx, "grad_w": gw}
        return out | ({"grad_up_bias": gub, "grad_down_bias": gdb} if c["bias"] else {})
