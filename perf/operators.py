"""The operators of fp8 layers whose scales cover blocks of 128, case by case.

  quantize   activations to fp8 e4m3 with one scale per row and 128 columns, of x or of SiLU(gate) * up
  gemm       x [m, k] times a weight [n, k], both fp8: one scale per row and 128 k, and per 128 x 128 of the weight
  route      the top-k experts of each token's logits, with their softmax weights
  few        a whole mixture-of-experts layer for a few tokens, from the router's logits on
  many       the experts' layer for many tokens, with the routing at hand

`run` computes each from elementary torch operations in 32 bits where `own` is false, and calls the library where
it is true.  `exact` computes the definition in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128
TOP = 448.0  # the largest e4m3 value
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- the cases --
def listed():
    return [
        # one decoded token's hidden state on its way into a layer
        {"name": "quantize 1x7168", "op": "quantize", "m": 1, "k": 7168, "silu": False, "act": "bf16"},
        # the intermediate of a long prompt, an odd number of tokens, between the two projections of an MLP
        {"name": "quantize silu 8191x2048", "op": "quantize", "m": 8191, "k": 2048, "silu": True, "act": "bf16"},
        # one decoded token through a projection
        {"name": "gemm 1x4096x7168", "op": "gemm", "m": 1, "n": 4096, "k": 7168, "act": "bf16"},
        # a decoded batch of odd size through a narrow projection whose columns end inside a scale block
        {"name": "gemm 33x576x7168", "op": "gemm", "m": 33, "n": 576, "k": 7168, "act": "f16"},
        # a short prompt, or a large decoded batch
        {"name": "gemm 200x14336x4096", "op": "gemm", "m": 200, "n": 14336, "k": 4096, "act": "bf16"},
        # a long prompt
        {"name": "gemm 4096x4096x7168", "op": "gemm", "m": 4096, "n": 4096, "k": 7168, "act": "bf16"},
        # one decoded token's routing
        {"name": "route 1x256", "op": "route", "t": 1, "experts": 256, "topk": 8, "renorm": True, "logits": "f32"},
        # a long prompt's routing, 16-bit logits with many ties
        {"name": "route 16383x160", "op": "route", "t": 16383, "experts": 160, "topk": 6, "renorm": False, "logits": "bf16"},
        # one decoded token through an experts' layer
        {"name": "few 1 of 256", "op": "few", "t": 1, "experts": 256, "topk": 8, "h": 7168, "inter": 256, "renorm": True, "act": "bf16"},
        # a decoded batch of odd size
        {"name": "few 13 of 256", "op": "few", "t": 13, "experts": 256, "topk": 8, "h": 7168, "inter": 256, "renorm": False, "act": "bf16"},
        # a short prompt: about sixteen rows for each expert
        {"name": "many 509 of 256", "op": "many", "t": 509, "experts": 256, "topk": 8, "h": 7168, "inter": 256, "act": "bf16"},
        # a long prompt
        {"name": "many 4096 of 256", "op": "many", "t": 4096, "experts": 256, "topk": 8, "h": 7168, "inter": 256, "act": "bf16"},
    ]


def _spread(rng, low, high):
    """A whole number in [low, high], even over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "route", "few", "few", "many"])
    act = rng.choice(["bf16", "bf16", "f16"])
    if op == "quantize":
        return {"op": op, "m": _spread(rng, 1, 8191), "k": BLOCK * _spread(rng, 1, 56), "silu": rng.random() < 0.5, "act": act}
    if op == "gemm":
        c = {"op": op, "m": _spread(rng, 1, 4096), "n": 16 * _spread(rng, 4, 896), "k": BLOCK * _spread(rng, 1, 64), "act": act}
        while c["m"] * c["n"] * c["k"] > 4096 * 4096 * 7168:
            c["m"] = c["m"] // 2
        return c
    if op == "route":
        experts = _spread(rng, 4, 512)
        return {"op": op, "t": _spread(rng, 1, 16383), "experts": experts, "topk": rng.randint(1, min(8, experts)),
                "renorm": rng.random() < 0.5, "logits": rng.choice(["f32", "bf16", "f16"])}
    experts = _spread(rng, 8, 256)
    c = {"op": op, "experts": experts, "topk": rng.randint(1, min(8, experts)), "h": BLOCK * _spread(rng, 4, 56),
         "inter": BLOCK * _spread(rng, 1, 8), "act": act}
    while c["experts"] * c["h"] * c["inter"] > 256 * 7168 * 256:
        c["inter"] = max(BLOCK, c["inter"] // 2 // BLOCK * BLOCK)
        c["experts"] = max(8, c["experts"] * 3 // 4)
    c["t"] = _spread(rng, 1, 16) if op == "few" else _spread(rng, 24, 4096)
    if op == "few":
        c["renorm"] = rng.random() < 0.5
    else:
        while c["t"] * c["topk"] * c["h"] * c["inter"] > 4096 * 8 * 7168 * 256:
            c["t"] = c["t"] // 2
    return c


# ---------------------------------------------------------------- the inputs --
def _gen(seed):
    g = torch.Generator("cuda" if torch.cuda.is_available() else "cpu")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=g.device)


def _hidden(g, m, k, dtype):
    """Hidden states: rows of different sizes, a few large columns, a block of zeros now and then."""
    x = _normal(g, m, k) * torch.exp(0.5 * _normal(g, m, 1))
    x = x * (1 + 15 * (torch.rand(1, k, generator=g, device=g.device) < 0.004))
    dead = torch.rand(m, k // BLOCK, 1, generator=g, device=g.device) < 0.002
    return (x.view(m, k // BLOCK, BLOCK) * ~dead).view(m, k).to(dtype)


def _weight(g, n, k, experts=None):
    """e4m3 codes and one scale per 128 x 128, as a checkpoint holds them; products come out of order one."""
    lead = () if experts is None else (experts,)
    codes = (_normal(g, *lead, n, k) * 96).clamp_(-TOP, TOP).to(torch.float8_e4m3fn)
    shape = lead + (-(-n // BLOCK), k // BLOCK)
    scales = (0.5 + torch.rand(*shape, generator=g, device=g.device)) / (96 * math.sqrt(k))
    return codes, scales


def _logits(g, t, experts, dtype):
    """Router logits with experts shut off (the lowest value) in some rows."""
    x = _normal(g, t, experts) + 0.5 * _normal(g, 1, experts)
    off = (torch.rand(t, 1, generator=g, device=g.device) < 0.05) & (torch.rand(t, experts, generator=g, device=g.device) < 0.5)
    return x.masked_fill(off, -math.inf).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    op = c["op"]
    s = {"case": c}
    if op == "quantize":
        s["x"] = _hidden(g, c["m"], (2 if c["silu"] else 1) * c["k"], DTYPES[c["act"]])
    elif op == "gemm":
        s["a"], s["a_scale"] = _quantize(_hidden(g, c["m"], c["k"], DTYPES[c["act"]]).float())
        s["w"], s["w_scale"] = _weight(g, c["n"], c["k"])
        if own:
            import bit_quantized_gemm_repack_amd as hq

            s["a"] = s["a"].view(torch.uint8)
            s["plan"] = hq.Plan(c["n"], c["k"], hq.w8a8_block(c["act"]), max_m=c["m"])
            s["w"] = s["plan"].repack(s["w"].view(torch.uint8), s.pop("w_scale"))
    elif op == "route":
        s["logits"] = _logits(g, c["t"], c["experts"], torch.float32 if c["logits"] == "f32" else DTYPES[c["logits"]])
    else:
        s["x"] = _hidden(g, c["t"], c["h"], DTYPES[c["act"]])
        s["w1"], s["s1"] = _weight(g, 2 * c["inter"], c["h"], c["experts"])
        s["w2"], s["s2"] = _weight(g, c["h"], c["inter"], c["experts"])
        s["logits"] = _logits(g, c["t"], c["experts"], torch.float32)
        if op == "many":
            s["ids"], s["weights"] = _route(s.pop("logits"), c["topk"], False)
        if own:
            import bit_quantized_gemm_repack_amd as hq

            quant = hq.w8a8_block(c["act"])
            s["gate_up"] = hq.MoePlan(2 * c["inter"], c["h"], quant, c["experts"], c["t"], "silu_mul_qfp8")
            s["down"] = hq.MoePlan(c["h"], c["inter"], quant, c["experts"], c["t"], "topk_combine")
            s["w1"] = s["gate_up"].repack(s["w1"].view(torch.uint8), s.pop("s1"))
            s["w2"] = s["down"].repack(s["w2"].view(torch.uint8), s.pop("s2"))
    return s


# ------------------------------------------------------------ the plain forms --
def _quantize(v):
    """fp32 [m, k] -> e4m3 values [m, k] and scales [k/128, m]."""
    b = v.view(v.shape[0], -1, BLOCK)
    top = b.abs().amax(-1, keepdim=True)
    # a tensor's division rounds correctly where one by a number may multiply by its reciprocal
    scale = torch.where(top > 0, top / torch.full_like(top, TOP), torch.ones_like(top))
    codes = (b / scale).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    return codes.view(v.shape), scale.squeeze(-1).t().contiguous()


def _rows(codes, scale):
    """The fp32 values of quantised rows."""
    return (codes.float().view(codes.shape[0], -1, BLOCK) * scale.t().unsqueeze(-1)).view(codes.shape)


def _values(codes, scales):
    """The fp32 values of weights [.., n, k] with a scale per 128 x 128."""
    n, k = codes.shape[-2:]
    by_row = scales.repeat_interleave(BLOCK, -2)[..., :n, :]
    return (codes.float().unflatten(-1, (k // BLOCK, BLOCK)) * by_row.unsqueeze(-1)).flatten(-2)


def _silu_mul(h):
    gate, up = h.chunk(2, -1)
    return gate / (1 + torch.exp(-gate)) * up


def _route(logits, topk, renorm):
    x = logits.float()
    best, ids = torch.sort(x, dim=-1, descending=True, stable=True)
    best, ids = best[:, :topk], ids[:, :topk].int()
    top = best[:, :1].clamp_min(torch.finfo(torch.float32).min)
    e = torch.exp(best - top)
    total = e.sum(-1, keepdim=True) if renorm else torch.exp(x - top).sum(-1, keepdim=True)
    none = best == -math.inf
    return ids.masked_fill(none, -1), (e / total).masked_fill(none, 0.0)


def _experts(s, ids, weights):
    """The experts' layer: each slot's row through its expert, the weighted rows summed per token."""
    c = s["case"]
    t, topk = ids.shape
    rows = _rows(*_quantize(s["x"].float()))
    flat = ids.reshape(-1).long()
    weight = torch.where(flat >= 0, weights.reshape(-1), torch.zeros_like(weights.reshape(-1)))
    flat = flat.clamp_min(0)
    token = torch.arange(t, device=ids.device).repeat_interleave(topk)
    if t * topk <= c["experts"]:  # few slots: each slot's own weights
        at, x = flat, rows[token].unsqueeze(1)
    else:  # many: an expert's slots side by side
        order = torch.argsort(flat, stable=True)
        count = torch.bincount(flat, minlength=c["experts"])
        place = torch.arange(t * topk, device=ids.device) - (count.cumsum(0) - count)[flat[order]]
        at = torch.arange(c["experts"], device=ids.device)
        x = rows.new_zeros(c["experts"], int(count.max()), c["h"])
        x[flat[order], place] = rows[token[order]]
    h = torch.bmm(x, _values(s["w1"].view(torch.uint8)[at].view(torch.float8_e4m3fn), s["s1"][at]).transpose(1, 2))
    a = _silu_mul(h)
    a = _rows(*_quantize(a.reshape(-1, c["inter"]))).view(a.shape)
    o = torch.bmm(a, _values(s["w2"].view(torch.uint8)[at].view(torch.float8_e4m3fn), s["s2"][at]).transpose(1, 2))
    if t * topk <= c["experts"]:
        o = o.squeeze(1)
    else:
        o = torch.empty(t * topk, c["h"], device=o.device).index_copy_(0, order, o[flat[order], place])
    return (o * weight.unsqueeze(-1)).view(t, topk, -1).sum(1).to(s["x"].dtype)


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import bit_quantized_gemm_repack_amd as hq

        if op == "quantize":
            codes, scales = hq.quantize_blocks(state["x"], silu_mul=c["silu"])
            return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales}
        if op == "gemm":
            return state["plan"].gemm(state["a"], *state["w"], a_scale=state["a_scale"])
        if op == "route":
            ids, weights = hq.route_topk(state["logits"], c["topk"], renormalize=c["renorm"])
            return {"ids": ids, "weights": weights}
        if op == "few":
            y, ids, weights = hq.moe_layer_routed(state["gate_up"], state["down"], state["x"], state["logits"], c["topk"],
                                                  *state["w1"], *state["w2"], renormalize=c["renorm"])
            return {"y": y, "ids": ids, "weights": weights}
        return hq.moe_layer(state["gate_up"], state["down"], state["x"], state["ids"], state["weights"], *state["w1"], *state["w2"])
    if op == "quantize":
        x = state["x"].float()
        codes, scales = _quantize(_silu_mul(x) if c["silu"] else x)
        return {"codes": codes, "scales": scales}
    if op == "gemm":
        y = _rows(state["a"], state["a_scale"]) @ _values(state["w"], state["w_scale"]).t()
        return y.to(DTYPES[c["act"]])
    if op == "route":
        ids, weights = _route(state["logits"], c["topk"], c["renorm"])
        return {"ids": ids, "weights": weights}
    if op == "few":
        ids, weights = _route(state["logits"], c["topk"], c["renorm"])
        return {"y": _experts(state, ids, weights), "ids": ids, "weights": weights}
    return _experts(state, state["ids"], state["weights"])


# ------------------------------------------------------------------ the work --
def _hit(c):
    """Experts that t * topk slots reach, on average over uniform routings."""
    return c["experts"] * (1 - (1 - c["topk"] / c["experts"]) ** c["t"])


def work(case):
    c = case
    if c["op"] == "quantize":
        n = c["m"] * c["k"]
        return {"bytes": (4 if c["silu"] else 2) * n + n + 4 * n // BLOCK, "flops": (8 if c["silu"] else 3) * n}
    if c["op"] == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": n * k + m * k + 4 * (-(-n // BLOCK) + m) * (k // BLOCK) + 2 * m * n, "flops": 2 * m * n * k}
    if c["op"] == "route":
        e = c["t"] * c["experts"]
        return {"bytes": (4 if c["logits"] == "f32" else 2) * e + 8 * c["t"] * c["topk"], "flops": 4 * e}
    per_expert = 3 * c["inter"] * c["h"] * (1 + 4 / BLOCK**2)
    moved = _hit(c) * per_expert + 4 * c["t"] * c["h"] + 8 * c["t"] * c["topk"] + (4 * c["t"] * c["experts"] if c["op"] == "few" else 0)
    return {"bytes": moved, "flops": 2 * c["t"] * c["topk"] * 3 * c["inter"] * c["h"]}


# ------------------------------------------------------- the definition in 64 --
def _exact_code(v):
    """The nearest e4m3 value of each v, ties to even, at most 448 in size."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0**-6))) - 3)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def _f32(v):
    return v.float().double()


def _exact_quantize(v):
    """The definition holds two roundings to fp32, since the scale is an fp32 number and 16-bit values over their
    block's largest fall on the midpoints of e4m3 often: the scale's, and the quotient's before it is coded."""
    b = v.unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1)
    scale = _f32(torch.where(top > 0, top / TOP, torch.ones_like(top)))
    return _exact_code(_f32(b / scale.unsqueeze(-1))).flatten(-2), scale


def _exact_act(h):
    half = h.shape[-1] // 2
    return h[..., :half] * torch.sigmoid(h[..., :half]) * h[..., half:]


def _exact_weight(codes, scales):
    n, k = codes.shape
    row = torch.arange(n, device=codes.device) // BLOCK
    col = torch.arange(k, device=codes.device) // BLOCK
    return codes.double() * scales.double()[row][:, col]


def _exact_route(logits, topk, renorm):
    p = logits.double()
    # one key for both orders: the place in a sort by value, the earlier index first
    rank = torch.argsort(torch.argsort(-p, dim=-1, stable=True), dim=-1, stable=True)
    ids = torch.argsort(rank, dim=-1)[:, :topk]
    chosen = torch.gather(p, 1, ids)
    norm = torch.logsumexp(chosen if renorm else p, -1, keepdim=True)
    none = torch.isinf(chosen)
    return ids.int().masked_fill(none, -1), torch.exp(chosen - norm).masked_fill(none, 0.0)


def exact(case, seed):
    global own
    was, own = own, False  # the inputs as they come, not the library's layout
    s = prepare(case, seed)
    own = was
    c = s["case"]
    if c["op"] == "quantize":
        v = s["x"].double()
        codes, scale = _exact_quantize(_exact_act(v) if c["silu"] else v)
        return {"codes": codes, "scales": scale.t().contiguous()}
    if c["op"] == "gemm":
        a = s["a"].double() * s["a_scale"].double().t().repeat_interleave(BLOCK, 1)
        return a @ _exact_weight(s["w"], s["w_scale"]).t()
    if c["op"] == "route":
        ids, weights = _exact_route(s["logits"], c["topk"], c["renorm"])
        return {"ids": ids, "weights": weights}
    ids, weights = (s["ids"], s["weights"].double()) if c["op"] == "many" else _exact_route(s["logits"], c["topk"], c["renorm"])
    codes, scale = _exact_quantize(s["x"].double())
    x = codes * scale.repeat_interleave(BLOCK, -1)
    y = torch.zeros(c["t"], c["h"], dtype=torch.float64, device=x.device)
    for e in torch.unique(ids).tolist():
        if e < 0:
            continue
        token, slot = torch.nonzero(ids == e, as_tuple=True)
        codes, scale = _exact_quantize(_exact_act(x[token] @ _exact_weight(s["w1"][e], s["s1"][e]).t()))
        o = (codes * scale.repeat_interleave(BLOCK, -1)) @ _exact_weight(s["w2"][e], s["s2"][e]).t()
        y.index_add_(0, token, o * weights[token, slot].unsqueeze(-1))
    return y if c["op"] == "many" else {"y": y, "ids": ids, "weights": weights}
