"""The operators of a layer of routed experts in 8 bits, as measured cases.

Four operators that such a layer needs around the library's GEMMs:

  route     gemm_route_*: softmax or sigmoid scores of a router's logits, a bias for
            balance, groups, the top k experts of each token with their weights, and
            the tokens' order by expert
  quantise  gemm_fp8_quantise_*: rows as E4M3 codes with a scale for each 128 values
  product   gemm_fp8_blocks*: the product of E4M3 matrices with a scale for each 1 x 128
            block of A and each 128 x 128 block of B
  experts   gemm_experts: the experts' gate, up and down products of the routed tokens
            and the weighted sum of each token's experts

``own`` selects the library's kernels; otherwise ``run`` computes the same values with
elementary torch operations, in 32 bits (in 64 where choices between experts are made).
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 128
QMAX = 448.0
SMALLEST = 2.0 ** -126      # a block whose scale would be below this stores zeros


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one user's decode step: a token's logits over 64 experts, latency counts
        dict(name="route 1 x 64", op="route", tokens=1, experts=64, top_k=8, dtype="bf16", score="softmax",
             bias=False, groups=1, top_groups=1, renormalise=True),
        # a batch of decoding users; balanced by a bias, 8 groups of which 4 are kept
        dict(name="route 64 x 256, groups", op="route", tokens=64, experts=256, top_k=8, dtype="f32",
             score="sigmoid", bias=True, groups=8, top_groups=4, renormalise=True),
        # prompts prefilled together, the same router
        dict(name="route 16384 x 256, groups", op="route", tokens=16384, experts=256, top_k=8, dtype="f32",
             score="sigmoid", bias=True, groups=8, top_groups=4, renormalise=True),
        # one token's activations before a product: latency counts
        dict(name="quantise 1 x 4096", op="quantise", rows=1, cols=4096, block_rows=1, dtype="bf16"),
        # the activations of a long prefill, 4096 values a token (the LLaMA-7B layer's)
        dict(name="quantise 16384 x 4096", op="quantise", rows=16384, cols=4096, block_rows=1, dtype="bf16"),
        # a decode step's product with the 7B layer's gate or up weight
        dict(name="product 1 x 11008 x 4096", op="product", rows=1, cols=11008, depth=4096, dtype="bf16"),
        # an odd number of tokens through the down weight, sums left in fp32
        dict(name="product 77 x 4096 x 11008, f32", op="product", rows=77, cols=4096, depth=11008, dtype="f32"),
        # a prefill's product
        dict(name="product 8192 x 11008 x 4096", op="product", rows=8192, cols=11008, depth=4096, dtype="bf16"),
        # the 7B layer's FFN cut into narrow experts (11008 / 8 wide): one user's token
        dict(name="experts 1 of 64", op="experts", tokens=1, experts=64, top_k=8, hidden=4096, width=1376),
        # a batch of decoding users: about 8 tokens an expert
        dict(name="experts 64 of 64", op="experts", tokens=64, experts=64, top_k=8, hidden=4096, width=1376),
        # a ragged prefill through few, wider experts
        dict(name="experts 777 of 8", op="experts", tokens=777, experts=8, top_k=2, hidden=2048, width=2752),
        # prompts prefilled together
        dict(name="experts 16384 of 64", op="experts", tokens=16384, experts=64, top_k=8, hidden=4096, width=1376),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["route", "quantise", "product", "product", "experts", "experts"])
    if op == "route":
        groups = rng.choice([1, 1, 1, 2, 4, 8])
        experts = groups * _spread(rng, 4, 384 // groups)
        top_groups = rng.randint(1, groups)
        top_k = min(rng.choice([1, 2, 4, 6, 8, 8, 10]), experts * top_groups // groups)
        return dict(op=op, tokens=_spread(rng, 1, 16384), experts=experts, top_k=top_k, dtype=rng.choice(["bf16", "f32"]),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                    top_groups=top_groups, renormalise=rng.random() < 0.7)
    if op == "quantise":
        cols = 8 * _spread(rng, 16, 1376)
        block_rows = rng.choice([1, 1, 1, 128])
        return dict(op=op, rows=min(_spread(rng, 1, 16384), 16384 * 4096 // cols), cols=cols, block_rows=block_rows,
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "product":
        cols, depth = 16 * _spread(rng, 16, 688), 16 * _spread(rng, 16, 688)
        most = 8192 * 11008 * 4096 // (cols * depth)
        return dict(op=op, rows=min(_spread(rng, 1, 16384), most), cols=cols, depth=depth, dtype=rng.choice(["bf16", "bf16", "f32"]))
    hidden, width = 16 * _spread(rng, 32, 256), 16 * _spread(rng, 16, 172)
    experts = rng.choice([4, 8, 16, 24, 32, 64, 64, 128])
    experts = max(1, min(experts, 64 * 4096 * 1376 // (hidden * width)))
    top_k = min(rng.choice([1, 2, 2, 4, 6, 8, 8]), experts)
    most = 16384 * 8 * 4096 * 1376 // (top_k * hidden * width)
    return dict(op=op, tokens=min(_spread(rng, 1, 16384), most), experts=experts, top_k=top_k, hidden=hidden, width=width)


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        return {"bytes": t * (e * (2 if case["dtype"] == "bf16" else 4) + 12 * k) + 4 * e * (2 if case["bias"] else 1), "flops": 8 * t * e}
    if case["op"] == "quantise":
        m, k = case["rows"], case["cols"]
        return {"bytes": m * k * (3 if case["dtype"] == "bf16" else 5) + 4 * -(-m // case["block_rows"]) * _blocks(k), "flops": 3 * m * k}
    if case["op"] == "product":
        m, n, k = case["rows"], case["cols"], case["depth"]
        return {"bytes": m * k + k * n + m * n * (2 if case["dtype"] == "bf16" else 4) + 4 * _blocks(k) * (m + _blocks(n)),
                "flops": 2 * m * n * k}
    t, e, k, h, w = (case[x] for x in ("tokens", "experts", "top_k", "hidden", "width"))
    met = e * (1.0 - (1.0 - k / e) ** t)                      # experts that have a token
    return {"bytes": 4 * t * h + met * 3 * (h * w + 4 * _blocks(h) * _blocks(w)) + 8 * t * k, "flops": 6 * t * k * h * w}


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _activations(g, rows, cols):
    """Normed activations: most values around one, some channels far larger, rows of their own size."""
    x = _randn(g, rows, cols) * torch.exp(0.5 * _randn(g, 1, cols))
    return x * torch.exp(0.3 * _randn(g, rows, 1))


def _weight(g, lead, k, n):
    """Codes and scales of a weight whose blocks are filled to the format's largest value."""
    codes = torch.empty(*lead, k, n, dtype=torch.float8_e4m3fn, device="cuda")
    flat = codes.view(-1, n)
    step = max(1, (1 << 27) // n)
    for at in range(0, flat.shape[0], step):
        part = flat[at:at + step]
        part.copy_((110.0 * _randn(g, *part.shape)).clamp_(-QMAX, QMAX))
    scale = torch.exp(0.2 * _randn(g, *lead, _blocks(k), _blocks(n))) / (110.0 * math.sqrt(k))
    return codes, scale


def prepare(case, seed):
    s = dict(case)
    s.update({"route": _prepare_route, "quantise": _prepare_quantise, "product": _prepare_product,
              "experts": _prepare_experts}[case["op"]](case, seed))
    if own and case["op"] == "experts":       # the handle on the weights that a serving program keeps
        import roofline_driven_optimisation_gb300 as lib
        s["handle"] = lib.ExpertWeights(*s["gate"], *s["up"], *s["down"])
    return s


def _prepare_route(case, seed):
    g = _gen(seed)
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    # some experts are more popular than others
    logits = (1.5 * _randn(g, t, e) + 0.5 * _randn(g, 1, e)).to(_type(case))
    ints = dict(dtype=torch.int32, device="cuda")
    return dict(logits=logits, bias_values=0.1 * _randn(g, e) if case["bias"] else None, ids=torch.empty(t, k, **ints),
                weights=torch.empty(t, k, device="cuda"), offsets=torch.empty(e + 1, **ints), order=torch.empty(t * k, **ints))


def _prepare_quantise(case, seed):
    g = _gen(seed)
    m, k = case["rows"], case["cols"]
    return dict(x=_activations(g, m, k).to(_type(case)), codes=torch.empty(m, k, dtype=torch.float8_e4m3fn, device="cuda"),
                scales=torch.empty(-(-m // case["block_rows"]), _blocks(k), device="cuda"))


def _prepare_product(case, seed):
    g = _gen(seed)
    m, n, k = case["rows"], case["cols"], case["depth"]
    a, a_scale = _plain_quantise(_activations(g, m, k).bfloat16(), 1)
    b, b_scale = _weight(g, (), k, n)
    return dict(a=a, a_scale=a_scale, b=b, b_scale=b_scale, c=torch.empty(m, n, dtype=_type(case), device="cuda"))


def _prepare_experts(case, seed):
    g = _gen(seed)
    t, e, k, h, w = (case[x] for x in ("tokens", "experts", "top_k", "hidden", "width"))
    logits = 1.5 * _randn(g, t, e) + 0.5 * _randn(g, 1, e)
    weights, ids = torch.softmax(logits, 1).topk(k, dim=1)
    weights = (weights / weights.sum(1, keepdim=True)).contiguous()
    offsets, order = _order(ids, e)
    return dict(x=_activations(g, t, h).bfloat16(), weights=weights, ids=ids.int(), offsets=offsets, order=order,
                most=int((offsets[1:] - offsets[:-1]).max()), gate=_weight(g, (e,), h, w), up=_weight(g, (e,), h, w),
                down=_weight(g, (e,), w, h), out=torch.empty(t, h, dtype=torch.bfloat16, device="cuda"))


# ------------------------------------------------------------------ one pass
def run(state):
    return {"route": _route, "quantise": _quantise, "product": _product, "experts": _experts}[state["op"]](state)


def _route(s):
    if own:
        import roofline_driven_optimisation_gb300 as lib
        lib.route(s["logits"], s["ids"], s["weights"], s["offsets"], s["order"], bias=s["bias_values"],
                  score=lib.ROUTE_SOFTMAX if s["score"] == "softmax" else lib.ROUTE_SIGMOID, groups=s["groups"],
                  top_groups=s["top_groups"], renormalise=s["renormalise"], scale=2.5)
        return {"ids": s["ids"], "weights": s["weights"], "offsets": s["offsets"], "order": s["order"]}
    return _plain_route(s)


def _quantise(s):
    if own:
        import roofline_driven_optimisation_gb300 as lib
        lib.fp8_quantise(s["x"], s["codes"], s["scales"], block_rows=s["block_rows"])
        return {"codes": s["codes"], "scales": s["scales"]}
    codes, scales = _plain_quantise(s["x"], s["block_rows"])
    return {"codes": codes, "scales": scales}


def _product(s):
    if own:
        import roofline_driven_optimisation_gb300 as lib
        return lib.fp8_blocks(s["a"], s["a_scale"], s["b"], s["b_scale"], s["c"])
    return (_values(s["a"], s["a_scale"], 1) @ _values(s["b"], s["b_scale"], BLOCK)).to(s["c"].dtype)


def _experts(s):
    if own:
        import roofline_driven_optimisation_gb300 as lib
        return lib.experts(s["handle"], s["x"], s["offsets"], s["order"], s["weights"], s["out"])
    return _plain_experts(s)


# ------------------------------------------------------------------ plain forms
def _order(ids, experts):
    """Where each expert's slots begin, and the slots (token * top_k + rank) by expert, tokens in order."""
    flat = ids.reshape(-1).long()
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.cumsum(torch.zeros(experts, dtype=torch.int64, device=ids.device).scatter_add_(
        0, flat, torch.ones_like(flat)), 0)
    return offsets, torch.sort(flat, stable=True).indices.int()


def _plain_route(s):
    tokens, experts = s["logits"].shape
    x = s["logits"].double()
    score = torch.softmax(x, 1) if s["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-x))
    choice = x if s["bias_values"] is None and s["groups"] == 1 else score
    if s["bias_values"] is not None:
        choice = score + s["bias_values"].double()
    if s["groups"] > 1:
        part = choice.view(tokens, s["groups"], -1)
        best = torch.sort(part, dim=2, descending=True).values[:, :, :2].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        seen = torch.zeros_like(best).scatter_(1, kept, 1.0) > 0
        choice = part.masked_fill(~seen[:, :, None], -math.inf).view(tokens, experts)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :s["top_k"]]
    weights = score.gather(1, ids)
    if s["renormalise"]:
        weights = weights / weights.sum(1, keepdim=True)
    offsets, order = _order(ids, experts)
    return {"ids": ids.int(), "weights": (2.5 * weights).float(), "offsets": offsets, "order": order}


def _plain_quantise(x, block_rows):
    rows, cols = x.shape
    x = x.float()
    padded = torch.nn.functional.pad(x, (0, -cols % BLOCK, 0, -rows % block_rows))
    big = padded.abs().view(-1, block_rows, _blocks(cols), BLOCK).amax((1, 3))
    scale = big / torch.full_like(big, QMAX)
    scale = torch.where(scale >= SMALLEST, scale, torch.zeros_like(scale))
    r = torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))
    codes = (x * _spread_out(r, block_rows, rows, cols)).clamp(-QMAX, QMAX).to(torch.float8_e4m3fn)
    return codes, scale


def _spread_out(scale, block_rows, rows, cols):
    """A scale for every value: [..., rows, cols] from [..., blocks of rows, blocks of cols]."""
    scale = scale.repeat_interleave(BLOCK, -1)[..., :cols]
    return scale if block_rows == 1 else scale.repeat_interleave(block_rows, -2)[..., :rows, :]


def _values(codes, scale, block_rows):
    return codes.float() * _spread_out(scale, block_rows, *codes.shape[-2:])


def _plain_experts(s):
    tokens, hidden = s["x"].shape
    top_k, experts, width = s["top_k"], s["experts"], s["width"]
    x = _values(*_plain_quantise(s["x"], 1), 1)
    slots = tokens * top_k
    if slots < experts:                       # fewer slots than experts: each slot's own weights
        of = s["ids"].reshape(-1).long()
        rows = x.repeat_interleave(top_k, 0)[:, None]
        place = torch.arange(slots, device="cuda")
    else:                                     # a padded batch of each expert's tokens
        of = torch.arange(experts, device="cuda")
        order, begin = s["order"].long(), s["offsets"].long()
        owner = torch.searchsorted(begin, torch.arange(slots, device="cuda"), right=True) - 1
        place = torch.empty_like(order)
        place[order] = owner * s["most"] + torch.arange(slots, device="cuda") - begin[owner]
        rows = torch.zeros(experts * s["most"], hidden, device="cuda")
        rows[place] = x.repeat_interleave(top_k, 0)
        rows = rows.view(experts, s["most"], hidden)

    def weight(w):
        codes, scale = w
        if slots < experts:
            codes, scale = codes.view(torch.int8)[of].view(codes.dtype), scale[of]
        return _values(codes, scale, BLOCK)
    gate, up = torch.bmm(rows, weight(s["gate"])), torch.bmm(rows, weight(s["up"]))
    inner = (gate / (1.0 + torch.exp(-gate)) * up).view(-1, width)
    inner = _values(*_plain_quantise(inner, 1), 1).view(rows.shape[0], -1, width)
    y = torch.bmm(inner, weight(s["down"])).view(-1, hidden)[place].view(tokens, top_k, hidden)
    return (y * s["weights"][:, :, None]).sum(1).bfloat16()


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"route": _exact_route, "quantise": _exact_quantise, "product": _exact_product,
            "experts": _exact_experts}[case["op"]](s)


def _exact_route(s):
    """Ranks found by counting the experts that are ahead of each."""
    x, bias, groups = s["logits"].double(), s["bias_values"], s["groups"]
    tokens, experts = x.shape
    if s["score"] == "softmax":
        score = torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
    else:
        score = torch.sigmoid(x)
    choice = score + bias.double() if bias is not None else score if groups > 1 else x

    def ahead(v):                     # how many of a row are ahead of each: larger, or as large and earlier
        n = v.shape[1]
        earlier = torch.arange(n, device=v.device)[:, None] < torch.arange(n, device=v.device)
        return torch.cat([((p[:, :, None] > p[:, None]) | ((p[:, :, None] == p[:, None]) & earlier)).sum(1)
                          for p in v.split(max(1, (1 << 28) // (n * n)))])
    if groups > 1:
        part = choice.view(tokens, groups, experts // groups)
        out = ahead(part.topk(min(2, experts // groups), 2).values.sum(2)) >= s["top_groups"]
        choice = choice.masked_fill(out.repeat_interleave(experts // groups, 1), -math.inf)
    rank = ahead(choice)
    ids = torch.empty_like(rank).scatter_(1, rank, torch.arange(experts, device="cuda").expand(tokens, -1))[:, :s["top_k"]]
    weights = score.gather(1, ids)
    if s["renormalise"]:
        weights = weights / weights.sum(1, keepdim=True)
    return {"ids": None, "weights": 2.5 * weights, "offsets": None, "order": None}


def _on_grid(x):
    """x rounded to E4M3's values (ties to even), in 64 bits: three bits after the leading
    one, and steps of 2^-9 below 2^-6."""
    step = torch.ldexp(torch.ones_like(x), torch.frexp(x).exponent.clamp_min(-5) - 4)
    return (torch.round(x / step) * step).clamp(-QMAX, QMAX)


def _exact_held(x, block_rows=1):
    """Codes and scales of x.  A scale, its reciprocal and the product with it are held in 32
    bits by the operator's definition: bf16 values meet the middle between two codes often."""
    x = x.double()
    scale = torch.empty(-(-x.shape[0] // block_rows), _blocks(x.shape[1]), dtype=torch.float64, device=x.device)
    codes = torch.empty_like(x)
    at_row = torch.arange(x.shape[0], device=x.device) // block_rows
    for b in range(scale.shape[1]):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        big = torch.zeros(scale.shape[0], dtype=torch.float64, device=x.device).scatter_reduce_(0, at_row, part.abs().amax(1), "amax")
        scale[:, b] = (big / QMAX).float().double()
        r = (1.0 / scale[:, b].clamp_min(SMALLEST)).float().double()
        codes[:, b * BLOCK:(b + 1) * BLOCK] = _on_grid((part * r[at_row, None]).float().double())
    return codes, scale


def _exact_quantise(s):
    codes, scale = _exact_held(s["x"], s["block_rows"])
    return {"codes": codes, "scales": scale}


def _exact_scaled(codes, scale):
    """The values of a weight's codes."""
    at = [torch.arange(n, device="cuda") // BLOCK for n in codes.shape]
    return codes.double() * scale.double()[at[0]][:, at[1]]


def _exact_rows(codes, scale):
    return codes.double() * scale.double()[:, torch.arange(codes.shape[1], device="cuda") // BLOCK]


def _exact_product(s):
    if 2 * s["rows"] * s["cols"] * s["depth"] > 6e12:
        return None
    return _exact_rows(s["a"], s["a_scale"]) @ _exact_scaled(s["b"], s["b_scale"])


def _exact_experts(s):
    tokens, hidden = s["x"].shape
    x = _exact_rows(*_exact_held(s["x"]))
    out = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda")
    begin = s["offsets"].tolist()
    for e in range(s["experts"]):
        slots = s["order"][begin[e]:begin[e + 1]].long()
        if not len(slots):
            continue
        of = slots // s["top_k"]
        gate, up, down = (_exact_scaled(codes[e], scale[e]) for codes, scale in (s["gate"], s["up"], s["down"]))
        a = x[of] @ gate
        inner = _exact_rows(*_exact_held(a * torch.sigmoid(a) * (x[of] @ up)))
        out.index_add_(0, of, (inner @ down) * s["weights"].reshape(-1)[slots, None].double())
    return out
