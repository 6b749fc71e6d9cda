"""The operators of a serving step, as measured cases.

Three operators that a decode step needs between and after its GEMMs:

  append     gemm_kv_append: rotate Q and K by position and store K, V in a paged
             8-bit cache with one scale for each page and head
  attention  gemm_kv_attention: attention of the newest tokens over that cache
  sample     gemm_sample_*: temperature, top-k, top-p and min-p sampling of the LM
             head's logits from given uniform numbers

``own`` selects the library's kernels; otherwise ``run`` computes the same values
with elementary torch operations in 32 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

E4M3, INT8 = "e4m3", "int8"
QMAX = {E4M3: 448.0, INT8: 127.0}
SMALLEST = 2.0 ** -126      # a page whose scale would be below this stores zeros
ONE = 2.0 ** 40             # the integer mass of a token whose weight is 1


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one user's decode step of a 32-head, 128-wide layer (the LLaMA-7B layer of
        # the repository's benchmark): 1 token, latency counts
        dict(name="append 1 token", op="append", seqs=1, base=1000, new=1, hq=32, hkv=32, dim=128,
             page=64, fmt=E4M3, interleaved=False),
        # a batch of 64 decoding users, grouped heads, INT8, interleaved rotation
        dict(name="append 64 x 1 token", op="append", seqs=64, base=2011, new=1, hq=32, hkv=8, dim=128,
             page=16, fmt=INT8, interleaved=True),
        # ragged prompts prefilled together, starting inside pages
        dict(name="append 7 x 611 tokens, d 64", op="append", seqs=7, base=93, new=611, hq=16, hkv=4,
             dim=64, page=32, fmt=INT8, interleaved=False),
        # one long prompt of the benchmark's layer
        dict(name="append 16384 tokens", op="append", seqs=1, base=0, new=16384, hq=32, hkv=32, dim=128,
             page=64, fmt=E4M3, interleaved=False),
        # one user with a short context: latency counts
        dict(name="attend 1 x 777", op="attention", seqs=1, ctx=777, new=1, hq=32, hkv=32, dim=128, page=64,
             fmt=E4M3),
        # one user with a very long context, grouped heads
        dict(name="attend 1 x 131071", op="attention", seqs=1, ctx=131071, new=1, hq=32, hkv=8, dim=128,
             page=64, fmt=E4M3),
        # checking 5 drafted tokens a user, narrow heads, small pages
        dict(name="attend 24 x 1500, 5 tokens", op="attention", seqs=24, ctx=1500, new=5, hq=16, hkv=4,
             dim=64, page=16, fmt=INT8),
        # a batch of the benchmark's layer, no grouping
        dict(name="attend 16 x 4096, 32 heads", op="attention", seqs=16, ctx=4096, new=1, hq=32, hkv=32,
             dim=128, page=64, fmt=INT8),
        # a large ragged batch with grouped heads
        dict(name="attend 128 x 8192", op="attention", seqs=128, ctx=8192, new=1, hq=32, hkv=8, dim=128,
             page=32, fmt=E4M3),
        # one user's token from the LM head (vocabulary 32000): latency counts
        dict(name="sample 1 x 32000", op="sample", rows=1, vocab=32000, dtype="bf16", mode="all"),
        # a batch, every row with settings of its own
        dict(name="sample 64 x 32000 mixed", op="sample", rows=64, vocab=32000, dtype="bf16", mode="mixed"),
        # a large batch over a large vocabulary in fp32 (an odd row length)
        dict(name="sample 384 x 131071", op="sample", rows=384, vocab=131071, dtype="f32", mode="all"),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "sample"])
    fmt = rng.choice([E4M3, INT8])
    page = rng.choice([16, 32, 64, 128])
    dim = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8, 8, 16, 32])
    hq = hkv * rng.choice([1, 1, 2, 4, 5, 8] if hkv < 16 else [1, 2])
    if op == "append":
        seqs = _spread(rng, 1, 256)
        # decoding (1 token each) or prompts, up to the largest listed case's tokens and bytes
        new = 1 if rng.random() < 0.4 else _spread(rng, 1, 16384)
        most = 16384 * 96 * 128 // ((hq + 2 * hkv) * dim)
        seqs = max(1, min(seqs, most // new))
        new = min(new, most)
        return dict(op=op, seqs=seqs, base=rng.randrange(0, 3000), new=new, hq=hq, hkv=hkv, dim=dim,
                    page=page, fmt=fmt, interleaved=rng.random() < 0.5)
    if op == "attention":
        seqs, ctx = _spread(rng, 1, 256), _spread(rng, 1, 131072)
        new = rng.choice([1, 1, 1, 2, 3, 4, 6, 8])
        # codes at most half of the largest listed case's, scores at most 2^27
        seqs = max(1, min(seqs, (128 * 8192 * 8 * 128 // 2) // (ctx * hkv * dim), (1 << 27) // (ctx * hq * new)))
        most = min((128 * 8192 * 8 * 128 // 2) // (seqs * hkv * dim), (1 << 27) // (seqs * hq * new))
        ctx = max(new, min(ctx, most))
        return dict(op=op, seqs=seqs, ctx=ctx, new=new, hq=hq, hkv=hkv, dim=dim, page=page, fmt=fmt)
    rows, vocab = _spread(rng, 1, 512), _spread(rng, 1000, 262144)
    rows = max(1, min(rows, 384 * 131071 // vocab))
    return dict(op=op, rows=rows, vocab=vocab, dtype=rng.choice(["bf16", "f32"]),
                mode=rng.choice(["all", "mixed", "mixed", "plain", "top_k", "top_p", "min_p"]))


def _ladder(n, mean, least=0):
    """n whole numbers around `mean`, from a quarter to seven quarters of it."""
    v = (mean * (0.25 + 1.5 * (torch.arange(n, dtype=torch.float64) + 0.5) / n)).round().long()
    return v.clamp_min(least)


def work(case):
    if case["op"] == "append":
        tokens = int(_ladder(case["seqs"], case["new"], 1).sum())
        hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
        pages = tokens / case["page"]
        return {"bytes": tokens * (2 * (hq + 2 * hkv) * dim + 2 * hq * dim + 2 * hkv * dim) + pages * hkv * 8 + tokens * dim * 4,
                "flops": tokens * (3 * (hq + hkv) * dim + 3 * hkv * dim)}
    if case["op"] == "attention":
        tokens = int(_ladder(case["seqs"], case["ctx"], case["new"]).sum())
        rows = case["seqs"] * case["new"] * case["hq"]
        return {"bytes": 2 * tokens * case["hkv"] * (case["dim"] + 4 / case["page"]) + 4 * rows * case["dim"],
                "flops": 4 * tokens * case["new"] * case["hq"] * case["dim"]}
    size = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": case["rows"] * (case["vocab"] * size + 28), "flops": case["rows"] * case["vocab"] * 4}


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _ints(values):
    return torch.as_tensor(values).to(device="cuda", dtype=torch.int32)


def _shuffled(g, *ladders):
    """The ladders in one random order."""
    order = torch.randperm(len(ladders[0]), generator=g, device="cuda")
    return [v.cuda()[order] for v in ladders]


def _page_table(lengths, page, g):
    """Random distinct pages for sequences that hold up to `lengths` tokens, and the number of pages."""
    need = (lengths + page - 1) // page
    total = int(need.sum()) + 5
    cols = max(1, int(need.max()))
    order = torch.randperm(total, generator=g, device="cuda").int()
    at = torch.cumsum(need, 0) - need
    col = torch.arange(cols, device="cuda")
    table = order[(at[:, None] + col).clamp_max(total - 1)]
    return torch.where(col < need[:, None], table, torch.zeros_like(table)).contiguous(), total


def _tables(positions, dim):
    """cos and sin of the position rotation, base 10000."""
    f = 10000.0 ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cos(a).float(), torch.sin(a).float()


def _code_type(fmt):
    return torch.float8_e4m3fn if fmt == E4M3 else torch.int8


def _random_cache(total, heads, page, dim, fmt, g):
    """A pool whose pages already hold quantised normal values, each page and head with its scale."""
    codes = torch.empty(total, heads, page, dim, dtype=_code_type(fmt), device="cuda")
    scale = torch.empty(total, heads, device="cuda")
    step = max(1, (1 << 26) // (heads * page * dim))
    for p in range(0, total, step):
        x = torch.randn(codes[p:p + step].shape, generator=g, device="cuda")
        s = x.abs().amax((2, 3)) / QMAX[fmt]
        x = x / s[:, :, None, None]
        codes[p:p + step] = (x.round() if fmt == INT8 else x).clamp(-QMAX[fmt], QMAX[fmt]).to(codes.dtype)
        # heads and pages differ in size, as keys' and values' do
        scale[p:p + step] = s * torch.exp(0.3 * torch.randn(s.shape, generator=g, device="cuda"))
    return codes, scale


def prepare(case, seed):
    state = dict(case)
    state.update({"append": _prepare_append, "attention": _prepare_attention, "sample": _prepare_sample}[case["op"]](case, seed))
    if own and case["op"] != "sample":      # the handle on the cache that a serving program keeps
        import roofline_driven_optimisation_gb300 as lib
        state["cache"] = lib.KVCache(state["k"], state["v"], state["k_scale"], state["v_scale"], state["table"])
    return state


def _prepare_append(case, seed):
    g = _gen(seed)
    seqs, page, dim, hq, hkv = (case[k] for k in ("seqs", "page", "dim", "hq", "hkv"))
    new, base = _shuffled(g, _ladder(seqs, case["new"], 1), _ladder(seqs, case["base"]))
    tokens = int(new.sum())
    table, total = _page_table(base + new, page, g)
    k, k_scale = _random_cache(total, hkv, page, dim, case["fmt"], g)
    v, v_scale = _random_cache(total, hkv, page, dim, case["fmt"], g)
    # one matrix, as the qkv GEMM leaves it: Q, K and V of a token side by side
    qkv = torch.randn(tokens, (hq + 2 * hkv) * dim, generator=g, device="cuda").bfloat16()
    start = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
    start[1:] = torch.cumsum(new, 0)
    cos, sin = _tables(int((base + new).max()), dim)
    return dict(k=k, v=v, k_scale=k_scale, v_scale=v_scale, table=table, base=_ints(base), start=start,
                most=int(new.max()), cos=cos, sin=sin, q_out=torch.empty(tokens, hq, dim, dtype=torch.bfloat16, device="cuda"),
                q_in=qkv[:, :hq * dim].unflatten(1, (hq, dim)), k_in=qkv[:, hq * dim:(hq + hkv) * dim].unflatten(1, (hkv, dim)),
                v_in=qkv[:, (hq + hkv) * dim:].unflatten(1, (hkv, dim)))


def _prepare_attention(case, seed):
    g = _gen(seed)
    seqs, page, dim, hq, hkv, new = (case[k] for k in ("seqs", "page", "dim", "hq", "hkv", "new"))
    lengths, = _shuffled(g, _ladder(seqs, case["ctx"], new))
    table, total = _page_table(lengths, page, g)
    k, k_scale = _random_cache(total, hkv, page, dim, case["fmt"], g)
    v, v_scale = _random_cache(total, hkv, page, dim, case["fmt"], g)
    # queries a little larger than keys, so that a row's softmax has a few large entries
    q = (1.5 * torch.randn(seqs * new, hq, dim, generator=g, device="cuda")).bfloat16()
    return dict(k=k, v=v, k_scale=k_scale, v_scale=v_scale, table=table, lengths=_ints(lengths),
                start=_ints(torch.arange(seqs + 1) * new), q_in=q, out=torch.empty_like(q))


def _prepare_sample(case, seed):
    g = _gen(seed)
    rows, vocab, mode = case["rows"], case["vocab"], case["mode"]
    logits = 2.5 * torch.randn(rows, vocab, generator=g, device="cuda")
    # a few likely tokens a row, and some that are forbidden
    at = torch.randint(vocab, (rows, 20), generator=g, device="cuda")
    logits.scatter_add_(1, at, 9.0 * torch.rand(rows, 20, generator=g, device="cuda"))
    logits.masked_fill_(torch.rand(rows, vocab, generator=g, device="cuda") < 0.01, -math.inf)
    if case["dtype"] == "bf16":
        logits = logits.bfloat16()

    def of(values):                       # a setting of each row's own
        return torch.tensor(values, device="cuda")[torch.randint(len(values), (rows,), generator=g, device="cuda")]
    mixed = mode == "mixed"
    return dict(
        logits=logits, u=torch.rand(rows, generator=g, device="cuda"),
        temperature=of([0.0, 0.3, 0.7, 1.0, 1.5]) if mixed else torch.full((rows,), 0.8, device="cuda"),
        top_k=of([0, 1, 5, 40, 50, 1000]).int() if mixed else _ints([50] * rows) if mode in ("all", "top_k") else None,
        top_p=of([0.1, 0.5, 0.9, 0.95, 1.0]) if mixed else torch.full((rows,), 0.95, device="cuda") if mode in ("all", "top_p") else None,
        min_p=of([0.0, 0.02, 0.1]) if mixed else torch.full((rows,), 0.03, device="cuda") if mode in ("all", "min_p") else None,
        token=torch.empty(rows, dtype=torch.int32, device="cuda"), logprob=torch.empty(rows, device="cuda"))


# ------------------------------------------------------------------ one pass
def run(state):
    return {"append": _append, "attention": _attention, "sample": _sample}[state["op"]](state)


def _append(s):
    if own:
        import roofline_driven_optimisation_gb300 as lib
        lib.kv_append(s["cache"], s["q_in"], s["k_in"], s["v_in"], s["cos"], s["sin"], s["base"], s["q_out"],
                      start=s["start"], max_new=s["most"], interleaved=s["interleaved"])
    else:
        _plain_append(s)
    return {"q": s["q_out"], "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _attention(s):
    if own:
        import roofline_driven_optimisation_gb300 as lib
        lib.kv_attention(s["cache"], s["q_in"], s["out"], s["lengths"], start=s["start"], max_new=s["new"])
        return s["out"]
    return _plain_attention(s)


def _sample(s):
    if own:
        import roofline_driven_optimisation_gb300 as lib
        lib.sample(s["logits"], s["u"], s["token"], s["logprob"], temperature=s["temperature"], top_k=s["top_k"],
                   top_p=s["top_p"], min_p=s["min_p"])
        return {"token": s["token"], "logprob": s["logprob"]}
    return _plain_sample(s)


# ------------------------------------------------------------------ plain forms
def _rotate(x, c, s, interleaved):
    x = x.float()
    c, s = c[:, None], s[:, None]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _codes(x, scale, fmt):
    """x held as codes: x / scale on the format's grid (the reciprocal is rounded once)."""
    r = torch.where(scale >= SMALLEST, 1.0 / scale, torch.zeros_like(scale))
    x = (x * r).clamp(-QMAX[fmt], QMAX[fmt])
    return (x.round() if fmt == INT8 else x).to(_code_type(fmt))


def _plain_append(s):
    fmt, page = s["fmt"], s["page"]
    base, start, table = s["base"].long(), s["start"].long(), s["table"].long()
    seqs = len(base)
    tokens = s["k_in"].shape[0]
    of = torch.searchsorted(start, torch.arange(tokens, device="cuda"), right=True) - 1   # token -> sequence
    pos = base[of] + torch.arange(tokens, device="cuda") - start[of]
    c, si = s["cos"][pos], s["sin"][pos]
    s["q_out"].copy_(_rotate(s["q_in"], c, si, s["interleaved"]))
    at, off = table[of, pos // page], pos % page
    # sequences whose first new token lands in a page that holds earlier ones
    first = table[torch.arange(seqs, device="cuda"), base // page]
    kept = (torch.arange(page, device="cuda") < (base % page)[:, None])[:, None, :, None]

    def store(x, codes, scale):
        big = torch.zeros_like(scale).scatter_reduce_(0, at[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
        written = torch.zeros_like(scale[:, 0]).index_fill_(0, at, 1.0)[:, None] > 0
        grown = big / torch.full_like(big, QMAX[fmt])
        grown = torch.where(grown >= SMALLEST, grown, torch.zeros_like(grown))
        old = scale[first]
        fresh = torch.where(written, grown, scale)
        fresh[first] = torch.where((base % page > 0)[:, None], torch.maximum(old, grown[first]), fresh[first])
        held = codes.view(torch.int8)                     # the codes' bytes, for indexing
        earlier = held[first]
        again = _codes(earlier.view(codes.dtype).float() * old[..., None, None], fresh[first][..., None, None], fmt)
        moved = kept & (fresh[first] > old)[..., None, None]
        held[first] = torch.where(moved, again.view(torch.int8), earlier)
        held[at, :, off] = _codes(x, fresh[at][..., None], fmt).view(torch.int8)
        scale.copy_(fresh)

    store(_rotate(s["k_in"], c, si, s["interleaved"]), s["k"], s["k_scale"])
    store(s["v_in"].float(), s["v"], s["v_scale"])


def _plain_attention(s):
    seqs, new, hq, hkv, dim, page = (s[k] for k in ("seqs", "new", "hq", "hkv", "dim", "page"))
    lengths, table = s["lengths"].long(), s["table"].long()
    keys = table.shape[1] * page

    def values(codes, scale):
        x = codes.view(torch.int8)[table].view(codes.dtype).float()          # seqs, pages, heads, page, dim
        x = x * scale[table][..., None, None]
        return x.transpose(1, 2).reshape(seqs, hkv, keys, dim)
    q = s["q_in"].float().view(seqs, new, hkv, hq // hkv, dim).permute(0, 2, 1, 3, 4).reshape(seqs, hkv, -1, dim)
    scores = (q @ values(s["k"], s["k_scale"]).transpose(2, 3)) / math.sqrt(dim)
    last = lengths[:, None] - new + torch.arange(new, device="cuda")           # the last key a query sees
    seen = torch.arange(keys, device="cuda") <= last[..., None]                # seqs, new, keys
    scores = scores.view(seqs, hkv, new, -1, keys).masked_fill(~seen[:, None, :, None], -math.inf)
    scores = torch.exp(scores - scores.amax(-1, keepdim=True))
    total = scores.sum(-1, keepdim=True)
    out = scores.reshape(seqs, hkv, -1, keys) @ values(s["v"], s["v_scale"])
    out = out.view(seqs, hkv, new, -1, dim) / total
    return out.permute(0, 2, 1, 3, 4).reshape(seqs * new, hq, dim).bfloat16()


def _plain_sample(s):
    logits, rows = s["logits"].float(), s["logits"].shape[0]
    vocab = logits.shape[1]
    greedy = s["temperature"] <= 0
    top = logits.amax(1, keepdim=True)
    one = torch.ones_like(s["temperature"])
    z = (logits - top) * (1.0 / torch.where(greedy, one, s["temperature"]))[:, None]
    weight = torch.exp(z)
    mass = (weight * ONE).long()
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices
    ranked = mass.gather(1, order)
    rank = torch.arange(vocab, device="cuda")
    if s["top_k"] is not None:
        k = torch.where(s["top_k"] > 0, s["top_k"], vocab)
        ranked = ranked * (rank < k[:, None])
    if s["top_p"] is not None:
        bound = s["top_p"].double() * ranked.sum(1).double()
        before = torch.cumsum(ranked, 1) - ranked
        ranked = ranked * ((before.double() < bound[:, None]) | (rank == 0))
    if s["min_p"] is not None:
        ranked = ranked * (weight.gather(1, order) >= s["min_p"][:, None])
    ranked = ranked * ((rank == 0) | ~greedy[:, None])
    kept = torch.zeros_like(mass).scatter_(1, order, ranked)
    running = torch.cumsum(kept, 1)
    total = running[:, -1]
    target = torch.minimum((s["u"].double() * total.double()).long(), total - 1)
    token = (running <= target[:, None]).sum(1)
    chosen = z.gather(1, token[:, None])[:, 0]
    logprob = chosen - torch.log((total.double() / ONE).float())
    return {"token": token.int(), "logprob": logprob.view(rows)}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"append": _exact_append, "attention": _exact_attention, "sample": _exact_sample}[case["op"]](s)


def _on_grid(x, fmt):
    """x rounded to the format's values (ties to even), in 64 bits."""
    x = x.clamp(-QMAX[fmt], QMAX[fmt])
    if fmt == INT8:
        return torch.round(x)
    # E4M3: three bits after the leading one, and steps of 2^-9 below 2^-6
    step = torch.ldexp(torch.ones_like(x), torch.frexp(x).exponent.clamp_min(-5) - 4)
    return torch.round(x / step) * step


def _exact_append(s):
    fmt, page, dim = s["fmt"], s["page"], s["dim"]
    cos, sin = s["cos"].double(), s["sin"].double()
    at = torch.arange(dim, device="cuda")
    i, j = (at[0::2], at[1::2]) if s["interleaved"] else (at[:dim // 2], at[dim // 2:])
    out = {"q": torch.zeros_like(s["q_out"], dtype=torch.float64)}
    for name in ("k", "v", "k_scale", "v_scale"):
        out[name] = s[name].double()

    def turned(x, first):
        y, n = torch.empty_like(x), len(x)
        c, t = cos[first:first + n, None], sin[first:first + n, None]
        y[..., i] = x[..., i] * c - x[..., j] * t
        y[..., j] = x[..., j] * c + x[..., i] * t
        return y
    base, start = s["base"].tolist(), s["start"].tolist()
    for b, first in enumerate(base):                 # one sequence after another
        rows = slice(start[b], start[b + 1])
        n = start[b + 1] - start[b]
        out["q"][rows] = turned(s["q_in"][rows].double(), first)
        held = first % page                          # earlier tokens of its first page
        last = -(-(first + n) // page)
        g = s["table"][b, first // page:last].long()
        for name, x in (("k", turned(s["k_in"][rows].double(), first)), ("v", s["v_in"][rows].double())):
            heads = x.shape[1]
            whole = torch.zeros(len(g) * page, heads, dim, dtype=torch.float64, device="cuda")
            whole[held:held + n] = x
            whole = whole.view(len(g), page, heads, dim).transpose(1, 2)
            scale = whole.abs().amax((2, 3)) / QMAX[fmt]
            old = out[name + "_scale"][g[0]]
            if held:
                scale[0] = torch.maximum(scale[0], old)
            codes = _on_grid(whole / torch.where(scale > 0, scale, 1.0)[..., None, None], fmt)
            before = out[name][g]
            if held:
                earlier = _on_grid(before[0] * (old / scale[0])[:, None, None], fmt)
                codes[0, :, :held] = torch.where((scale[0] > old)[:, None, None], earlier, before[0])[:, :held]
            used = held + n - (len(g) - 1) * page    # tokens of its last page, after the call
            codes[-1, :, used:] = before[-1, :, used:]
            out[name][g], out[name + "_scale"][g] = codes, scale
    if fmt == INT8:                     # whole numbers have no error
        out["k"] = out["v"] = None
    return out


def _exact_attention(s):
    new, hq, hkv, dim = (s[k] for k in ("new", "hq", "hkv", "dim"))
    out = torch.zeros(len(s["q_in"]), hq, dim, dtype=torch.float64, device="cuda")
    for b, length in enumerate(s["lengths"].tolist()):
        pages = s["table"][b, :-(-length // s["page"])].long()
        seen = torch.arange(length, device="cuda") <= length - new + torch.arange(new, device="cuda")[:, None]
        for h in range(hkv):
            k = (s["k"][pages, h].double() * s["k_scale"][pages, h].double()[:, None, None]).reshape(-1, dim)[:length]
            v = (s["v"][pages, h].double() * s["v_scale"][pages, h].double()[:, None, None]).reshape(-1, dim)[:length]
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            q = s["q_in"][b * new:(b + 1) * new, heads].double()
            p = torch.softmax((q @ k.T / math.sqrt(dim)).masked_fill(~seen[:, None], -math.inf), -1)
            out[b * new:(b + 1) * new, heads] = p @ v
    return out


def _exact_sample(s):
    logits = s["logits"].double().cpu().numpy()
    get = lambda name, none: none if s[name] is None else s[name].double().cpu().numpy()  # noqa: E731
    rows, vocab = logits.shape
    temperature, u = get("temperature", None), get("u", None)
    k, p, least = get("top_k", np.zeros(rows)), get("top_p", np.full(rows, 2.0)), get("min_p", np.zeros(rows))
    logprob = np.zeros(rows)
    for r in range(rows):
        x = logits[r] - logits[r].max()
        if temperature[r] <= 0:
            continue
        w = np.exp(x / temperature[r])
        order = np.argsort(-x, kind="stable")
        ranked = w[order]
        if k[r] > 0:
            ranked[int(k[r]):] = 0
        before = np.cumsum(ranked) - ranked
        keep = before < p[r] * ranked.sum()
        keep[0] = True
        ranked = np.where(keep & (ranked >= least[r]), ranked, 0)
        kept = np.zeros(vocab)
        kept[order] = ranked
        running = np.cumsum(kept)
        token = min(int(np.searchsorted(running, u[r] * running[-1], side="right")), vocab - 1)
        logprob[r] = x[token] / temperature[r] - math.log(running[-1])
    return {"token": None, "logprob": logprob}
