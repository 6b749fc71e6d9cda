"""gemm_kv_attention against the 64-bit oracle over the cache's exact values.

The result is rounded once to bf16 (8 significant bits): at most 2^-8 of the value's
own size.  Before that it may be off, in shares of the row's and head's largest
sum_j P_j |V_j|, by the fp16 rounding of the probabilities times the page's scale,
2^-11, and by the scores' fp32 sums and the exponential, which move every probability
by less than 2^-11 for the score sizes used here (|s| below 2^6, D at most 512
products)."""
import numpy as np
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from oracle import serving as S
from serving_util import Case, check_status

pytestmark = pytest.mark.gpu
ROUND, SUM = 2.0 ** -8, 2.0 ** -11 + 2.0 ** -11
FMTS = [g.KV_E4M3, g.KV_INT8]


def run(fmt, heads, hq, dim, page, lengths, new=None, scale=0.0, gap=0, q_scale=1.0, one=False, path=None, want=None,
        change=None, **kw):
    new = [1] * len(lengths) if new is None else new
    c = Case(fmt, heads, dim, page, lengths, **kw)
    if change is not None:
        change(c)
        c.put()
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    tokens = int(start[-1])
    x = torch.from_numpy((q_scale * c.rng.normal(size=(tokens, hq * dim + gap))).astype(np.float32)).bfloat16()
    Q = x.cuda()[:, :hq * dim].unflatten(1, (hq, dim))
    O = torch.full((tokens, hq * dim + gap), float("nan"), dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    args = dict(start=None if one else torch.from_numpy(start).cuda(), max_new=max(new, default=1), scale=scale)
    if path is not None:
        g.force_path(path)
    try:
        g.kv_attention(c.cache, Q, O[:, :hq * dim].unflatten(1, (hq, dim)), lens, **args)
        ran = g.last_path()
    finally:
        g.force_path(g.PATH_AUTO)
    check_status()
    again = torch.full_like(O, float("nan"))
    if path is None:
        g.kv_attention(c.cache, Q, again[:, :hq * dim].unflatten(1, (hq, dim)), lens, **args)
        check_status()
        assert torch.equal(O.view(torch.int16), again.view(torch.int16))       # the same bits
    got = O[:, :hq * dim].float().cpu().numpy().reshape(tokens, hq, dim)
    ref, size = S.attention(c.np, fmt, Q.float().cpu().numpy(), lengths, start, scale)
    assert np.isfinite(got).all()
    off = np.abs(got - ref) - ROUND * np.abs(ref)
    assert (off <= SUM * size[..., None]).all(), \
        f"{(off / np.maximum(size, 1e-30)[..., None]).max():.2e} > {SUM:.2e} (path {ran})"
    assert gap == 0 or torch.isnan(O[:, hq * dim:]).all()
    if want is not None:
        assert ran == want
    return got, ref


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,heads", [(2, 2), (8, 2), (10, 2), (8, 1)])
def test_one_token(cuda_lib, fmt, dim, page, hq, heads):
    # one key, a page's edges, a slab's edges, several pages
    run(fmt, heads, hq, dim, page, [1, 2, 15, 16, 17, 31, 33, 64, 127, 300], one=True, seed=page + hq)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq,heads", [(2, 2), (8, 2), (6, 2), (16, 1)])
def test_several_tokens(cuda_lib, fmt, dim, hq, heads):
    # ragged: as many queries as keys, one, none, several; more than a row tile holds
    run(fmt, heads, hq, dim, 32, [3, 200, 90, 64, 65, 333], [3, 1, 0, 5, 8, 9], seed=hq)


@pytest.mark.parametrize("fmt", FMTS)
def test_chunk_of_a_prompt(cuda_lib, fmt):
    run(fmt, 2, 8, 128, 64, [150, 77], [100, 77])


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_without_keys_are_zero(cuda_lib, fmt):
    got, _ = run(fmt, 2, 4, 64, 16, [0, 40, 2, 0], [1, 1, 4, 3])
    assert (got[0] == 0).all() and (got[2:4] == 0).all() and (got[6:] == 0).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim", [64, 128])
def test_long_contexts_are_split(cuda_lib, fmt, dim):
    run(fmt, 2, 8, dim, 64, [20011], one=True)
    run(fmt, 1, 2, dim, 16, [5000, 3, 9001, 700], [2, 1, 3, 1])


def test_many_short_sequences(cuda_lib):
    rng = np.random.default_rng(2)
    run(g.KV_INT8, 4, 8, 64, 16, rng.integers(0, 90, 300).tolist(), one=True)


@pytest.mark.parametrize("layout", ["pages_heads", "pages_tokens", "heads_pages"])
@pytest.mark.parametrize("extra", [0, 16, 5])
def test_cache_layouts(cuda_lib, layout, extra):
    run(g.KV_E4M3, 3, 6, 128, 16, [100, 37], [2, 1], layout=layout, extra=extra)
    run(g.KV_INT8, 3, 6, 64, 16, [100, 37], [2, 1], layout=layout, extra=extra)


@pytest.mark.parametrize("gap,offset", [(0, 1), (8, 0), (3, 0), (3, 7), (1, 16)])
def test_strides_and_alignment(cuda_lib, gap, offset):
    run(g.KV_E4M3, 2, 4, 128, 32, [100, 37], gap=gap, offset=offset)


@pytest.mark.parametrize("dim,page", [(80, 16), (96, 64), (128, 24), (64, 1), (6, 5), (1, 4), (256, 64), (512, 16),
                                      (128, 256)])
@pytest.mark.parametrize("fmt", FMTS)
def test_unusual_sizes(cuda_lib, dim, page, fmt):
    run(fmt, 2, 4, dim, page, [130, 1, 40], [3, 1, 2])


@pytest.mark.parametrize("fmt", FMTS)
def test_given_scale_and_peaked_rows(cuda_lib, fmt):
    run(fmt, 2, 4, 128, 64, [500, 70], scale=0.3)
    run(fmt, 2, 4, 128, 64, [500, 70], q_scale=8.0)


@pytest.mark.parametrize("fmt", FMTS)
def test_page_scales_of_many_sizes(cuda_lib, fmt):
    # scales from 1e-9 to 1e9 of one another in V, and pages of zeros
    def spread(c):
        e = c.rng.uniform(-9, 9, c.np["vs"].shape)
        c.np["vs"][:] = (10.0 ** e).astype(np.float32)
        c.np["vs"][c.used[::5]] = 0.0
        c.np["ks"][c.used[1::7]] = 0.0
    run(fmt, 2, 4, 128, 16, [500, 70, 16], change=spread)
    # a row all of whose weight is on small pages while a large one is masked out by its score
    def outlier(c):
        c.np["vs"][c.used[0]] = 3e4
        c.np["k"][c.used[0]] = c.np["k"][c.used[0]] & 0x7F if fmt == g.KV_E4M3 else 127
    run(fmt, 1, 2, 64, 16, [300], change=outlier)


def test_queries_of_any_size(cuda_lib):
    # tiny and huge rows: the power-of-two scaling of a row is exact
    for q_scale, scale in ((2.0 ** -100, 2.0 ** 98), (2.0 ** 60, 2.0 ** -62), (0.0, 0.0)):
        run(g.KV_INT8, 2, 4, 128, 32, [100], q_scale=q_scale, scale=scale)


def test_unused_rows_and_pages_never_matter(cuda_lib):
    # NaN codes, NaN and infinite scales wherever no visible token is
    def poison(c):
        seen = np.zeros((c.pages, c.page), bool)
        for b, n in enumerate([37, 5, 64]):
            for t in range(n):
                seen[c.np["table"][b, t // c.page], t % c.page] = True
        for name in ("k", "v"):
            c.np[name] = np.where(seen[:, None, :, None], c.np[name], 0x7F)
            c.np[name + "s"][~seen.any(1)] = [[np.nan, np.inf]]
    run(g.KV_E4M3, 2, 4, 128, 32, [37, 5, 64], change=poison)
    run(g.KV_E4M3, 2, 4, 64, 16, [37, 5, 64], [3, 2, 1], change=poison)


def test_later_tokens_never_reach_earlier_queries(cuda_lib):
    # the newest token's K and V are NaN: only its own query may be NaN
    c = Case(g.KV_E4M3, 1, 128, 32, [50])
    p = c.np["table"][0, 1]
    for name in ("k", "v"):
        c.np[name][p, 0, 49 - 32] = 0x7F
    c.put()
    Q = torch.randn(4, 2, 128, device="cuda").bfloat16()
    O = torch.empty_like(Q)
    g.kv_attention(c.cache, Q, O, torch.tensor([50], dtype=torch.int32, device="cuda"),
                   start=torch.tensor([0, 4], dtype=torch.int32, device="cuda"), max_new=4)
    check_status()
    assert torch.isfinite(O[:3]).all() and torch.isnan(O[3]).any()


def test_nan_shows_where_it_is_seen(cuda_lib):
    for where in ("q", "k", "v", "ks", "vs"):
        c = Case(g.KV_E4M3, 2, 64, 16, [40])
        p = c.np["table"][0, 1]
        if where in ("k", "v"):
            c.np[where][p, 0, 3, 5] = 0xFF
        elif where != "q":
            c.np[where][p, 0] = np.nan
        c.put()
        Q = torch.randn(1, 4, 64, device="cuda").bfloat16()
        if where == "q":
            Q[0, :2, 7] = float("nan")
        O = torch.empty_like(Q)
        g.kv_attention(c.cache, Q, O, torch.tensor([40], dtype=torch.int32, device="cuda"))
        check_status()
        assert torch.isnan(O[0, :2]).any(-1).all() and torch.isfinite(O[0, 2:]).all(), where


def test_offsets_past_32_bits(cuda_lib):
    pages, H, P, D = 36000, 8, 128, 128               # 4.7 GB
    k = torch.empty(pages, H, P, D, dtype=torch.int8, device="cuda")
    v = torch.empty_like(k)
    used = [pages - 1, 3, pages - 5, 20000]
    for t in (k, v):
        for p in used:
            t[p] = torch.randint(-127, 128, (H, P, D), device="cuda").to(torch.int8)
    s = torch.full((pages, H), 0.01, device="cuda")
    table = torch.tensor([used], dtype=torch.int32, device="cuda")
    Q = torch.randn(1, H, D, device="cuda").bfloat16()
    O = torch.empty_like(Q)
    length = 3 * P + 50
    g.kv_attention(g.KVCache(k, v, s, s, table), Q, O, torch.tensor([length], dtype=torch.int32, device="cuda"))
    check_status()
    small = {"k": k[used].cpu().numpy().view(np.uint8), "v": v[used].cpu().numpy().view(np.uint8),
             "ks": np.full((4, H), 0.01, np.float32), "vs": np.full((4, H), 0.01, np.float32),
             "table": np.array([[0, 1, 2, 3]])}
    ref, size = S.attention(small, g.KV_INT8, Q.float().cpu().numpy(), [length], [0, 1])
    assert (np.abs(O.float().cpu().numpy() - ref) <= ROUND * np.abs(ref) + SUM * size[..., None]).all()


def test_misfits_are_reported(cuda_lib):
    def call(lengths=(40,), start=(0, 1), table=None, max_new=1):
        c = Case(g.KV_INT8, 1, 64, 16, [40])
        if table is not None:
            c.table[0, 1] = table
        Q = torch.randn(1, 1, 64, device="cuda").bfloat16()
        O = torch.zeros_like(Q)
        g.kv_attention(c.cache, Q, O, torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                       start=torch.tensor(start, dtype=torch.int32, device="cuda"), max_new=max_new)
        torch.cuda.synchronize()
        return g.device_status()
    bad = (g.GEMM_ERR_INVALID_ARG, 61)
    assert call() == (0, 0)
    assert call(table=99) == bad and call(table=-5) == bad
    assert call(lengths=(49,)) == bad and call(lengths=(-2,)) == bad      # three columns of 16
    assert call(start=(0, 2), max_new=2) == bad and call(start=(1, 0)) == bad
    assert call() == (0, 0)


def test_streams_and_graph(cuda_lib):
    c = Case(g.KV_E4M3, 2, 128, 16, [4000, 20])
    lens = torch.tensor([4000, 20], dtype=torch.int32, device="cuda")
    Q = torch.randn(2, 8, 128, device="cuda").bfloat16()
    want = g.kv_attention(c.cache, Q, torch.empty_like(Q), lens).clone()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    torch.cuda.synchronize()
    for s in streams:                                 # each stream has a workspace of its own
        with torch.cuda.stream(s):
            outs.append(g.kv_attention(c.cache, Q, torch.empty_like(Q), lens))
    check_status()
    assert all(torch.equal(o, want) for o in outs)
    size = g.gemm_kv_attention_workspace(2, 2, 8, 128, 1)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    O = torch.empty_like(Q)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        g.kv_attention(c.cache, Q, O, lens, workspace=ws)
    for length in (4000, 7, 1234):
        lens[0] = length
        gr.replay()
        check_status()
        assert torch.equal(O, g.kv_attention(c.cache, Q, torch.empty_like(Q), lens))
