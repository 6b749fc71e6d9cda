"""gemm_kv_append against the oracle.

Every step of the operator has one rounding that its definition states (products
and sums of the rotation, one division, one reciprocal, one product, the format's
grid), so codes and scales must equal the oracle's fp32 form bit for bit.  Against
the 64-bit form: with y the exact rotated value and s the stored scale, the fp32
steps move x/s by at most 8 * 2^-24 of |x|/s, and the grid rounds to half a step:
INT8 0.5 s, E4M3 2^-4 |y| or 2^-10 s among the subnormals.  So
    |stored - y| <= half step + 2^-20 * (qmax * s)
holds with the exact y, and the rotated queries (bf16) hold to 2^-8 |y| + 2^-20 times
their row's size."""
import numpy as np
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from oracle import serving as S
from serving_util import Case, check_status

pytestmark = pytest.mark.gpu


def _angles(positions, pairs):
    f = 10000.0 ** (-np.arange(pairs) / max(1, pairs))
    a = np.arange(positions)[:, None] * f
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def _rows(rng, tokens, heads, dim, gap):
    """bf16 [tokens][heads][dim] inside wider rows, and its fp32 values."""
    x = torch.from_numpy(rng.normal(size=(tokens, heads * dim + gap)).astype(np.float32)).bfloat16()
    view = x[:, :heads * dim].unflatten(1, (heads, dim))
    return x.cuda()[:, :heads * dim].unflatten(1, (heads, dim)), view.float().numpy()


def run(fmt, heads, hq, dim, page, base, new, rot=None, interleaved=False, layout="pages_heads", gap=0, seed=0,
        one=False, path=None, **kw):
    rot = dim if rot is None else rot
    lengths = [b + n for b, n in zip(base, new)]
    c = Case(fmt, heads, dim, page, lengths, layout=layout, seed=seed, **kw)
    tokens = sum(new)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    Q, qn = _rows(c.rng, tokens, max(hq, 1), dim, gap)
    K, kn = _rows(c.rng, tokens, heads, dim, gap)
    V, vn = _rows(c.rng, tokens, heads, dim, gap)
    cos, sin = _angles(max(lengths) if lengths else 1, rot // 2)
    out = torch.full((tokens, hq, dim), float("nan"), dtype=torch.bfloat16, device="cuda") if hq else None
    pool = {n: t.clone() for n, t in c.flat.items()}
    if path is not None:
        g.force_path(path)
    try:
        g.kv_append(c.cache, Q if hq else None, K, V, torch.from_numpy(cos).cuda() if rot else None,
                    torch.from_numpy(sin).cuda() if rot else None, torch.tensor(base, dtype=torch.int32, device="cuda"),
                    out, start=None if one else torch.from_numpy(start).cuda(), max_new=max(new, default=0),
                    interleaved=interleaved)
        ran = g.last_path()
    finally:
        g.force_path(g.PATH_AUTO)
    check_status()
    q32 = S.append(c.np, fmt, qn if hq else None, kn, vn, cos, sin, base, start, interleaved, np.float32)
    for name in ("ks", "vs"):
        assert np.array_equal(c.got(name), c.np[name]), name
    for name in ("k", "v"):
        assert np.array_equal(c.got(name), c.np[name]), name
    # nothing else of the pool has moved: padding, other pages, other rows
    for name in ("k", "v"):
        view = c.views[name].view(torch.uint8)
        want = torch.as_strided(pool[name], view.shape, view.stride(), view.storage_offset())
        want.copy_(torch.from_numpy(c.np[name]))
        assert torch.equal(pool[name], c.flat[name])
    # 64-bit bounds on what is stored
    y = {"k": S.rotate(kn, cos[_pos(base, new)], sin[_pos(base, new)], interleaved), "v": vn.astype(np.float64)}
    for name in ("k", "v"):
        for b in range(len(base)):
            for i in range(new[b]):
                t = base[b] + i
                p, r = c.np["table"][b, t // page], t % page
                s = c.np[name + "s"][p].astype(np.float64)[:, None]
                x, v = y[name][start[b] + i], S.values(c.got(name)[p, :, r], fmt) * s
                half = 0.5 * s if fmt == g.KV_INT8 else np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10)
                assert (np.abs(v - x) <= half + 2.0 ** -20 * S.QMAX[fmt] * s).all()
    if hq:
        q64 = S.rotate(qn, cos[_pos(base, new)], sin[_pos(base, new)], interleaved)
        got = out.float().cpu().numpy()
        assert (np.abs(got - q64) <= 2.0 ** -8 * np.abs(q64) + 2.0 ** -20 * np.abs(qn).max()).all()
        assert np.array_equal(got, torch.from_numpy(q32).bfloat16().float().numpy())
    return ran


def _pos(base, new):
    return np.concatenate([b + np.arange(n) for b, n in zip(base, new)]).astype(int)


FMTS = [g.KV_E4M3, g.KV_INT8]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("base", [[0], [1], [63], [64], [130, 0, 17, 31]])
def test_one_token(cuda_lib, fmt, dim, interleaved, base):
    run(fmt, 2, 6, dim, 32, base, [1] * len(base), interleaved=interleaved, one=True, seed=base[0])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("most", [2, 5, 8, 9, 16, 17])
def test_a_few_tokens(cuda_lib, fmt, dim, most):
    # a few tokens each, across a page's edge, none at all
    for interleaved in (False, True):
        run(fmt, 2, 3, dim, 16, [0, 15, 14, 3, 32, 9], [most, most, 2, 0, 1, most], interleaved=interleaved, seed=most)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim,page", [(128, 16), (128, 64), (64, 32), (128, 128), (64, 16), (64, 128), (128, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_prompts(cuda_lib, fmt, dim, page, interleaved):
    # fresh pages, a page entered in its middle, a sequence with nothing, one token
    run(fmt, 3, 5, dim, page, [0, 7, page - 1, 40, page], [page * 2 + 3, 9, page + 1, 0, 1], interleaved=interleaved,
        seed=dim + page)


@pytest.mark.parametrize("layout", ["pages_heads", "pages_tokens", "heads_pages"])
@pytest.mark.parametrize("extra", [0, 16, 5])
def test_cache_layouts(cuda_lib, layout, extra):
    run(g.KV_E4M3, 4, 4, 128, 16, [5, 0], [20, 33], layout=layout, extra=extra)


@pytest.mark.parametrize("dim,page,rot,heads", [(80, 16, 80, 2), (96, 24, 96, 1), (128, 5, 128, 2), (64, 1, 64, 2),
                                                (128, 64, 32, 2), (64, 16, 0, 2), (6, 3, 2, 1), (1, 4, 0, 2),
                                                (256, 64, 256, 1), (512, 16, 128, 1), (128, 256, 128, 1)])
@pytest.mark.parametrize("fmt", FMTS)
def test_unusual_sizes(cuda_lib, dim, page, rot, heads, fmt):
    run(fmt, heads, heads, dim, page, [0, 3, 11], [13, 1, 7], rot=rot)


@pytest.mark.parametrize("gap,offset", [(0, 1), (8, 0), (3, 0), (3, 7)])
def test_strides_and_alignment(cuda_lib, gap, offset):
    run(g.KV_INT8, 2, 2, 128, 16, [9, 0], [30, 4], gap=gap, offset=offset)
    run(g.KV_INT8, 2, 2, 64, 16, [9, 0], [1, 1], gap=gap, offset=offset, one=True)


def test_no_queries_and_in_place(cuda_lib):
    run(g.KV_INT8, 2, 0, 128, 16, [9, 0], [30, 4])
    c = Case(g.KV_INT8, 1, 64, 16, [5])
    x = torch.randn(1, 2, 64, device="cuda").bfloat16()
    cos, sin = (torch.from_numpy(t).cuda() for t in _angles(8, 32))
    base = torch.tensor([4], dtype=torch.int32, device="cuda")
    apart, same = torch.empty_like(x), x.clone()
    g.kv_append(c.cache, x, x[:, :1], x[:, :1], cos, sin, base, apart)
    g.kv_append(c.cache, same, x[:, :1], x[:, :1], cos, sin, base)
    assert torch.equal(apart, same)


def test_many_sequences_find_their_pages(cuda_lib):
    rng = np.random.default_rng(3)
    base, new = rng.integers(0, 40, 700).tolist(), rng.integers(0, 4, 700).tolist()
    new[5], new[699] = 90, 50
    run(g.KV_INT8, 1, 1, 64, 16, base, new)


@pytest.mark.parametrize("fmt", FMTS)
def test_appending_again_changes_nothing(cuda_lib, fmt):
    c = Case(fmt, 2, 128, 16, [40])
    K = torch.randn(9, 2, 128, device="cuda").bfloat16()
    base = torch.tensor([31], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    g.kv_append(c.cache, None, K, K, None, None, base, start=start, max_new=9)
    one = {n: c.got(n).copy() for n in ("k", "v", "ks", "vs")}
    g.kv_append(c.cache, None, K, K, None, None, base, start=start, max_new=9)
    for n in one:
        assert np.array_equal(one[n], c.got(n))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("value", ["zeros", "tiny", "inf", "nan", "huge"])
def test_extreme_values(cuda_lib, fmt, value):
    for new in (1, 20):
        c = Case(fmt, 1, 64, 16, [3 + new])
        K = torch.randn(new, 1, 64).bfloat16()
        if value == "zeros":
            K.zero_()
        elif value == "tiny":
            K.copy_((K.float() * 2.0 ** -130).bfloat16())
        elif value == "huge":
            K[0, 0, 3] = 3e38
        else:
            K[0, 0, 3] = float(value)
        start = torch.tensor([0, new], dtype=torch.int32, device="cuda")
        g.kv_append(c.cache, None, K.cuda(), K.cuda(), None, None, torch.tensor([3], dtype=torch.int32, device="cuda"),
                    start=start, max_new=new)
        check_status()
        none = np.zeros((64, 0), np.float32)
        S.append(c.np, fmt, None, K.float().numpy(), K.float().numpy(), none, none, [3], [0, new], False, np.float32)
        for n in ("ks", "vs"):
            assert np.array_equal(c.got(n), c.np[n]) and np.isfinite(c.got(n)).all()
        for n in ("k", "v"):
            if fmt == g.KV_INT8 and value == "nan":      # stored as 0
                p = c.np["table"][0, 0]
                assert c.got(n)[p, 0, 3, 3] == 0
                c.np[n][p, 0, 3, 3] = 0
            assert np.array_equal(c.got(n), c.np[n])


def test_offsets_past_32_bits(cuda_lib):
    # pages 2^31 bytes apart and more: only the last page of a 4.5 GB pool is used
    pages, H, P, D = 1100, 32, 1024, 128
    k = torch.empty(pages, H, P, D, dtype=torch.int8, device="cuda")
    s = torch.zeros(pages, H, device="cuda")
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    k[pages - 1].zero_()
    v, vs = torch.empty_like(k), torch.zeros_like(s)
    v[pages - 1].zero_()
    cache = g.KVCache(k, v, s, vs, table)
    x = torch.randn(3, H, D, device="cuda").bfloat16()
    base = torch.tensor([1000], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    g.kv_append(cache, None, x, x, None, None, base, start=start, max_new=3)
    check_status()
    want = x.float().abs().amax((0, 2)) / torch.full((H,), 127.0, device="cuda")
    assert torch.equal(s[pages - 1], want) and torch.equal(vs[pages - 1], want)
    code = (x.float() * (1 / want)[None, :, None]).round().clamp(-127, 127).to(torch.int8)
    for t in (k, v):
        assert torch.equal(t[pages - 1, :, 1000:1003], code.transpose(0, 1))


def test_misfits_are_reported_and_skipped(cuda_lib):
    def call(base=(3,), start=(0, 2), table=None, positions=64, max_new=2):
        c = Case(g.KV_INT8, 1, 64, 16, [30])
        if table is not None:
            c.table[0, 0] = table
        before = {n: c.got(n).copy() for n in ("k", "v", "ks", "vs")}
        x = torch.randn(2, 1, 64, device="cuda").bfloat16()
        cos, sin = (torch.from_numpy(t).cuda() for t in _angles(positions, 32))
        g.kv_append(c.cache, None, x, x, cos, sin, torch.tensor(base, dtype=torch.int32, device="cuda"),
                    start=torch.tensor(start, dtype=torch.int32, device="cuda"), max_new=max_new)
        torch.cuda.synchronize()
        status, where = g.device_status()
        same = all(np.array_equal(before[n], c.got(n)) for n in before)
        return status, where, same
    bad = (g.GEMM_ERR_INVALID_ARG, 60, True)
    assert call(table=99) == bad and call(table=-1) == bad
    assert call(base=(40,)) == bad              # past the table's two columns
    assert call(base=(-1,)) == bad and call(positions=4) == bad
    assert call(start=(0, 3), max_new=3) == bad and call(start=(2, 0)) == bad and call(start=(-1, 1)) == bad
    status, _, same = call()
    assert status == 0 and not same


def test_other_stream_and_graph(cuda_lib):
    c = Case(g.KV_E4M3, 2, 128, 16, [40, 20], new=1)
    K = torch.randn(2, 2, 128, device="cuda").bfloat16()
    base = torch.tensor([40, 20], dtype=torch.int32, device="cuda")
    g.kv_append(c.cache, None, K, K, None, None, base)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    K2 = torch.randn(2, 2, 128, device="cuda").bfloat16()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=s):
        g.kv_append(c.cache, None, K, K, None, None, base)
    base += 0
    K.copy_(K2)
    gr.replay()
    check_status()
    graph = {n: c.got(n).copy() for n in ("k", "v", "ks", "vs")}
    g.kv_append(c.cache, None, K2, K2, None, None, base)
    check_status()
    assert all(np.array_equal(graph[n], c.got(n)) for n in graph)
