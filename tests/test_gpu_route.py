"""Routing to experts against the 64-bit oracle: ids, offsets and order are equal, weights
are within what fp32 may add.  A weight is a quotient of exponentials: each argument of up
to 24 (logits of up to 12) is rounded once, which moves exp by 24 half steps, exp and the
division by 2 each, and the sums of up to 1024 terms in groups of at most 32 and 5 levels
by 37 half steps; numerator, denominator and the renormalising sum together stay below 200
half steps (2^-24): 1.2e-5."""
import numpy as np
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from experts_util import check_status
from oracle import experts as ox

pytestmark = pytest.mark.gpu
TOL = 200 * ox.U32


def run(logits, top_k, plan=True, **kw):
    tokens, experts = logits.shape
    ids = torch.full((tokens, top_k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((tokens, top_k), float("nan"), device="cuda")
    offsets = order = None
    if plan:
        offsets = torch.full((experts + 1,), -7, dtype=torch.int32, device="cuda")
        order = torch.full((tokens * top_k,), -7, dtype=torch.int32, device="cuda")
    g.route(logits, ids, w, offsets, order, **kw)
    assert g.last_path() == g.PATH_ROUTE
    check_status()
    return ids, w, offsets, order


def check(logits, top_k, plan=True, **kw):
    ids, w, offsets, order = run(logits, top_k, plan, **kw)
    if kw.get("bias") is not None:
        kw["bias"] = kw["bias"].cpu().numpy()
    kw.pop("workspace", None)
    want, ww = ox.route(logits.float().cpu().numpy(), top_k, **kw)
    np.testing.assert_array_equal(ids.cpu().numpy(), want)
    got = w.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - ww) <= TOL * np.abs(ww) + 1e-37)
    if plan:
        o, r = ox.by_expert(want, logits.shape[1])
        np.testing.assert_array_equal(offsets.cpu().numpy(), o)
        np.testing.assert_array_equal(order.cpu().numpy(), r)


def logits(tokens, experts, dtype=torch.float32, seed=0, size=2.0):
    gen = torch.Generator().manual_seed(seed)
    return (size * torch.randn(tokens, experts, generator=gen)).clamp(-12, 12).to(dtype).cuda()


def bias(experts, seed=9, size=0.1):
    return size * torch.randn(experts, generator=torch.Generator().manual_seed(seed)).cuda()


@pytest.mark.parametrize("tokens,experts,top_k", [
    (1, 1, 1), (1, 64, 8), (3, 7, 3), (33, 32, 32), (128, 60, 6), (129, 64, 8), (1000, 160, 6), (5000, 256, 8),
    (40, 257, 9), (700, 512, 16), (33, 1000, 10), (1300, 1024, 32)])
@pytest.mark.parametrize("score", [g.ROUTE_SOFTMAX, g.ROUTE_SIGMOID])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sizes(tokens, experts, top_k, score, dtype):
    x = logits(tokens, experts, dtype, seed=tokens + experts)
    check(x, top_k, score=score)
    check(x, top_k, score=score, bias=bias(experts), renormalise=False, scale=2.5)


@pytest.mark.parametrize("tokens", [1, 64, 500])
@pytest.mark.parametrize("experts,groups,top_groups,top_k", [
    (256, 8, 4, 8), (160, 8, 3, 6), (60, 3, 1, 4), (64, 32, 5, 8), (32, 32, 8, 8), (1024, 32, 32, 32), (21, 7, 2, 5)])
@pytest.mark.parametrize("group_best", [1, 2])
def test_groups(tokens, experts, groups, top_groups, top_k, group_best):
    kw = dict(groups=groups, top_groups=top_groups, group_best=group_best)
    x = logits(tokens, experts, seed=experts)
    check(x, top_k, score=g.ROUTE_SIGMOID, bias=bias(experts), **kw)
    check(x, top_k, score=g.ROUTE_SOFTMAX, **kw)
    check(x.bfloat16(), top_k, score=g.ROUTE_SOFTMAX, bias=bias(experts, size=0.01), **kw)


@pytest.mark.parametrize("score", [g.ROUTE_SOFTMAX, g.ROUTE_SIGMOID])
def test_ties_go_to_the_lowest_index(score):
    x = torch.zeros(200, 96, device="cuda")
    x[50:100] = logits(50, 96).round()                       # many equal logits
    x[100:] = logits(100, 96, torch.bfloat16).float()
    for kw in (dict(), dict(bias=torch.zeros(96, device="cuda")), dict(bias=bias(96).round(decimals=1)),
               dict(groups=8, top_groups=3), dict(groups=8, top_groups=3, bias=torch.zeros(96, device="cuda"))):
        check(x, 8, score=score, **kw)


@pytest.mark.parametrize("score", [g.ROUTE_SOFTMAX, g.ROUTE_SIGMOID])
@pytest.mark.parametrize("experts", [60, 256, 512])
def test_rows_of_padding(experts, score):
    """Rows of one number among others, with groups, and biases that are all equal or all but one."""
    x = logits(400, experts, seed=2)
    x[::3] = 0
    x[1::7] = 1.5
    x[2::50] = float("-inf")
    x[5] = float("nan")
    x[7, 1:] = x[7, 0]
    x[8, 1:] = x[8, 0]
    x[8, experts // 2] += 1e-6
    check(x, 6, score=score, groups=4, top_groups=2)
    check(x, 6, score=score, groups=4, top_groups=2, bias=torch.full((experts,), 0.25, device="cuda"))
    b = torch.zeros(experts, device="cuda")
    b[experts - 1] = 1e-30
    check(x, 6, score=score, groups=4, top_groups=2, bias=b)
    check(x, 6, score=score, groups=4, top_groups=3, group_best=1, bias=b * 0)


def test_choices_that_fp32_cannot_tell_apart():
    """Sums of score and bias that differ by less than a step of fp32: the order is that
    of 64 bits."""
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(400, 64, generator=gen)
    b = (0.7 - 1.0 / (1.0 + torch.exp(-x[0].double()))).float()          # row 0: all choices near 0.7
    x[1::2] = x[0] + 1e-6 * torch.randn(200, 64, generator=gen)
    check(x.cuda(), 8, score=g.ROUTE_SIGMOID, bias=b.cuda())
    check(x.cuda(), 8, score=g.ROUTE_SIGMOID, bias=b.cuda(), groups=4, top_groups=2)
    s = torch.softmax(x[0].double(), 0)
    check(x.cuda(), 8, score=g.ROUTE_SOFTMAX, bias=(0.1 - s).float().cuda())


@pytest.mark.parametrize("step", [2.0 ** -22, 2.0 ** -18, 2.0 ** -15, 2.0 ** -12])
@pytest.mark.parametrize("experts,top_k", [(8, 3), (64, 8), (200, 1), (256, 8), (256, 31)])
def test_neighbours_close_to_each_other(experts, top_k, step):
    """Choices that lie `step` apart, in any order: more than a step of fp32 and less than
    one of the 16 bits that a choice near 1 has in a packed key, or just above it."""
    gen = torch.Generator().manual_seed(experts + top_k)
    place = torch.stack([torch.randperm(experts, generator=gen) for _ in range(300)]).double()
    near = (0.4 + step * place).float()                                   # fp32 values themselves
    check(near.cuda(), top_k, score=g.ROUTE_SIGMOID)
    check((near - 0.4).cuda(), top_k, score=g.ROUTE_SOFTMAX)
    b = 0.05 * torch.randn(experts, generator=gen)
    target = (0.9 + step * place).numpy()                                 # score and bias together
    x = torch.from_numpy(target) - b.double()
    x = torch.log(x / (1 - x)).float()
    check(x.cuda(), top_k, score=g.ROUTE_SIGMOID, bias=b.cuda())
    groups = 4 if experts % 4 == 0 and top_k <= experts // 2 else 1
    check(x.cuda(), top_k, score=g.ROUTE_SIGMOID, bias=b.cuda(), groups=groups, top_groups=max(1, groups // 2))


@pytest.mark.parametrize("score", [g.ROUTE_SOFTMAX, g.ROUTE_SIGMOID])
def test_peaked_scores(score):
    """Scores that underflow fp32, and choices then ruled by the bias."""
    x = logits(300, 64, size=60.0, seed=5) * 8
    ids, w, _, _ = run(x, 8, score=score, bias=bias(64))
    want, _ = ox.route(x.cpu().numpy(), 8, bias=bias(64).cpu().numpy(), score=score)
    np.testing.assert_array_equal(ids.cpu().numpy(), want)
    ids, w, _, _ = run(x, 8, score=score)
    want, _ = ox.route(x.cpu().numpy(), 8, score=score)
    np.testing.assert_array_equal(ids.cpu().numpy(), want)
    assert torch.isfinite(w).all()


@pytest.mark.parametrize("score", [g.ROUTE_SOFTMAX, g.ROUTE_SIGMOID])
@pytest.mark.parametrize("kw", [dict(), dict(groups=4, top_groups=2), dict(renormalise=False)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_infinities_and_nan(score, kw, with_bias):
    x = logits(12, 40, seed=8)
    x[0] = -float("inf")
    x[1] = float("nan")
    x[2, 5:9] = float("inf")
    x[3, ::2] = float("nan")
    x[4, 1:] = -float("inf")
    x[5, 3] = float("inf")
    x[6, 3], x[6, 30] = float("inf"), float("nan")
    if with_bias:
        b = bias(40)
        b[0], b[7], b[11], b[39] = -float("inf"), float("nan"), float("inf"), -3e38
        kw = dict(kw, bias=b)
    check(x, 6, score=score, **kw)


def test_strides_and_alignment():
    wide = logits(300, 300, torch.bfloat16)
    check(wide[:, 3:259], 8, bias=bias(256), score=g.ROUTE_SIGMOID)
    check(wide[::2, :256], 8)
    check(logits(50, 131)[:, 1:129], 4)
    x = logits(300, 64)
    ids, w, _, _ = run(x, 4, plan=False)
    np.testing.assert_array_equal(ids.cpu().numpy(), ox.route(x.cpu().numpy(), 4)[0])


def test_no_tokens():
    offsets = torch.full((65,), -7, dtype=torch.int32, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    g.route(torch.empty(0, 64, device="cuda"), none.view(0, 8), torch.empty(0, 8, device="cuda"), offsets, none)
    check_status()
    assert (offsets == 0).all()


def test_streams_graphs_and_repeats():
    x = logits(3000, 256)
    b = bias(256)
    kw = dict(bias=b, score=g.ROUTE_SIGMOID, groups=8, top_groups=4)
    first = run(x, 8, **kw)
    again = run(x, 8, **kw)
    for p, q in zip(first, again):
        assert torch.equal(p, q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(t) for t in first]
    with torch.cuda.stream(s):
        g.route(x, *outs, **kw)
    s.synchronize()
    for p, q in zip(first, outs):
        assert torch.equal(p, q)
    held = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.route(held, *outs, **kw)
    for seed in (1, 2):
        held.copy_(logits(3000, 256, seed=seed))
        graph.replay()
        want = run(held, 8, **kw)
        for p, q in zip(want, outs):
            assert torch.equal(p, q)
