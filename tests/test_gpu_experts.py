"""The experts' FFN of routed tokens against the fp64 oracle, element by element, within
what fp32 sums, codes that fall on the other side of a middle, and the roundings of y and
O to bf16 may add (oracle.experts.experts)."""
import numpy as np
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from experts_util import BF16, Layer, check_status, placed, routing
from oracle import experts as ox

pytestmark = pytest.mark.gpu


def inputs(tokens, hidden, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(tokens, hidden, generator=gen) * torch.exp(torch.randn(tokens, 1, generator=gen))).to(BF16)


def check(layer, tokens, top_k, logits=None, path=None, want=g.PATH_BLOCKS, seed=0, pad=0):
    ids, w, offsets, order = routing(tokens, layer.experts, top_k, seed, logits=logits)
    x = placed(inputs(tokens, layer.hidden, seed + 1), pad)
    out = placed(torch.full((tokens, layer.hidden), float("nan"), dtype=BF16), pad, fill=7.0)
    if path is not None:
        g.force_path(path)
    try:
        g.experts(layer.weights, x, offsets, order, w, out)
    finally:
        g.force_path(g.PATH_AUTO)
    assert g.last_path() == want
    check_status()
    layer.check(x, ids, w, out)
    if pad:
        assert (out.as_strided((tokens, layer.hidden + pad), out.stride())[:, layer.hidden:] == 7.0).all()
    return out


@pytest.mark.parametrize("experts,top_k,hidden,width", [
    (1, 1, 128, 128), (4, 2, 256, 144), (8, 2, 400, 272), (16, 4, 512, 1376), (40, 8, 144, 16)])
@pytest.mark.parametrize("tokens", [1, 5, 64, 300])
def test_sizes(tokens, experts, top_k, hidden, width):
    check(Layer(experts, hidden, width), tokens, top_k)


@pytest.mark.parametrize("rows", [128, 256])
@pytest.mark.parametrize("tokens,experts,top_k,hidden,width", [
    (1, 4, 2, 144, 16), (300, 4, 2, 272, 400), (260, 1, 1, 128, 128), (900, 3, 2, 400, 144)])
def test_each_kernel(tokens, experts, top_k, hidden, width, rows):
    g.force_tile_n(rows)
    try:
        check(Layer(experts, hidden, width), tokens, top_k)
        assert g.last_tile_n() == rows
    finally:
        g.force_tile_n(0)


def test_many_tokens():
    check(Layer(4, 272, 400), 1500, 2)


def test_one_token_splits_k():
    check(Layer(4, 4096, 128), 1, 2)
    check(Layer(4, 128, 4096), 1, 2)


@pytest.mark.parametrize("tokens", [7, 200])
def test_uneven_experts(tokens):
    """All tokens at the same experts: most experts have none, and some all."""
    x = torch.zeros(tokens, 24)
    x[:, 3] = 9
    x[:, 17] = 8
    x[::3, 23] = 12
    check(Layer(24, 256, 272), tokens, 2, logits=x)


@pytest.mark.parametrize("hidden,width", [(100, 72), (129, 130), (16, 9)])
def test_generic(hidden, width):
    for tokens in (1, 50):
        check(Layer(6, hidden, width), tokens, 3, want=g.PATH_GENERIC)


def test_forced_generic_and_padded():
    layer = Layer(6, 272, 144, pad=16)
    check(layer, 33, 3, pad=5)
    check(layer, 33, 3, pad=8)
    check(layer, 33, 3, path=g.PATH_GENERIC, want=g.PATH_GENERIC)


@pytest.mark.parametrize("rows", [0, 128, 256])
@pytest.mark.parametrize("tokens", [3, 500])
def test_odd_sizes_of_padded_weights(tokens, rows):
    # 270 and 142 columns in rows of 272 and 144
    g.force_tile_n(rows)
    try:
        check(Layer(3, 270, 142, pad=2), tokens, 2)
    finally:
        g.force_tile_n(0)


def test_zero_and_infinite_rows():
    layer = Layer(4, 256, 144)
    ids, w, offsets, order = routing(20, 4, 2)
    x = inputs(20, 256).cuda()
    x[3] = 0
    x[5, 7] = float("nan")
    out = torch.empty(20, 256, dtype=BF16, device="cuda")
    g.experts(layer.weights, x, offsets, order, w, out)
    check_status()
    assert (out[3] == 0).all() and torch.isnan(out[5]).any()
    rest = [t for t in range(20) if t != 5]
    ref, bound = ox.experts(x[rest].float().cpu().numpy(), ids.cpu().numpy()[rest], w.cpu().numpy()[rest], *layer.values)
    assert np.all(np.abs(out[rest].float().cpu().numpy() - ref) <= bound + 1e-30)


def test_forced_paths_that_cannot_run():
    layer = Layer(2, 129, 130)
    ids, w, offsets, order = routing(3, 2, 1)
    x = inputs(3, 129).cuda()
    out = torch.empty_like(x)
    for path in (g.PATH_SKINNY, g.PATH_BF16_TC):          # no such kernels; rows that no copy takes
        g.force_path(path)
        try:
            with pytest.raises(g.GemmError) as e:
                g.experts(layer.weights, x, offsets, order, w, out)
        finally:
            g.force_path(g.PATH_AUTO)
        assert e.value.code == g.GEMM_ERR_UNSUPPORTED


def test_no_tokens():
    layer = Layer(4, 256, 144)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    g.experts(layer.weights, torch.empty(0, 256, dtype=BF16, device="cuda"),
              torch.zeros(5, dtype=torch.int32, device="cuda"), none, torch.empty(0, 2, device="cuda"),
              torch.empty(0, 256, dtype=BF16, device="cuda"))
    check_status()


@pytest.mark.parametrize("rows", [0, 128, 256])
def test_slots_that_do_not_fit_are_skipped_and_reported(rows):
    g.force_tile_n(rows)
    try:
        _slots_that_do_not_fit()
    finally:
        g.force_tile_n(0)


def _slots_that_do_not_fit():
    layer = Layer(4, 256, 144)
    ids, w, offsets, order = routing(30, 4, 2)
    x = inputs(30, 256).cuda()
    out = torch.empty(30, 256, dtype=BF16, device="cuda")
    good = order.clone()
    for bad in (60, -1, 1 << 30):
        order.copy_(good)
        order[11] = bad
        g.experts(layer.weights, x, offsets, order, w, out)
        torch.cuda.synchronize()
        assert g.device_status()[0] == g.GEMM_ERR_INVALID_ARG
        t = int(good[11]) // 2
        rest = [i for i in range(30) if i != t]
        ref, bound = ox.experts(x.float().cpu().numpy(), ids.cpu().numpy(), w.cpu().numpy(), *layer.values)
        assert np.all((np.abs(out.float().cpu().numpy() - ref) <= bound + 1e-30)[rest])
    for at, bad in ((1, 61), (2, -5), (4, 1 << 30)):
        o = offsets.clone()
        o[at] = bad
        g.experts(layer.weights, x, o, good, w, out)
        torch.cuda.synchronize()
        assert g.device_status()[0] == g.GEMM_ERR_INVALID_ARG
    g.experts(layer.weights, x, offsets, good, w, out)
    check_status()


@pytest.mark.parametrize("rows", [0, 128, 256])
def test_ranges_that_overlap_are_reported(rows):
    layer = Layer(8, 256, 144)
    ids, w, offsets, order = routing(640, 8, 1)
    x = inputs(640, 256).cuda()
    out = torch.empty(640, 256, dtype=BF16, device="cuda")
    bad = torch.tensor([0, 640] * 4 + [0], dtype=torch.int32, device="cuda")
    g.force_tile_n(rows)
    try:
        for o in (bad, torch.zeros_like(bad) - 1):          # no range fits: no work at all
            g.experts(layer.weights, x, o, order, w, out)
            torch.cuda.synchronize()
            assert g.device_status()[0] == g.GEMM_ERR_INVALID_ARG
        for _ in range(3):
            g.experts(layer.weights, x, torch.zeros_like(bad) - 1, order, w, out)
            g.experts(layer.weights, x, offsets, order, w, out)
        torch.cuda.synchronize()
        assert g.device_status()[0] == g.GEMM_ERR_INVALID_ARG
    finally:
        g.force_tile_n(0)
    layer.check(x, ids, w, out)


def test_repeats_streams_and_graphs():
    layer = Layer(8, 272, 400)
    ids, w, offsets, order = routing(100, 8, 2)
    x = inputs(100, 272).cuda()
    outs = [torch.empty(100, 272, dtype=BF16, device="cuda") for _ in range(4)]
    g.experts(layer.weights, x, offsets, order, w, outs[0])
    need = g.gemm_experts_workspace(100, 2, 272, 400)
    g.experts(layer.weights, x, offsets, order, w, outs[1],
              workspace=torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g.experts(layer.weights, x, offsets, order, w, outs[2], stream=s.cuda_stream)
    s.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    held = [x.clone(), inputs(100, 272, 5).cuda()]
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            g.experts(layer.weights, held[i], offsets, order, w, outs[3] if i == 0 else outs[2])
    graphs[1].replay()
    graphs[0].replay()
    check_status()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[3])
    layer.check(held[1], ids, w, outs[2])
