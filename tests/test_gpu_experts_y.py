"""What experts() holds of y: fp32 in calls whose y takes 64 MB at most, bf16 in larger ones.
With y in fp32 an output is off by its own rounding and what fp32 sums may add; its bound is
the oracle's without a rounding of y, which is tight (within a tenth of the output's half step
and what rounding y would add) wherever no code of h can fall on the other side of a middle."""
import numpy as np
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from experts_util import BF16, Layer, check_status, routing
from oracle import experts as ox

pytestmark = pytest.mark.gpu


def call(layer, tokens, top_k, rows=0):
    ids, w, offsets, order = routing(tokens, layer.experts, top_k, seed=3)
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(tokens, layer.hidden, generator=gen).to(BF16).cuda()
    out = torch.empty_like(x)
    g.force_tile_n(rows)
    try:
        g.experts(layer.weights, x, offsets, order, w, out)
    finally:
        g.force_tile_n(0)
    check_status()
    return x.float().cpu().numpy(), ids.cpu().numpy(), w.cpu().numpy(), out.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("hidden,width", [(256, 16), (130, 9)])          # the second: generic kernels
@pytest.mark.parametrize("tokens,rows", [(1, 0), (64, 0), (300, 0), (300, 128), (300, 256)])
def test_small_calls_do_not_round_y(tokens, rows, hidden, width):
    layer = Layer(4, hidden, width)
    x, ids, w, got = call(layer, tokens, 2, rows)
    ref, bound = ox.experts(x, ids, w, *layer.values, y_bf16=False)
    assert np.all(np.abs(got - ref) <= bound + 1e-30)
    # Of many outputs the bound is their own rounding and little else, so that a rounding of
    # y would show.  (A number of the oracle's alone, 0.42 for 64 tokens: the other outputs
    # have a code of h near a middle, by the bound that the oracle puts on h.)
    _, loose = ox.experts(x, ids, w, *layer.values)
    tight = bound - ox.U16 * np.abs(ref) < 0.1 * (loose - bound)
    assert tokens == 1 or tight.mean() > 0.25


@pytest.mark.parametrize("tokens,y_bf16", [(2048, False), (2049, True)])
def test_both_sides_of_the_limit(tokens, y_bf16):
    layer = Layer(4, 2048, 144)                              # 4 slots of 2048: 64 MB at 2048 tokens
    x, ids, w, got = call(layer, tokens, 4)
    ref, bound = ox.experts(x, ids, w, *layer.values, y_bf16=y_bf16)
    assert np.all(np.abs(got - ref) <= bound + 1e-30)


def test_a_workspace_takes_every_smaller_call():
    layer = Layer(2, 4096, 16)
    need = g.gemm_experts_workspace(2049, 2, 4096, 16)
    space = torch.empty(need, dtype=torch.uint8, device="cuda")
    for tokens in (2049, 2048, 2047, 1):
        assert g.gemm_experts_workspace(tokens, 2, 4096, 16) <= need
        ids, w, offsets, order = routing(tokens, 2, 2)
        x = torch.randn(tokens, 4096, device="cuda").to(BF16)
        first, again = torch.empty_like(x), torch.empty_like(x)
        g.experts(layer.weights, x, offsets, order, w, first)
        g.experts(layer.weights, x, offsets, order, w, again, workspace=space)
        check_status()
        assert torch.equal(first, again)
