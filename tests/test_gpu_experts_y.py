"""What experts() holds of y: fp32, and in calls whose y takes more than 64 MB and whose rows are
many, fp16 with a scale for each 128 columns.  With y in fp32 an output is off by its own rounding and what fp32 sums may add; its bound is
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
    ref, bound = ox.experts(x, ids, w, *layer.values, y_half_step=ox.U32)
    assert np.all(np.abs(got - ref) <= bound + 1e-30)
    # Of many outputs the bound is their own rounding and little else, so that a rounding of
    # y would show.  (A number of the oracle's alone, 0.42 for 64 tokens: the other outputs
    # have a code of h near a middle, by the bound that the oracle puts on h.)
    _, loose = ox.experts(x, ids, w, *layer.values)
    tight = bound - ox.U16 * np.abs(ref) < 0.1 * (loose - bound)
    assert tokens == 1 or tight.mean() > 0.25


# 4 slots of 2048: 64 MB at 2048 tokens; 270 columns in rows of 272; tiles of 128 rows and
# generic kernels hold fp32 at any size
@pytest.mark.parametrize("hidden,tokens,rows,pad,half_step", [
    (2048, 2048, 0, 0, ox.U32), (2048, 2049, 0, 0, ox.UH), (2048, 2049, 128, 0, ox.U32), (270, 16000, 0, 2, ox.UH),
    (270, 16000, 256, 2, ox.UH), (262, 16500, 0, 0, ox.U32)])
def test_both_sides_of_the_limit(hidden, tokens, rows, pad, half_step):
    layer = Layer(4, hidden, 142, pad=pad)
    assert tokens * 4 * hidden * 4 > 64 << 20 or half_step == ox.U32
    x, ids, w, got = call(layer, tokens, 4, rows)
    ref, bound = ox.experts(x, ids, w, *layer.values, y_half_step=half_step)
    assert np.all(np.abs(got - ref) <= bound + 1e-30)


@pytest.mark.parametrize("size", [2.0 ** -70, 1.0, 2.0 ** 60, 2.0 ** 100])
def test_large_calls_of_every_magnitude(size):
    """Rows and columns of unlike sizes, zeros, infinities and NaN: each 128 columns of a row have a
    scale of their own."""
    layer = Layer(2, 528, 144)
    scale = torch.ones(2, 2, 5, device="cuda")
    scale[:, :, 1], scale[:, :, 2], scale[:, :, 4] = 2.0 ** -20, 0.0, 2.0 ** 10      # by 128 columns of down
    scale *= size
    layer.weights.tensors[5].mul_(scale)
    wide = ox.spread(scale[0].double().cpu().numpy(), 128, 144, 528)
    layer.values[2] = [v * wide for v in layer.values[2]]
    tokens = 16500
    ids, w, offsets, order = routing(tokens, 2, 2, seed=3)
    x = torch.randn(tokens, 528, generator=torch.Generator().manual_seed(4))
    x *= torch.exp2(torch.randint(-20, 10, (tokens, 1), generator=torch.Generator().manual_seed(5)))
    x[7] = 0
    x = x.to(BF16).cuda()
    x[11, 3] = float("nan")
    out = torch.full_like(x, 7.0)
    g.experts(layer.weights, x, offsets, order, w, out)
    assert g.last_tile_n() == 256
    check_status()
    assert (out[7] == 0).all() and torch.isnan(out[11]).any()
    keep = torch.ones(tokens, dtype=torch.bool)
    keep[11] = False
    ref, bound = ox.experts(x.float().cpu().numpy()[keep], ids.cpu().numpy()[keep], w.cpu().numpy()[keep], *layer.values,
                            y_half_step=ox.UH)
    got = out.float().cpu().numpy().astype(np.float64)[keep]
    # fp32 holds every sum on the way (both experts are each token's): the magnitudes added up
    xv = ox.dequantise(*ox.quantise(x.float().cpu().numpy()[keep]), 1)
    fits = np.ones(ref.shape, bool)
    for gate, up, down in zip(*layer.values):
        a = xv @ gate
        h = a / (1 + np.exp(-np.maximum(a, -700))) * (xv @ up)
        fits &= 1.1 * np.abs(h) @ np.abs(down) < 3e38
    assert np.all((np.abs(got - ref) <= bound + 1e-37)[fits]) and fits.mean() > 0.2


def test_large_calls_with_infinite_rows():
    """An infinite scale of down's makes infinities in its columns; those beside them, of one
    item or not, stay what they are."""
    layer = Layer(2, 528, 144)
    layer.weights.tensors[5][:, 0, 1] = float("inf")
    tokens = 16500
    ids, w, offsets, order = routing(tokens, 2, 2, seed=3)
    x = torch.randn(tokens, 528, generator=torch.Generator().manual_seed(4)).to(BF16).cuda()
    out = torch.full_like(x, 7.0)
    g.experts(layer.weights, x, offsets, order, w, out)
    check_status()
    ref, bound = ox.experts(x.float().cpu().numpy(), ids.cpu().numpy(), w.cpu().numpy(), *layer.values, y_half_step=ox.UH)
    got = out.float().cpu().numpy().astype(np.float64)
    rest = np.r_[0:128, 256:528]
    assert np.all(np.abs(got[:, rest] - ref[:, rest]) <= bound[:, rest] + 1e-30)
    assert not np.isfinite(got[:, 128:256]).any()


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
