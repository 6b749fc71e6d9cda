"""Slots that no expert's range covers, before the first or behind the last, are reported; the
other tokens' rows are right."""
import numpy as np
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from experts_util import BF16, Layer, check_status, routing
from oracle import experts as ox

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hidden,rows", [(256, 0), (256, 128), (256, 256), (4096, 0), (129, 0)])      # the last: generic
@pytest.mark.parametrize("tokens", [2, 40, 300])
def test_reported(tokens, hidden, rows):
    layer = Layer(6, hidden, 144)
    ids, w, offsets, order = routing(tokens, 6, 2)
    x = torch.randn(tokens, hidden, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    out = torch.empty_like(x)
    ref, bound = ox.experts(x.float().cpu().numpy(), ids.cpu().numpy(), w.cpu().numpy(), *layer.values)
    g.force_tile_n(rows)
    try:
        for at, by in ((0, 1), (6, -1)):
            o = offsets.clone()
            o[at] += by
            if at == 0:
                o[1:-1].clamp_(min=1)                          # still ascending
            else:
                o[1:-1].clamp_(max=int(o[-1]))
            g.experts(layer.weights, x, o, order, w, out)
            torch.cuda.synchronize()
            assert g.device_status()[0] == g.GEMM_ERR_INVALID_ARG
            lost = int(order[0 if at == 0 else -1]) // 2
            rest = [t for t in range(tokens) if t != lost]
            assert np.all((np.abs(out.float().cpu().numpy() - ref) <= bound + 1e-30)[rest])
        g.experts(layer.weights, x, offsets, order, w, out)
        check_status()
    finally:
        g.force_tile_n(0)
    layer.check(x, ids, w, out)


def test_no_token_of_the_first_and_the_last_expert_is_no_fault():
    layer = Layer(6, 256, 144)
    logits = torch.full((20, 6), -9.0)
    logits[:, 2:4] = 9.0
    ids, w, offsets, order = routing(20, 6, 2, logits=logits)
    x = torch.randn(20, 256, device="cuda").to(BF16)
    g.experts(layer.weights, x, offsets, order, w, torch.empty_like(x))
    check_status()
