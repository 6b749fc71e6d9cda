"""Routing of the most tokens."""
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from experts_util import BF16, check_status

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


def test_most_tokens(cuda_lib):
    # booleans are asserted, never tensors: a failed assertion would print 2^31 values
    x = torch.empty(MOST, 2, dtype=BF16, device="cuda")
    x.view(-1)[:2 ** 31].normal_(generator=torch.Generator(device="cuda").manual_seed(0))
    x.view(-1)[2 ** 31:].normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    ints = dict(dtype=torch.int32, device="cuda")
    ids, order, offsets = torch.full((MOST, 1), -7, **ints), torch.full((MOST,), -7, **ints), torch.full((3,), -7, **ints)
    w = torch.full((MOST, 1), float("nan"), device="cuda")
    g.route(x, ids, w, offsets, order, renormalise=True)
    check_status()
    # w * (1/w): the reciprocal is off by 2^-23 at most, the product by 2^-24
    off = float((w - 1).abs_().max())
    del w
    second = x[:, 1] > x[:, 0]
    del x
    wrong = int((ids[:, 0] != second).sum())
    first = MOST - int(second.sum())
    ends = offsets.tolist()
    ascending = bool((order[1:first] > order[:first - 1]).all()) and bool((order[first + 1:] > order[first:-1]).all())
    mixed = int(second[order[:first].long()].sum()) + int((~second[order[first:].long()]).sum())
    del ids, order, second
    assert off <= 3 * 2.0 ** -24 and wrong == 0
    assert ends == [0, first, MOST] and ascending and mixed == 0
