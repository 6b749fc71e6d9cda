"""Routing by scores that are denormal in fp32: which groups are kept, and their experts, are
those of 64 bits."""
import numpy as np
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from experts_util import check_status
from oracle import experts as ox

pytestmark = pytest.mark.gpu


def check(x, top_k, **kw):
    tokens = x.shape[0]
    ids = torch.empty(tokens, top_k, dtype=torch.int32, device="cuda")
    w = torch.empty(tokens, top_k, device="cuda")
    bias = kw.pop("bias", None)
    score = kw.pop("score", g.ROUTE_SOFTMAX)
    g.route(x.cuda(), ids, w, bias=None if bias is None else bias.cuda(), score=score, **kw)
    check_status()
    want, _ = ox.route(x.numpy(), top_k, score=score, bias=None if bias is None else bias.numpy(), **kw)
    np.testing.assert_array_equal(ids.cpu().numpy(), want)


def test_two_groups_a_step_apart():
    """fp32 has 4 steps of 2^-149 for the second group and 3 for the third, 64 bits 3.2 and 3.8."""
    x = torch.full((6, 6), -200.0)
    x[:, 0] = 0.0
    x[:, 2:4] = torch.tensor([-102.3234, -103.7897])
    x[:, 4:6] = torch.tensor([-102.4034, -102.9424])
    check(x, 4, groups=3, top_groups=2)
    check(x + 3.0, 3, groups=3, top_groups=2)


@pytest.mark.parametrize("low,high", [(86, 89), (88, 104), (92, 104), (100, 110)])
@pytest.mark.parametrize("experts,groups,top_groups", [(32, 8, 4), (256, 8, 4), (60, 6, 3), (512, 16, 9)])
@pytest.mark.parametrize("group_best", [1, 2])
def test_groups_far_below_the_largest(low, high, experts, groups, top_groups, group_best):
    gen = torch.Generator().manual_seed(low + experts)
    x = -(low + (high - low) * torch.rand(500, experts, generator=gen))
    x[:, ::experts // groups] += torch.where(torch.arange(groups) < 2, 90.0, 0.0)         # two groups with weight
    x += torch.randn(500, 1, generator=gen)
    check(x, 5, groups=groups, top_groups=top_groups, group_best=group_best)
    check(x, 5, groups=groups, top_groups=top_groups, group_best=group_best, bias=torch.zeros(experts))


def test_sigmoids_and_biases_below_2_to_minus_126():
    """1/(1 + e^88.6) is 3.3e-39, ahead of a bias of 3e-39."""
    x = torch.tensor([[-88.6, -300.0]]).repeat(5, 1)
    check(x, 1, bias=torch.tensor([0.0, 3e-39]), score=g.ROUTE_SIGMOID)
    x = torch.tensor([[-88.8, -88.6, -300.0]]).repeat(5, 1)
    check(x, 2, bias=torch.tensor([0.0, 0.0, 3e-39]), score=g.ROUTE_SIGMOID)
