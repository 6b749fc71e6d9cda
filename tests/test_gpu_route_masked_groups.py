"""Routing where a bias masks whole groups, by -inf or by finite numbers whose sum passes the
range of fp32: groups rank as their scores do in 64 bits."""
import numpy as np
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from experts_util import check_status
from oracle import experts as ox

pytestmark = pytest.mark.gpu
INF, LEAST = float("inf"), torch.finfo(torch.float32).min


def check(x, bias, top_k, score, **kw):
    tokens = x.shape[0]
    ids = torch.empty(tokens, top_k, dtype=torch.int32, device="cuda")
    w = torch.empty(tokens, top_k, device="cuda")
    g.route(x.cuda(), ids, w, bias=bias.cuda(), score=score, **kw)
    check_status()
    want, _ = ox.route(x.numpy(), top_k, score=score, bias=bias.numpy(), **kw)
    np.testing.assert_array_equal(ids.cpu().numpy(), want)


# masks of groups 1, 3, 4 and 6 of eight
MASKS = [(-2e38, -3.4e38, -1.9e38, -2e38), (LEAST, -2e38, -INF, -INF), (-INF, LEAST, LEAST, -2e38), (-INF,) * 4,
         (LEAST,) * 4, (-3e38, -1e38, -1.5e38, -1.8e38)]


@pytest.mark.parametrize("score", [g.ROUTE_SOFTMAX, g.ROUTE_SIGMOID])
@pytest.mark.parametrize("experts", [32, 56, 256, 512])
@pytest.mark.parametrize("masks", MASKS)
def test_masked_groups(masks, experts, score):
    gen = torch.Generator().manual_seed(experts)
    x = torch.randn(70, experts, generator=gen)
    bias = 0.1 * torch.randn(experts, generator=gen)
    size = experts // 8
    for group, v in zip((1, 3, 4, 6), masks):
        bias[group * size:(group + 1) * size] = v
    for top_groups in range(1, 8):
        for group_best in (1, 2):
            check(x, bias, min(6, size * top_groups), score, groups=8, top_groups=top_groups, group_best=group_best)
    bias[size + 1] = 0.3                                   # one expert of a masked group is not
    check(x, bias, 3, score, groups=8, top_groups=5)
    check(x, bias, 3, score, groups=8, top_groups=6)


def test_groups_of_one_expert():
    bias = torch.tensor([-2e38, -3e38, 0.1, LEAST, -INF, -3.1e38])
    check(torch.zeros(3, 6), bias, 3, g.ROUTE_SIGMOID, groups=6, top_groups=4, group_best=2)
