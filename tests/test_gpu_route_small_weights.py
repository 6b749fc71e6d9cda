"""Renormalised weights of experts whose scores fp32 holds in a few bits or not at all: they are
the quotients of 64 bits.  A weight may be off by 2^-23 of itself: the rounding to fp32 and the
product with the factor."""
import numpy as np
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from experts_util import check_status
from oracle import experts as ox

pytestmark = pytest.mark.gpu


def check(x, top_k, bias=None, **kw):
    tokens = x.shape[0]
    ids = torch.empty(tokens, top_k, dtype=torch.int32, device="cuda")
    w = torch.empty(tokens, top_k, device="cuda")
    g.route(x.cuda(), ids, w, bias=None if bias is None else bias.cuda(), **kw)
    check_status()
    want, ww = ox.route(x.float().numpy(), top_k, bias=None if bias is None else bias.numpy(), **kw)
    np.testing.assert_array_equal(ids.cpu().numpy(), want)
    got = w.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - ww) <= 2 * ox.U32 * np.abs(ww) + 1e-37)
    return got


@pytest.mark.parametrize("experts", [16, 256, 400])
@pytest.mark.parametrize("base", [-80.0, -90.0, -104.0, -120.0, -400.0, -700.0])
def test_sigmoids_that_underflow(base, experts):
    x = base + torch.randn(40, experts, generator=torch.Generator().manual_seed(1))
    got = check(x, 4, score=g.ROUTE_SIGMOID, scale=2.5)
    np.testing.assert_allclose(got.sum(1), 2.5, rtol=1e-6)
    check(x.bfloat16(), 4, score=g.ROUTE_SIGMOID)
    check(x, 4, score=g.ROUTE_SIGMOID, bias=torch.zeros(experts), groups=4, top_groups=2)


def test_scores_of_nothing_have_no_weight():
    x = torch.full((3, 16), -float("inf"))
    x[1] = -800.0                                       # 0 in 64 bits as well
    assert (check(x, 4, score=g.ROUTE_SIGMOID) == 0).all()


def test_softmax_of_experts_that_a_bias_chose():
    x = torch.randn(40, 64, generator=torch.Generator().manual_seed(2))
    x[:, :8] += 150.0
    bias = torch.zeros(64)
    bias[20:24] = 3.0
    got = check(x, 4, bias=bias, score=g.ROUTE_SOFTMAX)
    np.testing.assert_allclose(got.sum(1), 1.0, rtol=1e-6)
