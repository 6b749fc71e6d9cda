"""Abort paths of the block-scaled products' kernels: with gemm_test_stall the MMA issuer
of the first CTA or cluster waits on a barrier that nothing arrives at.  The bounded wait
runs out, the kernel reports its place and leaves (copies landed, tensor memory freed), and
the next call is right.  No address changes and no copy is skipped."""
import numpy as np
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from experts_util import BF16, Layer, check_status, codes, fp8, routing
from oracle import experts as ox

pytestmark = pytest.mark.gpu

SITE_DECODE, SITE_WIDE = 71, 77       # WaitSite values of the library
LIMIT_NS = 8_000_000                  # the stalled wait gives up after 2 ms


@pytest.fixture
def short_limit(cuda_lib):
    assert g.device_status()[0] == 0
    g.set_wait_timeout_ns(LIMIT_NS)
    try:
        yield
    finally:
        g.test_stall(0)
        g.set_wait_timeout_ns(0)
        g.force_tile_n(0)


def stalled(call):
    g.test_stall(1)
    try:
        call()
    finally:
        g.test_stall(0)
    torch.cuda.synchronize()
    return g.device_status()


@pytest.mark.parametrize("M,N,K,rows,split,site", [
    (4, 256, 4096, 0, True, SITE_DECODE), (4, 5000, 512, 0, False, SITE_DECODE), (60, 512, 1024, 0, None, SITE_DECODE),
    (300, 512, 1024, 128, False, SITE_DECODE), (300, 528, 1024, 256, False, SITE_WIDE)])
def test_products(short_limit, M, N, K, rows, split, site):
    rng = np.random.default_rng(0)
    a, b = codes(rng, M, K), codes(rng, K, -(-N // 16) * 16)
    sa = rng.uniform(0.5, 1, (M, ox.blocks(K))).astype(np.float32)
    sb = rng.uniform(0.5, 1, (ox.blocks(K), ox.blocks(N))).astype(np.float32)
    args = [fp8(a).cuda(), torch.from_numpy(sa).cuda(), fp8(b).cuda()[:, :N], torch.from_numpy(sb).cuda()]
    C = torch.empty(M, N, device="cuda")
    g.force_tile_n(rows)
    assert stalled(lambda: g.fp8_blocks(*args, C)) == (g.GEMM_ERR_DEVICE_TIMEOUT, site)
    assert split is None or (g.last_k_split() > 1) == split
    assert g.device_status()[0] == 0
    for _ in range(2):
        g.fp8_blocks(*args, C)
        check_status()
        want, bound = ox.product(ox.dequantise(a, sa, 1), ox.dequantise(b[:, :N], sb, 128))
        assert np.all(np.abs(C.cpu().numpy() - want) <= bound)


@pytest.mark.parametrize("tokens,rows,site", [(3, 0, SITE_DECODE), (200, 128, SITE_DECODE), (200, 256, SITE_WIDE)])
def test_experts(short_limit, tokens, rows, site):
    layer = Layer(4, 528, 1040)
    ids, w, offsets, order = routing(tokens, 4, 2)
    x = torch.randn(tokens, 528, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    out = torch.empty_like(x)
    g.force_tile_n(rows)
    status, where = stalled(lambda: g.experts(layer.weights, x, offsets, order, w, out))
    assert (status, where) == (g.GEMM_ERR_DEVICE_TIMEOUT, site)
    for _ in range(2):
        g.experts(layer.weights, x, offsets, order, w, out)
        check_status()
        layer.check(x, ids, w, out)
