"""The block-scaled pair kernel gives up in the middle of K: the warps that store rows of C
wait for a whole item, so that a limit shorter than an item ends their wait while all other
roles are at work.  The kernel reports it and leaves, and the next call is right."""
import numpy as np
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from experts_util import BF16, check_status, codes, fp8
from oracle import experts as ox

pytestmark = pytest.mark.gpu

SITE_ROWS = 81                        # WaitSite value of the library
LIMIT_NS = 1_000_000


@pytest.fixture
def short_limit(cuda_lib):
    assert g.device_status()[0] == 0
    g.set_wait_timeout_ns(LIMIT_NS)
    g.force_tile_n(256)
    try:
        yield
    finally:
        g.set_wait_timeout_ns(0)
        g.force_tile_n(0)


def product(M, N, K, C):
    """Random operands on the GPU, and the call."""
    A = torch.randint(0, 0x70, (M, K), dtype=torch.uint8, device="cuda")
    B = torch.randint(0, 0x70, (K, N), dtype=torch.uint8, device="cuda")
    sa = torch.ones(M, ox.blocks(K), device="cuda")
    sb = torch.ones(ox.blocks(K), ox.blocks(N), device="cuda")
    g.fp8_blocks(A, sa, B, sb, C)
    torch.cuda.synchronize()


# 2560 blocks of K take 1 ms; several items, so that warps are at the ends of some too
@pytest.mark.parametrize("M,N,blocks", [(300, 528, 6000), (2000, 4096, 4001)])
def test_product_gives_up_midway(short_limit, M, N, blocks):
    C = torch.empty(M, N, dtype=BF16, device="cuda")
    product(M, N, blocks * 128, C)
    status, where = g.device_status()
    assert (status, where) == (g.GEMM_ERR_DEVICE_TIMEOUT, SITE_ROWS)
    assert g.device_status()[0] == 0
    rng = np.random.default_rng(0)
    a, b = codes(rng, 300, 1024), codes(rng, 1024, 528)
    sa = rng.uniform(0.5, 1, (300, 8)).astype(np.float32)
    sb = rng.uniform(0.5, 1, (8, 5)).astype(np.float32)
    out = torch.empty(300, 528, dtype=BF16, device="cuda")
    g.fp8_blocks(fp8(a).cuda(), torch.from_numpy(sa).cuda(), fp8(b).cuda(), torch.from_numpy(sb).cuda(), out)
    check_status()
    want, bound = ox.product(ox.dequantise(a, sa, 1), ox.dequantise(b, sb, 128), bf16=True)
    assert np.all(np.abs(out.float().cpu().numpy() - want) <= bound)


# the limit ends near the end of K, and with all of K in the ring: the roles that copy and
# multiply may be through when another gives up
@pytest.mark.parametrize("blocks", [2500, 2600, 2700, 2800, 2900])
def test_product_gives_up_at_the_end(short_limit, blocks):
    C = torch.empty(256, 256, dtype=BF16, device="cuda")
    product(256, 256, blocks * 128, C)
    assert g.device_status()[0] in (0, g.GEMM_ERR_DEVICE_TIMEOUT)
    out = torch.empty(300, 528, dtype=BF16, device="cuda")
    for _ in range(3):
        product(300, 528, 512, out)
        check_status()


@pytest.mark.parametrize("M,rows", [(4, 0), (60, 0), (300, 128), (300, 256)])
@pytest.mark.parametrize("blocks", [1, 2, 4])
def test_stalled_with_all_of_k_in_the_ring(short_limit, M, rows, blocks):
    A, sa = codes(np.random.default_rng(1), M, blocks * 128), np.ones((M, blocks), np.float32)
    B, sb = codes(np.random.default_rng(2), blocks * 128, 528), np.ones((blocks, 5), np.float32)
    args = [fp8(A).cuda(), torch.from_numpy(sa).cuda(), fp8(B).cuda(), torch.from_numpy(sb).cuda()]
    out = torch.empty(M, 528, device="cuda")
    g.force_tile_n(rows)
    g.test_stall(1)
    try:
        g.fp8_blocks(*args, out)
    finally:
        g.test_stall(0)
    torch.cuda.synchronize()
    assert g.device_status()[0] == g.GEMM_ERR_DEVICE_TIMEOUT
    for _ in range(2):
        g.fp8_blocks(*args, out)
        check_status()
        want, bound = ox.product(ox.dequantise(A, sa, 1), ox.dequantise(B, sb, 128))
        assert np.all(np.abs(out.cpu().numpy() - want) <= bound)
