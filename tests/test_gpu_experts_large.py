"""Routing, block-scaled products and experts where offsets pass 32 bits."""
import numpy as np
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from experts_util import BF16, check_status, codes, fp8
from oracle import experts as ox

pytestmark = pytest.mark.gpu


def sparse(rows, cols, step, dtype):
    """[rows][cols] of rows `step` elements apart, in memory of no set contents."""
    return torch.empty(rows * step, dtype=dtype, device="cuda").view(rows, step)[:, :cols]


def test_route(cuda_lib):
    tokens, step = 4200, 1 << 20                       # the last row begins 4.4e9 elements in
    logits = sparse(tokens, 64, step, BF16)
    values = torch.randn(tokens, 64, generator=torch.Generator().manual_seed(0)).to(BF16)
    logits.copy_(values)
    ids = torch.empty(tokens, 4, dtype=torch.int32, device="cuda")
    g.route(logits, ids, torch.empty(tokens, 4, device="cuda"))
    check_status()
    assert np.array_equal(ids.cpu().numpy(), ox.route(values.float().numpy(), 4)[0])


@pytest.mark.parametrize("rows", [0, 128])
def test_product(cuda_lib, rows):
    M, N, K, step = 8300, 144, 272, 1 << 19
    rng = np.random.default_rng(0)
    a, b = codes(rng, M, K), codes(rng, K, N)
    sa = rng.uniform(0.5, 1, (M, 3)).astype(np.float32)
    sb = rng.uniform(0.5, 1, (3, 2)).astype(np.float32)
    A, C = sparse(M, K, step, torch.float8_e4m3fn), sparse(M, N, step, BF16)
    A.copy_(fp8(a))
    g.force_tile_n(rows)
    try:
        g.fp8_blocks(A, torch.from_numpy(sa).cuda(), fp8(b).cuda(), torch.from_numpy(sb).cuda(), C)
    finally:
        g.force_tile_n(0)
    check_status()
    want, bound = ox.product(ox.dequantise(a, sa, 1), ox.dequantise(b, sb, 128), bf16=True)
    assert np.all(np.abs(C.float().cpu().numpy() - want) <= bound)


@pytest.mark.parametrize("tokens", [7, 4100])
def test_experts(cuda_lib, tokens):
    E, H, F = 1024, 2048, 2112                         # 4.4e9 codes a weight
    gen = torch.Generator(device="cuda").manual_seed(0)
    parts = []
    for rows, cols in ((H, F), (H, F), (F, H)):
        w = torch.empty(E, rows, cols, dtype=torch.uint8, device="cuda")
        for e in range(0, E, 64):
            w[e:e + 64].random_(0, 0x70, generator=gen)          # positive codes ...
            w[e:e + 64] += (w[e:e + 64] & 1) << 7                # ... and negative ones
        parts += [w, torch.rand(E, -(-rows // 128), -(-cols // 128), generator=gen, device="cuda") * (0.05 / rows ** 0.5)]
    x = torch.randn(tokens, H, generator=gen, device="cuda").to(BF16)
    # each expert has a token and the last expert the most
    ids = (torch.arange(tokens, device="cuda") % E).int()
    ids[1::3] = E - 1
    w = torch.ones(tokens, 1, device="cuda")
    order = torch.argsort(ids, stable=True).int()
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(ids, minlength=E), 0)
    out = torch.empty_like(x)
    g.experts(g.ExpertWeights(*parts), x, offsets, order, w, out)
    check_status()
    chosen = [0, 1, 2, tokens - 2, tokens - 1]
    for t in chosen:
        e = int(ids[t])
        v = [ox.dequantise(parts[2 * i][e].cpu().numpy(), parts[2 * i + 1][e].cpu().numpy(), 128) for i in range(3)]
        want, bound = ox.experts(x[t:t + 1].float().cpu().numpy(), [[0]], [[1.0]], *([m] for m in v))
        assert np.all(np.abs(out[t].float().cpu().numpy() - want[0]) <= bound[0] + 1e-30)
