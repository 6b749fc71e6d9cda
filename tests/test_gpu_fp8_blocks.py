"""Block-scaled E4M3 products against the fp64 oracle, element by element, within what
fp32 sums and the one rounding to C's type may add (oracle.experts.product)."""
import numpy as np
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from experts_util import BF16, F32, check_status, codes, fp8, placed
from oracle import experts as ox

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, M, N, K, seed=0):
        rng = np.random.default_rng(seed + M + 7 * N + 31 * K)
        self.M, self.N, self.K = M, N, K
        self.a, self.b = codes(rng, M, K), codes(rng, K, N)
        self.sa = np.exp(rng.normal(0, 1, (M, ox.blocks(K)))).astype(np.float32)
        self.sb = np.exp(rng.normal(0, 1, (ox.blocks(K), ox.blocks(N)))).astype(np.float32)
        self.sa[rng.random(self.sa.shape) < 0.1] = 0
        self.c0 = torch.from_numpy(rng.normal(0, 100, (M, N)).astype(np.float32))

    def run(self, out, alpha=1.0, beta=0.0, pad=(0, 0, 0), offset=(0, 0, 0), path=None, want_path=None):
        A, B = placed(fp8(self.a), pad[0], offset[0], fill=0x7F), placed(fp8(self.b), pad[1], offset[1], fill=0x7F)
        c0 = self.c0.to(out)
        C = placed(c0 if beta else torch.full_like(c0, float("nan")), pad[2], offset[2], fill=7.0)
        if path is not None:
            g.force_path(path)
        try:
            g.fp8_blocks(A, torch.from_numpy(self.sa).cuda(), B, torch.from_numpy(self.sb).cuda(), C, alpha, beta)
        finally:
            g.force_path(g.PATH_AUTO)
        if want_path is not None:
            assert g.last_path() == want_path
        check_status()
        if pad[2]:
            assert (C.as_strided((self.M, self.N + pad[2]), C.stride())[:, self.N:] == 7.0).all()
        ref, bound = ox.product(ox.dequantise(self.a, self.sa, 1), ox.dequantise(self.b, self.sb, 128), alpha, beta,
                                c0.float().numpy(), out == BF16)
        off = np.abs(C.float().cpu().numpy().astype(np.float64) - ref)
        assert np.all(off <= bound), f"{(off > bound).sum()} of {off.size} off by up to {np.nanmax(off / bound):.2f} bounds"
        return C


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("N,K", [(16, 16), (128, 128), (144, 400), (1376, 512), (272, 2064), (4096, 256)])
@pytest.mark.parametrize("M", [1, 5, 16, 17, 33, 64, 77, 129, 300])
def test_sizes(M, N, K, out):
    Case(M, N, K).run(out, want_path=g.PATH_BLOCKS)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(513, 4096, 640), (1025, 2816, 384), (2100, 1040, 272)])
def test_many_rows(M, N, K, out):
    Case(M, N, K).run(out, want_path=g.PATH_BLOCKS)


@pytest.fixture(params=[128, 256])
def rows_a_tile(request):
    """Single CTAs with row tiles of 128, and CTA pairs, whatever the sizes ask for."""
    g.force_tile_n(request.param)
    yield request.param
    g.force_tile_n(0)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (130, 272, 144), (256, 256, 128), (257, 400, 1040), (700, 1376, 512)])
def test_each_kernel(M, N, K, out, rows_a_tile):
    c = Case(M, N, K)
    c.run(out, 1.0, 0.0, want_path=g.PATH_BLOCKS)
    assert g.last_tile_n() == rows_a_tile
    c.run(out, -1.5, 0.5, (16, 32, 3), (0, 16, 1))
    c.run(out, 2.0, 1.0, (0, 0, 8), (0, 0, 8))


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("M", [40, 290])
def test_odd_columns(M, out, rows_a_tile):
    """Rows of B that are whole vectors but for their last columns, and of C of any kind."""
    c = Case(M, 1003, 200)
    for pad_c in (0, 5, 13):
        c.run(out, 1.0, 0.0, (8, 5, pad_c), want_path=g.PATH_BLOCKS)
    c.run(out, 0.5, -1.0, (8, 5, 5), want_path=g.PATH_BLOCKS)


@pytest.mark.parametrize("M", [1, 40])
@pytest.mark.parametrize("N,K", [(1024, 8192), (128, 4096), (4096, 4096), (512, 1000)])
def test_split_k(M, N, K):
    """Few columns and rows: clusters share K (a tail block among them)."""
    if K == 1000:
        K = 1008
    Case(M, N, K).run(F32, want_path=g.PATH_BLOCKS)
    assert g.last_k_split() > 1


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("alpha,beta", [(1.0, 1.0), (-0.5, 0.25), (0.0, 1.0), (2.0, 0.0)])
@pytest.mark.parametrize("M", [3, 200])
def test_alpha_beta(M, alpha, beta, out):
    Case(M, 400, 384).run(out, alpha, beta)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("pad,offset", [((16, 32, 3), (0, 0, 0)), ((48, 16, 8), (16, 32, 1))])
def test_strides(out, pad, offset):
    for M in (9, 150):
        Case(M, 272, 400).run(out, 1.0, 0.5, pad, offset, want_path=g.PATH_BLOCKS)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("M,N,K,pad,offset", [
    (1, 1, 1, (0, 0, 0), (0, 0, 0)), (5, 37, 100, (0, 0, 0), (0, 0, 0)), (33, 129, 300, (1, 2, 3), (0, 0, 0)),
    (20, 144, 160, (0, 0, 0), (1, 0, 0)), (20, 144, 160, (0, 0, 0), (0, 8, 0)), (70, 200, 259, (0, 0, 0), (0, 0, 0))])
def test_generic(M, N, K, pad, offset, out):
    Case(M, N, K).run(out, 1.5, -0.5, pad, offset, want_path=g.PATH_GENERIC)


def test_forced_generic_agrees():
    Case(40, 272, 400).run(F32, path=g.PATH_GENERIC, want_path=g.PATH_GENERIC)


def test_nothing_to_add():
    """K == 0 gives beta * C; beta == 0 never reads C."""
    c = torch.full((5, 48), 3.0, device="cuda")
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    g.fp8_blocks(none.view(5, 0), torch.empty(5, 0, device="cuda"), none.view(0, 48), torch.empty(0, 1, device="cuda"),
                 c, beta=0.5)
    check_status()
    assert (c == 1.5).all()
    g.fp8_blocks(torch.empty(0, 64, dtype=torch.uint8, device="cuda"), torch.empty(0, 1, device="cuda"),
                 torch.zeros(64, 48, dtype=torch.uint8, device="cuda"), torch.ones(1, 1, device="cuda"),
                 torch.empty(0, 48, device="cuda"))


@pytest.mark.parametrize("M", [4, 100, 600])
def test_nan_and_infinite_scales_stay_in_their_rows(M):
    c = Case(M, 272, 400)
    A, B = fp8(c.a).cuda(), fp8(c.b).cuda()
    sa, sb = torch.from_numpy(c.sa).cuda(), torch.from_numpy(c.sb).cuda()
    clean, C = torch.empty(M, 272, device="cuda"), torch.empty(M, 272, device="cuda")
    g.fp8_blocks(A, sa, B, sb, clean)
    A.view(torch.uint8)[1, 200] = 0x7F
    sa[3, 1] = float("inf")
    g.fp8_blocks(A, sa, B, sb, C)
    check_status()
    rest = [m for m in range(M) if m not in (1, 3)]
    assert torch.isnan(C[1]).all() and not torch.isfinite(C[3]).all()
    assert torch.equal(C[rest], clean[rest])


def test_repeats_streams_and_graphs():
    c = Case(90, 1376, 1024)
    A, B = fp8(c.a).cuda(), fp8(c.b).cuda()
    sa, sb = torch.from_numpy(c.sa).cuda(), torch.from_numpy(c.sb).cuda()
    outs = [torch.empty(90, 1376, dtype=BF16, device="cuda") for _ in range(4)]
    g.fp8_blocks(A, sa, B, sb, outs[0])
    g.fp8_blocks(A, sa, B, sb, outs[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g.fp8_blocks(A, sa, B, sb, outs[2])
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.fp8_blocks(A, sa, B, sb, outs[3])
    graph.replay()
    check_status()
    for o in outs[1:]:
        assert torch.equal(outs[0], o)
