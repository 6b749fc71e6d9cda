"""Block-scaled products of the most columns and the longest K."""
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from experts_util import check_status

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 256


def zeros(*shape):
    return torch.zeros(*shape, dtype=torch.uint8, device="cuda")


def test_longest_k(cuda_lib):
    A, B = zeros(1, MOST), zeros(MOST, 16)[:, :1]
    sa = torch.ones(1, MOST // 128, device="cuda")
    sb = torch.ones(MOST // 128, 1, device="cuda")
    at = torch.tensor([0, 127, 128, 2 ** 30, 2 ** 30 + 5, MOST - 129, MOST - 1], device="cuda")
    A[0, at], B[at, 0] = 0x38, 0x40                           # 1.0 and 2.0
    sa[0, -1], sb[-1, 0], sb[2 ** 23, 0] = 8.0, 0.5, 16.0
    C = torch.full((1, 1), float("nan"), device="cuda")
    g.fp8_blocks(A, sa, B, sb, C)
    assert g.last_path() == g.PATH_BLOCKS
    check_status()
    # two of the seven lie in block 2^23, one in the last
    assert C.item() == 2 * (4 + 2 * 16 + 4)


@pytest.mark.parametrize("M,path", [(1, g.PATH_GENERIC), (2, g.PATH_BLOCKS)])     # a row of one column: no map takes it
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_most_columns(cuda_lib, dtype, M, path):
    A, B = zeros(M, 16)[:, :1], zeros(1, MOST)
    A[:] = 0x40
    B[0] = 0x38
    sb = (torch.arange(MOST // 128, device="cuda") % 127 + 1).float()[None]
    C = torch.full((M, MOST), float("nan"), dtype=dtype, device="cuda")
    g.fp8_blocks(A, torch.ones(M, 1, device="cuda"), B, sb, C)
    assert g.last_path() == path
    check_status()
    for row in C:
        got = row.view(-1, 128)
        assert torch.equal(got.amin(1).float(), 2 * sb[0]) and torch.equal(got.amax(1).float(), 2 * sb[0])
