"""Quantisation of the most columns and the most rows: a block along a row has the codes and
scale of a row of 128 values by itself, and so has a column of 128 rows."""
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from experts_util import BF16, check_status

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1
BLOCKS = 2 ** 24


@pytest.fixture(scope="module")
def values():
    """2^31 values, of which the last is left out below."""
    x = torch.empty(2 ** 31, dtype=BF16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(0))
    x[-1] = 0                                    # as a value that is not there
    codes, scales = torch.empty(2 ** 31, dtype=torch.uint8, device="cuda"), torch.empty(BLOCKS, device="cuda")
    g.fp8_quantise(x.view(BLOCKS, 128), codes.view(BLOCKS, 128), scales.view(BLOCKS, 1))
    check_status()
    return x, codes, scales


@pytest.mark.parametrize("shape,block_rows,scale_shape", [
    ((1, MOST), 1, (1, BLOCKS)), ((1, MOST), 128, (1, BLOCKS)), ((MOST, 1), 128, (BLOCKS, 1)),
    ((1, MOST - 127), 1, (1, BLOCKS - 1)), ((MOST - 127, 1), 128, (BLOCKS - 1, 1))])
def test_largest_sizes(cuda_lib, values, shape, block_rows, scale_shape):
    x, codes, scales = values
    n = shape[0] * shape[1]
    got = torch.full((2 ** 31,), 0x7F, dtype=torch.uint8, device="cuda")
    s = torch.full(scale_shape, float("nan"), device="cuda")
    g.fp8_quantise(x[:n].view(shape), got[:n].view(shape), s, block_rows=block_rows)
    check_status()
    whole = n // 128 * 128
    assert torch.equal(got[:n], codes[:n]) and (got[n:] == 0x7F).all()
    assert torch.equal(s.view(-1), scales[:s.numel()])
    assert whole in (n, n - 127)
