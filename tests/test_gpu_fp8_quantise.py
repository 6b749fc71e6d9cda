"""E4M3 codes with block scales against the oracle's fp32 arithmetic: the same bits."""
import numpy as np
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from experts_util import check_status, placed
from oracle import experts as ox

pytestmark = pytest.mark.gpu


def check(x, block_rows, pad=0, offset=0):
    rows, cols = x.shape
    codes = placed(torch.full((rows, cols), 0x55, dtype=torch.uint8), pad, offset, fill=0x55)
    scales = torch.full((-(-rows // block_rows), ox.blocks(cols)), float("nan"), device="cuda")
    g.fp8_quantise(x, codes, scales, block_rows)
    assert g.last_path() == g.PATH_QUANTISE
    check_status()
    want, s = ox.quantise(x.float().cpu().numpy(), block_rows)
    np.testing.assert_array_equal(scales.cpu().numpy(), s)
    got = codes.cpu().numpy()
    # NaN codes carry either sign
    got, want = (np.where((c & 0x7F) == 0x7F, 0x7F, c) for c in (got, want))
    np.testing.assert_array_equal(got, want)
    if pad:
        around = codes.as_strided((rows, cols + pad), codes.stride())[:, cols:]
        assert (around == 0x55).all()


def values(rows, cols, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=gen) * torch.exp(2 * torch.randn(rows, 1, generator=gen))
    return x.to(dtype)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (3, 127), (128, 128), (129, 136), (77, 1376), (300, 1000), (1000, 4096)])
def test_sizes(rows, cols, dtype, block_rows):
    check(values(rows, cols, dtype).cuda(), block_rows)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,offset", [(3, 0), (8, 0), (8, 1), (16, 8)])
def test_strides_and_alignment(pad, offset, dtype, block_rows):
    check(placed(values(140, 264, dtype), pad, offset), block_rows, pad, offset)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_special_values(dtype, block_rows):
    x = values(256, 512, dtype)
    x[0] = 0
    x[1, :128] = 0
    x[2, 5], x[2, 200] = float("inf"), -float("inf")
    x[3, 5] = float("nan")
    x[4, :128] = float("nan")
    x[5] *= 1e-38
    x[6] = 1e-40
    x[7] = 3e38
    x[128:, 128:256] = 0
    check(x.cuda(), block_rows)


def test_no_rows():
    g.fp8_quantise(torch.empty(0, 256, device="cuda"), torch.empty(0, 256, dtype=torch.uint8, device="cuda"),
                   torch.empty(0, 2, device="cuda"))
    check_status()


def test_offsets_past_32_bits():
    """2^31 values and more in a row of rows."""
    rows, cols = 70000, 32768
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = values(3, cols, torch.bfloat16).cuda()
    x[-3:] = tail
    codes = torch.full((rows, cols), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, cols // 128, device="cuda")
    g.fp8_quantise(x, codes, scales)
    check_status()
    want, s = ox.quantise(tail.float().cpu().numpy())
    np.testing.assert_array_equal(codes[-3:].cpu().numpy(), want)
    np.testing.assert_array_equal(scales[-3:].cpu().numpy(), s)
    assert int(codes[:-3].max()) == 0
