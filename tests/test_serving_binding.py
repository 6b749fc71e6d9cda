"""What the serving operators' binding makes of tensors before a call, on the CPU."""
import pytest
import torch

import roofline_driven_optimisation_gb300 as g


class OnGpu:
    """Stands for a CUDA tensor: what the binding looks at, without a GPU."""
    is_cuda = True

    def __init__(self, t):
        self.dtype, self.shape, self.stride = t.dtype, t.shape, t.stride


def heads(t, n, dim, tokens):
    g._torch()
    return g._heads(OnGpu(t), "Q", n, dim, tokens)


def test_rows_that_overlap_are_refused():
    # a stride below a row's width must not be replaced: the call would leave the tensor
    row = torch.zeros(1, 4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="apart"):
        heads(row.expand(3, 4, 8), 4, 8, 3)
    with pytest.raises(ValueError, match="apart"):
        heads(torch.zeros(200, dtype=torch.bfloat16).as_strided((3, 4, 8), (31, 8, 1)), 4, 8, 3)
    with pytest.raises(ValueError, match="apart"):
        g._ld(torch.zeros(1, 8).expand(3, 8))
    with pytest.raises(ValueError, match="apart"):
        g._ld(torch.zeros(40).as_strided((3, 8), (7, 1)))


def test_rows_that_do_not_overlap_are_taken():
    wide = torch.zeros(3, 50, dtype=torch.bfloat16)
    assert heads(wide[:, :32].unflatten(1, (4, 8)), 4, 8, 3) == 50
    assert heads(torch.zeros(3, 4, 8, dtype=torch.bfloat16), 4, 8, 3) == 32
    # the stride of a single row, or of none, is never taken
    assert heads(torch.zeros(1, 4, 8, dtype=torch.bfloat16).expand(1, 4, 8).as_strided((1, 4, 8), (0, 8, 1)), 4, 8, 1) == 32
    assert heads(torch.zeros(0, 4, 8, dtype=torch.bfloat16), 4, 8, 0) == 32
    assert g._ld(torch.zeros(1, 8).as_strided((1, 8), (0, 1))) == 8 and g._ld(torch.zeros(3, 9)[:, :8]) == 9
    assert g._ld(torch.zeros(3, 0)) == 1


def test_caches_that_overlap_are_refused():
    k = torch.zeros(2, 2, 16, 64, dtype=torch.int8)
    s, t = torch.zeros(2, 2), torch.zeros(3, 4, dtype=torch.int32)
    one = torch.zeros(2, 2, 1, 64, dtype=torch.int8).expand(2, 2, 16, 64)
    with pytest.raises(ValueError, match="apart"):
        g.KVCache(one, one, s, s, t)
    # one table row for several sequences
    with pytest.raises(ValueError, match="apart"):
        g.KVCache(k, k, s, s, t[:1].expand(3, 4))
    with pytest.raises(ValueError, match="CUDA"):      # nothing else is wrong with them
        g.KVCache(k, k, s, s, t)
