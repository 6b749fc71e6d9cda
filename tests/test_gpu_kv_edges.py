"""gemm_kv_append and gemm_kv_attention at the ends of what they take."""
import numpy as np
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from oracle import serving as S
from serving_util import Case, check_status

pytestmark = pytest.mark.gpu


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("new", [1, 2, 9])
def test_positions_up_to_the_last_of_32_bits(cuda_lib, new):
    # without a rotation any position will do; the last page ends at 2^31, and no table
    # reaches it: queries are taken over, keys and values reported
    c = Case(g.KV_INT8, 2, 64, 16, [30])
    before = {n: c.got(n).copy() for n in ("k", "v", "ks", "vs")}
    # a page's worth of rows behind the call's, which it must leave alone
    allQ, allK = torch.randn(new + 16, 3, 64, device="cuda").bfloat16(), torch.randn(new + 16, 2, 64, device="cuda").bfloat16()
    all_out = torch.zeros_like(allQ)
    Q, K, out = allQ[:new], allK[:new], all_out[:new]
    g.kv_append(c.cache, Q, K, K, None, None, ints(2 ** 31 - 1 - new), out, start=ints(0, new), max_new=new)
    torch.cuda.synchronize()
    assert g.device_status() == (g.GEMM_ERR_INVALID_ARG, 60)
    assert torch.equal(out, Q) and (all_out[new:] == 0).all()
    assert all(np.array_equal(before[n], c.got(n)) for n in before)
