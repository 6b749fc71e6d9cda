"""gemm_experts_workspace on the CPU: the workspace of a call takes every call of fewer tokens."""
import os
import shutil

import pytest


@pytest.fixture(scope="module")
def g():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from roofline_driven_optimisation_gb300 import _build
    _build.build()
    import roofline_driven_optimisation_gb300 as lib
    lib.load()
    return lib


@pytest.mark.parametrize("top_k,hidden,width", [(1, 1, 1), (8, 4096, 1376), (2, 2048, 2752), (32, 7168, 2048), (1, 100, 9)])
def test_more_tokens_never_need_less(g, top_k, hidden, width):
    # around the tokens from which y is held in bf16, and far from them
    edge = (64 << 20) // (4 * top_k * -(-hidden // 8) * 8)
    tokens = sorted({1, 2, 3, 100, 16384} | {max(1, edge + d) for d in range(-3, 4)} | {2 * edge, 2 * edge + 1, 3 * edge})
    sizes = [g.gemm_experts_workspace(t, top_k, hidden, width) for t in tokens]
    assert sizes == sorted(sizes) and sizes[0] > 0


def test_sizes_that_no_call_takes_need_none(g):
    most = 65535 * 1024
    assert g.gemm_experts_workspace(1, 1, most, 1) > 0 and g.gemm_experts_workspace(1, 1, 1, most) > 0
    # past 32 bits in every part, the largest that a call takes
    assert g.gemm_experts_workspace(2 ** 31 - 1, 1, most, most) >= (2 ** 31 - 1) * (most + most + 4 * most)
    for bad in ((1, 1, most + 1, 1), (1, 1, 1, most + 1), (1, 1, 2 ** 31 - 1, 1), (2 ** 31 - 1, 1, 2 ** 31 - 1, 2 ** 31 - 1)):
        assert g.gemm_experts_workspace(*bad) == 0
