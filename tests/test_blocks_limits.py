"""Sizes near 2^31 of block-scaled products, on the CPU: N and K above 2^31 - 256, whose blocks and
tiles do not count in 32 bits, are refused; the largest that are taken are refused for nothing
but their missing operands."""
import os
import shutil

import pytest

MOST = 2 ** 31 - 256
P = 1 << 20          # an aligned stand-in address (never dereferenced)


@pytest.fixture(scope="module")
def g():
    import torch
    if torch.cuda.is_available():
        pytest.skip("runs only where validation is all that can happen")
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from roofline_driven_optimisation_gb300 import _build
    _build.build()
    import roofline_driven_optimisation_gb300 as lib
    lib.load()
    return lib


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("N,K", [(1, MOST), (MOST, 1), (1, MOST + 1), (1, MOST + 129), (1, 2 ** 31 - 1), (MOST + 1, 1),
                                 (2 ** 31 - 4, 1), (2 ** 31 - 1, 1)])
def test_blocks_that_do_not_count_in_32_bits(g, N, K, bf16):
    fn = g.gemm_fp8_blocks if bf16 else g.gemm_fp8_blocks_f32out
    with pytest.raises(g.GemmError) as e:
        fn(1, N, K, 1.0, None, K, P, 1 << 25, P, N, P, 1 << 25, 0.0, P, 2 ** 31 - 1, 0)
    if N > MOST or K > MOST:
        assert e.value.code == g.GEMM_ERR_UNSUPPORTED and "above" in str(e.value)
    else:
        assert e.value.code == g.GEMM_ERR_INVALID_ARG and "NULL" in str(e.value)
