"""Sizes of the serving operators that pass 32 bits, on the CPU."""
import shutil
import os

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


@pytest.mark.parametrize("seqs,heads,group,max_new", [(1, 1, 1, 1), (7, 3, 5, 9), (1, 1, 65535, 2 ** 31 - 1),
                                                      (8192, 1, 65535, 2 ** 31 - 1), (8192, 8, 8, 2 ** 31 - 1)])
def test_workspace_has_a_counter_for_each_tile(g, seqs, heads, group, max_new):
    # a tile has 32 rows at most, and a sequence and head max_new * group rows
    size = g.gemm_kv_attention_workspace(seqs, heads, heads * group, 128, max_new) - \
        g.gemm_kv_attention_workspace(0, heads, heads * group, 128, max_new)
    least = 4 * seqs * heads * -(-max_new * group // 32)
    assert least <= size <= 4 * least + 16
