"""silu of the experts' epilogues on every fp32 gate, against 64 bits: relative errors from -87.3
on, and next to 0 below, where it is flushed; infinite and NaN gates.

Half steps (2^-24) of itself that a result may be off by: 8 of the fast form, which is what the
oracle's bounds take, and 6 of the generic one (expf by 2 units of 2^-23, a sum and a division by
half a step each); the product with `up` adds one."""
import ctypes
import os
import subprocess

import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from conftest import ROOT
from experts_util import BF16, Layer, check_status, routing

pytestmark = pytest.mark.gpu
OUT = os.path.join(ROOT, "roofline_driven_optimisation_gb300", "_build", "silu_check.so")


@pytest.fixture(scope="module")
def check(cuda_lib):
    from roofline_driven_optimisation_gb300 import _build
    os.makedirs(os.path.dirname(OUT), exist_ok=True)
    subprocess.run([_build.nvcc()] + _build.ARCH_FLAGS + _build.COMMON_FLAGS +
                   ["-shared", os.path.join(ROOT, "tests", "silu_check.cu"), "-o", OUT], check=True)
    lib = ctypes.CDLL(OUT)
    lib.silu_check.argtypes = [ctypes.c_uint32, ctypes.c_uint64, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p]

    def run(first, count, u):
        errors, wrong = (ctypes.c_float * 4)(), ctypes.c_uint(0)
        assert lib.silu_check(first, count, u, errors, ctypes.byref(wrong)) == 0
        return list(errors), wrong.value
    return run


@pytest.mark.parametrize("u", [1.0, -1.0, 1.5, 3.7e-3, -1.1e4])
def test_every_gate(check, u):
    errors, wrong = check(0, 1 << 32, u)
    more = 0 if abs(u) == 1 else 1
    assert wrong == 0
    assert errors[0] <= 8 + more and errors[2] <= 6 + more, errors
    # |g| e^-|g| falls from 87.3 on, where it is 1.1e-36: 2^-119.4
    assert errors[1] <= 2.0 ** -119 * abs(u) and errors[3] <= 2.0 ** -119 * abs(u), errors


@pytest.mark.parametrize("hidden,width", [(256, 144), (129, 70)])          # the second: generic kernels
@pytest.mark.parametrize("tokens,rows", [(3, 0), (300, 0), (300, 256)])
def test_experts_with_large_gates(cuda_lib, tokens, rows, hidden, width):
    layer = Layer(4, hidden, width)
    layer.weights.tensors[1].mul_(512.0)                  # gates of some hundreds on both sides
    layer.values[0] = [v * 512.0 for v in layer.values[0]]
    ids, w, offsets, order = routing(tokens, 4, 2)
    x = torch.randn(tokens, hidden, generator=torch.Generator().manual_seed(5)).to(BF16).cuda()
    out = torch.empty_like(x)
    g.force_tile_n(rows)
    try:
        g.experts(layer.weights, x, offsets, order, w, out)
    finally:
        g.force_tile_n(0)
    check_status()
    layer.check(x, ids, w, out)
