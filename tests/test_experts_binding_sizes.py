"""Sizes that do not fit the C ABI's integers, and workspaces whose elements are not their bytes:
the routed experts' binding refuses them (ctypes would pass a number's last 32 bits)."""
import os
import shutil

import pytest
import torch

BIG = 2 ** 32 + 3


@pytest.fixture(scope="module")
def g():
    if torch.cuda.is_available():
        pytest.skip("runs only where validation is all that can happen")
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from roofline_driven_optimisation_gb300 import _build
    _build.build()
    import roofline_driven_optimisation_gb300 as lib
    lib.load()
    lib._torch()
    return lib


class OnGpu:
    """Stands for a CUDA tensor without memory: what the binding looks at."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.float32, step=None):
        t = torch.empty(shape, dtype=dtype, device="meta")
        self.t = t if step is None else t.as_strided(shape, (step, 1))

    def get_device(self):
        return 0

    def data_ptr(self):
        return 1 << 20

    def __getattr__(self, name):
        return getattr(self.t, name)


E4M3, I32, BF16, U8 = torch.float8_e4m3fn, torch.int32, torch.bfloat16, torch.uint8


@pytest.fixture(autouse=True)
def no_stream(g, monkeypatch):
    monkeypatch.setattr(g, "_raw_stream", lambda index: 0)


def test_route(g):
    for tokens, experts, top_k in ((BIG, 8, 2), (2 ** 31, 8, 2), (3, BIG, 2)):
        with pytest.raises(ValueError, match="at most"):
            g.route(OnGpu(tokens, experts), OnGpu(tokens, top_k, dtype=I32), OnGpu(tokens, top_k))


def test_quantise(g):
    for rows, cols in ((BIG, 8), (2, BIG), (2 ** 31, 1)):
        with pytest.raises(ValueError, match="at most"):
            g.fp8_quantise(OnGpu(rows, cols), OnGpu(rows, cols, dtype=E4M3), OnGpu(rows, -(-cols // 128)))


def test_blocks(g):
    def call(M, N, K, **step):
        kb, nb = -(-K // 128), -(-N // 128)
        g.fp8_blocks(OnGpu(M, K, dtype=E4M3, step=step.get("a")), OnGpu(M, kb, step=step.get("sa")),
                     OnGpu(K, N, dtype=E4M3, step=step.get("b")), OnGpu(kb, nb, step=step.get("sb")),
                     OnGpu(M, N, step=step.get("c")))
    for sizes in ((BIG, 8, 8), (8, BIG, 8), (8, 8, BIG)):
        with pytest.raises(ValueError, match="at most"):
            call(*sizes)
    for name in ("a", "sa", "b", "sb", "c"):
        for step in (2 ** 31, 2 ** 32 + 512):
            with pytest.raises(ValueError, match="at most"):
                call(300, 300, 300, **{name: step})
    with pytest.raises(g.GemmError):                          # as far as the device, where there is none
        call(300, 300, 300, a=2 ** 31 - 1, c=2 ** 31 - 1)


def test_expert_weights(g):
    for experts, hidden, width in ((BIG, 16, 16), (2, BIG, 16), (2, 16, BIG)):
        up, down = OnGpu(experts, hidden, width, dtype=U8), OnGpu(experts, width, hidden, dtype=U8)
        s = OnGpu(experts, 1, 1)
        with pytest.raises(ValueError, match="at most"):
            g.ExpertWeights(up, s, up, s, down, s)


def test_strides_that_nothing_steps_over(g):
    """gate and up of one expert, or one row, may differ in the strides of it."""
    def weights(shape, step_gate, step_up):
        def make(shape, step):
            t = OnGpu(*shape, dtype=U8)
            t.t, t.device = t.t.as_strided(shape, step), "cuda:0"
            return t
        down = make((shape[0], shape[2], shape[1]), (shape[1] * shape[2], shape[1], 1))
        s = OnGpu(shape[0], 1, 1)
        s.device = "cuda:0"
        return g.ExpertWeights(make(shape, step_gate), s, make(shape, step_up), s, down, s)
    for shape, gate, up in (((1, 16, 32), (512, 32, 1), (4096, 32, 1)), ((3, 1, 32), (32, 32, 1), (32, 64, 1))):
        assert weights(shape, gate, up).experts == shape[0]
    for shape, gate, up in (((2, 16, 32), (512, 32, 1), (4096, 32, 1)), ((1, 16, 32), (512, 32, 1), (512, 48, 1))):
        with pytest.raises(ValueError, match="strides"):
            weights(shape, gate, up)


class Weights:
    experts, hidden, width, device, index, address = 4, 64, 32, torch.device("cpu"), 0, 0


def experts(g, tokens=3, top_k=2, workspace=None):
    g.experts(Weights(), OnGpu(tokens, 64, dtype=BF16), OnGpu(5, dtype=I32), OnGpu(tokens * top_k, dtype=I32),
              OnGpu(tokens, top_k), OnGpu(tokens, 64, dtype=BF16), workspace=workspace)


def test_experts(g):
    for tokens, top_k in ((BIG, 1), (1, BIG)):
        with pytest.raises(ValueError, match="at most"):
            experts(g, tokens, top_k)


def test_workspaces(g):
    spread = OnGpu(1, dtype=U8)
    spread.t = spread.t.expand(1 << 20)                       # a byte that looks like many
    gaps = OnGpu(1 << 21, dtype=U8)
    gaps.t = gaps.t[::2]
    for bad in (spread, gaps, OnGpu(1 << 20), OnGpu(1 << 20, dtype=torch.int8)):
        with pytest.raises(TypeError, match="workspace"):
            experts(g, workspace=bad)
        with pytest.raises(TypeError, match="workspace"):
            g.route(OnGpu(300, 8), OnGpu(300, 2, dtype=I32), OnGpu(300, 2), OnGpu(9, dtype=I32), OnGpu(600, dtype=I32),
                    workspace=bad)
