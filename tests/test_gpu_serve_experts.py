"""Routing, quantisation, block-scaled products and experts as they are used together: in
the serving example, in a captured step, and by calls on two streams at once."""
import os
import sys

import numpy as np
import pytest
import torch

from conftest import ROOT

import roofline_driven_optimisation_gb300 as g
from experts_util import BF16, Layer, check_status
from oracle import experts as ox

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example(cuda_lib):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import serve_step
    return serve_step


def test_serving_with_experts_runs_and_repeats(example):
    prompts = [[1, 5, 9], list(range(100, 400)), [7], list(range(64))]
    layer = example.Layer(heads=8, kv_heads=2, dim=64, ffn=272, vocab=1000, experts=8, top_k=3)
    token, logprob = example.serve(prompts, 6, layer)
    again, _ = example.serve(prompts, 6, layer)
    check_status()
    assert token.shape == (4, 6) and torch.equal(token, again)
    assert ((token >= 0) & (token < 1000)).all() and torch.isfinite(logprob).all() and (logprob <= 0).all()


class Step:
    """A layer's step: x through a block-scaled product into the router's logits, routed
    to 3 of 16 experts; every buffer its own."""

    def __init__(self, layer, tokens, seed):
        rng = np.random.default_rng(seed)
        H, E = layer.hidden, layer.experts
        self.layer, self.tokens = layer, tokens
        self.x = torch.empty(tokens, H, dtype=BF16, device="cuda")
        self.router = rng.normal(size=(H, E)).astype(np.float32)
        self.rq = torch.empty(H, E, dtype=torch.float8_e4m3fn, device="cuda")
        self.rs = torch.empty(-(-H // 128), 1, device="cuda")
        g.fp8_quantise(torch.from_numpy(self.router).cuda(), self.rq, self.rs, 128)
        self.xq = torch.empty(tokens, H, dtype=torch.float8_e4m3fn, device="cuda")
        self.xs = torch.empty(tokens, -(-H // 128), device="cuda")
        self.logits = torch.empty(tokens, E, device="cuda")
        ints = dict(dtype=torch.int32, device="cuda")
        self.ids, self.w = torch.empty(tokens, 3, **ints), torch.empty(tokens, 3, device="cuda")
        self.offsets, self.order = torch.empty(E + 1, **ints), torch.empty(tokens * 3, **ints)
        self.out = torch.empty(tokens, H, dtype=BF16, device="cuda")

    def run(self, stream=None):
        g.fp8_quantise(self.x, self.xq, self.xs, stream=stream)
        g.fp8_blocks(self.xq, self.xs, self.rq, self.rs, self.logits, alpha=0.1, stream=stream)
        g.route(self.logits, self.ids, self.w, self.offsets, self.order, groups=2, top_groups=1, score=g.ROUTE_SIGMOID,
                stream=stream)
        g.experts(self.layer.weights, self.x, self.offsets, self.order, self.w, self.out, stream=stream)

    def fill(self, seed):
        gen = torch.Generator().manual_seed(seed)
        self.x.copy_(torch.randn(self.x.shape, generator=gen))
        self.out.fill_(float("nan"))

    def check(self):
        x = self.x.float().cpu().numpy()
        logits, bound = ox.product(ox.dequantise(*ox.quantise(x), 1), ox.dequantise(*ox.quantise(self.router, 128), 128), 0.1)
        got = self.logits.cpu().numpy()
        assert np.all(np.abs(got - logits) <= bound)
        ids, w = ox.route(got, 3, score=ox.SIGMOID, groups=2, top_groups=1)
        assert np.array_equal(self.ids.cpu().numpy(), ids) and np.allclose(self.w.cpu().numpy(), w, rtol=1e-5, atol=0)
        offsets, order = ox.by_expert(ids, self.layer.experts)
        assert np.array_equal(self.offsets.cpu().numpy(), offsets) and np.array_equal(self.order.cpu().numpy(), order)
        self.layer.check(self.x, self.ids, self.w, self.out)


@pytest.mark.parametrize("tokens", [1, 40, 700])
def test_a_layer_called_captured_and_replayed(tokens):
    step = Step(Layer(16, 272, 144), tokens, 1)
    step.fill(1)
    step.run()
    check_status()
    step.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    for seed in (2, 3):
        step.fill(seed)
        graph.replay()
        check_status()
        step.check()


def test_weights_written_right_before_the_call():
    # weights, scales and routing are written by the calls just before on the same stream,
    # over other ones that would give other results
    layer = Layer(16, 1024, 512, seed=3)
    step = Step(layer, 5, 2)
    step.fill(4)
    step.run()
    check_status()
    want = step.out.clone()
    kept = [t.clone() for t in layer.weights.tensors]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for t in layer.weights.tensors:
            t.view(torch.uint8).zero_()
        step.order.zero_()
        step.offsets.zero_()
        for t, k in zip(layer.weights.tensors, kept):
            t.view(torch.uint8).copy_(k.view(torch.uint8))
        step.run()
    for _ in range(3):
        graph.replay()
        check_status()
        assert torch.equal(step.out, want)


def test_two_streams_at_once():
    layer = Layer(16, 272, 400)
    steps = [Step(layer, n, n) for n in (30, 700)]
    streams = [torch.cuda.Stream() for _ in steps]
    for i, s in enumerate(steps):
        s.fill(i)
    torch.cuda.synchronize()
    for _ in range(10):
        for s, on in zip(steps, streams):
            s.run(on.cuda_stream)
    check_status()
    for s in steps:
        s.check()
