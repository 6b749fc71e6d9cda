"""The example's serving loop: decoding a sequence a token at a time gives the logits of
prefilling it at once, and a run repeats itself."""
import os
import sys

import pytest
import torch

from conftest import ROOT

import roofline_driven_optimisation_gb300 as g

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example(cuda_lib):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import serve_step
    return serve_step


def test_decoding_matches_prefilling_everything(example):
    # the logits of a token-by-token run against those of one prefill of the same tokens:
    # both append the same values to their caches, page scales included once the pages
    # are full, so they differ by the order of bf16 roundings only
    layer = example.Layer(heads=8, kv_heads=2, dim=64, ffn=512, vocab=1000)
    gen = torch.Generator().manual_seed(3)
    tokens = torch.randint(1000, (40,), generator=gen).int().cuda()
    ints = dict(dtype=torch.int32, device="cuda")
    whole = example.new_cache(layer, [64])
    logits = layer.step(whole, tokens, torch.zeros(1, **ints), torch.tensor([40], **ints),
                        torch.tensor([0, 40], **ints), 40)
    cache = example.new_cache(layer, [64])
    one = [layer.step(cache, tokens[i:i + 1], torch.tensor([i], **ints), torch.tensor([i + 1], **ints), None, 1)
           for i in range(40)]
    torch.cuda.synchronize()
    assert g.device_status()[0] == 0
    one = torch.cat(one)
    # E4M3 keys and values at two scales: 2^-4 of each value at most, averaged over keys
    scale = logits.std()
    assert (one - logits).abs().max() < 0.5 * scale and (one - logits).std() < 0.05 * scale


def test_serve_runs_and_repeats(example):
    prompts = [[1, 5, 9], list(range(100, 400)), [7], list(range(64))]
    layer = example.Layer()
    token, logprob = example.serve(prompts, 12, layer)
    again, _ = example.serve(prompts, 12, layer)
    torch.cuda.synchronize()
    assert g.device_status()[0] == 0
    assert token.shape == (4, 12) and torch.equal(token, again)
    assert ((token >= 0) & (token < layer.vocab)).all() and torch.isfinite(logprob).all() and (logprob <= 0).all()
    # other numbers, other tokens
    other, _ = example.serve(prompts, 12, layer, seed=2)
    assert not torch.equal(token, other)
