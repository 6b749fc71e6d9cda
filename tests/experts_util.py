"""Helpers of the routed experts' tests: tensors on the GPU in several layouts, and the
same as the oracle's arrays."""
from __future__ import annotations

import numpy as np
import torch

import roofline_driven_optimisation_gb300 as g
from oracle import experts as ox

BF16, F32 = torch.bfloat16, torch.float32


def check_status():
    torch.cuda.synchronize()
    status, where = g.device_status()
    assert status == 0, f"device status {status} at site {where}"


def placed(x, pad=0, offset=0, fill=None):
    """x on the GPU as a view with `pad` columns more a row, `offset` elements behind an
    aligned address; what is around it holds `fill`."""
    rows, cols = x.shape
    flat = torch.zeros(offset + rows * (cols + pad) + 32, dtype=x.dtype)
    if fill is not None:
        (flat.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else flat).fill_(fill)
    view = flat[offset:offset + rows * (cols + pad)].view(rows, cols + pad)
    view[:, :cols] = x
    return flat.cuda()[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


def codes(rng, rows, cols):
    """Random E4M3 codes (no NaN) as uint8."""
    c = rng.integers(0, 256, (rows, cols)).astype(np.uint8)
    c[(c & 0x7F) == 0x7F] = 0x3A
    return c


def fp8(c):
    return torch.from_numpy(np.ascontiguousarray(c)).view(torch.float8_e4m3fn)


class Layer:
    """Experts with random weights; some blocks of weights are 0."""

    def __init__(self, experts, hidden, width, seed=0, pad=0):
        rng = np.random.default_rng(seed)
        self.experts, self.hidden, self.width = experts, hidden, width
        self.values, tensors = [], []
        for k, n in ((hidden, width), (hidden, width), (width, hidden)):
            c = codes(rng, experts * k, n).reshape(experts, k, n)
            s = rng.uniform(0.2, 1.0, (experts, ox.blocks(k), ox.blocks(n))).astype(np.float32) / (100 * np.sqrt(k))
            s = s.astype(np.float32)
            s[rng.random(s.shape) < 0.05] = 0
            self.values.append([ox.dequantise(c[e], s[e], 128) for e in range(experts)])
            wide = torch.zeros(experts, k, n + pad, dtype=torch.uint8)
            wide[:, :, :n] = torch.from_numpy(c)
            tensors += [wide.cuda().view(torch.float8_e4m3fn)[:, :, :n], torch.from_numpy(s).cuda()]
        self.weights = g.ExpertWeights(*tensors)

    def check(self, x, ids, weights, got):
        ref, bound = ox.experts(x.float().cpu().numpy(), ids.cpu().numpy(), weights.cpu().numpy(), *self.values)
        got = got.float().cpu().numpy().astype(np.float64)
        off = np.abs(got - ref)
        assert np.all(off <= bound + 1e-30), \
            f"{(off > bound).sum()} of {off.size} off by up to {np.nanmax(off / (bound + 1e-30)):.2f} bounds"
        return float(np.max(off / (bound + 1e-30))) if off.size else 0.0


def routing(tokens, experts, top_k, seed=0, score=None, logits=None):
    """ids, weights, offsets and order from the library's own router."""
    gen = torch.Generator().manual_seed(seed)
    if logits is None:
        logits = torch.randn(tokens, experts, generator=gen)
    ids = torch.empty(tokens, top_k, dtype=torch.int32, device="cuda")
    w = torch.empty(tokens, top_k, device="cuda")
    offsets = torch.empty(experts + 1, dtype=torch.int32, device="cuda")
    order = torch.empty(tokens * top_k, dtype=torch.int32, device="cuda")
    g.route(logits.cuda(), ids, w, offsets, order, score=g.ROUTE_SOFTMAX if score is None else score)
    return ids, w, offsets, order
