"""gemm_kv_attention gives the same bits on every run, also where items are split over
blocks: which block arrives last, and what else it has to add, is not the same twice."""
import numpy as np
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from serving_util import Case, check_status

pytestmark = pytest.mark.gpu


def ragged(rng, seqs, longest, one=1):
    return [int(n) for n in np.where(rng.random(seqs) < 0.6, rng.integers(0, longest, seqs), rng.choice([0, one, 16], seqs))]


@pytest.mark.parametrize("fmt", [g.KV_E4M3, g.KV_INT8])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,group,new", [(3, 2, 1), (8, 3, 1), (8, 2, 1), (1, 2, 2), (2, 3, 8), (3, 1, 8), (3, 5, 1)])
def test_runs_repeat_bit_for_bit(cuda_lib, fmt, dim, heads, group, new):
    rng = np.random.default_rng(heads * 100 + group * 10 + new)
    for seqs, longest in ((7, 2500), (16, 2500), (30, 18000)):
        lengths = ragged(rng, seqs, longest)
        c = Case(fmt, heads, dim, 32, [0] * seqs, new=max(lengths), seed=seqs)
        if fmt == g.KV_E4M3:                          # no NaN codes among what is read
            for n in ("k", "v"):
                c.np[n][(c.np[n] & 0x7F) == 0x7F] = 0
            c.put()
        lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        gen = torch.Generator(device="cuda").manual_seed(seqs)
        Q = torch.randn(seqs * new, heads * group, dim, generator=gen, device="cuda").bfloat16()
        start = torch.arange(seqs + 1, dtype=torch.int32, device="cuda") * new
        outs = [torch.empty_like(Q) for _ in range(40)]
        for o in outs:
            g.kv_attention(c.cache, Q, o, lens, start=start, max_new=new)
        check_status()
        assert torch.isfinite(outs[0]).all()
        differ = [i for i, o in enumerate(outs) if not torch.equal(o.view(torch.int16), outs[0].view(torch.int16))]
        assert not differ, f"runs {differ} of {len(outs)} differ from the first"
