"""gemm_sample_* where a cut, a bound or a list is at its limit: held, token for token,
to the rule written out in torch with the same whole-number masses."""
import math

import numpy as np
import pytest
import torch

from test_gpu_sample import _rule, call

pytestmark = pytest.mark.gpu


def _logprob(l, token, temperature, top_k, top_p):
    """The token's log-probability among the kept, from the rule in 64 bits."""
    out = []
    for r, x in enumerate(l.double().numpy()):
        z = (x - x.max()) / float(temperature[r])
        order = np.argsort(-x, kind="stable")
        w = np.exp(z[order])
        if top_k[r] > 0:
            w[int(top_k[r]):] = 0
        before = np.cumsum(w) - w
        keep = before < float(top_p[r]) * w.sum()
        keep[0] = True
        out.append(z[token[r]] - math.log(w[keep].sum()))
    return np.array(out)


@pytest.mark.parametrize("rows", [6, 40])
@pytest.mark.parametrize("vocab", [300000, 360448])
def test_top_p_cuts_once_where_the_kept_lie_side_by_side(cuda_lib, vocab, rows):
    # an index bin is ceil(vocab / 512) wide, so that more than 512 kept tokens fit into
    # one: the draw then sorts a list that top-p has cut already
    gen = torch.Generator().manual_seed(vocab)
    l = torch.randn(rows, vocab, generator=gen)
    width = -(-vocab // 512)
    l[:, :width] = 10.0 + torch.rand(rows, width, generator=gen)
    l[rows // 2:, :width] = l[rows // 2:, :width].flip(1)
    u = ((np.arange(rows) + 0.5) / rows).astype(np.float32)
    t, k, p = torch.ones(rows), torch.full((rows,), width + 114), torch.full((rows,), 0.97)
    token, logprob = call(l, u, temperature=t.tolist(), top_k=k.tolist(), top_p=p.tolist())
    assert np.array_equal(token, _rule(l, u, t, k, p, torch.zeros(rows)))
    # the cut falls on a token of about 1/600 of the mass: one token more or less
    assert np.abs(logprob - _logprob(l, token, t, k, p)).max() < 2.5 / 500


@pytest.mark.parametrize("vocab", [16385, 40960, 50257, 65537, 100277])
def test_top_p_alone_where_a_block_has_nothing(cuda_lib, vocab):
    # rows whose last blocks begin behind the vocabulary's end, and rows of which one
    # block's whole part is forbidden; top_p that keeps the first rank only among them
    rows = 12
    gen = torch.Generator().manual_seed(vocab)
    l = 2.5 * torch.randn(rows, vocab, generator=gen)
    l[4:8, :8192 * (vocab // 16385)] = -math.inf
    l[8:, 8192:] = -math.inf
    u = np.random.default_rng(vocab).random(rows).astype(np.float32)
    t, k, m = torch.full((rows,), 0.8), torch.zeros(rows, dtype=torch.int64), torch.zeros(rows)
    for p in (torch.tensor([0.0, -1.0, math.nan, 1e-30]), torch.tensor([0.5, 0.9, 0.999, 0.05])):
        p = p.repeat(rows // 4)
        for top_k in (k, k + 2 * vocab):                      # off, or all of the vocabulary
            token, logprob = call(l, u, temperature=t.tolist(), top_k=top_k.tolist(), top_p=p.tolist())
            assert np.array_equal(token, _rule(l, u, t, k, p, m))
            assert np.isfinite(logprob).all() and (logprob <= 0).all()
            assert (logprob[~(p > 1e-20).numpy()] == 0).all()      # one rank is kept


@pytest.mark.parametrize("vocab", [20000, 40000, 131071])
def test_both_cuts_where_the_lowest_logit_is_shared(cuda_lib, vocab):
    # logits clipped from below, a top-k beyond all that is not forbidden, then top-p: the
    # cut by count ends at the third level of keys, with every equal logit kept, and the
    # cut by mass begins at once with the histogram that the blocks have just read
    rows = 12
    gen = torch.Generator().manual_seed(vocab)
    l = torch.full((rows, vocab), -math.inf)
    at = torch.randperm(vocab, generator=gen)
    l[:, at[:3000]] = 1.0                                       # the lowest, 3000 times
    # the same bin of logits, 2^20 keys and fewer above it
    l[:, at[3000:3400]] = 1.0 + 1e-3 * torch.rand(rows, 400, generator=gen)
    l[:, at[3400:3410]] = 2.0 + 9.0 * torch.rand(rows, 10, generator=gen)
    u = np.random.default_rng(vocab).random(rows).astype(np.float32)
    t, m = torch.tensor([1.0, 3.0, 30.0]).repeat(rows // 3), torch.zeros(rows)
    for k in (3410, 4000, 9000):
        for p in (0.2, 0.9, 0.9999):
            kk, pp = torch.full((rows,), k), torch.full((rows,), p)
            want = _rule(l, u, t, kk, pp, m)
            for _ in range(4):
                token, _ = call(l, u, temperature=t.tolist(), top_k=kk.tolist(), top_p=pp.tolist())
                assert np.array_equal(token, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab", [(5, 3000), (5, 40000), (333, 40000)])
@pytest.mark.parametrize("size", [1e-36, 3e-37, 1e-38, 1e-40])
def test_logits_that_differ_by_next_to_nothing(cuda_lib, dtype, rows, vocab, size):
    # 512 bins over such a range are narrower than fp32's largest number can count
    gen = torch.Generator().manual_seed(vocab)
    l = (size * torch.rand(rows, vocab, generator=gen)).to(dtype)
    u = ((np.arange(rows) + 0.5) / rows).astype(np.float32)
    t, m = torch.ones(rows), torch.zeros(rows)
    for k, p in ((5, 1.0), (64, 0.5), (300, 0.9), (3000, 0.99), (0, 0.001)):
        k, p = torch.full((rows,), k), torch.full((rows,), p)
        token, _ = call(l, u, temperature=t.tolist(), top_k=k.tolist(), top_p=p.tolist())
        assert np.array_equal(token, _rule(l, u, t, k, p, m))


@pytest.mark.parametrize("rows,vocab", [(6, 100), (6, 50257), (333, 40000), (2, 400003)])
def test_settings_that_are_no_numbers_keep_the_first_rank(cuda_lib, rows, vocab):
    gen = torch.Generator().manual_seed(vocab)
    l = torch.randn(rows, vocab, generator=gen).bfloat16()
    u = np.random.default_rng(vocab).random(rows).astype(np.float32)
    nan = [math.nan] * rows
    first = l.float().argmax(1).numpy()
    for kw in (dict(temperature=nan), dict(top_p=nan), dict(min_p=nan), dict(min_p=[1.5] * rows), dict(top_p=[0.0] * rows),
               dict(top_k=[7] * rows, top_p=nan), dict(top_k=[700] * rows, min_p=nan), dict(temperature=nan, top_p=[0.5] * rows)):
        token, logprob = call(l, u, **kw)
        assert np.array_equal(token, first), kw
        assert (logprob == 0).all(), kw
