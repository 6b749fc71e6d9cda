"""gemm_sample_* against the 64-bit oracle.

Weights are fp32 exponentials (relative error 2^-21 at most, the argument's two
roundings included for the sizes used here) cut to 2^-40, so every share of mass that
a decision compares is within SHARE of the exact one; where the oracle's nearest
decision is closer than that the row has no one right answer and is not compared.
Where the masses are the same on both sides -- the rule written out in torch, with
torch's exponential -- tokens must be equal without exception."""
import math

import numpy as np
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from oracle import serving as S
from serving_util import check_status

pytestmark = pytest.mark.gpu
SHARE = 2.0 ** -20 + 2.0 ** -22          # 2^18 tokens of 2^-40 each, and the exponentials
LOGPROB = 2.0 ** -19                      # of z below 2^5 and the logarithm, in fp32


def call(logits, u, ld=None, **kw):
    rows, vocab = logits.shape
    x = logits
    if ld is not None:
        wide = torch.full((rows, ld), float("inf"), dtype=logits.dtype)      # never read
        wide[:, :vocab] = logits
        x = wide.cuda()[:, :vocab]
    else:
        x = x.cuda()
    dev = {k: None if v is None else torch.tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32, device="cuda")
           for k, v in kw.items()}
    token = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    logprob = torch.full((rows,), float("nan"), device="cuda")
    u = torch.as_tensor(u, dtype=torch.float32).cuda()
    g.sample(x, u, token, logprob, **dev)
    assert g.last_path() == g.PATH_SAMPLE
    check_status()
    return token.cpu().numpy(), logprob.cpu().numpy()


def compare(logits, u, least=0.9, **kw):
    token, logprob = call(logits, u, **kw)
    kw.pop("ld", None)
    x = logits.float().numpy()
    clear = 0
    for r in range(len(x)):
        setting = {k: v[r] for k, v in kw.items() if v is not None}
        exact = {k: float(np.float32(v)) if k != "top_k" else v for k, v in setting.items()}
        want, lp, margin, doubt = S.sample(x[r], float(np.float32(u[r])), share=SHARE, **exact)
        if margin <= SHARE:
            continue
        clear += 1
        assert token[r] == want, (r, setting, token[r], want, margin)
        assert abs(logprob[r] - lp) <= LOGPROB * max(1.0, abs(lp)) + 2 * doubt
    assert clear >= least * len(x)
    return token


def make(rows, vocab, dtype, seed, spread=2.5):
    gen = torch.Generator().manual_seed(seed)
    l = spread * torch.randn(rows, vocab, generator=gen)
    l.scatter_add_(1, torch.randint(vocab, (rows, min(20, vocab)), generator=gen),
                   9 * torch.rand(rows, min(20, vocab), generator=gen))
    return l.to(dtype), np.random.default_rng(seed).random(rows).astype(np.float32)


SETTINGS = {
    "plain": {}, "temperature": dict(temperature=0.7), "hot": dict(temperature=30.0), "cold": dict(temperature=0.02),
    "top_k": dict(top_k=40), "top_p": dict(top_p=0.9), "min_p": dict(min_p=0.05),
    "all": dict(temperature=0.8, top_k=50, top_p=0.95, min_p=0.03), "wide_p": dict(top_p=0.9999),
    "narrow_p": dict(top_p=1e-6), "k1": dict(top_k=1), "k_all": dict(top_k=10 ** 6, top_p=0.5),
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", sorted(SETTINGS))
@pytest.mark.parametrize("vocab", [1, 2, 33, 1000, 32000])
def test_rules(cuda_lib, dtype, name, vocab):
    rows = 6
    l, u = make(rows, vocab, dtype, vocab + len(name))
    # a wide-open draw has thousands of boundaries; most are still clear
    compare(l, u, least=0.3, **{k: [v] * rows for k, v in SETTINGS[name].items()})


@pytest.mark.parametrize("vocab", [32768, 32769, 65537, 131071, 262144])
def test_large_vocabularies(cuda_lib, vocab):
    l, u = make(3, vocab, torch.float32, vocab)
    compare(l, u, least=0.3, temperature=[0.8, 1.0, 0.3], top_k=[50, 0, 2000], top_p=[0.95, 0.5, 1.0],
            min_p=[0.0, 0.1, 0.01])


def test_each_row_has_its_settings(cuda_lib):
    l, u = make(64, 5000, torch.bfloat16, 5)
    rng = np.random.default_rng(5)
    compare(l, u, least=0.8, temperature=rng.choice([0.0, 0.3, 1.0, 1.7], 64).tolist(),
            top_k=rng.choice([0, 1, 5, 100], 64).tolist(), top_p=rng.choice([0.1, 0.9, 1.0], 64).tolist(),
            min_p=rng.choice([0.0, 0.1], 64).tolist())


def _rule(l, u, temperature, top_k, top_p, min_p):
    """The header's rule in torch on the GPU, with the same whole-number masses."""
    l, u = l.cuda().float(), torch.as_tensor(u).cuda()
    vocab = l.shape[1]
    w = torch.exp((l - l.amax(1, keepdim=True)) * (1 / temperature.cuda())[:, None])
    mass = (w * 2.0 ** 40).long()
    order = torch.sort(l, dim=1, descending=True, stable=True).indices
    m, rank = mass.gather(1, order), torch.arange(vocab, device="cuda")
    k = torch.where(top_k > 0, top_k, vocab).cuda()
    m = m * (rank < k[:, None])
    before = torch.cumsum(m, 1) - m
    m = m * ((before.double() < (top_p.cuda().double() * m.sum(1).double())[:, None]) | (rank == 0))
    m = m * ((w.gather(1, order) >= min_p.cuda()[:, None]) | (rank == 0))
    run = torch.cumsum(torch.zeros_like(m).scatter_(1, order, m), 1)
    target = torch.minimum((u.double() * run[:, -1].double()).long(), run[:, -1] - 1)
    return (run <= target[:, None]).sum(1).int().cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [17, 4099, 32000, 100003])
def test_tokens_equal_the_written_rule(cuda_lib, dtype, vocab):
    rows = 192
    l, u = make(rows, vocab, dtype, vocab, spread=1.5)
    l[::7, ::3] = -math.inf
    gen = torch.Generator().manual_seed(1)

    def of(*v):
        return torch.tensor(v)[torch.randint(len(v), (rows,), generator=gen)]
    t, k, p, m = of(0.3, 0.8, 1.0, 2.0, 9.0), of(0, 0, 7, 50, 3000), of(1.0, 0.99, 0.8, 0.3), of(0.0, 0.0, 0.01, 0.2)
    token, _ = call(l, u, temperature=t.tolist(), top_k=k.tolist(), top_p=p.tolist(), min_p=m.tolist())
    assert np.array_equal(token, _rule(l, u, t, k, p, m))


def test_ties_go_to_the_lowest_index(cuda_lib):
    # every logit equal, then two values: cuts fall inside a run of equal ones
    for vocab in (100, 32000, 70000):
        l = torch.zeros(8, vocab)
        u = np.array([0.0, 0.1, 0.3, 0.5, 0.7, 0.9, 0.99, 0.999], np.float32)
        token, _ = call(l, u, top_k=[10] * 8)
        assert token.tolist() == [int(x * 10) for x in u.astype(np.float64)]
        token, _ = call(l, u, top_p=[0.25] * 8)
        assert (token == np.floor(u.astype(np.float64) * (vocab // 4))).all()
        l[:, vocab // 2:] = 1.0
        token, _ = call(l, u, top_k=[7] * 8)
        assert token.tolist() == [vocab // 2 + int(x * 7) for x in u.astype(np.float64)]
    l = torch.tensor([[1.0, 3.0, 3.0, 2.0]])
    assert call(l, [0.99], temperature=[0.0])[0][0] == 1 and call(l, [0.99], top_k=[1])[0][0] == 1
    zeros = torch.tensor([[-0.0, 0.0, -0.0, 0.0]])
    assert call(zeros, [0.99], top_k=[2])[0][0] == 1


def test_infinities_nan_and_empty_rows(cuda_lib):
    inf, nan = math.inf, math.nan
    l = torch.tensor([[-inf, -inf, -inf, -inf], [nan, nan, -inf, nan], [-inf, 2.0, -inf, nan], [1.0, inf, 3.0, inf],
                      [nan, 0.0, 0.0, -3e38], [-3e38, -3e38, -inf, -inf]])
    u = np.full(6, 0.6, np.float32)
    for kw in ({}, dict(top_p=[0.999] * 6), dict(top_k=[3] * 6), dict(temperature=[1e30] * 6),
               dict(temperature=[math.inf] * 6), dict(min_p=[0.5] * 6)):
        token, logprob = call(l, u, **kw)
        assert token[:2].tolist() == [-1, -1] and (logprob[:2] == -inf).all()
        assert token[2] == 1 and logprob[2] == 0.0
        assert token[3] == 3 and abs(logprob[3] + math.log(2)) < 1e-6
        assert token[5] == 1
        if "temperature" not in kw:
            assert token[4] == 2
    for t in (0.0, -1.0, nan, 1e-45):                      # greedy
        token, logprob = call(l, u, temperature=[t] * 6)
        assert token.tolist() == [-1, -1, 1, 1, 1, 0] and (logprob[2:] == 0).all()


def test_given_numbers_at_their_ends(cuda_lib):
    l = torch.log(torch.tensor([[0.25, 0.5, 0.25]] * 7))
    token, _ = call(l, np.array([0.0, 1.0, 1.5, -1.0, math.nan, math.inf, 1 - 2.0 ** -24], np.float32))
    assert token.tolist() == [0, 2, 2, 0, 0, 2, 2]


def test_parameters_at_their_ends(cuda_lib):
    l = torch.log(torch.tensor([[0.2, 0.5, 0.3]] * 4))
    u = np.full(4, 0.99, np.float32)
    assert call(l, u, top_p=[0.0, -1.0, math.nan, 2.0])[0].tolist() == [1, 1, 1, 2]
    assert call(l, u, min_p=[2.0, 0.55, -1.0, math.nan])[0][:3].tolist() == [1, 2, 2]
    assert call(l, u, top_k=[-5, 1, 2, 99])[0].tolist() == [2, 1, 2, 2]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab,ld", [(1000, 1001), (32000, 32007), (777, 1024), (70001, 70003)])
def test_row_strides(cuda_lib, dtype, vocab, ld):
    l, u = make(5, vocab, dtype, ld)
    compare(l, u, ld=ld, least=0.5, temperature=[0.6] * 5, top_k=[30] * 5, top_p=[0.9] * 5)


def test_draws_follow_the_distribution(cuda_lib):
    # a fine ladder of u walks through the kept tokens in shares of their mass
    l, _ = make(1, 3001, torch.float32, 9)
    n = 2048
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    token, logprob = call(l.expand(n, -1).contiguous(), u, top_k=[6] * n)
    assert (np.diff(token) >= 0).all()
    ids, count = np.unique(token, return_counts=True)
    assert set(ids) == set(np.argsort(-l[0].numpy())[:6])
    for i, c in zip(ids, count):
        assert abs(c / n - math.exp(logprob[token == i][0])) <= 2 / n
        assert len(set(logprob[token == i])) == 1


def test_without_logprob_and_in_a_graph(cuda_lib):
    l, u = make(4, 32000, torch.bfloat16, 3)
    x, v = l.cuda(), torch.from_numpy(u).cuda()
    token, lp = torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty(4, device="cuda")
    g.sample(x, v, token)
    want = g.sample(x, v, torch.empty_like(token), lp).clone()
    assert torch.equal(token, want)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        g.sample(x, v, token, lp)
    x.copy_(make(4, 32000, torch.bfloat16, 4)[0])
    gr.replay()
    check_status()
    assert torch.equal(token, g.sample(x, v, torch.empty_like(token)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab,ld", [(8000, None), (16384, None), (40000, 40003), (40004, 40008), (131071, None)])
def test_many_long_rows(cuda_lib, dtype, vocab, ld):
    # a row for each SM and more: rows with few ranks stream through one block each, the
    # others and those that do not suit it go to a second kernel
    rows = 333
    gen = torch.Generator().manual_seed(vocab)
    l = 2.5 * torch.randn(rows, vocab, generator=gen)
    l.masked_fill_(torch.rand(rows, vocab, generator=gen) < 0.01, -math.inf)
    l[1] = l[1].sort().values                       # ascending: every tile beats the ones before
    l[2] = 0.5                                      # all equal
    l[3, :20000] = -math.inf                        # the first tile has nothing (the shortest: the row)
    l[4] = -math.inf
    l[4, vocab - 1] = 1.0
    l[5, :9000] -= 50.0
    l[6] = torch.arange(vocab) / vocab
    l[7] = -torch.arange(vocab) / vocab
    l = l.to(dtype)
    u = np.random.default_rng(vocab).random(rows).astype(np.float32)

    def of(*v):
        x = torch.tensor(v)[torch.randint(len(v), (rows,), generator=gen)]
        x[1:8] = v[-1]
        return x
    t, k, p, m = of(0.3, 2.0, 0.8), of(0, 1, 3, 64, 65, 900, 50), of(1.0, 0.5, 0.95), of(0.0, 0.2, 0.01)
    token, logprob = call(l, u, ld=ld, temperature=t.tolist(), top_k=k.tolist(), top_p=p.tolist(), min_p=m.tolist())
    some = (l > -math.inf).any(1).numpy()           # row 3 of short ones has none
    assert np.array_equal(token, np.where(some, _rule(l, u, t, k, p, m), -1))
    assert np.isfinite(logprob[some]).all() and (logprob <= 0).all() and (logprob[~some] == -math.inf).all()
    greedy, lp = call(l, u, ld=ld, temperature=[0.0] * rows)
    assert np.array_equal(greedy, np.where(some, l.float().argmax(1).numpy(), -1)) and (lp[some] == 0).all()
    l[0] = math.nan
    none, lp = call(l[:1].expand(rows, -1).contiguous(), u, top_k=[5] * rows)
    assert (none == -1).all() and (lp == -math.inf).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab", [(41, 131071), (76, 65536), (100, 40001), (152, 32000), (17, 260001), (304, 32001)])
@pytest.mark.parametrize("first", [0, 1, 3])
def test_rows_over_several_blocks(cuda_lib, dtype, rows, vocab, first):
    # fewer long rows: each is streamed by one, two or four blocks; rows begin at any
    # element, with what must not be read on either side
    gen = torch.Generator().manual_seed(vocab + first)
    l = 2.5 * torch.randn(rows, vocab, generator=gen)
    l[1] = l[1].sort().values
    l[2] = 0.5
    l[3, :vocab - 7] = -math.inf
    l[4] = -math.inf
    l[5] = l[5].sort(descending=True).values
    l[6, vocab // 2:] = math.nan
    l[7, 8192 * 3:] += 40.0                          # a later block's part has all
    l[8] = -math.inf
    l[8, 0] = l[8, vocab - 1] = -3.0
    l[9, 20:] = -math.inf
    l = l.to(dtype)
    wide = torch.full((rows, vocab + 6), math.inf, dtype=dtype)
    wide[:, first:first + vocab] = l
    x = wide.cuda()[:, first:first + vocab]
    u = np.random.default_rng(vocab).random(rows).astype(np.float32)
    some = (l > -math.inf).any(1).numpy()
    clean = torch.where(l.isnan(), -math.inf, l.float()).to(dtype)
    for k in (1, 7, 64):
        t, kk, p, m = torch.full((rows,), 0.8), torch.full((rows,), k), torch.full((rows,), 0.95), torch.full((rows,), 0.01)
        token = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
        logprob = torch.full((rows,), math.nan, device="cuda")
        g.sample(x, torch.as_tensor(u).cuda(), token, logprob, temperature=t.cuda(), top_k=kk.int().cuda(), top_p=p.cuda(),
                 min_p=m.cuda())
        check_status()
        assert np.array_equal(token.cpu().numpy(), np.where(some, _rule(clean, u, t, kk, p, m), -1))
        assert (logprob.cpu().numpy()[some] <= 0).all() and (logprob.cpu().numpy()[~some] == -math.inf).all()


def test_offsets_past_32_bits(cuda_lib):
    # rows that begin 2^31 elements into a tensor and later
    rows, vocab, ld = 17500, 1000, 131071
    wide = torch.zeros(rows * ld, dtype=torch.bfloat16, device="cuda")
    x = wide.as_strided((rows, vocab), (ld, 1))
    gen = torch.Generator().manual_seed(1)
    last, u = make(40, vocab, torch.bfloat16, 5)
    x[-40:] = last.cuda()
    for k in (1, 20, 0):
        token = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
        kk = torch.full((rows,), k, dtype=torch.int32)
        p = torch.full((rows,), 0.9)
        uu = torch.rand(rows, generator=gen)
        uu[-40:] = torch.as_tensor(u)
        g.sample(x, uu.cuda(), token, top_k=kk.cuda(), top_p=p.cuda())
        check_status()
        want = _rule(last, u, torch.ones(40), kk[-40:], p[-40:], torch.zeros(40))
        assert np.array_equal(token[-40:].cpu().numpy(), want)
    del wide, x
    full = torch.zeros(8300, 1 << 18, dtype=torch.bfloat16, device="cuda")       # 2^31, in rows that stream
    at = torch.randint(1 << 18, (8300,), generator=gen).cuda()
    full.scatter_(1, at[:, None], 5.0)
    kk = torch.full((8300,), 1, dtype=torch.int32)
    token = g.sample(full, torch.rand(8300, generator=gen).cuda(), torch.full((8300,), -7, dtype=torch.int32, device="cuda"),
                     top_k=kk.cuda())
    check_status()
    assert torch.equal(token.long(), at)


@pytest.mark.parametrize("vocab", [400003, 1 << 20])
def test_largest_vocabularies(cuda_lib, vocab):
    # longer than a cluster's shared memory holds
    rows = 5
    l, u = make(rows, vocab, torch.bfloat16, vocab)
    t, k = torch.tensor([0.8, 1.0, 0.5, 1.0, 2.0]), torch.tensor([50, 0, 0, 1000, 7])
    p, m = torch.tensor([0.95, 1.0, 0.7, 0.9, 1.0]), torch.tensor([0.0, 0.1, 0.0, 0.0, 0.0])
    token, _ = call(l, u, temperature=t.tolist(), top_k=k.tolist(), top_p=p.tolist(), min_p=m.tolist())
    assert np.array_equal(token, _rule(l, u, t, k, p, m))


@pytest.mark.parametrize("vocab", [5000, 32000, 131071])
def test_crowded_bins(cuda_lib, vocab):
    # runs of equal and of nearly equal logits where the cuts and the draw fall
    rows = 64
    gen = torch.Generator().manual_seed(vocab)
    l = torch.randn(rows, vocab, generator=gen)
    at = torch.randperm(vocab, generator=gen)
    l[:16, at[:1500]] = 6.0                                   # equal, anywhere
    l[16:32, :1500] = 6.0                                     # equal, side by side
    l[32:40, at[:2000]] = 6.0 + 1e-6 * torch.rand(8, 2000, generator=gen)
    l[40:48] = torch.round(l[40:48])                          # a few values in all
    l[48:52] = 1.0
    l[52:, :3] += 30.0                                        # a few far above
    u = np.random.default_rng(vocab).random(rows).astype(np.float32)

    def of(*v):
        return torch.tensor(v)[torch.arange(rows) % len(v)]
    for t, k, p in ((of(1.0, 0.7), of(1000, 700, 300), of(1.0, 0.9, 0.5, 0.99, 0.2)),
                    (of(1.0, 3.0, 0.2), of(0), of(0.9, 0.5, 0.99, 0.05)), (of(1.0), of(50, 64, 3000), of(0.97, 0.5, 1.0, 0.1))):
        m = of(0.0, 0.0, 0.3)
        token, _ = call(l, u, temperature=t.tolist(), top_k=k.tolist(), top_p=p.tolist(), min_p=m.tolist())
        assert np.array_equal(token, _rule(l, u, t, k, p, m))
