"""kv_attention without a workspace argument: calls in graphs and outside of them never
share counters, whatever runs first."""
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from serving_util import Case, check_status

pytestmark = pytest.mark.gpu


def case(lengths, seed=0):
    c = Case(g.KV_E4M3, 2, 128, 16, lengths, seed=seed)
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    Q = torch.randn(len(lengths), 8, 128, device="cuda").bfloat16()
    want = g.kv_attention(c.cache, Q, torch.empty_like(Q), lens,
                          workspace=torch.zeros(g.gemm_kv_attention_workspace(len(lengths), 2, 8, 128, 1),
                                                dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    return c, lens, Q, want


def capture(c, lens, Q, stream):
    O = torch.empty_like(Q)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=stream):
        g.kv_attention(c.cache, Q, O, lens)
        g.kv_attention(c.cache, Q, O, lens)
    return gr, O


def run(gr, O, want):
    O.fill_(float("nan"))
    gr.replay()
    check_status()
    assert torch.equal(O, want)


def test_graphs_replay_in_any_order_and_beside_eager_calls(cuda_lib):
    # split over blocks, so that every call counts arrivals
    cases = [case([5000, 40], 1), case([9000], 2), case([3000, 700, 2000], 3)]
    s = torch.cuda.Stream()
    graphs = [capture(*c[:3], s) for c in cases]
    # eager calls on the capture's stream before any replay, then a larger one
    with torch.cuda.stream(s):
        for c, lens, Q, want in cases:
            O = torch.full_like(Q, float("nan"))
            g.kv_attention(c.cache, Q, O, lens)
            check_status()
            assert torch.equal(O, want)
        many = case([33] * 4000, 4)
        O = torch.full_like(many[2], float("nan"))
        g.kv_attention(many[0].cache, many[2], O, many[1])
        check_status()
        assert torch.equal(O, many[3])
    # tensors where a dropped workspace could have been
    other = [torch.full((1 << 22,), i + 1, dtype=torch.int32, device="cuda") for i in range(24)]
    for i in (2, 0, 1, 1, 2, 0):
        run(*graphs[i], cases[i][3])
    assert all((t == i + 1).all() for i, t in enumerate(other))
    # two graphs of one capture stream, side by side on two others
    torch.cuda.synchronize()
    for _ in range(10):
        for i, stream in ((0, torch.cuda.Stream()), (1, torch.cuda.Stream())):
            with torch.cuda.stream(stream):
                graphs[i][0].replay()
        check_status()
        assert torch.equal(graphs[0][1], cases[0][3]) and torch.equal(graphs[1][1], cases[1][3])


def test_a_stream_that_is_not_the_current_one(cuda_lib):
    c, lens, Q, want = case([5000, 40])
    s = torch.cuda.Stream()
    for stream in (s.cuda_stream, 0):
        O = torch.full_like(Q, float("nan"))
        torch.cuda.synchronize()
        g.kv_attention(c.cache, Q, O, lens, stream=stream)
        check_status()
        assert torch.equal(O, want)
    with torch.cuda.stream(s):
        O = torch.full_like(Q, float("nan"))
        s.synchronize()
        g.kv_attention(c.cache, Q, O, lens, stream=0)
        check_status()
        assert torch.equal(O, want)


def test_overlapping_rows_are_refused(cuda_lib):
    c, lens, Q, _ = case([50, 40])
    for q, o in ((Q[:1].expand(2, 8, 128), torch.empty_like(Q)), (Q, torch.empty_like(Q)[:1].expand(2, 8, 128))):
        with pytest.raises(ValueError, match="apart"):
            g.kv_attention(c.cache, q, o, lens)
    with pytest.raises(ValueError, match="apart"):
        g.KVCache(c.views["k"], c.views["v"], c.views["ks"], c.views["vs"], c.table[:1].expand(2, -1))
    l = torch.randn(1, 1000, device="cuda").expand(3, 1000)
    with pytest.raises(ValueError, match="apart"):
        g.sample(l, torch.rand(3, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda"))


def test_after_a_timeout_the_counters_are_zero_again(cuda_lib):
    # counts as a call that gave up leaves them: the status that reports it ends their use
    c, lens, Q, want = case([9000, 40])
    O = torch.empty_like(Q)
    g.kv_attention(c.cache, Q, O, lens)
    check_status()
    for w in g._kv_workspaces.values():
        w.view(torch.int32).fill_(1)
    g.selftest_wait_timeout(2_000_000)
    torch.cuda.synchronize()
    assert g.device_status()[0] == g.GEMM_ERR_DEVICE_TIMEOUT
    for _ in range(2):
        O.fill_(float("nan"))
        g.kv_attention(c.cache, Q, O, lens)
        check_status()
        assert torch.equal(O, want)


def test_counters_past_32_bits(cuda_lib):
    # max_new is a bound, and every tile that it allows has a counter: 2.7 billion here,
    # those of the long sequence's items behind 2^31
    lengths, heads, hq, most = [40, 3, 0, 17, 5000], 32, 256, 1 << 26
    c = Case(g.KV_INT8, heads, 128, 64, lengths)
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    Q = torch.randn(5, hq, 128, device="cuda").bfloat16()
    start = torch.arange(6, dtype=torch.int32, device="cuda")
    want = g.kv_attention(c.cache, Q, torch.empty_like(Q), lens, start=start, max_new=1)
    size = g.gemm_kv_attention_workspace(5, heads, hq, 128, most)
    assert size > 10 * 2 ** 30
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        O = torch.full_like(Q, float("nan"))
        g.kv_attention(c.cache, Q, O, lens, start=start, max_new=most, workspace=ws)
        check_status()
        # other tiles, so another order of sums: each side a bf16 rounding (2^-8) and
        # 2^-10 of its row's size, at most the largest value (127 codes of 0.02), off
        assert ((O.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 2.0 ** -9 * 2.54).all()
    assert (ws[g.gemm_kv_attention_workspace(0, heads, hq, 128, most):].view(torch.int32) == 0).all()
