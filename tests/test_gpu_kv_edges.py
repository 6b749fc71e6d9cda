"""gemm_kv_append and gemm_kv_attention at the ends of what they take."""
import numpy as np
import pytest
import torch

import roofline_driven_optimisation_gb300 as g
from oracle import serving as S
from serving_util import Case, check_status

pytestmark = pytest.mark.gpu


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("new", [1, 2, 9])
def test_positions_up_to_the_last_of_32_bits(cuda_lib, new):
    # without a rotation any position will do; the last page ends at 2^31, and no table
    # reaches it: queries are taken over, keys and values reported
    c = Case(g.KV_INT8, 2, 64, 16, [30])
    before = {n: c.got(n).copy() for n in ("k", "v", "ks", "vs")}
    # a page's worth of rows behind the call's, which it must leave alone
    allQ, allK = torch.randn(new + 16, 3, 64, device="cuda").bfloat16(), torch.randn(new + 16, 2, 64, device="cuda").bfloat16()
    all_out = torch.zeros_like(allQ)
    Q, K, out = allQ[:new], allK[:new], all_out[:new]
    g.kv_append(c.cache, Q, K, K, None, None, ints(2 ** 31 - 1 - new), out, start=ints(0, new), max_new=new)
    torch.cuda.synchronize()
    assert g.device_status() == (g.GEMM_ERR_INVALID_ARG, 60)
    assert torch.equal(out, Q) and (all_out[new:] == 0).all()
    assert all(np.array_equal(before[n], c.got(n)) for n in before)


@pytest.mark.parametrize("length", [2 ** 31 - 16, 2 ** 31 - 19])
def test_contexts_up_to_the_last_position_of_32_bits(cuda_lib, length):
    # 4097 pages under a table of 2^27 - 1 columns; the last column has a page of its own,
    # whose keys have all the weight (scores of 40 and more against 0 of 2^31 others,
    # e^40 > 10^8 * 2^31), and behind the length keys with still more
    cols, P, D = 2 ** 27 - 1, 16, 64
    rng = np.random.default_rng(length)
    table = torch.arange(cols, dtype=torch.int32, device="cuda").remainder_(4096)
    table[-1] = 4096
    k = torch.zeros(4097, 1, P, D, dtype=torch.int8, device="cuda")
    code = 100 + rng.integers(0, 4, P)
    code[length % P or P:] = 127
    k[4096, 0] = torch.from_numpy(code.astype(np.int8)).cuda()[:, None]
    v = torch.randint(-127, 128, (4097, 1, P, D), device="cuda", dtype=torch.int8)
    scale = torch.full((4097, 1), 0.05, device="cuda")
    cache = g.KVCache(k, v, scale, scale, table[None])
    Q = torch.ones(1, 4, D, device="cuda").bfloat16()
    O = g.kv_attention(cache, Q, torch.empty_like(Q), ints(length))
    assert g.last_path() == g.PATH_KV
    check_status()
    n = length % P or P
    s = code[:n] * 0.05 * D / np.sqrt(D)
    p = np.exp(s - s.max())
    x = v[4096, 0, :n].double().cpu().numpy() * float(np.float32(0.05))
    want = (p / p.sum()) @ x
    # the bounds of test_gpu_kv_attention: one rounding to bf16, P in fp16 and the scores
    size = (p / p.sum()) @ np.abs(x)
    off = np.abs(O[0].float().cpu().numpy() - want)
    assert (off <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * size.max() + 1e-6).all()


# new tokens a sequence and the width that is turned: the kernel of a few tokens, the
# kernel of pages, the generic one
KERNELS = [(2, 64), (24, 64), (3, 32)]


@pytest.mark.parametrize("new,turned", KERNELS)
def test_a_sequence_past_the_angles_is_skipped_as_a_whole(cuda_lib, new, turned):
    # the second sequence's last row has no angles: its other rows are not stored either,
    # and its queries are not written; the others are not touched by that
    base, rows = [3, 40, 0], 3 * new
    c = Case(g.KV_INT8, 2, 64, 16, [b + new for b in base])
    start = np.arange(4) * new
    angle = np.random.default_rng(1).normal(size=(40 + new - 1, turned // 2)).astype(np.float32)
    cos, sin = np.cos(angle), np.sin(angle)
    Q, K = torch.randn(rows, 3, 64).bfloat16(), torch.randn(rows, 2, 64).bfloat16()
    out = torch.full((rows, 3, 64), 7.0, device="cuda").bfloat16()
    g.kv_append(c.cache, Q.cuda(), K.cuda(), K.cuda(), torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda(), ints(*base),
                out, start=ints(*start), max_new=new)
    assert (g.last_path() == g.PATH_KV) == (turned == 64)
    torch.cuda.synchronize()
    assert g.device_status() == (g.GEMM_ERR_INVALID_ARG, 60)
    none = np.array([0, new, new, 2 * new])            # the call without that sequence's rows
    keep = np.r_[0:new, 2 * new:rows]
    want = S.append(c.np, g.KV_INT8, *(t.float().numpy()[keep] for t in (Q, K, K)), cos, sin, base, none, False, np.float32)
    for n in ("k", "v", "ks", "vs"):
        assert np.array_equal(c.got(n), c.np[n])
    out = out.float().cpu()
    assert (out[new:2 * new] == 7).all() and torch.equal(out[keep], torch.from_numpy(want).bfloat16().float())


@pytest.mark.parametrize("new,turned", KERNELS)
def test_queries_of_tokens_without_a_page_are_turned(cuda_lib, new, turned):
    # a table that ends before the new tokens do, and a page number that is none
    c = Case(g.KV_INT8, 2, 64, 16, [16])
    before = {n: c.got(n).copy() for n in ("k", "v", "ks", "vs")}
    angle = np.random.default_rng(1).normal(size=(64, turned // 2)).astype(np.float32)
    cos, sin = np.cos(angle), np.sin(angle)
    Q, K = torch.randn(new, 3, 64).bfloat16(), torch.randn(new, 2, 64).bfloat16().cuda()
    for base, page in ((16, None), (0, 99)):
        if page is not None:
            c.table[0, 0] = page
        out = torch.full((new, 3, 64), 7.0, device="cuda").bfloat16()
        g.kv_append(c.cache, Q.cuda(), K, K, torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda(), ints(base), out,
                    start=ints(0, new), max_new=new)
        torch.cuda.synchronize()
        assert g.device_status() == (g.GEMM_ERR_INVALID_ARG, 60)
        pos = base + np.arange(new)
        want = S.rotate(Q.float().numpy(), cos[pos], sin[pos], False, np.float32)
        assert torch.equal(out.float().cpu(), torch.from_numpy(want).bfloat16().float())
        assert all(np.array_equal(before[n], c.got(n)) for n in before)


@pytest.mark.parametrize("fmt", [g.KV_E4M3, g.KV_INT8])
def test_pages_filled_a_token_at_a_time(cuda_lib, fmt):
    # every growth of a scale rounds what the page holds: the same bits as the oracle's
    # after each token, for tokens of growing size
    c = Case(fmt, 2, 128, 16, [0, 5], new=20)
    rng = np.random.default_rng(fmt)
    none = np.zeros((64, 0), np.float32)
    for t in range(20):
        x = torch.from_numpy((rng.normal(size=(2, 2, 128)) * 1.2 ** t).astype(np.float32)).bfloat16()
        g.kv_append(c.cache, None, x.cuda(), x.cuda(), None, None, ints(t, 5 + t))
        S.append(c.np, fmt, None, x.float().numpy(), x.float().numpy(), none, none, [t, 5 + t], [0, 1, 2], False, np.float32)
        check_status()
        for n in ("k", "v", "ks", "vs"):
            assert np.array_equal(c.got(n), c.np[n]), (t, n)


def test_small_query_values_keep_their_bits(cuda_lib):
    # a row's largest value is scaled to 2^14 and more, so a bf16 value 2^31 times smaller
    # ends at fp16's smallest step, 2^-24: all of its weight is there
    c = Case(g.KV_INT8, 1, 64, 16, [40])
    c.np["k"][:, :, :, 0] = 0
    c.np["k"][:, :, :, 1] = c.rng.integers(-127, 128, c.np["k"][:, :, :, 1].shape).astype(np.int8).view(np.uint8)
    c.np["k"][:, :, :, 2:] = 0
    c.np["ks"][:] = 1.0
    c.put()
    for e in (-30, -31):
        Q = torch.zeros(1, 2, 64)
        Q[0, :, 0], Q[0, 0, 1], Q[0, 1, 1] = 1.0, 2.0 ** e * 255 / 128, -2.0 ** e * 129 / 128
        O = torch.empty(1, 2, 64, dtype=torch.bfloat16, device="cuda")
        # scores up to 31: the last of the value's eight bits is a share of 0.2 of a weight
        scale = 2.0 ** (-3 - e)
        g.kv_attention(c.cache, Q.bfloat16().cuda(), O, ints(40), scale=scale)
        check_status()
        want, size = S.attention(c.np, g.KV_INT8, Q.numpy(), [40], [0, 1], scale)
        assert (np.abs(O.float().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * size[..., None]).all()
