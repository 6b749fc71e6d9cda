"""Refusals of the paged-cache and sampling entry points, on the CPU: each bad call
returns its gemm_status and a message before any device access, and empty calls are
no-ops that touch nothing."""
import os
import shutil

import pytest


@pytest.fixture(scope="module")
def g():
    import torch
    if torch.cuda.is_available():
        pytest.skip("runs only where validation is all that can happen")
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from roofline_driven_optimisation_gb300 import _build
    _build.build()
    import roofline_driven_optimisation_gb300 as lib
    lib.load()
    return lib


P = 1 << 20          # an aligned stand-in address (never dereferenced)


def cache(g, **kw):
    f = dict(k=P, v=P, k_scale=P, v_scale=P, table=P, page_stride=4096, head_stride=2048, token_stride=128,
             table_stride=4, format=0, pages=9, page_tokens=16, heads=2, dim=128, seqs=3, table_cols=4)
    f.update(kw)
    return g.KVCacheStruct(**f)


def append(g, c=None, tokens=3, Hq=4, Q=P, ldq=512, K=P, ldk=256, V=P, ldv=256, Qo=P, ldqo=512, cos=P, sin=P,
           positions=64, rotated=128, base=P, start=0, max_new=1):
    g.gemm_kv_append(cache(g) if c is None else c, tokens, Hq, Q, ldq, K, ldk, V, ldv, Qo, ldqo, cos, sin, positions,
                     rotated, 0, base, start or None, max_new, 0)


def attend(g, c=None, tokens=3, Hq=4, Q=P, ldq=512, O=P, ldo=512, lengths=P, start=0, max_new=1, scale=0.0, ws=P,
           size=1 << 40):
    g.gemm_kv_attention(cache(g) if c is None else c, tokens, Hq, Q, ldq, O, ldo, lengths, start or None, max_new, scale,
                        ws, size, 0)


def sample(g, rows=2, vocab=8, logits=P, ld=8, u=P, token=P, f32=True, **kw):
    fn = g.gemm_sample_f32 if f32 else g.gemm_sample_bf16
    fn(rows, vocab, logits, ld, kw.get("temperature"), kw.get("top_k"), kw.get("top_p"), kw.get("min_p"), u, token,
       kw.get("logprob"), 0)


CACHE = [
    (dict(format=2), "INVALID_ARG", "format"), (dict(page_tokens=0), "INVALID_ARG", "cache sizes"),
    (dict(heads=0), "INVALID_ARG", "cache sizes"), (dict(dim=0), "INVALID_ARG", "cache sizes"),
    (dict(pages=-1), "INVALID_ARG", "cache sizes"), (dict(seqs=-1), "INVALID_ARG", "cache sizes"),
    (dict(dim=513), "UNSUPPORTED", "512"), (dict(token_stride=127), "INVALID_ARG", "strides"),
    (dict(page_stride=-1), "INVALID_ARG", "strides"), (dict(table_stride=3), "INVALID_ARG", "strides"),
    (dict(table_cols=1 << 28, table_stride=1 << 28), "UNSUPPORTED", "positions"),
    (dict(k=0), "INVALID_ARG", "NULL"), (dict(v_scale=0), "INVALID_ARG", "NULL"), (dict(table=0), "INVALID_ARG", "NULL"),
    (dict(k_scale=P + 2), "MISALIGNED", "4 bytes"), (dict(table=P + 1), "MISALIGNED", "4 bytes"),
]


@pytest.mark.parametrize("call", [append, attend])
@pytest.mark.parametrize("bad,status,text", CACHE)
def test_bad_caches(g, call, bad, status, text):
    with pytest.raises(g.GemmError) as e:
        call(g, cache(g, **bad))
    assert e.value.code == getattr(g, "GEMM_ERR_" + status) and text in str(e.value)


CALLS = [
    (append, dict(tokens=-1), "INVALID_ARG", "negative"), (append, dict(tokens=4), "INVALID_ARG", "without start"),
    (append, dict(start=P, max_new=0), "INVALID_ARG", "at most 0"), (append, dict(start=P + 2), "MISALIGNED", "start"),
    (append, dict(rotated=3), "INVALID_ARG", "rotated"), (append, dict(rotated=130), "INVALID_ARG", "rotated"),
    (append, dict(positions=-1), "INVALID_ARG", "negative"), (append, dict(Hq=65535, ldq=1 << 24, ldqo=1 << 24),
                                                              "UNSUPPORTED", "65535"),
    (append, dict(ldk=255), "INVALID_ARG", "leading"), (append, dict(ldqo=511), "INVALID_ARG", "leading"),
    (append, dict(K=0), "INVALID_ARG", "NULL"), (append, dict(Qo=0), "INVALID_ARG", "NULL"),
    (append, dict(base=0), "INVALID_ARG", "NULL"), (append, dict(sin=0), "INVALID_ARG", "cos or sin"),
    (append, dict(V=P + 1), "MISALIGNED", "element size"), (append, dict(cos=P + 2), "MISALIGNED", "element size"),
    (attend, dict(tokens=-2), "INVALID_ARG", "negative"), (attend, dict(Hq=3), "INVALID_ARG", "multiple"),
    (attend, dict(Hq=65536, ldq=1 << 24, ldo=1 << 24), "UNSUPPORTED", "65535"),
    (attend, dict(scale=-1.0), "INVALID_ARG", "scale"), (attend, dict(scale=float("nan")), "INVALID_ARG", "scale"),
    (attend, dict(ldo=500), "INVALID_ARG", "leading"), (attend, dict(O=0), "INVALID_ARG", "NULL"),
    (attend, dict(lengths=0), "INVALID_ARG", "NULL"), (attend, dict(Q=P + 1), "MISALIGNED", "element size"),
    (attend, dict(ws=0), "INVALID_ARG", "workspace"), (attend, dict(size=8), "INVALID_ARG", "workspace"),
    (attend, dict(ws=P + 8), "MISALIGNED", "16 bytes"),
    (sample, dict(rows=-1), "INVALID_ARG", "negative"), (sample, dict(vocab=0), "INVALID_ARG", "empty"),
    (sample, dict(vocab=(1 << 20) + 1, ld=1 << 21), "UNSUPPORTED", "vocab"), (sample, dict(ld=7), "INVALID_ARG", "leading"),
    (sample, dict(u=0), "INVALID_ARG", "NULL"), (sample, dict(token=0), "INVALID_ARG", "NULL"),
    (sample, dict(logits=P + 2), "MISALIGNED", "element size"), (sample, dict(top_p=P + 2), "MISALIGNED", "element size"),
    (sample, dict(f32=False, logits=P + 1), "MISALIGNED", "element size"),
]


@pytest.mark.parametrize("call,bad,status,text", CALLS)
def test_bad_arguments(g, call, bad, status, text):
    with pytest.raises(g.GemmError) as e:
        call(g, **bad)
    assert e.value.code == getattr(g, "GEMM_ERR_" + status), str(e.value)
    assert text in str(e.value)


def test_empty_calls_are_no_ops(g):
    none = dict(k=0, v=0, k_scale=0, v_scale=0, table=0, seqs=0, pages=0)
    append(g, cache(g, **none), tokens=0, Q=0, K=0, V=0, Qo=0, base=0)
    attend(g, cache(g, **none), tokens=0, Q=0, O=0, lengths=0, ws=0, size=0)
    sample(g, rows=0, logits=0, u=0, token=0)


def test_real_calls_need_a_device(g):
    for call in (append, attend, sample):
        with pytest.raises(g.GemmError) as e:
            call(g)
        assert e.value.code in (g.GEMM_ERR_CUDA, g.GEMM_ERR_UNSUPPORTED)


def test_workspace_size(g):
    assert g.gemm_kv_attention_workspace(4, 8, 32, 128, 1) >= 16
    for bad in ((-1, 8, 32, 128, 1), (4, 0, 32, 128, 1), (4, 8, 31, 128, 1), (4, 8, 32, 0, 1), (4, 8, 32, 128, -1)):
        assert g.gemm_kv_attention_workspace(*bad) == 0


def test_binding_refuses_tensors_that_do_not_fit(g):
    import torch
    with pytest.raises(TypeError):
        g.KVCache(torch.zeros(2, 2, 2), torch.zeros(2, 2, 2), None, None, None)
    k = torch.zeros(2, 2, 16, 64, dtype=torch.int8)
    s, t = torch.zeros(2, 2), torch.zeros(1, 1, dtype=torch.int32)
    for args, error in (((k, k.view(torch.uint8), s, s, t), TypeError), ((k, k[:1], s, s, t), ValueError),
                        ((k, k, s[:1], s, t), TypeError), ((k, k, s, s, t.long()), TypeError),
                        ((k, k, s, s, t, g.KV_E4M3), TypeError), ((k, k, s, s, t), ValueError)):
        with pytest.raises(error):
            g.KVCache(*args)
    with pytest.raises(ValueError):
        g.sample(torch.zeros(1, 4), torch.zeros(1), torch.zeros(1, dtype=torch.int32))
