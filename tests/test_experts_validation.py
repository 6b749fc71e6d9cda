"""Refusals of the routing, quantisation, block-scaled product and experts entry points, on
the CPU: each bad call returns its gemm_status and a message before any device access, and
empty calls are no-ops that touch nothing."""
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


def route(g, tokens=3, experts=8, top_k=2, logits=P, ld=8, bias=P, score=0, groups=1, top_groups=1, group_best=2,
          scale=1.0, ids=P, weights=P, offsets=P, order=P, ws=P, size=1 << 30, f32=True):
    fn = g.gemm_route_f32 if f32 else g.gemm_route_bf16
    fn(tokens, experts, top_k, logits, ld, bias, score, groups, top_groups, group_best, 1, scale, ids, weights,
       offsets or None, order or None, ws, size, 0)


def quantise(g, rows=3, cols=200, X=P, ldx=200, codes=P, ldq=200, scales=P, lds=2, block_rows=1, f32=True):
    fn = g.gemm_fp8_quantise_f32 if f32 else g.gemm_fp8_quantise_bf16
    fn(rows, cols, X, ldx, codes, ldq, scales, lds, block_rows, 0)


def blocks(g, M=3, N=200, K=300, A=P, lda=304, a_scale=P, ldsa=3, B=P, ldb=208, b_scale=P, ldsb=2, C=P, ldc=200,
           f32=True):
    fn = g.gemm_fp8_blocks_f32out if f32 else g.gemm_fp8_blocks
    fn(M, N, K, 1.0, A, lda, a_scale, ldsa, B, ldb, b_scale, ldsb, 0.0, C, ldc, 0)


def experts(g, w=None, tokens=3, top_k=2, X=P, ldx=64, offsets=P, order=P, weights=P, O=P, ldo=64, ws=P, size=1 << 40,
            **kw):
    f = dict(gate=P, up=P, down=P, gate_scale=P, up_scale=P, down_scale=P, ld_up=32, stride_up=2048, ld_down=64,
             stride_down=2048, experts=4, hidden=64, width=32)
    f.update(kw)
    g.gemm_experts(g.ExpertWeightsStruct(**f), tokens, top_k, X, ldx, offsets, order, weights, O, ldo, ws, size, 0)


CALLS = [
    (route, dict(tokens=-1), "INVALID_ARG", "bad sizes"), (route, dict(experts=0), "INVALID_ARG", "bad sizes"),
    (route, dict(top_k=0), "INVALID_ARG", "bad sizes"), (route, dict(top_k=9), "INVALID_ARG", "kept groups"),
    (route, dict(experts=1025, ld=2000), "UNSUPPORTED", "1024"), (route, dict(top_k=33, experts=64, ld=64), "UNSUPPORTED", "32"),
    (route, dict(score=2), "INVALID_ARG", "score"), (route, dict(score=-1), "INVALID_ARG", "score"),
    (route, dict(groups=3), "INVALID_ARG", "groups"), (route, dict(groups=0), "INVALID_ARG", "groups"),
    (route, dict(groups=2, top_groups=3), "INVALID_ARG", "kept"), (route, dict(groups=2, top_groups=0), "INVALID_ARG", "kept"),
    (route, dict(experts=66, ld=66, groups=33, top_groups=2), "UNSUPPORTED", "32"),
    (route, dict(groups=4, top_groups=1, top_k=3), "INVALID_ARG", "kept groups"),
    (route, dict(group_best=0), "INVALID_ARG", "1 or 2"), (route, dict(group_best=3), "INVALID_ARG", "1 or 2"),
    (route, dict(scale=float("nan")), "INVALID_ARG", "scale"), (route, dict(scale=float("inf")), "INVALID_ARG", "scale"),
    (route, dict(ld=7), "INVALID_ARG", "leading"), (route, dict(offsets=0), "INVALID_ARG", "together"),
    (route, dict(order=0), "INVALID_ARG", "together"), (route, dict(tokens=1 << 30), "UNSUPPORTED", "2^31"),
    (route, dict(logits=0), "INVALID_ARG", "NULL"), (route, dict(ids=0), "INVALID_ARG", "NULL"),
    (route, dict(weights=0), "INVALID_ARG", "NULL"), (route, dict(logits=P + 2), "MISALIGNED", "element size"),
    (route, dict(logits=P + 1, f32=False), "MISALIGNED", "element size"),
    (route, dict(bias=P + 2), "MISALIGNED", "element size"), (route, dict(ids=P + 1), "MISALIGNED", "element size"),
    (route, dict(tokens=300, ws=0), "INVALID_ARG", "workspace"), (route, dict(tokens=300, size=8), "INVALID_ARG", "workspace"),
    (route, dict(tokens=300, ws=P + 8), "MISALIGNED", "16 bytes"),
    (quantise, dict(rows=-1), "INVALID_ARG", "negative"), (quantise, dict(cols=-1), "INVALID_ARG", "negative"),
    (quantise, dict(block_rows=64), "INVALID_ARG", "128"), (quantise, dict(block_rows=0), "INVALID_ARG", "128"),
    (quantise, dict(ldx=199), "INVALID_ARG", "leading"), (quantise, dict(ldq=199), "INVALID_ARG", "leading"),
    (quantise, dict(lds=1), "INVALID_ARG", "leading"), (quantise, dict(X=0), "INVALID_ARG", "NULL"),
    (quantise, dict(codes=0), "INVALID_ARG", "NULL"), (quantise, dict(scales=0), "INVALID_ARG", "NULL"),
    (quantise, dict(X=P + 2), "MISALIGNED", "element size"), (quantise, dict(X=P + 1, f32=False), "MISALIGNED", "element size"),
    (quantise, dict(scales=P + 2), "MISALIGNED", "element size"),
    (blocks, dict(M=-1), "INVALID_ARG", "negative"), (blocks, dict(N=-1), "INVALID_ARG", "negative"),
    (blocks, dict(K=-1), "INVALID_ARG", "negative"), (blocks, dict(lda=299), "INVALID_ARG", "leading"),
    (blocks, dict(ldb=199), "INVALID_ARG", "leading"), (blocks, dict(ldc=199), "INVALID_ARG", "leading"),
    (blocks, dict(ldsa=2), "INVALID_ARG", "leading"), (blocks, dict(ldsb=1), "INVALID_ARG", "leading"),
    (blocks, dict(C=0), "INVALID_ARG", "NULL"), (blocks, dict(A=0), "INVALID_ARG", "NULL"),
    (blocks, dict(B=0), "INVALID_ARG", "NULL"), (blocks, dict(a_scale=0), "INVALID_ARG", "NULL"),
    (blocks, dict(b_scale=0), "INVALID_ARG", "NULL"), (blocks, dict(C=P + 2), "MISALIGNED", "element size"),
    (blocks, dict(C=P + 1, f32=False), "MISALIGNED", "element size"), (blocks, dict(b_scale=P + 2), "MISALIGNED", "element size"),
    (experts, dict(tokens=-1), "INVALID_ARG", "bad sizes"), (experts, dict(top_k=0), "INVALID_ARG", "bad sizes"),
    (experts, dict(experts=0), "INVALID_ARG", "bad sizes"), (experts, dict(hidden=0), "INVALID_ARG", "bad sizes"),
    (experts, dict(width=0), "INVALID_ARG", "bad sizes"), (experts, dict(experts=1025), "UNSUPPORTED", "1024"),
    (experts, dict(tokens=1 << 30), "UNSUPPORTED", "2^31"),
    (experts, dict(hidden=1 << 27, ldx=1 << 28, ldo=1 << 28, ld_down=1 << 28), "UNSUPPORTED", "hidden"),
    (experts, dict(ld_up=1 << 40), "UNSUPPORTED", "leading"), (experts, dict(ld_down=1 << 40), "UNSUPPORTED", "leading"),
    (experts, dict(ld_up=31), "INVALID_ARG", "leading"), (experts, dict(ld_down=63), "INVALID_ARG", "leading"),
    (experts, dict(ldx=63), "INVALID_ARG", "leading"), (experts, dict(ldo=63), "INVALID_ARG", "leading"),
    (experts, dict(stride_up=-1), "INVALID_ARG", "leading"), (experts, dict(stride_up=2047), "INVALID_ARG", "overlap"),
    (experts, dict(stride_down=2047), "INVALID_ARG", "overlap"), (experts, dict(gate=0), "INVALID_ARG", "NULL"),
    (experts, dict(down_scale=0), "INVALID_ARG", "NULL"), (experts, dict(X=0), "INVALID_ARG", "NULL"),
    (experts, dict(O=0), "INVALID_ARG", "NULL"), (experts, dict(order=0), "INVALID_ARG", "NULL"),
    (experts, dict(X=P + 1), "MISALIGNED", "element size"), (experts, dict(offsets=P + 2), "MISALIGNED", "element size"),
    (experts, dict(up_scale=P + 2), "MISALIGNED", "element size"), (experts, dict(ws=0), "INVALID_ARG", "workspace"),
    (experts, dict(size=64), "INVALID_ARG", "workspace"), (experts, dict(ws=P + 8), "MISALIGNED", "16 bytes"),
]


@pytest.mark.parametrize("call,bad,status,text", CALLS)
def test_bad_arguments(g, call, bad, status, text):
    with pytest.raises(g.GemmError) as e:
        call(g, **bad)
    assert e.value.code == getattr(g, "GEMM_ERR_" + status), str(e.value)
    assert text in str(e.value)


def test_null_weights(g):
    assert g.load().gemm_experts(None, 1, 1, P, 8, P, P, P, P, 8, P, 1 << 30, None) == g.GEMM_ERR_INVALID_ARG


def test_empty_calls_are_no_ops(g):
    route(g, tokens=0, logits=0, bias=0, ids=0, weights=0, offsets=0, order=0, ws=0, size=0)
    quantise(g, rows=0, X=0, codes=0, scales=0)
    quantise(g, cols=0, X=0, codes=0, scales=0)
    for none in (dict(M=0), dict(N=0)):
        blocks(g, A=0, B=0, C=0, a_scale=0, b_scale=0, **none)
    experts(g, tokens=0, X=0, offsets=0, order=0, weights=0, O=0, ws=0, size=0, gate=0, up=0, down=0)


def test_real_calls_need_a_device(g):
    for call in (route, quantise, blocks, experts):
        with pytest.raises(g.GemmError) as e:
            call(g)
        assert e.value.code in (g.GEMM_ERR_CUDA, g.GEMM_ERR_UNSUPPORTED)


def test_forced_paths(g):
    g.force_path(g.PATH_SKINNY)
    try:
        with pytest.raises(g.GemmError) as e:
            blocks(g)
        assert e.value.code == g.GEMM_ERR_UNSUPPORTED
        with pytest.raises(g.GemmError) as e:
            experts(g)
        assert e.value.code in (g.GEMM_ERR_UNSUPPORTED, g.GEMM_ERR_CUDA)        # a device comes first
        g.force_path(g.PATH_BF16_TC)
        with pytest.raises(g.GemmError) as e:
            blocks(g, lda=303)
        assert e.value.code == g.GEMM_ERR_UNSUPPORTED and "forced" in str(e.value)
    finally:
        g.force_path(g.PATH_AUTO)


def test_workspace_sizes(g):
    assert g.gemm_route_workspace(256, 64) == 0 and g.gemm_route_workspace(257, 64) >= 4 * 64
    for bad in ((-1, 8), (4, 0), (4, 1025)):
        assert g.gemm_route_workspace(*bad) == 0
    # codes and scales of every slot's x and h, y in bf16, and a place for each slot
    assert g.gemm_experts_workspace(3, 2, 64, 32) >= 6 * (64 + 4 + 32 + 4 + 2 * 64 + 4)
    size = g.gemm_experts_workspace(1 << 20, 32, 65535, 65535)
    assert size >= (1 << 25) * 65535 * 4                       # past 32 bits
    for bad in ((-1, 2, 64, 32), (3, 0, 64, 32), (3, 2, 0, 32), (3, 2, 64, 0), (1 << 30, 2, 64, 32)):
        assert g.gemm_experts_workspace(*bad) == 0


class OnGpu:
    """Stands for a CUDA tensor: what the binding looks at, without a GPU."""
    is_cuda = True

    def __init__(self, t, index=0):
        self.t, self.index = t, index

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_binding_refuses_tensors_that_do_not_fit(g, monkeypatch):
    import torch
    g._torch()
    monkeypatch.setattr(g, "_raw_stream", lambda index: 0)
    f32, i32, bf16, e4m3 = torch.float32, torch.int32, torch.bfloat16, torch.float8_e4m3fn

    def t(*shape, dtype=f32, index=0):
        return OnGpu(torch.zeros(shape, dtype=dtype), index)

    def wide(rows, cols, step, dtype=f32):
        return OnGpu(torch.zeros(rows * cols + 64, dtype=dtype).as_strided((rows, cols), (step, 1)))
    ids, w = t(3, 2, dtype=i32), t(3, 2)
    for args, error in (((t(3, 8, dtype=torch.float16), ids, w), TypeError), ((t(3, 8), t(3, 2, dtype=torch.int64), w), TypeError),
                        ((t(3, 8), t(4, 2, dtype=i32), w), TypeError), ((t(3, 8), ids, t(3, 2, dtype=bf16)), TypeError),
                        ((t(3, 8), ids, OnGpu(torch.zeros(2, 3).T)), TypeError), ((t(3, 8, index=1), ids, w), ValueError),
                        ((t(3, 8, index=-1), t(3, 2, dtype=i32, index=-1), t(3, 2, index=-1)), ValueError),
                        ((OnGpu(torch.zeros(8, 3).T), ids, w), ValueError), ((wide(3, 8, 4), ids, w), ValueError),
                        ((t(3, 8), ids, w, t(8, dtype=i32), t(6, dtype=i32)), (TypeError, ValueError)),
                        ((t(3, 8), ids, w, t(9, dtype=i32), t(5, dtype=i32)), (TypeError, ValueError)),
                        ((t(3, 8), ids, w, t(9, dtype=i32), t(6, dtype=i32), t(7)), (TypeError, ValueError))):
        with pytest.raises(error):
            g.route(*args)
    x, c, s = t(3, 200), t(3, 200, dtype=e4m3), t(3, 2)
    for args, error in (((t(3, 200, dtype=torch.float16), c, s), TypeError), ((x, t(3, 200, dtype=torch.int8), s), TypeError),
                        ((x, t(3, 201, dtype=e4m3), s), ValueError), ((x, c, t(2, 2)), ValueError), ((x, c, t(3, 2, dtype=bf16)), TypeError),
                        ((x, c, s, 64), ValueError), ((x, c, s, 128), ValueError), ((wide(3, 200, 0), c, s), ValueError),
                        ((x, t(3, 200, dtype=e4m3, index=1), s), ValueError)):
        with pytest.raises(error):
            g.fp8_quantise(*args)
    a, b, sa, sb, out = t(3, 300, dtype=e4m3), t(300, 200, dtype=e4m3), t(3, 3), t(3, 2), t(3, 200)
    for args, error in (((a, sa, t(301, 200, dtype=e4m3), sb, out), ValueError), ((a, sa, b, sb, t(3, 201)), ValueError),
                        ((a, sa, b, sb, t(3, 200, dtype=torch.float16)), TypeError), ((t(3, 300), sa, b, sb, out), TypeError),
                        ((a, t(3, 2), b, sb, out), ValueError), ((a, sa, b, t(3, 3), out), ValueError),
                        ((a, sa, b, sb, wide(3, 200, 100)), ValueError), ((a, t(3, 3, index=1), b, sb, out), ValueError)):
        with pytest.raises(error):
            g.fp8_blocks(*args)


def test_expert_weights_that_do_not_fit(g):
    import torch

    def make(gate=(4, 64, 32), up=(4, 64, 32), down=(4, 32, 64), s=(4, 1, 1), dtype=torch.uint8, sdtype=torch.float32):
        z = lambda shape: torch.zeros(shape, dtype=dtype)   # noqa: E731
        return [z(gate), torch.zeros(s, dtype=sdtype), z(up), torch.zeros(s, dtype=sdtype), z(down),
                torch.zeros(s, dtype=sdtype)]
    for kw, error in ((dict(dtype=torch.int8), TypeError), (dict(up=(4, 64, 33)), ValueError), (dict(down=(4, 64, 32)), ValueError),
                      (dict(s=(4, 1, 2)), TypeError), (dict(sdtype=torch.bfloat16), TypeError), (dict(gate=(64, 32)), TypeError)):
        with pytest.raises(error):
            g.ExpertWeights(*make(**kw))
    w = make()
    one = torch.zeros(1, 64, 32, dtype=torch.uint8).expand(4, 64, 32)
    with pytest.raises(ValueError, match="overlap"):
        g.ExpertWeights(one, w[1], one, *w[3:])
    with pytest.raises(ValueError, match="CUDA"):            # nothing else is wrong with them
        g.ExpertWeights(*w)


def test_experts_refuses_tensors_that_do_not_fit(g, monkeypatch):
    import torch
    g._torch()
    monkeypatch.setattr(g, "_raw_stream", lambda index: 0)
    bf16, i32 = torch.bfloat16, torch.int32

    class Weights:
        experts, hidden, width, device, index, address = 4, 64, 32, torch.device("cpu"), 0, 0

    def t(*shape, dtype=bf16, index=0):
        return OnGpu(torch.zeros(shape, dtype=dtype), index)
    good = dict(X=t(3, 64), offsets=t(5, dtype=i32), order=t(6, dtype=i32), token_weights=t(3, 2, dtype=torch.float32),
                O=t(3, 64), workspace=t(1, dtype=torch.uint8))
    for bad, error in ((dict(X=t(3, 64, dtype=torch.float32)), TypeError), (dict(O=t(3, 64, dtype=torch.float16)), TypeError),
                       (dict(token_weights=t(3, 2)), TypeError), (dict(X=t(4, 64)), ValueError), (dict(O=t(3, 65)), ValueError),
                       (dict(offsets=t(4, dtype=i32)), (TypeError, ValueError)), (dict(order=t(5, dtype=i32)), (TypeError, ValueError)),
                       (dict(order=t(6, dtype=torch.int64)), (TypeError, ValueError)), (dict(X=t(3, 64, index=1)), ValueError)):
        with pytest.raises(error):
            g.experts(Weights(), **dict(good, **bad))
