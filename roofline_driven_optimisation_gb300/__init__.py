"""GB300 dense GEMM: Python binding of the C-ABI library ``libgb300gemm.so``.

The binding only marshals arguments (device pointers, sizes, leading
dimensions, the CUDA stream handle) to the C entry points declared in
``include/gb300gemm.h``; every step of the computation runs in the library's
CUDA kernels.  There is no CPU fallback: if the library is missing or cannot
be loaded, every call raises.

Low-level calls (same names and argument order as the C ABI; pointers and the
stream are integers):

    gemm_f32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)
    gemm_bf16(...), gemm_bf16_f32out(...)

Tensor convenience wrapper (reads pointers, strides and the current stream):

    gemm(A, B, C, alpha=1.0, beta=0.0)
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import _build

GEMM_OK = 0
GEMM_ERR_INVALID_ARG = 1
GEMM_ERR_MISALIGNED = 2
GEMM_ERR_UNSUPPORTED = 3
GEMM_ERR_CUDA = 4
GEMM_ERR_DEVICE_TIMEOUT = 5

PATH_AUTO, PATH_GENERIC, PATH_F32_SIMT, PATH_BF16_TC, PATH_SKINNY, PATH_INT4, PATH_W4, PATH_ATTN, \
    PATH_KV, PATH_SAMPLE = range(10)
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU = range(4)
FP8_E4M3, FP8_E5M2 = 0, 1
KV_E4M3, KV_INT8 = 0, 1
PATH_NAMES = {PATH_AUTO: "none", PATH_GENERIC: "generic", PATH_F32_SIMT: "f32_simt",
              PATH_BF16_TC: "bf16_tc", PATH_SKINNY: "skinny", PATH_INT4: "int4", PATH_W4: "w4",
              PATH_ATTN: "attention", PATH_KV: "kv", PATH_SAMPLE: "sample"}

# every symbol the public header declares
EXPORTS = ("gemm_f32", "gemm_f32_noalloc", "gemm_bf16", "gemm_bf16_f32out", "gemm_f32_ex", "gemm_bf16_ex",
           "gemm_bf16_f32out_ex", "gemm_bf16_swiglu", "gemm_fp8", "gemm_fp8_f32out",
           "gemm_int4_dequant", "gemm_int4_dequant_f32", "gemm_w4a16", "gemm_w4a16_f32out",
           "gemm_int4_repack", "gemm_w4_packed_bytes", "gemm_attention", "gemm_kv_append", "gemm_kv_attention",
           "gemm_kv_attention_workspace", "gemm_sample_bf16", "gemm_sample_f32", "gemm_get_last_error",
           "gemm_device_status", "gemm_force_path", "gemm_last_path", "gemm_force_tile_n",
           "gemm_last_tile_n", "gemm_force_tc_pair", "gemm_last_tc_pair", "gemm_force_split_tiles",
           "gemm_last_k_split", "gemm_set_wait_timeout_ns",
           "gemm_selftest_wait_timeout", "gemm_test_stall")

_lib = None
_lock = threading.Lock()


class KVCacheStruct(ctypes.Structure):
    """gemm_kv_cache of the C ABI."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("page_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong),
                ("token_stride", ctypes.c_longlong), ("table_stride", ctypes.c_longlong),
                ("format", ctypes.c_int), ("pages", ctypes.c_int), ("page_tokens", ctypes.c_int),
                ("heads", ctypes.c_int), ("dim", ctypes.c_int), ("seqs", ctypes.c_int),
                ("table_cols", ctypes.c_int)]


class GemmError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"gemm error {code}: {message}")
        self.code = code


def library_path() -> str:
    return _build.LIB_PATH


def build(force: bool = False) -> str:
    return _build.build(force=force)


def load(path: str | None = None):
    """Load the C library (built in-tree by ``build()``) and declare signatures."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or library_path()
        if not os.path.exists(p):
            raise RuntimeError(f"CUDA GEMM library not built: {p} (run __graft_entry__.build())")
        lib = ctypes.CDLL(p)
        vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        for name in ("gemm_f32", "gemm_f32_noalloc", "gemm_bf16", "gemm_bf16_f32out"):
            fn = getattr(lib, name)
            fn.argtypes = [i, i, i, f, vp, i, vp, i, f, vp, i, vp]
            fn.restype = i
        for name in ("gemm_f32_ex", "gemm_bf16_ex", "gemm_bf16_f32out_ex"):
            fn = getattr(lib, name)
            fn.argtypes = [i, i, i, f, vp, i, vp, i, f, vp, i, vp, i, vp]
            fn.restype = i
        lib.gemm_bf16_swiglu.argtypes = [i, i, i, vp, i, vp, vp, i, vp, i, vp]
        lib.gemm_bf16_swiglu.restype = i
        for name in ("gemm_int4_dequant", "gemm_int4_dequant_f32"):
            fn = getattr(lib, name)
            fn.argtypes = [vp, i, i, i, vp, i, i, i, vp, i, vp]
            fn.restype = i
        for name in ("gemm_w4a16", "gemm_w4a16_f32out"):
            fn = getattr(lib, name)
            fn.argtypes = [i, i, i, f, vp, i, vp, vp, i, i, i, f, vp, i, vp]
            fn.restype = i
        lib.gemm_int4_repack.argtypes = [vp, i, i, i, vp, vp]
        lib.gemm_int4_repack.restype = i
        lib.gemm_attention.argtypes = [i, i, i, i, i, i, vp, vp, vp, vp, f, i, vp]
        lib.gemm_attention.restype = i
        ll, sz = ctypes.c_longlong, ctypes.c_size_t
        lib.gemm_kv_append.argtypes = [vp, i, i, vp, ll, vp, ll, vp, ll, vp, ll, vp, vp, i, i, i, vp, vp, i, vp]
        lib.gemm_kv_append.restype = i
        lib.gemm_kv_attention.argtypes = [vp, i, i, vp, ll, vp, ll, vp, vp, i, f, vp, sz, vp]
        lib.gemm_kv_attention.restype = i
        lib.gemm_kv_attention_workspace.argtypes = [i, i, i, i, i]
        lib.gemm_kv_attention_workspace.restype = sz
        for name in ("gemm_sample_bf16", "gemm_sample_f32"):
            fn = getattr(lib, name)
            fn.argtypes = [i, i, vp, ll, vp, vp, vp, vp, vp, vp, vp, vp]
            fn.restype = i
        lib.gemm_w4_packed_bytes.argtypes = [i, i]
        lib.gemm_w4_packed_bytes.restype = ctypes.c_size_t
        for name in ("gemm_fp8", "gemm_fp8_f32out"):
            fn = getattr(lib, name)
            fn.argtypes = [i, i, i, f, vp, i, i, vp, i, i, f, vp, i, vp]
            fn.restype = i
        lib.gemm_get_last_error.argtypes = []
        lib.gemm_get_last_error.restype = ctypes.c_char_p
        lib.gemm_device_status.argtypes = [vp, ctypes.POINTER(i)]
        lib.gemm_device_status.restype = i
        lib.gemm_force_path.argtypes = [i]
        lib.gemm_force_path.restype = i
        lib.gemm_last_path.argtypes = []
        lib.gemm_last_path.restype = i
        lib.gemm_force_tile_n.argtypes = [i]
        lib.gemm_force_tile_n.restype = i
        lib.gemm_last_tile_n.argtypes = []
        lib.gemm_last_tile_n.restype = i
        lib.gemm_force_tc_pair.argtypes = [i]
        lib.gemm_force_tc_pair.restype = i
        lib.gemm_last_tc_pair.argtypes = []
        lib.gemm_last_tc_pair.restype = i
        lib.gemm_force_split_tiles.argtypes = [i]
        lib.gemm_force_split_tiles.restype = i
        lib.gemm_last_k_split.argtypes = []
        lib.gemm_last_k_split.restype = i
        lib.gemm_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
        lib.gemm_set_wait_timeout_ns.restype = i
        lib.gemm_selftest_wait_timeout.argtypes = [ctypes.c_uint64, vp]
        lib.gemm_selftest_wait_timeout.restype = i
        lib.gemm_test_stall.argtypes = [i]
        lib.gemm_test_stall.restype = i
        _lib = lib
        return lib


def _check(rc: int):
    if rc != GEMM_OK:
        msg = _lib.gemm_get_last_error().decode(errors="replace")
        raise GemmError(rc, msg)


def gemm_f32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0):
    _check(load().gemm_f32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream))


def gemm_f32_noalloc(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0):
    _check(load().gemm_f32_noalloc(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream))


def gemm_bf16(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0):
    _check(load().gemm_bf16(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream))


def gemm_bf16_f32out(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0):
    _check(load().gemm_bf16_f32out(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream))


def gemm_f32_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias, act, stream=0):
    _check(load().gemm_f32_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias, act, stream))


def gemm_bf16_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias, act, stream=0):
    _check(load().gemm_bf16_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias, act, stream))


def gemm_bf16_f32out_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias, act, stream=0):
    _check(load().gemm_bf16_f32out_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias, act,
                                      stream))


def gemm_bf16_swiglu(M, N, K, A, lda, Bgate, Bup, ldb, C, ldc, stream=0):
    _check(load().gemm_bf16_swiglu(M, N, K, A, lda, Bgate, Bup, ldb, C, ldc, stream))


def gemm_fp8(M, N, K, alpha, A, fmt_a, lda, B, fmt_b, ldb, beta, C, ldc, stream=0):
    _check(load().gemm_fp8(M, N, K, alpha, A, fmt_a, lda, B, fmt_b, ldb, beta, C, ldc, stream))


def gemm_fp8_f32out(M, N, K, alpha, A, fmt_a, lda, B, fmt_b, ldb, beta, C, ldc, stream=0):
    _check(load().gemm_fp8_f32out(M, N, K, alpha, A, fmt_a, lda, B, fmt_b, ldb, beta, C, ldc,
                                  stream))


def gemm_int4_dequant(q, K, N, ldq, scales, lds, group, zero, W, ldw, stream=0):
    _check(load().gemm_int4_dequant(q, K, N, ldq, scales, lds, group, zero, W, ldw, stream))


def gemm_int4_dequant_f32(q, K, N, ldq, scales, lds, group, zero, W, ldw, stream=0):
    _check(load().gemm_int4_dequant_f32(q, K, N, ldq, scales, lds, group, zero, W, ldw, stream))


def gemm_w4a16(M, N, K, alpha, X, ldx, qk, scales, lds, group, zero, beta, C, ldc, stream=0):
    _check(load().gemm_w4a16(M, N, K, alpha, X, ldx, qk, scales, lds, group, zero, beta, C, ldc,
                             stream))


def gemm_w4a16_f32out(M, N, K, alpha, X, ldx, qk, scales, lds, group, zero, beta, C, ldc, stream=0):
    _check(load().gemm_w4a16_f32out(M, N, K, alpha, X, ldx, qk, scales, lds, group, zero, beta, C, ldc,
                                    stream))


def gemm_w4_packed_bytes(K, N) -> int:
    return int(load().gemm_w4_packed_bytes(K, N))


def gemm_int4_repack(q, K, N, ldq, qk, stream=0):
    _check(load().gemm_int4_repack(q, K, N, ldq, qk, stream))


def gemm_attention(B, Hq, Hkv, Sq, Sk, D, Q, K, V, O, scale=0.0, causal=0, stream=0):
    _check(load().gemm_attention(B, Hq, Hkv, Sq, Sk, D, Q, K, V, O, scale, causal, stream))


def gemm_kv_append(cache, tokens, Hq, Q, ldq, K, ldk, V, ldv, Qout, ldqo, cos, sin, positions, rotated,
                   interleaved, base, start, max_new, stream=0):
    """`cache`: a KVCacheStruct."""
    _check(load().gemm_kv_append(ctypes.addressof(cache), tokens, Hq, Q, ldq, K, ldk, V, ldv, Qout, ldqo, cos, sin,
                                 positions, rotated, interleaved, base, start, max_new, stream))


def gemm_kv_attention(cache, tokens, Hq, Q, ldq, O, ldo, lengths, start, max_new, scale, workspace, workspace_bytes,
                      stream=0):
    """`cache`: a KVCacheStruct."""
    _check(load().gemm_kv_attention(ctypes.addressof(cache), tokens, Hq, Q, ldq, O, ldo, lengths, start, max_new,
                                    scale, workspace, workspace_bytes, stream))


def gemm_kv_attention_workspace(seqs, heads, Hq, dim, max_new) -> int:
    return int(load().gemm_kv_attention_workspace(seqs, heads, Hq, dim, max_new))


def gemm_sample_bf16(rows, vocab, logits, ld, temperature, top_k, top_p, min_p, u, token, logprob, stream=0):
    _check(load().gemm_sample_bf16(rows, vocab, logits, ld, temperature, top_k, top_p, min_p, u, token, logprob,
                                   stream))


def gemm_sample_f32(rows, vocab, logits, ld, temperature, top_k, top_p, min_p, u, token, logprob, stream=0):
    _check(load().gemm_sample_f32(rows, vocab, logits, ld, temperature, top_k, top_p, min_p, u, token, logprob,
                                  stream))


def device_status(stream=0) -> tuple[int, int]:
    """(status code, location code) of the device status word; clears it."""
    where = ctypes.c_int(0)
    rc = load().gemm_device_status(stream, ctypes.byref(where))
    if rc != GEMM_OK:
        # A call that gave up a wait leaves counts in its workspace, and the word holds
        # the first failure alone: the next calls get new ones.
        _kv_workspaces.clear()
    return rc, where.value


def force_path(path: int):
    _check(load().gemm_force_path(path))


def last_path() -> int:
    return load().gemm_last_path()


def force_tile_n(bn: int):
    _check(load().gemm_force_tile_n(bn))


def last_tile_n() -> int:
    return load().gemm_last_tile_n()


def force_tc_pair(mode: int):
    _check(load().gemm_force_tc_pair(mode))


def last_tc_pair() -> int:
    return load().gemm_last_tc_pair()


def force_split_tiles(enable: int):
    _check(load().gemm_force_split_tiles(enable))


def last_k_split() -> int:
    return load().gemm_last_k_split()


def set_wait_timeout_ns(ns: int):
    _check(load().gemm_set_wait_timeout_ns(ns))


def selftest_wait_timeout(ns: int, stream=0):
    _check(load().gemm_selftest_wait_timeout(ns, stream))


def test_stall(enable: int):
    """Test hook: later calls on this thread make one role of the first CTA
    wait on a barrier nothing arrives at, so the kernel's abort path runs."""
    _check(load().gemm_test_stall(int(enable)))

def _ld(t) -> int:
    """Leading dimension of a row-major 2-D tensor (unit stride along columns)."""
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError("expected a 2-D row-major tensor with unit column stride")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"rows of {t.shape[1]} values lie {t.stride(0)} apart (an expanded tensor?)")
    return max(int(t.stride(0)), int(t.shape[1]), 1)


def gemm(A, B, C, alpha: float = 1.0, beta: float = 0.0, stream=None, bias=None,
         act: int = ACT_NONE):
    """C = act(alpha*A@B + beta*C + bias) for CUDA tensors (fp32/fp32/fp32,
    bf16/bf16/bf16 or bf16/bf16/fp32; bias: N fp32 values or None).
    Argument marshalling only."""
    import torch
    M, K = A.shape
    K2, N = B.shape
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError(f"shape mismatch {tuple(A.shape)} @ {tuple(B.shape)} -> {tuple(C.shape)}")
    if not (A.is_cuda and B.is_cuda and C.is_cuda):
        raise ValueError("gemm() takes CUDA tensors")
    s = stream if stream is not None else torch.cuda.current_stream(A.device).cuda_stream
    args = (M, N, K, float(alpha), A.data_ptr(), _ld(A), B.data_ptr(), _ld(B), float(beta),
            C.data_ptr(), _ld(C))
    if bias is not None:
        if bias.dtype != torch.float32 or not bias.is_cuda or bias.numel() != N or \
                (bias.dim() == 1 and bias.stride(0) != 1):
            raise ValueError("bias must be N contiguous fp32 values on the GPU")
    plain = bias is None and act == ACT_NONE
    ex = (bias.data_ptr() if bias is not None else None, int(act), s)
    if A.dtype == torch.float32 and B.dtype == torch.float32 and C.dtype == torch.float32:
        gemm_f32(*args, s) if plain else gemm_f32_ex(*args, *ex)
    elif A.dtype == torch.bfloat16 and B.dtype == torch.bfloat16 and C.dtype == torch.bfloat16:
        gemm_bf16(*args, s) if plain else gemm_bf16_ex(*args, *ex)
    elif A.dtype == torch.bfloat16 and B.dtype == torch.bfloat16 and C.dtype == torch.float32:
        gemm_bf16_f32out(*args, s) if plain else gemm_bf16_f32out_ex(*args, *ex)
    else:
        raise TypeError(f"unsupported dtypes {A.dtype}, {B.dtype} -> {C.dtype}")
    return C


def swiglu(A, Bgate, Bup, C, stream=None):
    """C = silu(A@Bgate) * (A@Bup) for bf16 CUDA tensors; Bgate and Bup share
    one shape and leading dimension.  Argument marshalling only."""
    import torch
    M, K = A.shape
    K2, N = Bgate.shape
    if K2 != K or tuple(Bup.shape) != (K, N) or tuple(C.shape) != (M, N):
        raise ValueError(f"shape mismatch {tuple(A.shape)} @ {tuple(Bgate.shape)}, "
                         f"{tuple(Bup.shape)} -> {tuple(C.shape)}")
    if _ld(Bgate) != _ld(Bup):
        raise ValueError("Bgate and Bup must have the same leading dimension")
    if not all(t.is_cuda and t.dtype == torch.bfloat16 for t in (A, Bgate, Bup, C)):
        raise TypeError("swiglu() takes bf16 CUDA tensors")
    s = stream if stream is not None else torch.cuda.current_stream(A.device).cuda_stream
    gemm_bf16_swiglu(M, N, K, A.data_ptr(), _ld(A), Bgate.data_ptr(), Bup.data_ptr(), _ld(Bgate),
                     C.data_ptr(), _ld(C), s)
    return C


def gemm_fp8_tensors(A, fmt_a: int, B, fmt_b: int, C, alpha: float = 1.0, beta: float = 0.0,
                     stream=None):
    """C = alpha*dec(A)@dec(B) + beta*C for CUDA tensors of FP8 codes (uint8)
    and a bf16 or fp32 C.  Argument marshalling only."""
    import torch
    M, K = A.shape
    K2, N = B.shape
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError(f"shape mismatch {tuple(A.shape)} @ {tuple(B.shape)} -> {tuple(C.shape)}")
    if A.dtype != torch.uint8 or B.dtype != torch.uint8 or not (A.is_cuda and B.is_cuda and C.is_cuda):
        raise TypeError("gemm_fp8_tensors() takes uint8 FP8 codes on the GPU")
    s = stream if stream is not None else torch.cuda.current_stream(A.device).cuda_stream
    args = (M, N, K, float(alpha), A.data_ptr(), int(fmt_a), _ld(A), B.data_ptr(), int(fmt_b), _ld(B),
            float(beta), C.data_ptr(), _ld(C), s)
    if C.dtype == torch.bfloat16:
        gemm_fp8(*args)
    elif C.dtype == torch.float32:
        gemm_fp8_f32out(*args)
    else:
        raise TypeError(f"unsupported output dtype {C.dtype}")
    return C


def int4_dequant(q, scales, N: int, group: int, zero: int, W, stream=None):
    """W = scales[k // group][n] * (q[k][n] - zero) for CUDA tensors: q K x ceil(N/2)
    uint8 codes, scales bf16, W bf16 or fp32 (K x N).  Argument marshalling only."""
    import torch
    K = q.shape[0]
    if W.shape[0] != K or W.shape[1] != N or q.dtype != torch.uint8 or scales.dtype != torch.bfloat16:
        raise ValueError("int4_dequant(): shape or dtype mismatch")
    s = stream if stream is not None else torch.cuda.current_stream(q.device).cuda_stream
    args = (q.data_ptr(), K, N, _ld(q), scales.data_ptr(), _ld(scales), group, zero, W.data_ptr(),
            _ld(W), s)
    if W.dtype == torch.bfloat16:
        gemm_int4_dequant(*args)
    elif W.dtype == torch.float32:
        gemm_int4_dequant_f32(*args)
    else:
        raise TypeError(f"unsupported output dtype {W.dtype}")
    return W



def int4_repack(q, K: int, N: int, stream=None):
    """Tiled copy (a new flat CUDA uint8 tensor of gemm_w4_packed_bytes(K, N))
    of INT4 codes q (K x ceil(N/2) bytes, packed along n).  Argument
    marshalling only."""
    import torch
    qk = torch.empty((max(gemm_w4_packed_bytes(K, N), 16),), dtype=torch.uint8, device=q.device)
    s = stream if stream is not None else torch.cuda.current_stream(q.device).cuda_stream
    gemm_int4_repack(q.data_ptr(), K, N, _ld(q), qk.data_ptr(), s)
    return qk


def w4a16(X, qk, scales, group: int, zero: int, C, alpha: float = 1.0, beta: float = 0.0,
          stream=None):
    """C = alpha * X @ W + beta * C with W = scales[k // group] * (q - zero) given
    as K-packed codes qk (from int4_repack); X bf16, C bf16 or fp32.  Argument
    marshalling only."""
    import torch
    M, K = X.shape
    N = C.shape[1]
    if C.shape[0] != M or qk.numel() < gemm_w4_packed_bytes(K, N) or X.dtype != torch.bfloat16:
        raise ValueError("w4a16(): shape or dtype mismatch")
    s = stream if stream is not None else torch.cuda.current_stream(X.device).cuda_stream
    args = (M, N, K, float(alpha), X.data_ptr(), _ld(X), qk.data_ptr(), scales.data_ptr(),
            _ld(scales), int(group), int(zero), float(beta), C.data_ptr(), _ld(C), s)
    if C.dtype == torch.bfloat16:
        gemm_w4a16(*args)
    elif C.dtype == torch.float32:
        gemm_w4a16_f32out(*args)
    else:
        raise TypeError(f"unsupported output dtype {C.dtype}")
    return C


def attention(Q, K, V, O, scale: float = 0.0, causal: bool = False, stream=None):
    """O = softmax(Q K^T * scale) V for contiguous bf16 CUDA tensors Q, O
    [B][Hq][Sq][D] and K, V [B][Hkv][Sk][D] (scale 0: 1/sqrt(D)).  Argument
    marshalling only."""
    import torch
    B, Hq, Sq, D = Q.shape
    Hkv, Sk = K.shape[1], K.shape[2]
    for t in (Q, K, V, O):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise TypeError("attention() takes contiguous bf16 CUDA tensors")
    if tuple(V.shape) != tuple(K.shape) or tuple(O.shape) != tuple(Q.shape) or K.shape[0] != B or K.shape[3] != D:
        raise ValueError("attention(): shape mismatch")
    s = stream if stream is not None else torch.cuda.current_stream(Q.device).cuda_stream
    gemm_attention(B, Hq, Hkv, Sq, Sk, D, Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(),
                   float(scale), int(bool(causal)), s)
    return O


class KVCache:
    """A paged key/value cache of CUDA tensors held in 8 bits (gemm_kv_cache).

    k, v: [pages][heads][page_tokens][dim] codes, any strides with dim contiguous
    and the same for both: float8_e4m3fn or int8, or uint8 with `fmt` (KV_E4M3,
    KV_INT8).  k_scale, v_scale: [pages][heads] fp32.  table: [seqs][columns]
    int32 page numbers, the columns contiguous.  The tensors are the caller's and
    are used in place; `rows(n)` is the same cache with the first n table rows.
    """

    def __init__(self, k, v, k_scale, v_scale, table, fmt: int | None = None):
        import torch
        fmts = {torch.float8_e4m3fn: KV_E4M3, torch.int8: KV_INT8, torch.uint8: fmt}
        if k.dim() != 4 or fmts.get(k.dtype) is None or v.dtype != k.dtype:
            raise TypeError("KVCache: k and v are 4-D tensors of float8_e4m3fn, int8 or (with fmt) uint8 codes")
        if fmt is not None and fmts[k.dtype] != fmt:
            raise TypeError("KVCache: fmt does not fit the codes' type")
        pages, heads, page_tokens, dim = k.shape
        if v.shape != k.shape or v.stride() != k.stride() or (dim > 1 and k.stride(3) != 1):
            raise ValueError("KVCache: k and v have one shape and one set of strides, with dim contiguous")
        if page_tokens > 1 and k.stride(2) < dim:
            raise ValueError(f"KVCache: tokens of {dim} values lie {k.stride(2)} apart (an expanded tensor?)")
        for s in (k_scale, v_scale):
            if s.dtype != torch.float32 or tuple(s.shape) != (pages, heads) or not s.is_contiguous():
                raise TypeError("KVCache: scales are contiguous fp32 [pages][heads]")
        if table.dtype != torch.int32 or table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
            raise TypeError("KVCache: table is int32 [seqs][columns] with contiguous columns")
        if table.shape[0] > 1 and table.stride(0) < table.shape[1]:
            raise ValueError(f"KVCache: table rows of {table.shape[1]} lie {table.stride(0)} apart (an expanded tensor?)")
        if not all(t.is_cuda and t.device == k.device for t in (k, v, k_scale, v_scale, table)):
            raise ValueError("KVCache takes CUDA tensors of one device")
        self.k, self.v, self.k_scale, self.v_scale, self.table = k, v, k_scale, v_scale, table
        self.heads, self.dim, self.seqs, self.device = heads, dim, table.shape[0], k.device
        self.struct = KVCacheStruct(
            k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), table.data_ptr(), k.stride(0),
            k.stride(1), max(k.stride(2), dim), max(table.stride(0), table.shape[1]), fmts[k.dtype], pages,
            page_tokens, heads, dim, table.shape[0], table.shape[1])
        self.address, self.index = ctypes.addressof(self.struct), k.device.index

    def rows(self, n: int) -> "KVCache":
        return KVCache(self.k, self.v, self.k_scale, self.v_scale, self.table[:n], self.struct.format)


def _torch():
    """torch, and the types that the calls below compare with (looked up once)."""
    global _t, _bf16, _f32, _i32, _raw_stream
    import torch
    _t, _bf16, _f32, _i32 = torch, torch.bfloat16, torch.float32, torch.int32
    # the current stream's handle without a Stream object around it
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda index: torch.cuda.current_stream(index).cuda_stream)
    return torch


_t = _bf16 = _f32 = _i32 = _raw_stream = None


def _heads(t, name: str, heads: int, dim: int, tokens: int) -> int:
    """Elements between the rows of a bf16 CUDA tensor [tokens][heads][dim] whose
    heads lie side by side."""
    if t.dtype is not _bf16 or not t.is_cuda:
        raise TypeError(f"{name} is a bf16 CUDA tensor")
    if t.shape != (tokens, heads, dim):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {(tokens, heads, dim)}")
    row, head, one = t.stride()
    if (one != 1 and dim > 1) or (head != dim and heads > 1):
        raise ValueError(f"{name}: a row's heads lie side by side")
    if row < heads * dim:
        if tokens > 1:
            raise ValueError(f"{name}: rows of {heads * dim} values lie {row} apart (an expanded tensor?)")
        row = heads * dim                             # of a single row it says nothing
    return row


def _values(t, name: str, n: int, dtype) -> int:
    if t.dtype is not dtype or not t.is_cuda or t.shape != (n,) or not t.is_contiguous():
        raise TypeError(f"{name} is a contiguous {dtype} CUDA tensor of {n} values")
    return t.data_ptr()


def kv_append(cache: KVCache, Q, K, V, cos, sin, base, Qout=None, start=None, max_new: int = 1,
              interleaved: bool = False, stream=None):
    """Store new tokens' K and V ([tokens][heads][dim] bf16) in the cache behind
    the base[b] tokens that sequence b has there, with Q ([tokens][Hq][dim], into
    Qout, default Q itself; or None) and K rotated by position with the tables cos
    and sin (fp32 [positions][pairs]; None: no rotation).  Sequence b's rows are
    start[b] .. start[b+1]-1, at most max_new (start None: row b).  Argument
    marshalling only."""
    if _t is None:
        _torch()
    H, D, seqs = cache.heads, cache.dim, cache.seqs
    tokens = K.shape[0]
    ldk, ldv = _heads(K, "K", H, D, tokens), _heads(V, "V", H, D, tokens)
    Hq = ldq = ldo = q = o = 0
    if Q is not None:
        if Qout is None:
            Qout = Q
        Hq = Q.shape[1]
        ldq, ldo = _heads(Q, "Q", Hq, D, tokens), _heads(Qout, "Qout", Hq, D, tokens)
        q, o = Q.data_ptr(), Qout.data_ptr()
    positions, pairs, c, s = 0x7fffffff, 0, 0, 0
    if cos is not None:
        if cos.dtype is not _f32 or sin.dtype is not _f32 or cos.dim() != 2 or cos.shape != sin.shape or \
                not (cos.is_cuda and sin.is_cuda and cos.is_contiguous() and sin.is_contiguous()):
            raise TypeError("cos and sin are contiguous fp32 CUDA tensors [positions][pairs]")
        positions, pairs = cos.shape
        c, s = cos.data_ptr(), sin.data_ptr()
    rc = (_lib or load()).gemm_kv_append(
        cache.address, tokens, Hq, q, ldq, K.data_ptr(), ldk, V.data_ptr(), ldv, o, ldo, c, s, positions, 2 * pairs,
        interleaved, _values(base, "base", seqs, _i32),
        None if start is None else _values(start, "start", seqs + 1, _i32), max_new,
        _raw_stream(cache.index) if stream is None else stream)
    if rc:
        _check(rc)
    return Qout


# kv_attention's workspaces, one for each device and stream (the C ABI leaves them
# to the caller): zeroed when made, ready again after every call, dropped by
# device_status() when a call has failed.  Calls that are being captured into a graph
# never get one of these.
_kv_workspaces: dict = {}


def _kv_workspace(device, stream: int, *sizes):
    """The workspace of one call on `stream`; sizes: the arguments of
    gemm_kv_attention_workspace."""
    if stream == _raw_stream(device.index):
        return _kv_workspace_here(device, stream, *sizes)
    # made on the stream that uses it, so that the zeros are there before the call and
    # the old one's memory is not reused before its last call
    with _t.cuda.stream(_t.cuda.ExternalStream(stream, device=device)):
        return _kv_workspace_here(device, stream, *sizes)


def _kv_workspace_here(device, stream: int, seqs: int, *sizes):
    size = (_lib or load()).gemm_kv_attention_workspace
    need = size(seqs, *sizes)
    if _t.cuda.is_current_stream_capturing():
        # The graph's own: its memory is of the graph's pool, and its counters (what lies
        # behind the workspace of no sequences) are set to zero by every replay.
        w = _t.empty((need,), dtype=_t.uint8, device=device)
        w[size(0, *sizes):].zero_()
        return w
    key = (device.index, stream)
    w = _kv_workspaces.get(key)
    if w is None or w.numel() < need:
        w = _kv_workspaces[key] = _t.zeros((max(need, 1 << 20),), dtype=_t.uint8, device=device)
    return w


def kv_attention(cache: KVCache, Q, O, lengths, start=None, max_new: int = 1, scale: float = 0.0, workspace=None,
                 stream=None):
    """O = softmax(Q K^T * scale) V of each sequence's newest tokens over the
    cache (scale 0: 1/sqrt(dim)).  Q, O: [tokens][Hq][dim] bf16; lengths[b] tokens
    are in the cache, the newest of them with queries in rows start[b] ..
    start[b+1]-1, at most max_new (start None: one token, row b); query i of n
    sees keys j <= lengths[b] - n + i.  workspace: zeroed uint8 tensor of
    gemm_kv_attention_workspace() bytes, or None for one that this module keeps
    for the stream.  A call captured by torch.cuda.graph gets one of the graph's own,
    zeroed by every replay; a capture that torch does not know of needs `workspace`.
    Argument marshalling only."""
    if _t is None:
        _torch()
    D, seqs = cache.dim, cache.seqs
    tokens, Hq = Q.shape[0], Q.shape[1]
    ldq, ldo = _heads(Q, "Q", Hq, D, tokens), _heads(O, "O", Hq, D, tokens)
    st = _raw_stream(cache.index) if stream is None else stream
    lib = _lib or load()
    if workspace is None:
        workspace = _kv_workspace(cache.device, st, seqs, cache.heads, Hq, D, max_new)
    rc = lib.gemm_kv_attention(
        cache.address, tokens, Hq, Q.data_ptr(), ldq, O.data_ptr(), ldo, _values(lengths, "lengths", seqs, _i32),
        None if start is None else _values(start, "start", seqs + 1, _i32), max_new, scale, workspace.data_ptr(),
        workspace.numel(), st)
    if rc:
        _check(rc)
    return O


def sample(logits, u, token, logprob=None, temperature=None, top_k=None, top_p=None, min_p=None, stream=None):
    """One token of each row of logits ([rows][vocab], bf16 or fp32) from the
    uniform numbers u: token (int32) and, if given, its log-probability among the
    kept.  temperature, top_p, min_p (fp32) and top_k (int32) are CUDA tensors of
    one value a row, or None (1, off).  Argument marshalling only."""
    if _t is None:
        _torch()
    rows, vocab = logits.shape
    if not logits.is_cuda:
        raise ValueError("sample() takes CUDA tensors")
    lib = _lib or load()
    if logits.dtype is _bf16:
        fn = lib.gemm_sample_bf16
    elif logits.dtype is _f32:
        fn = lib.gemm_sample_f32
    else:
        raise TypeError(f"unsupported logits dtype {logits.dtype}")
    rc = fn(rows, vocab, logits.data_ptr(), _ld(logits),
            None if temperature is None else _values(temperature, "temperature", rows, _f32),
            None if top_k is None else _values(top_k, "top_k", rows, _i32),
            None if top_p is None else _values(top_p, "top_p", rows, _f32),
            None if min_p is None else _values(min_p, "min_p", rows, _f32),
            _values(u, "u", rows, _f32), _values(token, "token", rows, _i32),
            None if logprob is None else _values(logprob, "logprob", rows, _f32),
            _raw_stream(logits.device.index) if stream is None else stream)
    if rc:
        _check(rc)
    return token
