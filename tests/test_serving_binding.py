"""What the serving operators' binding makes of tensors before a call, on the CPU."""
import contextlib

import pytest
import torch

import roofline_driven_optimisation_gb300 as g


class OnGpu:
    """Stands for a CUDA tensor: what the binding looks at, without a GPU."""
    is_cuda = True

    def __init__(self, t):
        self.dtype, self.shape, self.stride = t.dtype, t.shape, t.stride


def heads(t, n, dim, tokens):
    g._torch()
    return g._heads(OnGpu(t), "Q", n, dim, tokens)


def test_rows_that_overlap_are_refused():
    # a stride below a row's width must not be replaced: the call would leave the tensor
    row = torch.zeros(1, 4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="apart"):
        heads(row.expand(3, 4, 8), 4, 8, 3)
    with pytest.raises(ValueError, match="apart"):
        heads(torch.zeros(200, dtype=torch.bfloat16).as_strided((3, 4, 8), (31, 8, 1)), 4, 8, 3)
    with pytest.raises(ValueError, match="apart"):
        g._ld(torch.zeros(1, 8).expand(3, 8))
    with pytest.raises(ValueError, match="apart"):
        g._ld(torch.zeros(40).as_strided((3, 8), (7, 1)))


def test_rows_that_do_not_overlap_are_taken():
    wide = torch.zeros(3, 50, dtype=torch.bfloat16)
    assert heads(wide[:, :32].unflatten(1, (4, 8)), 4, 8, 3) == 50
    assert heads(torch.zeros(3, 4, 8, dtype=torch.bfloat16), 4, 8, 3) == 32
    # the stride of a single row, or of none, is never taken
    assert heads(torch.zeros(1, 4, 8, dtype=torch.bfloat16).expand(1, 4, 8).as_strided((1, 4, 8), (0, 8, 1)), 4, 8, 1) == 32
    assert heads(torch.zeros(0, 4, 8, dtype=torch.bfloat16), 4, 8, 0) == 32
    assert g._ld(torch.zeros(1, 8).as_strided((1, 8), (0, 1))) == 8 and g._ld(torch.zeros(3, 9)[:, :8]) == 9
    assert g._ld(torch.zeros(3, 0)) == 1


def test_caches_that_overlap_are_refused():
    k = torch.zeros(2, 2, 16, 64, dtype=torch.int8)
    s, t = torch.zeros(2, 2), torch.zeros(3, 4, dtype=torch.int32)
    one = torch.zeros(2, 2, 1, 64, dtype=torch.int8).expand(2, 2, 16, 64)
    with pytest.raises(ValueError, match="apart"):
        g.KVCache(one, one, s, s, t)
    # one table row for several sequences
    with pytest.raises(ValueError, match="apart"):
        g.KVCache(k, k, s, s, t[:1].expand(3, 4))
    with pytest.raises(ValueError, match="CUDA"):      # nothing else is wrong with them
        g.KVCache(k, k, s, s, t)


class Calls:
    """Stands for the C library: workspaces of 100 bytes and one for each sequence, and
    what each attention call was given."""

    def __init__(self):
        self.workspaces = []

    def gemm_kv_attention_workspace(self, seqs, heads, Hq, dim, max_new):
        return 100 + seqs

    def gemm_kv_attention(self, *args):
        self.workspaces.append((args[11], args[12]))
        return 0


class Cache:
    def __init__(self, seqs):
        self.heads, self.dim, self.seqs, self.address, self.index = 1, 8, seqs, 0, 0
        self.device = torch.device("cuda", 0)


class Torch:
    """Stands for torch: CPU tensors, and a stream that may be capturing."""
    uint8 = torch.uint8

    def __init__(self):
        self.capturing, self.made = False, []
        self.cuda = self

    def is_current_stream_capturing(self):
        return self.capturing

    def ExternalStream(self, stream, device):
        return stream

    def stream(self, stream):
        return contextlib.nullcontext()

    def _make(self, fill, shape, dtype, device):
        self.made.append(torch.full(shape, fill, dtype=dtype))
        return self.made[-1]

    def empty(self, shape, dtype, device):
        return self._make(7, shape, dtype, device)

    def zeros(self, shape, dtype, device):
        return self._make(0, shape, dtype, device)


@pytest.fixture
def stubs(monkeypatch):
    g._torch()
    calls, fake = Calls(), Torch()
    monkeypatch.setattr(g, "_lib", calls)
    monkeypatch.setattr(g, "_t", fake)
    monkeypatch.setattr(g, "_raw_stream", lambda index: 5)
    monkeypatch.setattr(g, "_kv_workspaces", {})
    monkeypatch.setattr(g, "_values", lambda *a: 0)
    monkeypatch.setattr(g, "_heads", lambda *a: 8)
    return calls, fake


def attend(seqs):
    q = torch.zeros(seqs, 1, 8, dtype=torch.bfloat16)
    g.kv_attention(Cache(seqs), q, q, None)


def test_captured_calls_have_workspaces_of_their_own(stubs):
    calls, fake = stubs
    fake.capturing = True
    attend(3)
    attend(3)
    fake.capturing = False
    attend(3)
    attend(2)
    attend(1 << 20)                                    # outgrows the kept one
    at = [p for p, _ in calls.workspaces]
    assert at[0] != at[1] and at[2] == at[3] and len(set(at)) == 4
    for w in fake.made[:2]:                            # the counters are zeroed, the rest needs no value
        assert w.numel() == 103 and (w[100:] == 0).all() and (w[:100] == 7).all()
    # nothing that a graph uses is kept, so nothing of it can be handed out or dropped
    assert [w.data_ptr() for w in g._kv_workspaces.values()] == at[4:]


def test_kept_workspaces_are_of_the_stream(stubs, monkeypatch):
    calls, _ = stubs
    attend(3)
    monkeypatch.setattr(g, "_raw_stream", lambda index: 6)
    attend(3)
    monkeypatch.setattr(g, "_raw_stream", lambda index: 5)
    attend(3)
    at = [p for p, _ in calls.workspaces]
    assert at[0] == at[2] != at[1]


@pytest.mark.parametrize("status", [g.GEMM_ERR_DEVICE_TIMEOUT, g.GEMM_ERR_INVALID_ARG])
def test_a_failure_on_the_device_drops_the_kept_workspaces(stubs, status):
    # a call that gave up leaves counts behind, and the status names the first failure only
    calls, fake = stubs
    word = [0]

    def gemm_device_status(stream, where):
        got, word[0] = word[0], 0
        return got
    calls.gemm_device_status = gemm_device_status
    attend(3)
    fake.made[-1].fill_(1)
    assert g.device_status()[0] == g.GEMM_OK
    attend(3)
    assert len(fake.made) == 1                         # no failure: kept
    word[0] = status
    assert g.device_status()[0] == status
    attend(3)
    assert len(fake.made) == 2 and (fake.made[1] == 0).all()
    assert calls.workspaces[2][0] == fake.made[1].data_ptr()
