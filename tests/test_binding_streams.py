"""Memory that a call of the binding allocates for itself belongs to the stream that the call runs on: the caching allocator
hands a freed block to the next allocation made for the same stream, which may run before another stream is done with it.
No GPU: tensors without storage, a library and streams that only take notes."""
import contextlib

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from quant_int8_quantized_gb300 import mq

pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


class Notes:
    """Stands in for the library; `made` holds, per allocation, the stream that was current."""

    def __init__(self):
        self.current, self.made, self.calls = 0, [], []

    def mq_attn_ws_bytes(self, *a):
        return 4096

    def mq_q6k_packed_row_bytes(self, K):
        return K // 256 * 224

    def __getattr__(self, name):
        def call(*a):
            self.calls.append((name, a[-1].value or 0))
            return mq.MQ_OK
        return call


@pytest.fixture
def notes(monkeypatch):
    n = Notes()

    @contextlib.contextmanager
    def stream(s):
        was, n.current = n.current, s.cuda_stream
        yield
        n.current = was

    empty = torch.empty
    monkeypatch.setattr(mq, "_lib", n)
    monkeypatch.setattr(mq, "_current_stream", lambda: mq.ctypes.c_void_p(0))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    with FakeTensorMode():
        yield n, lambda: monkeypatch.setattr(torch, "empty", lambda *a, **k: (n.made.append(n.current), empty(*a, **k))[1])


@pytest.mark.parametrize("stream,handle", [(Stream(77), 77), (78, 78), (None, 0)])
def test_attention_workspace(notes, stream, handle):
    n, watch = notes
    q = torch.empty((2, 1, 4, 64), dtype=torch.float16, device="cuda")
    own = mq.KV.empty(2, 10, 2, 64)
    length, out = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty_like(q)
    watch()
    mq.mq_attn_prefix(q, None, own, length, out, stream=stream)
    assert n.calls == [("mq_attn_prefix", handle)] and n.made == [handle] and n.current == 0


def test_a_workspace_of_the_caller_is_taken_as_it_is(notes):
    n, watch = notes
    q = torch.empty((2, 1, 4, 64), dtype=torch.float16, device="cuda")
    own = mq.KV.empty(2, 10, 2, 64)
    length, out = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty_like(q)
    ws = mq.attn_workspace(2, 1, 4, 2, 64, 0, 10)
    watch()
    mq.mq_attn_prefix(q, None, own, length, out, ws=ws, stream=Stream(5))
    assert n.calls == [("mq_attn_prefix", 5)] and n.made == []


@pytest.mark.parametrize("stream,handle", [(Stream(77), 77), (None, 0)])
def test_prepacked_rows(notes, stream, handle):
    n, watch = notes
    w = torch.empty((64, 210), dtype=torch.uint8, device="cuda")
    watch()
    mq.mq_prepack_q6k(w, 64, 256, stream=stream)
    assert n.calls == [("mq_prepack_q6k", handle)] and n.made == [handle] and n.current == 0
