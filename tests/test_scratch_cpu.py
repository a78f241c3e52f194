"""Where a call takes the workspace from that it allocates itself: the caching allocator
gives memory out again in the order of the stream it came from, so it has to come from the
stream that the call runs on.  Streams and the library are fakes here."""
import contextlib
import types

import pytest
import torch

import paged_kv_cache_190_gb300 as pa
from paged_kv_cache_190_gb300 import _lib


PREPARED = _lib.PreparedCall


class Stream:
    def __init__(self, cuda_stream=77, device=None):
        self.cuda_stream = cuda_stream


class Block(types.SimpleNamespace):
    pass


class Raw:                                  # a stream of another library: only its handle
    cuda_stream = 99


@pytest.fixture
def taken(monkeypatch):
    """Streams that were current, innermost last, when uint8 memory was asked for."""
    current, taken = [], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream.cuda_stream)
        yield
        current.pop()

    def empty(n, **kw):
        taken.append(current[-1] if current else None)
        block = Block(numel=lambda: n, element_size=lambda: 1, data_ptr=lambda: 256,
                      record_stream=lambda s: None)
        return block

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream(0))
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(_lib, "_step", types.SimpleNamespace(span_decode=lambda *a: 0))
    monkeypatch.setattr(_lib, "PreparedCall", lambda name, args, keep=None: lambda: None)
    monkeypatch.setattr(_lib, "_need_cuda_contig", lambda *a: None)
    return taken


def tensor(*shape, dtype=torch.bfloat16):
    t = torch.zeros(shape, dtype=dtype)
    return types.SimpleNamespace(shape=t.shape, dtype=t.dtype, device=t.device, is_cuda=True, dim=t.dim,
                                 numel=t.numel, data_ptr=lambda: 256, element_size=t.element_size,
                                 is_contiguous=lambda: True)


def window(**kw):
    q, c = tensor(2, 4, 128), tensor(3, 2, 16, 128)
    i = tensor(2, 2, dtype=torch.int32)
    return pa.pa_decode_window(q, q, c, c, i, i, 1.0, 2, 16, 8, **kw)


def page_scaled(**kw):
    q, c, s = tensor(2, 4, 128), tensor(3, 2, 16, 128, dtype=torch.uint8), tensor(3, 2, dtype=torch.float32)
    i = tensor(2, 2, dtype=torch.int32)
    return pa.pa_decode_fp8_block(q, q, c, c, i, i, 1.0, s, s, 2, 16, **kw)


def full(**kw):
    q, c = tensor(2, 4, 128), tensor(3, 2, 16, 128)
    i = tensor(2, 2, dtype=torch.int32)
    return pa.pa_decode(q, q, c, c, i, i, 1.0, 2, 16, **kw)


def multi(**kw):
    q, c = tensor(2, 2, 4, 128), tensor(3, 2, 16, 128)
    i = tensor(2, 2, dtype=torch.int32)
    return pa.pa_decode_multi(q, q, c, c, i, i, 1.0, 2, 16, **kw)


def fixed_scale(**kw):
    q, c, s = tensor(2, 4, 128), tensor(3, 2, 16, 128, dtype=torch.uint8), tensor(2, dtype=torch.float32)
    i = tensor(2, 2, dtype=torch.int32)
    return pa.pa_decode_fp8(q, q, c, c, i, i, 1.0, s, s, 2, 16, **kw)


@pytest.mark.parametrize("call", [window, page_scaled, full, multi, fixed_scale])
def test_workspace_comes_from_the_stream_of_the_call(taken, call):
    call(stream=Stream(7))
    call()
    call(stream=Raw())
    assert taken == [7, None, 99]


def cascade(**kw):
    q, c = tensor(2, 4, 128), tensor(3, 2, 16, 128)
    i, g = tensor(2, 2, dtype=torch.int32), tensor(2, dtype=torch.int32)
    return pa.pa_decode_cascade(q, q, c, c, i, i, g, tensor(1, dtype=torch.int32), 1.0, 2, 16, workspace=None, **kw)


@pytest.mark.parametrize("call", [full, multi, fixed_scale, cascade])
def test_a_prepared_call_keeps_the_workspace_that_it_allocated(monkeypatch, taken, call):
    """Its pointer is in the call's arguments: given out again, every later call of the
    prepared one would write into another tensor."""
    import weakref
    blocks = []
    empty = torch.empty

    def watched(*a, **kw):
        block = empty(*a, **kw)
        blocks.append(weakref.ref(block))
        return block

    monkeypatch.setattr(torch, "empty", watched)
    monkeypatch.setattr(_lib, "PreparedCall", PREPARED)
    monkeypatch.setattr(_lib, "pa_decode_cascade_workspace_size", lambda *a: 4096)
    prepared = call(prepare=True)
    assert len(blocks) == 1 and blocks[0]() is not None
    del prepared
    assert blocks[0]() is None
