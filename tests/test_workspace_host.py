"""Which calls share the binding's scratch buffer (host logic; the stream handles and captures
are given, the buffers lie in host memory)."""
import ctypes

import pytest

import bit_weight_only_w4_b200 as w4
from bit_weight_only_w4_b200 import build


@pytest.fixture
def on(monkeypatch):
    """on(stream, capture): the current stream's handle, and the capture that records it."""
    import torch
    build.build()
    now = [0, 0]
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: now[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: now[1] != 0, raising=False)
    monkeypatch.setattr(w4, "_capture_id", lambda index, handle: now[1], raising=False)
    monkeypatch.setattr(w4, "_ws_cache", {})
    monkeypatch.setattr(w4, "_ws_captured", {}, raising=False)
    monkeypatch.setattr(w4, "_workspace_size", lambda index, fn, *a: 4096)   # zeroed at the front of a capture's buffer
    dev = torch.device("cpu", 0)

    def ask(stream, capture=0, nbytes=1 << 21):
        now[:] = [stream, capture]
        return w4.workspace_for(dev, nbytes)
    return ask


def test_calls_on_a_stream_share_a_buffer(on):
    a = on(16)
    assert a.numel() >= 1 << 21 and not a.any()
    assert on(16) is a and on(16, nbytes=64) is a
    grown = on(16, nbytes=1 << 22)
    assert grown is not a and grown.numel() >= 1 << 22 and on(16) is grown


def test_streams_do_not_share(on):
    assert on(16) is not on(32)
    assert on(16) is on(16)


def test_captures_do_not_share(on):
    """A graph's buffer serves the calls of its own capture only."""
    eager = on(16)
    first = on(16, capture=5)
    assert first is not eager and not first[:4096].any()
    assert on(16, capture=5) is first and on(16, capture=5, nbytes=1 << 20) is first
    assert on(32, capture=5) is not first      # another stream of the same capture may run beside it
    assert on(16, capture=6) is not first
    assert on(16) is eager                     # eager calls after (or during) a capture


def test_capture_id_refusals():
    build.build()
    L = w4.lib()
    assert L.w4_stream_capture_id(None, None) == w4.W4_ERR_INVALID_ARG
    out = ctypes.c_uint64(7)
    assert L.w4_stream_capture_id(None, ctypes.byref(out)) == w4.W4_OK and out.value == 0
