"""Memory that a call allocates for itself belongs to the stream that the call runs on: the caching
allocator hands out blocks that the current stream alone may still use, so scratch taken from another
stream than the call's can be written by both. Seen without a GPU: which stream is current when
each call allocates."""
import contextlib
import types

import pytest
import torch


class Current:
    """Stands in for torch's current stream: `names` holds those that were made current."""

    def __init__(self, m, monkeypatch):
        self.names, self.at_empty = [], []
        real = torch.empty

        @contextlib.contextmanager
        def stream(s):
            self.names.append(s)
            try:
                yield
            finally:
                self.names.pop()

        def empty(*shape, dtype=None, device=None):
            self.at_empty.append(self.names[-1] if self.names else "current")
            return real(*shape, dtype=dtype)

        monkeypatch.setattr(torch.cuda, "stream", stream)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: f"stream {handle}")
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=0))
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: None)
        monkeypatch.setattr(torch, "empty", empty)


@pytest.fixture
def m():
    import token_eviction_b200
    return token_eviction_b200


@pytest.fixture
def current(m, monkeypatch):
    return Current(m, monkeypatch)


HANDLE = 0x7F00


@pytest.mark.parametrize("stream,want", [(None, "current"), (HANDLE, f"stream {HANDLE}")])
def test_paged_cache_scratch(m, current, monkeypatch, stream, want):
    calls = []
    for name in ("attend", "evict"):
        monkeypatch.setattr(m._kvp_binding, name, lambda *a, name=name: calls.append((name, a[-1])) or 0)
    monkeypatch.setattr(m, "_device_of", lambda t: torch.device("cpu"))
    sh = m.make_cache_shape(1, 4, 2, 64, 16, 8, 4)
    t = torch.zeros(1)
    m.kvp_cache_attend(sh, t, t, t, t, t, t, stream=stream)
    m.kvp_cache_evict(sh, m.make_evict(8), t, t, t, t, t, t, t, stream=stream)
    assert calls == [("attend", stream), ("evict", stream)]
    assert current.at_empty == [want, want]
