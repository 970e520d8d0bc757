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


class Library:
    """The C library, whose launching calls succeed without launching anything."""

    def __init__(self, lib):
        self.lib = lib

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.lib, name)
        return lambda *a: 0


@pytest.mark.parametrize("stream,want", [(None, "current"), (HANDLE, f"stream {HANDLE}")])
def test_prefill_scratch_and_outputs(m, current, monkeypatch, stream, want):
    monkeypatch.setattr(m, "_lib", Library(m._lib))
    monkeypatch.setattr(m, "_ptr", lambda *a, **k: 16)
    sh = m.make_shape(1, 4, 2, 64, 128, 16, 32)
    q, k = torch.zeros(1, 4, 16, 64), torch.zeros(1, 2, 128, 64)
    m.kvp_score(sh, q, k, k, k, stream=stream)
    m.kvp_select(sh, k, k, stream=stream)
    m.kvp_leverage(sh, k, k, torch.zeros(64, 8), k, stream=stream)
    m.kvp_select_adaptive(sh, 0.2, k, k, k, stream=stream)
    assert current.at_empty == [want] * 4
    # evict_layer's outputs and workspace: at least these
    m.evict_layer(q, k, k, 16, 32, stream=stream)
    assert len(current.at_empty) > 7 and set(current.at_empty) == {want}
