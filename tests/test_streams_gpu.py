"""Calls that allocate their own scratch, on another stream than the current one, while the current
stream still writes to a block of that size which was just given back."""
import numpy as np
import pytest
import torch

from tests.cache_utils import Cache, bits, kvp

pytestmark = pytest.mark.gpu


def busy(nbytes):
    """The current stream's allocator gets a block of `nbytes` back that its queue writes to yet."""
    block = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(20_000_000)
    for _ in range(20):
        block.fill_(0x7F)


STREAMS = {"stream": lambda s: s, "handle": lambda s: s.cuda_stream, "default": lambda s: 0, "none": lambda s: None}


@pytest.mark.parametrize("given", STREAMS)
@pytest.mark.parametrize("width", [None, 300])
def test_attend(given, width):
    m = kvp()
    c = Cache(1, 1, 8, 2, 64, 16, [900, 333], width=width)
    side = torch.cuda.Stream()
    n = m.attend_workspace_for(c.shape, True).numel()
    got = []
    for stream in (None, STREAMS[given](side)):
        q, k, v, table, lens, acc = c.gpu("q", "k", "v", "table", "lens", "acc")
        out, lse = torch.empty_like(q), torch.empty((c.b, c.hq), device="cuda")
        torch.cuda.synchronize()
        if stream is not None:
            busy(n)
        m.kvp_cache_attend(c.shape, q, k, v, table, lens, out, lse, acc, stream=stream)
        torch.cuda.synchronize()
        got.append([bits(t) for t in (out, lse, acc)])
    for x, y in zip(*got):
        assert np.array_equal(x, y)


@pytest.mark.parametrize("given", STREAMS)
@pytest.mark.parametrize("rows,budget", [(900, 400), (9000, 5000)])
def test_evict(given, rows, budget):
    m = kvp()
    c = Cache(2, 1, 2, 2, 64, 16, [rows, rows - 9])
    side, ev = torch.cuda.Stream(), m.make_evict(budget, 4, 16)
    n = m.evict_workspace_for(c.shape, ev).numel()
    got = []
    for stream in (None, STREAMS[given](side)):
        k, v, acc, table, lens = c.gpu("k", "v", "acc", "table", "lens")
        torch.cuda.synchronize()
        if stream is not None:
            busy(n)
        m.kvp_cache_evict(c.shape, ev, k, v, acc, acc, table, lens, lens, stream=stream)
        torch.cuda.synchronize()
        got.append([bits(t) for t in (k, v, acc, lens)])
    for x, y in zip(*got):
        assert np.array_equal(x, y)


@pytest.mark.parametrize("given", STREAMS)
def test_prefill(given):
    """Score, select and compact by evict_layer, and the leverage scores."""
    m = kvp()
    b, hq, hkv, d, L, w, B = 1, 8, 2, 64, 1500, 16, 200
    g = torch.Generator().manual_seed(3)
    q, k, v, r = (torch.randn(s, generator=g).to(torch.bfloat16).cuda()
                  for s in ((b, hq, w, d), (b, hkv, L, d), (b, hkv, L, d), (d, 16)))
    sh = m.make_shape(b, hq, hkv, d, L, w, B)
    side, n = torch.cuda.Stream(), m.kvp_workspace_bytes(sh)
    got = []
    for stream in (None, STREAMS[given](side)):
        lev = torch.empty((b, hkv, L), device="cuda")
        torch.cuda.synchronize()
        for call in ("layer", "leverage"):
            if stream is not None:
                busy(n)
            if call == "layer":
                buf = m.evict_layer(q, k, v, w, B, stream=stream)
            else:
                m.kvp_leverage(sh, k, v, r, lev, stream=stream)
        torch.cuda.synchronize()
        got.append([bits(t) for t in (buf.score, buf.idx, buf.k_out, buf.v_out, lev)])
    for x, y in zip(*got):
        assert np.array_equal(x, y)
