"""LayerCache with a budget of its own for every head."""
import numpy as np
import pytest
import torch

import synth
from tests.cache_utils import evict_ref, kvp
from tests.parity_utils import to_dev

pytestmark = pytest.mark.gpu


def test_adaptive_counts_survive_decoding():
    """Rows kept under adaptive budgets fill a cache; tokens later every head still has its own count, and
    each eviction is the plain form's at that head's budget."""
    m = kvp()
    wl = synth.small("llama8b_32k", hq=8, hkv=2, seq_len=1500, window=16, budget=200)
    inp = synth.make_inputs(wl)
    q, k, v = to_dev(inp.q_win), to_dev(inp.k), to_dev(inp.v)
    b, hq, hkv, d, L, w, B = wl.shape_tuple()
    sh = m.make_shape(b, hq, hkv, d, L, w, B)
    buf = m.LayerBuffers(sh, "cuda")
    m.evict_layer(q, k, v, w, B, buf)
    idx = torch.empty((b, hkv * B), dtype=torch.int32, device="cuda")
    counts = torch.empty((b, hkv), dtype=torch.int32, device="cuda")
    ko, vo = (torch.empty((b, hkv * B, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m.kvp_select_adaptive(sh, 0.2, buf.score, idx, counts)
    m.kvp_compact_ragged(sh, k, v, idx, counts, ko, vo)
    most = int(counts.max())
    assert most > B > int(counts.min()) > 4 + w              # heads that were given more, and less
    cache = m.LayerCache(b, hq, hkv, d, most + 64, 16, m.make_evict(most, 4, w), budgets=counts)
    cache.append(ko, vo, counts=counts)
    assert torch.equal(cache.lens, counts)
    g = torch.Generator().manual_seed(6)
    n = b * hkv
    table = cache.table.view(n, -1).cpu().long()
    row = (table[:, :, None] * 16 + torch.arange(16)).view(n, -1)
    for step in range(12):
        x, kn, vn = (torch.randn(s, generator=g).to(torch.bfloat16).cuda()
                     for s in ((b, hq, d), (b, hkv, 1, d), (b, hkv, 1, d)))
        cache.append(kn, vn)
        cache.attend(x)
        lens, acc, keys = cache.lens.view(-1).tolist(), cache.acc.cpu().view(-1), cache.k_pages.cpu().view(-1, d)
        cache.evict()
        assert torch.equal(cache.lens, counts)
        after, weights = cache.k_pages.cpu().view(-1, d), cache.acc.cpu().view(-1)
        for u in range(n):
            t = int(counts.view(-1)[u])
            src = torch.from_numpy(evict_ref(acc[row[u, :lens[u]]].numpy(), lens[u], t, 4, w))
            assert len(src) == t == lens[u] - 1
            assert torch.equal(after[row[u, :t]], keys[row[u, src]])
            assert np.array_equal(weights[row[u, :t]].numpy(), acc[row[u, src]].numpy())
