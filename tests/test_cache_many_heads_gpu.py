"""The three calls on more heads than a grid's second dimension holds: every head's result is that of
the same head among few."""
import numpy as np
import pytest
import torch

from tests.cache_utils import Cache, bits, kvp

pytestmark = pytest.mark.gpu

FEW, TIMES = 100, 700


def test_seventy_thousand_heads():
    m = kvp()
    page, d, budget = 16, 64, 12
    got = []
    for times in (1, TIMES):
        c = Cache(1, FEW, 2, 1, d, page, [(7 * i) % 16 for i in range(FEW)], spare=0)
        heads = FEW * times
        sh = m.make_cache_shape(heads, 2, 1, d, page, heads, 1)
        again = lambda t: t.cuda().repeat((times,) + (1,) * (t.dim() - 1))
        k, v, acc = again(c.k), again(c.v), again(c.acc)
        table = again(c.table) + FEW * torch.arange(times, dtype=torch.int32, device="cuda").repeat_interleave(FEW).view(-1, 1, 1)
        lens, q = again(c.lens), again(c.q)
        kn = again(torch.randn((FEW, 1, 1, d), generator=torch.Generator().manual_seed(2)).to(c.dtype))
        out, lse = torch.empty_like(q), torch.empty((heads, 2), device="cuda")
        src = torch.empty((heads, 1, budget), dtype=torch.int32, device="cuda")
        m.kvp_cache_append(sh, kn, kn, k, v, table.to(torch.int32), lens, lens, acc)
        m.kvp_cache_attend(sh, q, k, v, table.to(torch.int32), lens, out, lse, acc)
        m.kvp_cache_evict(sh, m.make_evict(budget, 1, 2), k, v, acc, acc, table.to(torch.int32), lens, lens, src)
        torch.cuda.synchronize()
        got.append([bits(t) for t in (k, v, acc, lens, out, lse, src)])
    for one, many in zip(*got):
        assert np.array_equal(np.tile(one, (TIMES,) + (1,) * (one.ndim - 1)), many)
