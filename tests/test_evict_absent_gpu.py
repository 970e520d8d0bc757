"""Eviction of caches some of whose pages are not there, by each of its variants.

A row without a page weighs zero, and of equal rows the lower stay: where one past t - w is kept, so is every
candidate below it, and there is no hole that it would fill. So only the window's rows can
arrive without a page; they leave their place as it was, and acc_out there untouched."""
import pytest
import torch

from tests.cache_utils import Cache
from tests.test_cache_gpu import run_evict

pytestmark = pytest.mark.gpu

VARIANTS = {
    "picked one by one": (1, 3, 16, 70, 64, 5),
    "fetched while it selects": (1, 3, 16, 100, 64, 8),
    "copied by the selecting CTA": (38, 4, 16, 500, 200, 16),
    "copied by a second kernel": (1, 3, 16, 900, 400, 20),
    "copied by a second kernel, a long window": (1, 3, 16, 900, 400, 300),
    "a cluster a head, 8 keys a thread": (1, 3, 16, 9000, 5000, 32),
    "a cluster a head, to few rows": (1, 2, 64, 20000, 600, 32),
    "a cluster a head, 16 keys a thread": (40, 1, 32, 30000, 15000, 16),
    "long": (1, 2, 64, 140000, 60000, 32),
    "longer than shared memory": (1, 1, 256, 450000, 200000, 70),
}


@pytest.mark.parametrize("share", [0.2, 0.7])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("variant", VARIANTS)
def test_absent_pages(variant, in_place, share):
    b, hkv, page, rows, budget, window = VARIANTS[variant]
    c = Cache(rows + window, b, hkv, hkv, 64, page, [rows - 3 * (i % 2) for i in range(b * hkv)], garbage=0.0,
              outliers=False)
    g = torch.Generator().manual_seed(rows)
    gone = torch.rand(c.table.shape, generator=g) < share
    c.table[gone] = torch.where(torch.rand(c.table.shape, generator=g) < 0.5, -1, c.num_pages).to(torch.int32)[gone]
    c.acc *= torch.rand(c.acc.shape, generator=g) < 0.6             # ties at zero with rows that are there
    run_evict(c, budget, 2, window, in_place=in_place)
    run_evict(c, rows - 5 if window < rows - 10 else budget, 2, window, in_place=in_place)
