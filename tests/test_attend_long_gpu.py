"""kvp_cache_attend where runs are long: the last eighth of the tiles cut into short runs, two blocks
that weigh a share, tile counts past 32-bit products; and tables of any width."""
import numpy as np
import pytest
import torch

from tests.cache_utils import Cache, kvp
from tests.test_attend_gpu import attend, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,dtype", [(16, torch.bfloat16), (48, torch.float16)])
def test_runs_of_unequal_length(hq, dtype):
    """Over 9472 tiles (32 for each of the 296 CTAs that are resident): 80 long heads, whose units lie across
    the border between long and short runs, and short ones before, between and after them."""
    short = [0, 1, 63, 64, 65, 500, 0, 0, 128, 17, 4096, 2, 0, 1000, 0, 33]
    lens = []
    for i in range(80):
        lens.append(9900 - 37 * i)
        if i % 5 == 4:
            lens.append(short[i // 5])
    assert sum(-(-n // 64) for n in lens) > 32 * 296
    c = Cache(hq, 24, hq, 4, 64, 64, lens, dtype)
    check(c, attend(c))
    out, lse, _ = attend(c, acc=False)
    check(c, (out, lse, None))


@pytest.mark.parametrize("hq,hkv,d,lens", [(12, 3, 64, [110000, 109000, 108001]), (6, 6, 128, [131072, 60000, 1, 50000, 40000, 70000])])
def test_shares_of_over_a_thousand_rows(hq, hkv, d, lens):
    """Two blocks of the join weigh each share's rows."""
    c = Cache(hkv, 1, hq, hkv, d, 128, lens)
    check(c, attend(c))


@pytest.mark.parametrize("heads,G,least", [(32, 8, 1 << 23), (16, 24, 1 << 23), (64, 4, 1 << 22)])
def test_more_tiles_than_32_bit_products_hold(heads, G, least):
    """2^22 tiles and more: heads of up to 2^23 rows, of whose pages all but a few are not there. The result is
    that of a cache of those few pages."""
    m, page, d, held = kvp(), 256, 64, 6
    rng = np.random.default_rng(heads)
    lens = [least if least == 1 << 23 else int(rng.integers(least, (1 << 23) + 1)) for _ in range(heads)]
    width = (1 << 23) // page
    assert sum(-(-n // 64) for n in lens) * -(-G // 16) >= 1 << 22
    ends = [(n - 1) % page + 1 for n in lens]                       # rows of the last page
    c = Cache(heads + G, heads, G, 1, d, page, [(held - 1) * page + e for e in ends], width=held)
    table = torch.full((heads, width), -1, dtype=torch.int32)
    for u, n in enumerate(lens):
        last = (n - 1) // page
        at = [0, 1] + sorted(rng.choice(np.arange(2, last), held - 3, replace=False).tolist()) + [last]
        table[u, at] = c.table[u, 0]
    sh = m.make_cache_shape(heads, G, 1, d, page, c.num_pages, width)
    q, k, v = c.gpu("q", "k", "v")
    out, lse = torch.empty_like(q), torch.empty((heads, G), device="cuda")
    m.kvp_cache_attend(sh, q, k, v, table.view(heads, 1, width).cuda(), torch.tensor(lens, dtype=torch.int32).view(heads, 1).cuda(),
                       out, lse)
    torch.cuda.synchronize()
    check(c, (out, lse, None))


@pytest.mark.parametrize("width", [63, 256, 257, 300, 4096])
def test_a_table_of_any_width(width):
    """Room for more rows selects another kernel or cut, whose bits may differ, within the same bound."""
    c = Cache(9, 1, 8, 2, 128, 16, [1000, 333], width=width, spare=0)
    check(c, attend(c))
