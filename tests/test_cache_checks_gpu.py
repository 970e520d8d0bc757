"""The paged cache's edge cases on the build whose kernels check their own indices (list places, table
rows, parts, logits), and canaries around everything that the calls write."""
import ctypes

import numpy as np
import pytest
import torch

from tests.cache_utils import Cache, kvp
from tests.test_attend_gpu import EDGES, attend, both, check, width_of
from tests.test_bounds_gpu import Arena
from tests.test_cache_gpu import run_append, run_evict
from tests.test_timeout_gpu import checks_library

pytestmark = pytest.mark.gpu

UNITS = {"append": 5, "attend": 6, "evict": 7}


def address(lib, name):
    return ctypes.cast(getattr(lib, name), ctypes.c_void_p).value


CALLS = ("kvp_cache_append", "kvp_cache_attend", "kvp_cache_evict")


@pytest.fixture
def checked():
    """The package's calls enter the checking build; at the end no check has failed."""
    m, lib = kvp(), checks_library()
    lib.kvp_debug_take_check_unit.argtypes = [ctypes.c_int, ctypes.c_void_p]
    lib.kvp_debug_take_check_unit.restype = ctypes.c_int
    got = np.zeros(4, dtype=np.int32)

    def failed():
        torch.cuda.synchronize()
        found = {}
        for name, unit in UNITS.items():
            assert lib.kvp_debug_take_check_unit(unit, got.ctypes.data) == 0
            if got[0]:
                found[name] = got[:3].tolist()
        return found

    failed()
    m._kvp_binding.use(*(address(lib, n) for n in CALLS))
    try:
        yield
        assert not failed()
    finally:
        m._kvp_binding.use(*(address(m._lib, n) for n in CALLS))


@both
@pytest.mark.parametrize("hq,hkv,d,page", [(4, 2, 64, 16), (7, 1, 128, 64), (24, 2, 128, 16), (17, 1, 64, 16), (64, 1, 128, 256)])
def test_attend(checked, hq, hkv, d, page, long_table):
    b = -(-len(EDGES) // hkv)
    c = Cache(hq * d, b, hq, hkv, d, page, (EDGES + [5] * hkv)[:b * hkv], width=width_of(long_table, page))
    check(c, attend(c))


@pytest.mark.parametrize("b,hq,hkv,d,page,lens", [
    (1, 8, 1, 128, 64, [50000]), (1, 40, 1, 128, 32, [12345]), (4, 5, 1, 64, 128, [1, 0, 64, 12000]),
    (3, 28, 4, 128, 32, [5000, 1, 0, 777, 4096, 4095, 64, 9, 0, 0, 0, 20000]), (1, 12, 1, 64, 256, [4096]),
    (300, 4, 4, 64, 16, [0] * 1100 + [70] * 100), (1, 66, 2, 64, 64, [4200, 200])])
def test_attend_lengths(checked, b, hq, hkv, d, page, lens):
    c = Cache(b + hq, b, hq, hkv, d, page, lens)
    check(c, attend(c))
    out, lse, _ = attend(c, acc=False)
    check(c, (out, lse, None))


@pytest.mark.parametrize("in_place", [False, True])
def test_append(checked, in_place):
    c = Cache(3, 2, 4, 4, 128, 16, [0, 15, 16, 40, 0, 1, 2, 3], width=8)
    for counts in ([[3, 0, 9, 4], [4, 4, 4, 4]], [[30, 5, 0, 0], [-3, 8, 8, 8]], [[0, 0, 0, 0], [0, 0, 0, 16]]):
        run_append(c, 4, counts, in_place=in_place)
    c = Cache(4, 2, 2, 2, 64, 16, [30, 47, 60, 1], width=4)
    c.table[0, 0, 2], c.table[1, 1, 0] = -1, c.num_pages
    run_append(c, 40, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("b,hkv,page,rows,budget,window", [
    (2, 4, 16, 33, 32, 8), (2, 4, 16, 200, 1, 0), (2, 4, 32, 300, 40, 40), (38, 4, 16, 500, 200, 16), (38, 4, 16, 68, 64, 5),
    (38, 4, 64, 120, 90, 34), (1, 3, 16, 900, 400, 300), (1, 8, 64, 9000, 8999, 32), (1, 2, 64, 20000, 600, 32),
    (40, 1, 32, 30000, 15000, 16), (1, 1, 64, 140000, 60000, 32), (1, 1, 256, 450000, 200000, 70)])
def test_evict(checked, b, hkv, page, rows, budget, window, in_place):
    c = Cache(rows, b, hkv, hkv, 64, page, [max(0, rows - 3 * (i % 5)) for i in range(b * hkv)])
    run_evict(c, budget, 0, window, in_place=in_place)
    run_evict(c, budget, 0, window, budgets=[max(1, budget - i % 7) for i in range(b * hkv)], in_place=in_place)


@pytest.mark.parametrize("b,hq,hkv,d,page,rows,budget,dtype", [
    (1, 8, 2, 64, 16, 70, 64, torch.bfloat16), (1, 8, 2, 128, 16, 900, 400, torch.float16), (38, 16, 4, 64, 16, 300, 200, torch.bfloat16),
    (1, 32, 2, 128, 64, 9000, 5000, torch.bfloat16), (1, 1, 1, 64, 256, 140000, 90000, torch.float16),
    (2, 28, 4, 128, 32, 5000, 4990, torch.float16), (1, 64, 1, 64, 16, 4100, 100, torch.bfloat16)])
def test_no_write_outside_buffers(b, hq, hkv, d, page, rows, budget, dtype):
    m = kvp()
    n = 3
    lens = [rows - 2 * (i % 3) for i in range(b * hkv)]
    c = Cache(rows + d, b, hq, hkv, d, page, lens, dtype, width=-(-(rows + n) // page))
    sh, ev = c.shape, m.make_evict(budget, 1, 7)
    heads, pool = b * hkv, c.num_pages * page
    ws = [m.attend_workspace_for(sh, False).numel(), m.attend_workspace_for(sh, True).numel(), m.evict_workspace_for(sh, ev).numel()]
    ar = Arena({"k": pool * d * 2, "v": pool * d * 2, "acc": pool * 4, "acc_out": pool * 4, "lens": heads * 4,
                "lens_out": heads * 4, "src": heads * budget * 4, "out": b * hq * d * 2, "lse": b * hq * 4,
                "ws0": ws[0], "ws1": ws[1], "ws2": ws[2]})
    k, v = ar.view("k", dtype, (c.num_pages, page, d)), ar.view("v", dtype, (c.num_pages, page, d))
    acc, acc_out = (ar.view(x, torch.float32, (c.num_pages, page)) for x in ("acc", "acc_out"))
    len0, len1 = (ar.view(x, torch.int32, (b, hkv)) for x in ("lens", "lens_out"))
    src = ar.view("src", torch.int32, (b, hkv, budget))
    out, lse = ar.view("out", dtype, (b, hq, d)), ar.view("lse", torch.float32, (b, hq))
    q, table = c.gpu("q", "table")
    k.copy_(c.k), v.copy_(c.v), acc.copy_(c.acc), len0.copy_(c.lens)
    kn = torch.randn((b, hkv, n, d), device="cuda").to(dtype)
    m.kvp_cache_append(sh, kn, kn, k, v, table, len0, len1, acc)
    m.kvp_cache_append(sh, kn[:, :, :1].contiguous(), kn[:, :, :1].contiguous(), k, v, table, len0, len0, acc)
    m.kvp_cache_attend(sh, q, k, v, table, len0, out, lse, None, ar.view("ws0", torch.uint8, (ws[0],)))
    m.kvp_cache_attend(sh, q, k, v, table, len0, out, lse, acc, ar.view("ws1", torch.uint8, (ws[1],)))
    m.kvp_cache_evict(sh, ev, k, v, acc, acc_out, table, len0, len1, src, workspace=ar.view("ws2", torch.uint8, (ws[2],)))
    m.kvp_cache_evict(sh, ev, k, v, acc, acc, table, len0, len0, None, workspace=ar.view("ws2", torch.uint8, (ws[2],)))
    torch.cuda.synchronize()
    ar.check()
    assert (len0 <= budget).all()
