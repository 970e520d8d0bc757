"""What the paged-cache calls refuse, on the host and before any launch (no GPU needed); and the plain
forms that the GPU tests compare with, on cases worked out by hand."""
import ctypes

import numpy as np
import pytest
import torch

from tests.cache_utils import evict_ref

OK, NULL, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4


def m():
    import token_eviction_b200
    return token_eviction_b200


GOOD = dict(batch=2, hq=8, hkv=2, head_dim=128, page_size=16, num_pages=64, max_pages=16)

BAD_SHAPES = [dict(batch=0), dict(hkv=0), dict(hq=7), dict(hq=0), dict(hq=130), dict(head_dim=96),
              dict(head_dim=256), dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(page_size=0),
              dict(num_pages=0), dict(max_pages=0), dict(max_pages=(1 << 19) + 1), dict(batch=1 << 20),
              dict(max_pages=-1), dict(batch=-1)]


def shape(**over):
    return m().make_cache_shape(**{**GOOD, **over})


def append(sh, k=16, v=16, n=1, counts=None, weight=None, kp=16, vp=16, acc=16, table=16, lens=16, lens_out=16):
    return m()._lib.kvp_cache_append(ctypes.byref(sh) if sh else None, k, v, n, counts, weight, kp, vp, acc, table,
                                     lens, lens_out, None)


def attend(sh, q=16, k=16, v=16, table=16, lens=16, out=16, lse=None, acc=None, ws=16, nbytes=1 << 40):
    return m()._lib.kvp_cache_attend(ctypes.byref(sh) if sh else None, q, k, v, table, lens, out, lse, acc, ws,
                                     nbytes, None)


def evict(sh, ev=(32, 4, 8), budgets=None, k=16, v=16, acc=16, acc_out=16, table=16, lens=16, lens_out=16,
          src=None, ws=16, nbytes=1 << 40):
    e = m().make_evict(*ev) if ev else None
    return m()._lib.kvp_cache_evict(ctypes.byref(sh) if sh else None, ctypes.byref(e) if e else None, budgets, k, v,
                                    acc, acc_out, table, lens, lens_out, src, ws, nbytes, None)


@pytest.mark.parametrize("over", BAD_SHAPES)
def test_bad_shapes(over):
    sh = shape(**over)
    assert append(sh) == SHAPE and attend(sh) == SHAPE and evict(sh) == SHAPE
    lib = m()._lib
    assert lib.kvp_cache_attend_workspace_bytes(ctypes.byref(sh), 0) == 0
    ev = m().make_evict(32, 4, 8)
    assert lib.kvp_cache_evict_workspace_bytes(ctypes.byref(sh), ctypes.byref(ev)) == 0


def test_bad_dtype():
    sh = shape()
    sh.dtype = 2
    assert append(sh) == SHAPE and attend(sh) == SHAPE and evict(sh) == SHAPE
    with pytest.raises(ValueError):
        m().make_cache_shape(**GOOD, dtype=torch.float32)


@pytest.mark.parametrize("ev", [(0, 0, 0), (-1, 0, 0), (32, -1, 0), (32, 0, -1), (32, 30, 3),
                                (32, 2 ** 31 - 1, 2 ** 31 - 1), ((1 << 23) + 1, 0, 0)])
def test_bad_eviction_policies(ev):
    assert evict(shape(), ev) == SHAPE


@pytest.mark.parametrize("name", ["k", "v", "kp", "vp", "table", "lens", "lens_out"])
def test_append_pointers(name):
    assert append(shape(), **{name: None}) == NULL
    assert append(shape(), **{name: 24}) == ALIGN


def test_append_other_refusals():
    assert append(None) == NULL
    assert append(shape(), n=-1) == SHAPE
    assert append(shape(), n=(1 << 23) + 1) == SHAPE
    assert append(shape(hq=2 ** 10, hkv=2 ** 10), n=1 << 22) == SHAPE           # hkv n past 2^31
    assert append(shape(), weight=16, acc=None) == SHAPE
    for name in ("counts", "weight", "acc"):
        assert append(shape(), **{name: 8}) == ALIGN


@pytest.mark.parametrize("name", ["q", "k", "v", "table", "lens", "out"])
def test_attend_pointers(name):
    assert attend(shape(), **{name: None}) == NULL
    assert attend(shape(), **{name: 8}) == ALIGN


def test_attend_other_refusals():
    assert attend(None) == NULL
    assert attend(shape(), lse=4) == ALIGN and attend(shape(), acc=4) == ALIGN
    assert attend(shape(), ws=None) == WORKSPACE and attend(shape(), ws=8) == ALIGN
    need = [m()._lib.kvp_cache_attend_workspace_bytes(ctypes.byref(shape()), x) for x in (0, 1)]
    assert 0 < need[0] < need[1]
    assert attend(shape(), nbytes=need[0] - 1) == WORKSPACE
    assert attend(shape(), acc=16, nbytes=need[0]) == WORKSPACE                  # the logits need room too


def test_attend_refuses_more_tiles_than_it_counts():
    sh = shape(batch=1 << 18, max_pages=1 << 19)                                 # 2^19 heads of 2^23 rows
    assert m()._lib.kvp_cache_attend_workspace_bytes(ctypes.byref(sh), 0) == 0
    assert attend(sh) == SHAPE


@pytest.mark.parametrize("name", ["k", "v", "acc", "acc_out", "table", "lens", "lens_out"])
def test_evict_pointers(name):
    assert evict(shape(), **{name: None}) == NULL
    assert evict(shape(), **{name: 8}) == ALIGN


def test_evict_other_refusals():
    assert evict(None) == NULL and evict(shape(), None) == NULL
    assert evict(shape(), src=8) == ALIGN and evict(shape(), budgets=8) == ALIGN
    assert evict(shape(), ws=None) == WORKSPACE and evict(shape(), ws=8) == ALIGN
    ev = m().make_evict(32, 4, 8)
    need = m()._lib.kvp_cache_evict_workspace_bytes(ctypes.byref(shape()), ctypes.byref(ev))
    assert need > 0 and evict(shape(), nbytes=need - 1) == WORKSPACE


def test_binding_refuses_host_tensors_and_missing_ones():
    sh = shape()
    pool = torch.zeros((64, 16, 128), dtype=torch.bfloat16)
    table, lens = torch.zeros((2, 2, 16), dtype=torch.int32), torch.zeros((2, 2), dtype=torch.int32)
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        m().kvp_cache_attend(sh, q, pool, pool, table, lens, q, workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError):
        m().kvp_cache_attend(sh, q, pool, pool, table, lens, None)
    with pytest.raises(ValueError):
        m().kvp_cache_append(sh, q, q, pool, pool, table, lens, lens)            # neither [b, hkv, n, d] nor counts
    with pytest.raises(ValueError):
        m().kvp_cache_evict(sh, dict(budget=32), pool, pool, None, None, table, lens, lens)


def test_evict_plain_form_by_hand():
    acc = np.array([5, 1, 4, 0, 3, 2, 9, 7, 1, 8], dtype=np.float32)
    # 10 rows to 6, first 1 and last 2 stay: of rows 1..7 the heaviest three are 6 (9), 7 (7), 2 (4)
    assert evict_ref(acc, 10, 6, 1, 2).tolist() == [0, 6, 2, 7, 8, 9]
    # nothing but the window
    assert evict_ref(acc, 10, 3, 0, 3).tolist() == [7, 8, 9]
    # ties go to the lower row
    assert evict_ref(np.ones(8, dtype=np.float32), 8, 4, 0, 1).tolist() == [0, 1, 2, 7]
    assert evict_ref(acc, 4, 6, 1, 2).tolist() == [0, 1, 2, 3]
