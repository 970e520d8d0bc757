"""kvp_cache_attend against float64: types, group sizes, pages, lengths from none to long ones, pages
that are not there, garbage behind the rows, streams, graphs and far offsets."""
import numpy as np
import pytest
import torch

from tests.cache_utils import Cache, attend_ref, bits, f64, kvp

pytestmark = pytest.mark.gpu

# Few heads whose tables hold at most 4096 rows are attended by a cluster of CTAs each; tables that
# hold more, by runs of rows cut over all SMs. Both are put to the same cases.
both = pytest.mark.parametrize("long_table", [False, True])


def width_of(long_table, page):
    return 4096 // page + 1 if long_table else None


def attend(c, acc=True, table=None, lens=None, k=None, v=None, stream=None, workspace=None):
    m = kvp()
    q = c.gpu("q")
    kk, vv = (c.gpu("k") if k is None else k), (c.gpu("v") if v is None else v)
    out = torch.full_like(q, float("nan"))
    lse = torch.full((c.b, c.hq), float("nan"), device="cuda")
    a = c.gpu("acc") if acc else None
    table = c.gpu("table") if table is None else table
    lens = c.gpu("lens") if lens is None else lens
    m.kvp_cache_attend(c.shape, q, kk, vv, table, lens, out, lse, a, workspace, stream)
    torch.cuda.synchronize()
    return out, lse, a


def check(c, got, present=None, lens=None):
    out, lse, a = got
    r_out, r_lse, r_w, t_out, t_lse, t_w = attend_ref(c, lens=lens, present=present)
    err = np.abs(f64(out) - r_out)
    assert (err <= t_out).all(), f"out off by {(err / np.maximum(t_out, 1e-300)).max():.2f} of the bound"
    g_lse = f64(lse)
    none = np.isneginf(r_lse)
    assert (np.isneginf(g_lse) == none).all()
    assert (np.abs(g_lse[~none] - r_lse[~none]) <= t_lse[~none]).all()
    if a is not None:
        before, after = f64(c.acc).reshape(-1), f64(a).reshape(-1)
        same = np.ones(before.size, dtype=bool)
        for u in range(c.b * c.hkv):
            r = c.rows(u, int((c.lens if lens is None else lens).view(-1)[u])).numpy()
            here = np.ones(len(r), dtype=bool) if present is None else present[u][:len(r)]
            rr = r[here]
            same[rr] = False
            want = before[rr] + r_w[u][here].sum(1)
            tol = t_w[u][here].sum(1) + (want + r_w[u].shape[1]) * 2.0 ** -23
            assert (np.abs(after[rr] - want) <= tol).all()
        # what no head holds is left as it was, bit for bit
        assert np.array_equal(bits(a).reshape(-1)[same], bits(c.acc).reshape(-1)[same])


EDGES = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 300]


@both
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hkv,d,page", [(4, 2, 64, 16), (8, 8, 128, 32), (7, 1, 128, 64), (16, 2, 64, 128),
                                           (24, 2, 128, 16), (16, 1, 128, 256), (17, 1, 64, 16), (64, 1, 128, 64),
                                           (66, 2, 64, 32)])
def test_edges_of_length(dtype, hq, hkv, d, page, long_table):
    b = -(-len(EDGES) // hkv)
    lens = (EDGES + [5] * hkv)[:b * hkv]
    c = Cache(hq * d + page, b, hq, hkv, d, page, lens, dtype, width_of(long_table, page))
    check(c, attend(c))
    out, lse, _ = attend(c, acc=False)
    check(c, (out, lse, None))


@pytest.mark.parametrize("b,hq,hkv,d,page,lens", [
    (1, 32, 8, 128, 16, [2111] * 8),                              # an evicted layer
    (1, 32, 8, 128, 64, [32768] * 8),                             # the 32K layer
    (1, 1, 1, 128, 16, [40001]),                                  # one head over all of the card
    (3, 28, 4, 128, 32, [5000, 1, 0, 777, 4096, 4095, 64, 9, 0, 0, 0, 20000]),
    (40, 8, 8, 64, 16, list(range(0, 640, 2))),                   # many short heads
    (300, 4, 4, 64, 16, [0] * 1100 + [70] * 100),                 # long stretches of empty heads
    (1, 4, 2, 64, 16, [512, 512]),                                # the small layer
    (1, 32, 8, 128, 16, [4096, 1, 4095, 0, 513, 4000, 512, 511]),   # the most that a cluster takes
    (1, 16, 1, 128, 16, [4090]),                                  # the same, 16 query heads
    (1, 12, 1, 64, 256, [4096]),
    (16, 1, 1, 64, 16, [i * 100 for i in range(16)]),             # one head too many for clusters
    (1, 12, 1, 64, 256, [4097]),                                  # one row too many
])
def test_real_lengths(b, hq, hkv, d, page, lens):
    c = Cache(b + d, b, hq, hkv, d, page, lens)
    check(c, attend(c))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("b,hq,hkv,d,page,lens", [
    (1, 8, 1, 128, 64, [50000]),                                  # more parts than a warp reads at a time
    (1, 1, 1, 64, 16, [4160]),                                    # fewer than the eight joining blocks would have each
    (1, 16, 1, 64, 16, [9001]),
    (1, 40, 1, 128, 32, [12345]),                                 # three units, the last of 8 query heads
    (1, 64, 1, 64, 256, [30000]),
    (2, 24, 2, 128, 16, [0, 70, 20000, 4097]),                    # none, one tile, some cut
    (4, 5, 1, 64, 128, [1, 0, 64, 12000]),
    (1, 66, 2, 64, 64, [4200, 200]),                              # six units: more than few
])
def test_few_heads_over_the_card(b, hq, hkv, d, page, lens, dtype):
    c = Cache(b + hq, b, hq, hkv, d, page, lens, dtype)
    check(c, attend(c))
    out, lse, _ = attend(c, acc=False)
    check(c, (out, lse, None))


@pytest.mark.parametrize("hq", [2, 34])
def test_a_workspace_used_again_with_other_lengths(hq):
    """What a call wrote of the units it cut is not taken for the next call's."""
    m = kvp()
    c = Cache(hq, 1, hq, 2, 64, 32, [20000, 20000])
    ws = m.attend_workspace_for(c.shape, True)
    for lens in ([20000, 6000], [64, 6000], [0, 0], [20000, 0], [5, 40], [3000, 20000]):
        at = torch.tensor([lens], dtype=torch.int32)
        check(c, attend(c, lens=at.cuda(), workspace=ws), lens=at)


@both
def test_all_heads_empty(long_table):
    c = Cache(1, 3, 8, 2, 64, 16, [0] * 6, width=width_of(long_table, 16))
    out, lse, a = attend(c)
    assert (f64(out) == 0).all() and np.isneginf(f64(lse)).all()
    assert np.array_equal(bits(a), bits(c.acc))


@pytest.mark.parametrize("most", [48, 4112])
def test_lengths_outside_the_table_are_clamped(most):
    c = Cache(2, 1, 4, 4, 64, 16, [most, most, 20, 0])
    wild = torch.tensor([[2 ** 30, most + 1, 20, -5]], dtype=torch.int32)
    clamped = torch.tensor([[most, most, 20, 0]], dtype=torch.int32)
    check(c, attend(c, lens=wild.cuda()), lens=clamped)


@both
@pytest.mark.parametrize("bad", [-1, -2 ** 31, "past", 2 ** 31 - 1])
def test_entries_that_are_no_page(bad, long_table):
    """Rows of an entry outside the pool draw no weight; a head with no page at all is an empty one."""
    c = Cache(3, 2, 8, 2, 128, 16, [100, 64, 33, 200], width=width_of(long_table, 16))
    bad = c.num_pages if bad == "past" else bad
    table = c.table.clone().view(4, -1)
    table[0, 2], table[1, :], table[2, 2], table[3, 0], table[3, 12] = bad, bad, bad, bad, bad
    present = [(table[u][torch.arange(int(c.lens.view(-1)[u])) // 16] == c.table.view(4, -1)[u][
        torch.arange(int(c.lens.view(-1)[u])) // 16]).numpy() for u in range(4)]
    got = attend(c, table=table.view_as(c.table).cuda())
    check(c, got, present=present)
    assert (f64(got[0])[0, 4:] == 0).all()


@both
def test_output_in_place_of_the_queries(long_table):
    c = Cache(4, 4, 28, 4, 128, 16, [(37 * i) % 900 for i in range(16)], width=width_of(long_table, 16))
    out, lse, _ = attend(c, acc=False)
    q = c.gpu("q")
    k, v, table, lens = c.gpu("k", "v", "table", "lens")
    kvp().kvp_cache_attend(c.shape, q, k, v, table, lens, q)
    assert np.array_equal(bits(q), bits(out))


@both
def test_infinite_and_nan_rows_behave_as_in_a_softmax(long_table):
    """A key that makes a head's logit -inf has no weight; a NaN among a head's rows makes that head's
    output NaN and no other's."""
    width = width_of(long_table, 16)
    c = Cache(5, 1, 3, 3, 64, 16, [100, 100, 100], garbage=0.0, outliers=False, width=width)
    c.q[:] = c.q.abs() + 0.5
    low = c.rows(0)[::3]
    c.k.view(-1, 64)[low] = float("-inf")
    present = [np.ones(100, dtype=bool) for _ in range(3)]
    present[0][::3] = False
    c.k.view(-1, 64)[c.rows(1)[50], 7] = float("nan")
    out, lse, a = attend(c)
    o = f64(out)
    assert np.isnan(o[0, 1]).all() and np.isnan(f64(lse)[0, 1])
    assert np.isnan(f64(a).reshape(-1)[c.rows(1).numpy()]).all()
    ref = Cache(5, 1, 3, 3, 64, 16, [100, 100, 100], garbage=0.0, outliers=False, width=width)
    ref.q[:] = ref.q.abs() + 0.5
    r_out, _, r_w, t_out, _, t_w = attend_ref(ref, present=present)
    for h in (0, 2):
        assert (np.abs(o[0, h] - r_out[0, h]) <= t_out[0, h]).all()
    drawn = f64(a).reshape(-1)[c.rows(0).numpy()] - f64(c.acc).reshape(-1)[c.rows(0).numpy()]
    assert (drawn[::3] == 0).all()


@both
def test_every_logit_minus_infinity_is_an_empty_row(long_table):
    c = Cache(6, 1, 2, 1, 64, 16, [40], garbage=0.0, width=width_of(long_table, 16))
    c.q[:] = 1.0
    c.k.view(-1, 64)[c.rows(0)] = float("-inf")
    out, lse, a = attend(c)
    assert (f64(out) == 0).all() and np.isneginf(f64(lse)).all()
    assert np.array_equal(bits(a), bits(c.acc))


@both
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_far_apart_logits(dtype, long_table):
    """One row far above the others, near the start and near the end of the cache: the running
    maximum jumps, and the others' weights fall below what a float holds."""
    for at in (3, 700):
        c = Cache(7, 1, 4, 1, 128, 32, [777], dtype, outliers=False, width=width_of(long_table, 32))
        c.q[:] = c.q * 2
        c.k.view(-1, 128)[c.rows(0)[at]] = (c.q[0, 0].float() * 4).to(dtype)
        check(c, attend(c))


@both
def test_repeat_calls_agree_bit_for_bit(long_table):
    c = Cache(8, 2, 32, 8, 128, 16, [(997 * i) % (6000 if long_table else 4000) for i in range(16)])
    first = attend(c)
    for _ in range(3):
        again = attend(c)
        for x, y in zip(first, again):
            assert np.array_equal(bits(x), bits(y))


def test_split_does_not_depend_on_the_table_width():
    """A long table with room for yet more rows gives the same bits (only lens says what there is)."""
    c = Cache(9, 1, 8, 2, 128, 16, [1000, 333], width=300)
    wide = Cache(9, 1, 8, 2, 128, 16, [1000, 333], width=4096, spare=0)
    wide.num_pages, wide.k, wide.v, wide.acc, wide.q = c.num_pages, c.k, c.v, c.acc, c.q
    table = torch.full((1, 2, 4096), -1, dtype=torch.int32)
    table[:, :, :c.width] = c.table
    wide.table = table
    for x, y in zip(attend(c), attend(wide)):
        assert np.array_equal(bits(x), bits(y))


@both
def test_two_streams_with_a_workspace_each(long_table):
    cs = [Cache(10 + i, 1, 32, 8, 128, 16, [4000 + i] * 8, width=width_of(long_table, 16)) for i in range(2)]
    want = [attend(c) for c in cs]
    m = kvp()
    streams = [torch.cuda.Stream() for _ in cs]
    held = []
    for c in cs:
        held.append(dict(zip(("q", "k", "v", "table", "lens", "acc"), c.gpu("q", "k", "v", "table", "lens", "acc"))))
    torch.cuda.synchronize()
    got = []
    for c, h, s in zip(cs, held, streams):
        ws = m.attend_workspace_for(c.shape, True)
        out, lse = torch.empty_like(h["q"]), torch.empty((c.b, c.hq), device="cuda")
        torch.cuda.synchronize()
        got.append((out, lse, h["acc"], ws, s, c, h))
    for out, lse, acc, ws, s, c, h in got:
        m.kvp_cache_attend(c.shape, h["q"], h["k"], h["v"], h["table"], h["lens"], out, lse, acc, ws, s)
    torch.cuda.synchronize()
    for (out, lse, acc, *_), w in zip(got, want):
        for x, y in zip((out, lse, acc), w):
            assert np.array_equal(bits(x), bits(y))


@pytest.mark.parametrize("width", [40, 200])
def test_captured_and_replayed_with_new_lengths(width):
    """A graph reads lens and the table when it runs: lengths may change between replays."""
    c = Cache(11, 2, 8, 4, 128, 32, [500, 3, 0, 64, 900, 17, 260, 1], width=width)
    c2 = Cache(11, 2, 8, 4, 128, 32, [500, 3, 0, 64, 900, 17, 260, 1], width=width)
    m = kvp()
    q, k, v, table, lens, acc = c.gpu("q", "k", "v", "table", "lens", "acc")
    out, lse = torch.empty_like(q), torch.empty((c.b, c.hq), device="cuda")
    ws = m.attend_workspace_for(c.shape, True)
    m.kvp_cache_attend(c.shape, q, k, v, table, lens, out, lse, None, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.kvp_cache_attend(c.shape, q, k, v, table, lens, out, lse, acc, ws)
    for shorter in (False, True):
        if shorter:
            new = (c2.lens.float() * 0.7).to(torch.int32)
            lens.copy_(new)
            c2.lens = new
        acc.copy_(c2.acc)
        graph.replay()
        torch.cuda.synchronize()
        check(c2, (out, lse, acc))


def test_far_offsets():
    """Rows past 2^31 elements of the pool."""
    c = Cache(12, 1, 8, 2, 128, 16, [150, 90], spare=0)
    pages = (2 ** 31) // (16 * 128) + 64
    k = torch.zeros((pages, 16, 128), dtype=c.dtype, device="cuda")
    v = torch.zeros_like(k)
    far = pages - c.num_pages
    k[far:], v[far:] = c.gpu("k", "v")
    want = attend(c)
    m = kvp()
    sh = m.make_cache_shape(1, 8, 2, 128, 16, pages, c.width)
    q, lens = c.gpu("q", "lens")
    acc = torch.zeros((pages, 16), device="cuda")
    acc[far:] = c.gpu("acc")
    out, lse = torch.empty_like(q), torch.empty((1, 8), device="cuda")
    m.kvp_cache_attend(sh, q, k, v, (c.table + far).cuda(), lens, out, lse, acc)
    torch.cuda.synchronize()
    for x, y in zip((out, lse, acc[far:]), want):
        assert np.array_equal(bits(x), bits(y))
