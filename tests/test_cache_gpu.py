"""kvp_cache_append and kvp_cache_evict against plain forms, bit for bit, and the three calls together
through LayerCache on what evict_layer kept."""
import numpy as np
import pytest
import torch

import synth
from tests.cache_utils import Cache, attend_ref, bits, evict_ref, f64, kvp
from tests.parity_utils import to_dev

pytestmark = pytest.mark.gpu


# ---- append

def append_ref(c, k_new, v_new, weight, counts, n):
    """Pools, acc and lens after the append, on the host."""
    k, v, acc = c.k.clone().view(-1, c.d), c.v.clone().view(-1, c.d), c.acc.clone().view(-1)
    lens = c.lens.clone().view(-1)
    kn, vn = k_new.reshape(c.b, -1, c.d), v_new.reshape(c.b, -1, c.d)
    wn = torch.zeros(kn.shape[:2]) if weight is None else weight.reshape(c.b, -1)
    cap = c.width * c.page
    for s in range(c.b):
        at = 0
        for h in range(c.hkv):
            u = s * c.hkv + h
            cnt = n if counts is None else min(max(int(counts[s, h]), 0), c.hkv * n - at)
            old = min(max(int(lens[u]), 0), cap)
            for i in range(cnt):
                j = old + i
                if j >= cap:
                    break
                page = int(c.table[s, h, j // c.page])
                if 0 <= page < c.num_pages:
                    r = page * c.page + j % c.page
                    k[r], v[r], acc[r] = kn[s, at + i], vn[s, at + i], wn[s, at + i]
            at += cnt
            lens[u] = min(old + cnt, cap)
    return k.view_as(c.k), v.view_as(c.v), acc.view_as(c.acc), lens.view_as(c.lens)


def run_append(c, n, counts=None, weight=True, in_place=False, seed=0):
    m = kvp()
    g = torch.Generator().manual_seed(seed)
    shape = (c.b, c.hkv, n, c.d) if counts is None else (c.b, c.hkv * n, c.d)
    kn, vn = torch.randn(shape, generator=g).to(c.dtype), torch.randn(shape, generator=g).to(c.dtype)
    w = torch.rand(shape[:-1], generator=g) if weight else None
    k, v, acc, table, lens = c.gpu("k", "v", "acc", "table", "lens")
    lens_out = lens if in_place else torch.full_like(lens, -7)
    m.kvp_cache_append(c.shape, kn.cuda(), vn.cuda(), k, v, table, lens, lens_out, acc,
                       None if w is None else w.cuda(),
                       None if counts is None else torch.as_tensor(counts, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    want = append_ref(c, kn, vn, w, None if counts is None else np.asarray(counts), n)
    for got, ref, name in zip((k, v, acc, lens_out), want, ("k", "v", "acc", "lens")):
        assert np.array_equal(bits(got), bits(ref)), name


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("b,hkv,d,page,n", [(1, 2, 64, 16, 1), (5, 8, 128, 16, 1), (2, 3, 128, 32, 7),
                                            (1, 8, 128, 64, 500), (3, 1, 64, 256, 130), (2, 2, 64, 16, 0)])
def test_append_uniform(dtype, b, hkv, d, page, n, in_place):
    lens = [(13 * i) % 70 for i in range(b * hkv)]
    c = Cache(n + d, b, hkv, hkv, d, page, lens, dtype, width=-(-(70 + n) // page))
    run_append(c, n, in_place=in_place)
    run_append(c, n, weight=False, in_place=in_place, seed=1)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("counts", [[[3, 0, 9, 4], [4, 4, 4, 4]], [[16, 0, 0, 0], [0, 0, 0, 16]],
                                    [[1, 2, 3, 4], [0, 0, 0, 0]],          # fewer rows than there is room for
                                    [[30, 5, 0, 0], [-3, 8, 8, 8]]])       # more than there are; a negative one
def test_append_ragged(counts, in_place):
    c = Cache(3, 2, 4, 4, 128, 16, [0, 15, 16, 40, 0, 1, 2, 3], width=8)
    run_append(c, 4, counts, in_place=in_place)


def test_append_past_the_table_and_without_pages():
    c = Cache(4, 2, 2, 2, 64, 16, [30, 47, 60, 1], width=4)
    c.table[0, 0, 2], c.table[1, 1, 0] = -1, c.num_pages
    run_append(c, 40)
    run_append(c, 40, in_place=True)


def test_append_far_offsets():
    m = kvp()
    pages = (2 ** 31) // (16 * 128) + 8
    k = torch.zeros((pages, 16, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    sh = m.make_cache_shape(1, 1, 1, 128, 16, pages, 1)
    table = torch.tensor([[[pages - 1]]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([[3]], dtype=torch.int32, device="cuda")
    kn, vn = torch.randn((2, 1, 1, 5, 128), device="cuda").to(torch.bfloat16)
    m.kvp_cache_append(sh, kn, vn, k, v, table, lens, lens)
    assert torch.equal(k[-1, 3:8], kn[0, 0]) and torch.equal(v[-1, 3:8], vn[0, 0])
    assert lens.item() == 8 and not k[-1, :3].any() and not k[-1, 8:].any() and not k[:8].any()


# ---- evict

def run_evict(c, budget, sinks, window, budgets=None, in_place=False, want_src=True):
    m = kvp()
    k, v, acc, table, lens = c.gpu("k", "v", "acc", "table", "lens")
    acc_out = acc if in_place else torch.full_like(acc, -1.0)
    lens_out = lens if in_place else torch.full_like(lens, -7)
    src = torch.full((c.b, c.hkv, budget), -9, dtype=torch.int32, device="cuda") if want_src else None
    b = None if budgets is None else torch.as_tensor(budgets, dtype=torch.int32).view(c.b, c.hkv).cuda()
    m.kvp_cache_evict(c.shape, m.make_evict(budget, sinks, window), k, v, acc, acc_out, table, lens, lens_out,
                      src, b)
    torch.cuda.synchronize()
    # on the host, a head at a time
    cap = c.width * c.page
    wk, wv = c.k.clone().view(-1, c.d), c.v.clone().view(-1, c.d)
    wacc = (c.acc.clone() if in_place else torch.full_like(c.acc, -1.0)).view(-1)
    acc0 = c.acc.view(-1)
    for u in range(c.b * c.hkv):
        n = min(max(int(c.lens.view(-1)[u]), 0), cap)
        t = budget if budgets is None else min(max(int(budgets[u]), sinks + window, 1), budget)
        pages = c.table.view(-1, c.width)[u].long()
        there = ((pages >= 0) & (pages < c.num_pages)).repeat_interleave(c.page)[:n]
        rows = (pages.clamp(0, c.num_pages - 1)[:, None] * c.page + torch.arange(c.page)).view(-1)[:n]
        weight = torch.where(there, acc0[rows], 0.0).numpy()
        ref = torch.from_numpy(evict_ref(weight, n, t, sinks, window))
        assert int(lens_out.view(-1)[u]) == len(ref) == min(n, t)
        if want_src:
            got = src.view(-1, budget)[u].cpu()
            assert torch.equal(got[:len(ref)].long(), ref) and (got[len(ref):] == -1).all()
        ok = there[ref] & there[:len(ref)]
        to, frm = rows[:len(ref)][ok], rows[ref][ok]
        moved = to != frm
        wk[to[moved]], wv[to[moved]] = c.k.view(-1, c.d)[frm[moved]], c.v.view(-1, c.d)[frm[moved]]
        wacc[to] = acc0[frm]
        # a place whose new row had no page: its own old weight, if any, stays
        left = there[:len(ref)] & ~there[ref]
        at = rows[:len(ref)][left]
        keeps = torch.arange(len(ref))[left] < (t - window if n > t else n)
        wacc[at[keeps]] = acc0[at[keeps]]
    for got, want, name in ((k, wk, "k"), (v, wv, "v"), (acc_out, wacc, "acc")):
        assert np.array_equal(bits(got).reshape(-1), bits(want).reshape(-1)), name


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("page,budget,sinks,window,lens", [
    (16, 32, 4, 8, [0, 1, 31, 32, 33, 40, 48, 200]),
    (16, 1, 0, 0, [0, 1, 2, 17, 100, 3, 9, 50]),              # a single row stays
    (32, 40, 0, 40, [41, 80, 39, 300, 100, 40, 60, 45]),      # the window alone
    (32, 20, 20, 0, [41, 80, 39, 300, 100, 40, 60, 21]),      # the sinks alone
    (64, 100, 3, 70, [101, 171, 169, 300, 130, 102, 99, 240]),  # a window longer than what is given up
    (256, 700, 4, 32, [700, 701, 1500, 2047, 733, 732, 731, 900]),
    (16, 500, 0, 0, [501, 1000, 502, 999, 750, 500, 640, 513]),
])
def test_evict_edges(page, budget, sinks, window, lens, in_place):
    for d, dtype in ((64, torch.float16), (128, torch.bfloat16)):
        c = Cache(budget + d, 2, 4, 4, d, page, lens, dtype)
        run_evict(c, budget, sinks, window, in_place=in_place)


@pytest.mark.parametrize("b,hkv,rows,budget,spread", [(1, 8, 32768, 2048, False), (1, 2, 32768, 22937, False),
                                                      (64, 8, 2064, 2048, True), (1, 1, 131072, 91750, False),
                                                      (1, 1, 450000, 1000, False), (2, 2, 9000, 8999, True),
                                                      (160, 1, 8000, 4000, True), (1, 1, 200000, 60000, False),
                                                      (80, 1, 16384, 5000, True), (1, 8, 4200, 4100, False),
                                                      (100, 2, 900, 700, True), (3, 1, 65536, 300, True)])
def test_evict_sizes(b, hkv, rows, budget, spread):
    """The sizes that select each variant: one CTA or a cluster a head, keys in registers, in shared
    memory or read again from the cache."""
    over = rows - budget
    lens = [budget + (over * i // max(1, b * hkv - 1) if spread else over) for i in range(b * hkv)]
    c = Cache(rows, b, hkv, hkv, 64, 64, lens)
    run_evict(c, budget, 4, 32, in_place=True)


@pytest.mark.parametrize("heads,rows,budget", [(20, 30000, 15000), (36, 10000, 9000), (37, 10000, 9000), (15, 60000, 800),
                                               (18, 8192, 8000)])
def test_evict_heads_and_clusters(heads, rows, budget):
    """More clusters than run at once, and the numbers of heads and rows about which they are used."""
    c = Cache(heads, heads, 1, 1, 64, 128, [rows - 3 * i for i in range(heads)])
    run_evict(c, budget, 0, 16)
    run_evict(c, budget, 5, 0, in_place=True)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("d,page,budget,window,over", [(64, 16, 150, 8, 150), (128, 32, 100, 0, 40), (128, 64, 90, 90, 300),
                                                       (128, 16, 700, 32, 352), (64, 256, 40, 5, 400)])
def test_evict_many_heads(d, page, budget, window, over, in_place):
    """Heads enough to fill the card copy their rows themselves, up to some hundreds of them."""
    lens = [budget + over * i // 151 for i in range(152)]
    run_evict(Cache(d + over, 38, 4, 4, d, page, lens), budget, 2 if window < budget else 0, window, in_place=in_place)


@pytest.mark.parametrize("equal", [False, True])
def test_evict_a_few_rows(equal):
    """Up to about ten rows over the budget, tied and not, absent pages among them."""
    c = Cache(13, 3, 4, 4, 64, 16, [65, 66, 67, 68, 69, 70, 71, 72, 73, 74, 64, 0])
    if equal:
        c.acc[:] = torch.where(torch.arange(c.acc.numel()).view_as(c.acc) % 2 == 0, 1.0, 0.0)
    run_evict(c, 64, 2, 5)
    c.table[0, 1, 1], c.table[1, 2, 4] = -1, c.num_pages
    c.k[:], c.v[:], c.acc[:] = (torch.nan_to_num(t) for t in (c.k, c.v, c.acc))
    run_evict(c, 64, 2, 5, in_place=True)
    run_evict(c, 64, 0, 64, in_place=True)
    run_evict(c, 64, 64, 0)
    run_evict(c, 60, 0, 0, budgets=[64, 60, 59, 60, 1, 60, 63, 60, 61, 60, 60, 2])


@pytest.mark.parametrize("fill", ["equal", "zeros", "two", "nan", "negative", "inf", "near"])
def test_evict_ties_and_odd_weights(fill):
    c = Cache(9, 2, 2, 2, 64, 16, [300, 65, 640, 513])
    live = c.acc.view(-1)
    n = live.numel()
    if fill == "equal":
        c.acc[:] = 0.7
    elif fill == "zeros":
        c.acc[:] = 0.0
    elif fill == "two":
        c.acc[:] = torch.where(torch.arange(n).view_as(c.acc) % 3 == 0, 1.0, 0.5)
    elif fill == "nan":
        live[::4] = float("nan")
    elif fill == "negative":
        live[::3] *= -1
        live[1::7] = -0.0
    elif fill == "inf":
        live[::90] = float("inf")
        live[1::50] = 1e-42                                  # subnormal weights order as numbers too
        live[2::50] = 2e-42
    else:
        c.acc[:] = (torch.arange(n).view_as(c.acc) * 7919 % n).float() * 2.0 ** -23 + 1.0
    for in_place in (False, True):
        run_evict(c, 64, 2, 5, in_place=in_place)


def test_evict_budgets_per_head():
    c = Cache(10, 2, 4, 4, 128, 16, [100, 200, 300, 400, 50, 60, 70, 80])
    run_evict(c, 90, 4, 8, budgets=[90, 50, 12, 1000, -4, 0, 70, 33])
    run_evict(c, 90, 0, 0, budgets=[90, 50, 12, 1000, -4, 0, 70, 33], in_place=True, want_src=False)


def test_evict_without_pages():
    c = Cache(11, 1, 2, 2, 64, 16, [200, 150], garbage=0.0)
    c.table[0, 0, 3], c.table[0, 0, 11], c.table[0, 1, 0] = -1, c.num_pages, -1
    run_evict(c, 40, 2, 10)
    run_evict(c, 40, 2, 10, in_place=True)


def test_evict_at_budget_changes_nothing():
    c = Cache(12, 1, 4, 4, 128, 32, [64, 10, 0, 63])
    run_evict(c, 64, 4, 8, in_place=True)


# ---- together

@pytest.mark.parametrize("adaptive", [False, True])
def test_decode_after_a_prefill_eviction(adaptive):
    """evict_layer's rows (or the adaptive budgets' ragged ones) fill a LayerCache; then tokens are
    decoded against it. Every step's attention is checked in float64 over the rows held, every
    eviction against the plain form on the weights held."""
    m = kvp()
    wl = synth.small("llama8b_32k", hq=8, hkv=2, seq_len=1500, window=16, budget=200)
    inp = synth.make_inputs(wl)
    q, k, v = to_dev(inp.q_win), to_dev(inp.k), to_dev(inp.v)
    b, hq, hkv, d, L, w, B = wl.shape_tuple()
    ev = m.make_evict(B, 4, 16)
    cache = m.LayerCache(b, hq, hkv, d, 2 * B, 16, ev)
    sh = m.make_shape(b, hq, hkv, d, L, w, B)
    buf = m.LayerBuffers(sh, "cuda", want_s1_s2=True)
    m.evict_layer(q, k, v, w, B, buf)
    if adaptive:
        idx = torch.empty((b, hkv * B), dtype=torch.int32, device="cuda")
        counts = torch.empty((b, hkv), dtype=torch.int32, device="cuda")
        ko = torch.empty((b, hkv * B, d), dtype=torch.bfloat16, device="cuda")
        vo = torch.empty_like(ko)
        m.kvp_select_adaptive(sh, 0.2, buf.score, idx, counts)
        m.kvp_compact_ragged(sh, k, v, idx, counts, ko, vo)
        cache.append(ko, vo, counts=counts)
        assert torch.equal(cache.lens, counts.clamp(max=cache.shape.max_pages * 16))
    else:
        cache.append(buf.k_out, buf.v_out, weight=buf.s1.gather(2, buf.idx.long()))
        assert (cache.lens == B).all()
    c = Cache(0, b, hq, hkv, d, 16, [1] * (b * hkv), width=cache.shape.max_pages)
    c.num_pages = cache.shape.num_pages
    c.table = cache.table.cpu()
    g = torch.Generator().manual_seed(5)
    for step in range(20):
        c.q = torch.randn((b, hq, d), generator=g).to(torch.bfloat16)
        kn, vn = (torch.randn((b, hkv, 1, d), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
        cache.append(kn, vn)
        before = cache.acc.clone()
        out = cache.attend(c.q.cuda())
        c.k, c.v, c.lens = cache.k_pages.cpu(), cache.v_pages.cpu(), cache.lens.cpu()
        r_out, r_lse, r_w, t_out, t_lse, t_w = attend_ref(c)
        assert (np.abs(f64(out) - r_out) <= t_out).all()
        assert (np.abs(f64(cache.lse) - r_lse) <= t_lse).all()
        gained = f64(cache.acc).reshape(-1) - f64(before).reshape(-1)
        held = f64(cache.acc).reshape(-1)
        for u in range(b * hkv):
            r = c.rows(u).numpy()
            assert torch.equal(c.k.view(-1, d)[r[-1]], kn.view(-1, d)[u].cpu())
            tol = t_w[u].sum(1) + (held[r] + hq) * 2.0 ** -22
            assert (np.abs(gained[r] - r_w[u].sum(1)) <= tol).all()
        weights, rows = cache.acc.cpu(), [c.rows(u) for u in range(b * hkv)]
        cache.evict()
        for u in range(b * hkv):
            src = evict_ref(weights.view(-1)[rows[u]].numpy(), len(rows[u]), B, 4, 16)
            assert int(cache.lens.view(-1)[u]) == len(src)
            for pool, old in ((cache.k_pages, c.k), (cache.v_pages, c.v)):
                assert torch.equal(pool.cpu().view(-1, d)[rows[u][:len(src)]], old.view(-1, d)[rows[u][src]])
            assert torch.equal(cache.acc.cpu().view(-1)[rows[u][:len(src)]], weights.view(-1)[rows[u][src]])


def test_refused_tensors():
    """Types, shapes, strides and devices are checked before anything is launched."""
    m = kvp()
    c = Cache(1, 2, 4, 2, 64, 16, [20, 30, 0, 9])
    sh = c.shape
    q, k, v, table, lens, acc = c.gpu("q", "k", "v", "table", "lens", "acc")
    out, lens2, kn = torch.empty_like(q), torch.empty_like(lens), torch.zeros((2, 2, 1, 64), dtype=q.dtype, device="cuda")
    ws = m.attend_workspace_for(sh, True)
    attend = dict(q=q, k_pages=k, v_pages=v, table=table, lens=lens, out=out, lse=None, acc=acc, workspace=ws)
    append = dict(k_new=kn, v_new=kn, k_pages=k, v_pages=v, table=table, lens=lens, lens_out=lens2, acc=acc)
    evict = dict(evict=m.make_evict(8, 1, 2), k_pages=k, v_pages=v, acc=acc, acc_out=acc, table=table, lens=lens,
                 lens_out=lens2)
    before = [t.clone() for t in (q, k, v, lens, acc)]
    for call, good in ((m.kvp_cache_attend, attend), (m.kvp_cache_append, append), (m.kvp_cache_evict, evict)):
        for name, t in good.items():
            if not isinstance(t, torch.Tensor) or name == "workspace":
                continue
            wrong = [t.cpu(), t.to(torch.float64), t[:0] if t.dim() else t, None, 3]
            wrong.append(torch.empty(t.shape + (2,), dtype=t.dtype, device="cuda")[..., 0])        # strided
            if name == "acc" and call is not m.kvp_cache_evict:
                wrong.remove(None)
            for bad in wrong:
                with pytest.raises(ValueError):
                    call(sh, **{**good, name: bad})
        with pytest.raises(ValueError):
            call(m.make_shape(1, 8, 2, 64, 128, 16, 32), **good)                     # another call's shape
    with pytest.raises(ValueError):
        m.kvp_cache_evict(sh, **{**evict, "evict": m.make_policy()})
    with pytest.raises(m.KvpError) as e:
        m.kvp_cache_attend(sh, **{**attend, "workspace": ws[:ws.numel() - 256]})
    assert e.value.status == 4
    with pytest.raises(m.KvpError) as e:
        m.kvp_cache_evict(sh, **{**evict, "evict": m.make_evict(8, 6, 3)}, workspace=ws)
    assert e.value.status == 2
    with pytest.raises(ValueError):
        m.LayerCache(1, 4, 2, 64, 64, 16, m.make_evict(64, 1, 2))
    torch.cuda.synchronize()
    for t, b in zip((q, k, v, lens, acc), before):
        assert np.array_equal(bits(t), bits(b))


def test_a_captured_step_replays():
    """A whole step (append, attend, evict) in a graph: lens advances on the device from replay to
    replay, and the results are those of steps called one by one."""
    m = kvp()
    ev = m.make_evict(60, 2, 8)
    g = torch.Generator().manual_seed(1)
    fill = [torch.randn((2, 4, 55, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    steps = [[torch.randn(s, generator=g).to(torch.bfloat16).cuda() for s in ((2, 8, 128), (2, 4, 1, 128), (2, 4, 1, 128))]
             for _ in range(12)]
    one, two = (m.LayerCache(2, 8, 4, 128, 80, 16, ev) for _ in range(2))
    for cache in (one, two):
        cache.append(*fill)
    want = []
    for q, k, v in steps:
        want.append(one.step(q, k, v).clone())
    q, k, v = (t.clone() for t in steps[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        two.step(q, k, v)
    for (a, b, c), w in zip(steps, want):
        q.copy_(a), k.copy_(b), v.copy_(c)
        graph.replay()
        assert torch.equal(two.out, w)
    assert torch.equal(one.lens, two.lens) and torch.equal(one.acc, two.acc)
    assert (one.lens == 60).all()
