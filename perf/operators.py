"""The decode-side operators on a paged key-value cache: appending rows, attending with one new
token, evicting by accumulated attention weight. What is measured of them, their plain forms
and their values in 64 bits.

A cache is a pool of pages ``[num_pages, page_size, head_dim]`` of keys and one of values, a
table ``[batch, hkv, max_pages]`` of page numbers (pages belong to one KV head of one
sequence, since heads keep different rows), the rows in use ``lens [batch, hkv]`` and, per
cached row, the attention weight it has drawn so far, ``acc [num_pages, page_size]``.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # the smallest call: a small layer's 512 rows, where launches and latencies count
        dict(name="attend tiny", op="attend", dtype="bf16", batch=1, hq=4, hkv=2, d=64, page=16,
             rows=512, ragged=False, acc=True),
        # the everyday decode step of one sequence whose prefill was evicted to 2048 rows a head
        dict(name="attend 2k", op="attend", dtype="bf16", batch=1, hq=32, hkv=8, d=128, page=16,
             rows=2111, ragged=False, acc=True),
        # the same layer not evicted: one long cache, split over all of the card
        dict(name="attend 32k", op="attend", dtype="bf16", batch=1, hq=32, hkv=8, d=128, page=64,
             rows=32768, ragged=False, acc=False),
        # a serving batch with GQA-7 and a different length for every head, one of them empty
        dict(name="attend ragged gqa7", op="attend", dtype="fp16", batch=24, hq=28, hkv=4, d=128,
             page=32, rows=16383, ragged=True, acc=True),
        # the largest: a full batch of caches, 2 GB read in one pass
        dict(name="attend batch64", op="attend", dtype="bf16", batch=64, hq=32, hkv=8, d=128,
             page=16, rows=8192, ragged=False, acc=True),
        # one decoded token of every sequence of a batch
        dict(name="append token", op="append", dtype="bf16", batch=64, hkv=8, d=128, page=16,
             rows=8192, n=1, ragged=False),
        # a prefill's kept rows under adaptive budgets, packed head after head, into a new cache
        dict(name="append adaptive", op="append", dtype="bf16", batch=1, hkv=8, d=128, page=16,
             rows=4096, n=2048, ragged=True),
        # a batch of prefills kept at 1024 rows a head
        dict(name="append batch8", op="append", dtype="fp16", batch=8, hkv=4, d=128, page=64,
             rows=1500, n=1024, ragged=False),
        # a decode loop's eviction: caches up to a page over their budget
        dict(name="evict step", op="evict", dtype="bf16", batch=64, hkv=8, d=128, page=16,
             budget=2048, rows=2064, sinks=4, window=32, spread=True),
        # the first eviction of a long cache down to a small budget
        dict(name="evict 32k", op="evict", dtype="bf16", batch=1, hkv=8, d=128, page=64,
             budget=2048, rows=32768, sinks=4, window=32, spread=False),
        # a mild eviction of a very long cache: much to move
        dict(name="evict 128k b70", op="evict", dtype="bf16", batch=1, hkv=8, d=128, page=128,
             budget=91750, rows=131072, sinks=0, window=32, spread=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "evict"])
    dtype = rng.choice(["bf16", "fp16"])
    hq, hkv = rng.choice([(4, 2), (32, 8), (28, 4), (8, 1), (8, 8), (24, 2)])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    batch = _log_int(rng, 1, 64)
    units = batch * hkv
    if op == "attend":
        most = min(131072, 64 * 8 * 8192 // units)
        rows = _log_int(rng, 1, most)
        return dict(op=op, dtype=dtype, batch=batch, hq=hq, hkv=hkv, d=d, page=page, rows=rows,
                    ragged=rng.random() < 0.5, acc=rng.random() < 0.6)
    if op == "append":
        n = _log_int(rng, 1, min(4096, 131072 // units))
        return dict(op=op, dtype=dtype, batch=batch, hkv=hkv, d=d, page=page, n=n,
                    rows=n + rng.randint(2 * n, 2 * n + 3000), ragged=rng.random() < 0.4)
    rows = _log_int(rng, 16, min(131072, 8 * 131072 // units))
    window = rng.randint(0, min(64, rows // 4))
    sinks = rng.choice([0, 0, 4])
    budget = min(rows, max(sinks + window + 1, int(rows * rng.uniform(0.05, 1.0))))
    return dict(op=op, dtype=dtype, batch=batch, hkv=hkv, d=d, page=page, rows=rows, budget=budget,
                sinks=min(sinks, budget - window), window=window, spread=rng.random() < 0.5)


# ------------------------------------------------------------------------------ inputs

def _even(units, most, gen, device):
    """Row counts spread evenly from 0 to `most` (from `most` alone where there is one unit),
    dealt to the units at random: their sum does not depend on the seed."""
    if units == 1:
        return torch.full((1,), most, dtype=torch.int32, device=device)
    v = torch.arange(units, device=device, dtype=torch.int64) * most // (units - 1)
    return v[torch.randperm(units, generator=gen, device=device)].to(torch.int32)


def _even_sum(units, most):
    return most if units == 1 else sum(i * most // (units - 1) for i in range(units))


def _uneven(hkv, n):
    """hkv counts around n that sum to hkv * n, from n / 4 to 7 n / 4."""
    got = [n] * hkv
    for i in range(hkv // 2):
        off = (3 * n * (hkv - 1 - 2 * i)) // (4 * max(1, hkv - 1))
        got[i], got[hkv - 1 - i] = n - off, n + off
    return got


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    b, hkv, d, page, rows = case["batch"], case["hkv"], case["d"], case["page"], case["rows"]
    units, width = b * hkv, -(-rows // page)
    pages = units * width + 3

    def normal(*shape, outliers=0):
        t = torch.randn(shape, generator=gen, device=dev, dtype=dt)
        if outliers:                       # a few channels with large activations
            at = torch.randperm(d, generator=gen, device=dev)[:outliers]
            t[..., at] *= 20
        return t

    s = dict(case=case, op=case["op"], page=page)
    s["table"] = torch.randperm(pages, generator=gen, device=dev)[:units * width].to(
        torch.int32).view(b, hkv, width)
    s["k_pages"] = normal(pages, page, d, outliers=d // 32)
    s["v_pages"] = normal(pages, page, d, outliers=d // 32)
    # heavy-tailed weights, zeros among them: some rows have drawn nothing yet
    u = torch.rand((pages, page), generator=gen, device=dev)
    s["acc"] = torch.where(u < 0.03, 0.0, 4 * u ** 8)
    if case["op"] == "attend":
        s["q"] = normal(b, case["hq"], d)
        s["lens"] = (_even(units, rows, gen, dev) if case["ragged"] else
                     torch.full((units,), rows, dtype=torch.int32, device=dev)).view(b, hkv)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((b, case["hq"]), dtype=torch.float32, device=dev)
        if not case["acc"]:
            s["acc"] = None
    elif case["op"] == "append":
        n = case["n"]
        shape = (b, hkv * n, d) if case["ragged"] else (b, hkv, n, d)
        s["k_new"], s["v_new"] = normal(*shape, outliers=d // 32), normal(*shape, outliers=d // 32)
        s["weight"] = torch.rand(shape[:-1], generator=gen, device=dev) if n > 1 else None
        s["counts"] = None
        if case["ragged"]:
            c = torch.tensor(_uneven(hkv, n), dtype=torch.int32, device=dev)
            at = torch.rand((b, hkv), generator=gen, device=dev).argsort(-1)
            s["counts"] = c[at].contiguous()
        room = rows - (2 * n if case["ragged"] else n)
        s["lens"] = torch.randint(0, room + 1, (b, hkv), generator=gen, device=dev, dtype=torch.int32)
        s["lens_out"] = torch.empty_like(s["lens"])
    else:
        over = rows - case["budget"]
        s["lens"] = ((case["budget"] + _even(units, over, gen, dev)) if case["spread"] else
                     torch.full((units,), rows, dtype=torch.int32, device=dev)).to(torch.int32).view(b, hkv)
        s["lens_out"] = torch.empty_like(s["lens"])
        s["acc_out"] = torch.zeros_like(s["acc"])
        s["src"] = torch.empty((b, hkv, case["budget"]), dtype=torch.int32, device=dev)
    return s


# ------------------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    return {"attend": _attend, "append": _append, "evict": _evict}[s["op"]](s)


def _run_own(s):
    import token_eviction_b200 as kvp
    if "shape" not in s:       # the handle and workspace that a program keeps beside its cache
        c = s["case"]
        s["shape"] = kvp.make_cache_shape(c["batch"], c.get("hq", c["hkv"]), c["hkv"], c["d"], c["page"],
                                          s["k_pages"].shape[0], s["table"].shape[2], s["k_pages"].dtype)
        if s["op"] == "attend":
            s["workspace"] = kvp.attend_workspace_for(s["shape"], s["acc"] is not None)
        elif s["op"] == "evict":
            s["policy"] = kvp.make_evict(c["budget"], c["sinks"], c["window"])
            s["workspace"] = kvp.evict_workspace_for(s["shape"], s["policy"])
    if s["op"] == "attend":
        kvp.kvp_cache_attend(s["shape"], s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                             s["out"], s["lse"], s["acc"], s["workspace"])
        return (s["out"], s["lse"]) if s["acc"] is None else (s["out"], s["lse"], s["acc"])
    if s["op"] == "append":
        kvp.kvp_cache_append(s["shape"], s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], s["table"],
                             s["lens"], s["lens_out"], s["acc"], s["weight"], s["counts"])
        return s["k_pages"], s["v_pages"], s["acc"], s["lens_out"]
    kvp.kvp_cache_evict(s["shape"], s["policy"], s["k_pages"], s["v_pages"], s["acc"], s["acc_out"],
                        s["table"], s["lens"], s["lens_out"], s["src"], workspace=s["workspace"])
    return s["k_pages"], s["v_pages"], s["acc_out"], s["lens_out"], s["src"]


def _row_ids(s):
    """[units, width * page]: where each of a unit's rows lies in the flattened pool."""
    t = s["table"].long().flatten(0, 1)
    p = s["page"]
    return (t[..., None] * p + torch.arange(p, device=t.device)).flatten(1)


def _attend(s):
    """o = softmax(q k^T / sqrt(d)) v over each head's rows, lse, and acc += the weights."""
    c = s["case"]
    g, d = c["hq"] // c["hkv"], c["d"]
    ids, n = _row_ids(s), s["lens"].flatten().long()
    live = torch.arange(ids.shape[1], device=ids.device) < n[:, None]                 # [U, L]
    k = s["k_pages"].view(-1, d)[ids].float()                                         # [U, L, d]
    q = s["q"].float().view(-1, g, d)
    logits = torch.matmul(q, k.transpose(1, 2)) / math.sqrt(d)                         # [U, g, L]
    del k
    logits = logits.masked_fill(~live[:, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    lse = top + torch.log(total)
    p = p / torch.where(total > 0, total, 1.0)
    v = s["v_pages"].view(-1, d)[ids].float().masked_fill(~live[..., None], 0.0)
    out = torch.matmul(p, v).to(s["q"].dtype).view(s["q"].shape)
    del v
    lse = lse.view(s["lse"].shape)
    if s["acc"] is None:
        return out, lse
    flat = s["acc"].view(-1)
    flat[ids] = flat[ids] + p.sum(1)                                                  # 0 past a head's rows
    return out, lse, s["acc"]


def _append(s):
    """Row i of a head's new rows goes to its row lens + i, with its weight (0 where none is given)."""
    c = s["case"]
    d, n, units, hkv = c["d"], c["n"], c["batch"] * c["hkv"], c["hkv"]
    ids, lens = _row_ids(s), s["lens"].flatten().long()
    k, v = s["k_new"].reshape(-1, d), s["v_new"].reshape(-1, d)
    w = torch.zeros(units * n, device=k.device) if s["weight"] is None else s["weight"].reshape(-1)
    r = torch.arange(units * n, device=k.device)
    if s["counts"] is None:
        counts = torch.full_like(lens, n)
        unit = r // n
        at = r - unit * n
    else:
        counts = s["counts"].flatten().long()
        ends = counts.view(-1, hkv).cumsum(-1)                                        # within a sequence
        seq = r // (hkv * n)
        inside = r - seq * (hkv * n)
        head = (ends[seq] <= inside[:, None]).sum(-1)
        unit = seq * hkv + head
        at = inside - (ends - counts.view(-1, hkv))[seq, head]
    to = ids[unit, lens[unit] + at]
    s["k_pages"].view(-1, d)[to] = k
    s["v_pages"].view(-1, d)[to] = v
    s["acc"].view(-1)[to] = w
    s["lens_out"].copy_((lens + counts).to(torch.int32).view_as(s["lens"]))
    return s["k_pages"], s["v_pages"], s["acc"], s["lens_out"]


def _evict(s):
    """Each head's first `sinks` rows, its last `window` rows and the heaviest between them, `budget`
    in all. Kept rows below budget - window stay; the holes among them, ascending, take the kept
    rows from there on, ascending; the window's rows follow."""
    c = s["case"]
    d, t, w, sinks = c["d"], c["budget"], c["window"], c["sinks"]
    ids, n = _row_ids(s), s["lens"].flatten().long()[:, None]
    at = torch.arange(ids.shape[1], device=ids.device)[None]
    weight = s["acc"].view(-1)[ids]
    full = n > t
    cand = (at >= sinks) & (at < n - w)
    key = torch.where(cand, torch.where(weight > 0, weight, 0.0), -1.0)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, at.expand_as(order))
    kept = cand & (rank < t - w - sinks)
    low = at < t - w
    hole = full & low & (at >= sinks) & ~kept
    high = full & kept & ~low
    # the i-th hole takes the i-th kept row at or past t - w: a stable sort lists those first
    high_at = torch.sort((~high).to(torch.int8), dim=-1, stable=True).indices
    nth = (hole.long().cumsum(-1) - 1).clamp_min(0)
    src = torch.where(hole, high_at.gather(1, nth), at)
    src = torch.where(full & ~low, n - t + at, src)[:, :t]
    new = torch.minimum(n, torch.full_like(n, t))
    live = at[:, :t] < new
    src = torch.where(live, src, at[:, :t])
    to, frm = ids[:, :t], ids.gather(1, src)
    for pool in (s["k_pages"], s["v_pages"]):
        flat = pool.view(-1, d)
        flat[to] = flat[frm]
    s["acc_out"].view(-1)[to] = torch.where(live, s["acc"].view(-1)[frm], 0.0)
    s["lens_out"].copy_(new.to(torch.int32).view_as(s["lens"]))
    s["src"].copy_(torch.where(live, src, -1).to(torch.int32).view_as(s["src"]))
    return s["k_pages"], s["v_pages"], s["acc_out"], s["lens_out"], s["src"]


# ------------------------------------------------------------------------------ work

def work(case):
    b, hkv, d, rows = case["batch"], case["hkv"], case["d"], case["rows"]
    units, row = b * hkv, 2 * 2 * d                       # bytes of a row of keys and one of values
    if case["op"] == "attend":
        total = _even_sum(units, rows) if case["ragged"] else units * rows
        nbytes = total * (row + (8 if case["acc"] else 0)) + total // case["page"] * 4 + units * 4
        nbytes += b * case["hq"] * (4 * d + 4)
        return {"bytes": nbytes, "flops": 4 * (case["hq"] // hkv) * d * total}
    if case["op"] == "append":
        total = units * case["n"]
        return {"bytes": total * (2 * row + 4 + (4 if case["n"] > 1 else 0)) + units * 12, "flops": 0}
    t, w, s = case["budget"], case["window"], case["sinks"]
    over = rows - t
    read = units * t + (_even_sum(units, over) if case["spread"] else units * over)
    gone = read / units - t                               # rows that a head gives up, on average
    part = (t - s - w) / max(1, t + gone - s - w)         # of the candidates, those that stay
    moved = part * gone + (w if gone > 0 else 0)          # kept rows past t - w, and the window
    return {"bytes": int(units * (moved * 2 * row + t * 8 + 8) + read * 4), "flops": 0}


# ------------------------------------------------------------------------------ values in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    hkv, d, page = case["hkv"], case["d"], case["page"]
    units = case["batch"] * hkv
    table = s["table"].view(units, -1).cpu()
    lens = s["lens"].flatten().tolist()

    def rows_of(u, first, last):
        j = torch.arange(first, last)
        return (table[u, j // page].long() * page + j % page).to("cuda")

    if case["op"] == "attend":
        g = case["hq"] // hkv
        out = torch.zeros(units, g, d, dtype=torch.float64, device="cuda")
        lse = torch.full((units, g), -math.inf, dtype=torch.float64, device="cuda")
        acc = None if s["acc"] is None else s["acc"].double().flatten()
        q = s["q"].double().view(units, g, d)
        for u in range(units):
            if lens[u] == 0:
                continue
            r = rows_of(u, 0, lens[u])
            x = (s["k_pages"].view(-1, d)[r].double() @ q[u].T) * d ** -0.5           # [rows, g]
            lse[u] = torch.logsumexp(x, 0)
            p = torch.exp(x - lse[u])
            out[u] = p.T @ s["v_pages"].view(-1, d)[r].double()
            if acc is not None:
                acc[r] += p.sum(1)
        got = (out.view(s["q"].shape), lse.view(s["lse"].shape))
        return got if acc is None else got + (acc.view_as(s["acc"]),)

    k, v = s["k_pages"].view(-1, d).clone(), s["v_pages"].view(-1, d).clone()
    if case["op"] == "append":
        n = case["n"]
        acc = s["acc"].double().flatten()
        counts = [n] * units if s["counts"] is None else s["counts"].flatten().tolist()
        at = 0
        kn, vn = s["k_new"].view(-1, d), s["v_new"].view(-1, d)
        for u in range(units):
            r = rows_of(u, lens[u], lens[u] + counts[u])
            k[r], v[r] = kn[at:at + counts[u]], vn[at:at + counts[u]]
            acc[r] = 0.0 if s["weight"] is None else s["weight"].flatten()[at:at + counts[u]].double()
            at += counts[u]
        after = torch.tensor([a + b for a, b in zip(lens, counts)], dtype=torch.int32)
        return (k.double().view(s["k_pages"].shape), v.double().view(s["v_pages"].shape),
                acc.view_as(s["acc"]), after.view(s["lens"].shape))

    t, w, first = case["budget"], case["window"], case["sinks"]
    acc_out = s["acc_out"].double().flatten()
    src_all = torch.full((units, t), -1, dtype=torch.int32)
    for u in range(units):
        n = lens[u]
        r = rows_of(u, 0, n)
        weight = s["acc"].flatten()[r].double()
        if n <= t:
            src = list(range(n))
        else:
            vals = weight.cpu().numpy()
            inner = sorted(range(first, n - w), key=lambda j: (-vals[j], j))[:t - w - first]
            keep = set(range(first)) | set(inner)
            spare = iter(sorted(j for j in keep if j >= t - w))
            src = [j if j in keep else next(spare) for j in range(t - w)] + list(range(n - w, n))
        frm = r[torch.tensor(src, dtype=torch.long, device="cuda")] if src else r[:0]
        to = r[:len(src)]
        k[to], v[to] = s["k_pages"].view(-1, d)[frm], s["v_pages"].view(-1, d)[frm]
        acc_out[to] = s["acc"].flatten()[frm].double()
        src_all[u, :len(src)] = torch.tensor(src, dtype=torch.int32)
    after = torch.tensor([min(n, t) for n in lens], dtype=torch.int32)
    return (k.double().view(s["k_pages"].shape), v.double().view(s["v_pages"].shape),
            acc_out.view_as(s["acc_out"]), after.view(s["lens"].shape), src_all.view(s["src"].shape))
