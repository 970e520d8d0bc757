"""Plain 64-bit forms of the paged-cache calls (numpy, one head at a time), the bounds that the
kernels' arithmetic keeps, and a cache builder."""
import numpy as np
import torch

F64 = np.float64


def kvp():
    import token_eviction_b200 as m
    return m


class Cache:
    """A pool with shuffled pages, table and lengths; rows past the lengths and unused pages hold
    garbage (NaN by default), so that reading one shows."""

    def __init__(self, seed, b, hq, hkv, d, page, lens, dtype=torch.bfloat16, width=None, garbage=float("nan"),
                 spare=3, outliers=True, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.b, self.hq, self.hkv, self.d, self.page, self.dtype = b, hq, hkv, d, page, dtype
        lens = torch.as_tensor(lens, dtype=torch.int32).reshape(b, hkv)
        self.width = width or max(1, -(-int(lens.max()) // page))
        self.num_pages = b * hkv * self.width + spare
        self.table = torch.randperm(self.num_pages, generator=g)[:b * hkv * self.width].to(torch.int32).view(
            b, hkv, self.width)
        self.lens = lens

        def rows(*shape):
            t = torch.randn(shape, generator=g)
            if outliers:
                t[..., torch.randperm(d, generator=g)[:d // 32]] *= 20
            return t.to(dtype)

        self.k, self.v = rows(self.num_pages, page, d), rows(self.num_pages, page, d)
        self.acc = torch.rand((self.num_pages, page), generator=g) ** 4
        live = torch.zeros((self.num_pages, page), dtype=torch.bool)
        for u in range(b * hkv):
            live.view(-1)[self.rows(u)] = True
        for t in (self.k, self.v, self.acc):
            t[~live] = garbage
        self.live = live
        self.q = rows(b, hq, d)
        self.device = device

    def rows(self, u, n=None):
        """Pool rows of head u's rows [0, n) (default: its length)."""
        n = int(self.lens.view(-1)[u]) if n is None else n
        j = torch.arange(n)
        return self.table.view(-1, self.width)[u, j // self.page].long() * self.page + j % self.page

    @property
    def shape(self):
        return kvp().make_cache_shape(self.b, self.hq, self.hkv, self.d, self.page, self.num_pages, self.width,
                                      self.dtype)

    def gpu(self, *names):
        got = [getattr(self, n).to(self.device).contiguous() for n in names]
        return got[0] if len(got) == 1 else got


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def attend_ref(c, q=None, k=None, v=None, lens=None, present=None):
    """out, lse, weights (a list of [rows, G] per head), and the bounds on each: see `bounds`."""
    q = f64(c.q if q is None else q).reshape(c.b * c.hkv, -1, c.d)
    k, v = f64(c.k if k is None else k).reshape(-1, c.d), f64(c.v if v is None else v).reshape(-1, c.d)
    lens = (c.lens if lens is None else lens).view(-1).tolist()
    G = q.shape[1]
    out = np.zeros((c.b * c.hkv, G, c.d))
    lse = np.full((c.b * c.hkv, G), -np.inf)
    tol_out, tol_lse = np.zeros_like(out), np.zeros_like(lse)
    weights, tol_w = [], []
    for u in range(c.b * c.hkv):
        r = c.rows(u, lens[u]).numpy()
        here = np.ones(len(r), dtype=bool) if present is None else present[u][:len(r)]
        w, tw = np.zeros((len(r), G)), np.zeros((len(r), G))
        kr, vr = k[r[here]], v[r[here]]
        if len(kr):
            t = kr @ q[u].T / np.sqrt(c.d)
            top = t.max(0)
            e = np.exp(t - top)
            s = e.sum(0)
            p = e / s
            out[u], lse[u] = p.T @ vr, top + np.log(s)
            w[here] = p
            rel, d_lse = bounds(c, q[u], kr, lse[u])
            half = torch.finfo(c.dtype).eps / 2
            tol_out[u] = 1.01 * half * np.abs(out[u]) + rel[:, None] * (p.T @ np.abs(vr))
            # a result below the type's smallest normal number is rounded to a fixed step
            tol_out[u] += float(torch.finfo(c.dtype).smallest_normal) * half
            tol_lse[u] = d_lse
            tw[here] = rel * p + 2.0 ** -126
        weights.append(w)
        tol_w.append(tw)
    shape = (c.b, c.hkv * G)
    return (out.reshape(shape + (c.d,)), lse.reshape(shape), weights,
            tol_out.reshape(shape + (c.d,)), tol_lse.reshape(shape), tol_w)


def bounds(c, q, k, lse):
    """Relative error of a weight times its value's share, and absolute error of lse.

    A logit is a sum of d exact products, accumulated in fp32 with at most one unit (2^-23) lost an
    addition, against the sum of the products' magnitudes; scaling it to log2 units rounds
    twice more. A weight 2^(t - m) has the logit's error (natural units), 2^-22 of ex2 and the
    rounding of t - m. A sum over n rows loses at most n / 4 units along one warp's chain (four
    warps share the rows) and a few in the joins. Weights that multiply V: rounded to the type
    (half a step) past 8 query heads, else kept to the square of that."""
    G, n = q.shape[0], len(k)
    half = torch.finfo(c.dtype).eps / 2
    u = 2.0 ** -23
    mag = (np.abs(k) @ np.abs(q).T).max(0) / np.sqrt(c.d)                 # per query head
    d_logit = (c.d + 4) * u * mag
    chain = (n / 4 + 64) * u
    # the spread of the logits, in log2 units, is rounded in t - m
    rel = 2 * d_logit + chain + 2 * u * (2 * mag * 1.45 + 4) + (half if G > 8 else 4 * half * half) + 2 * u
    return rel, d_logit + chain + (np.abs(lse) + 8) * 4 * u


def evict_ref(acc, n, t, s, w):
    """src of one head: acc its rows' weights (fp32), n of them, t its budget."""
    if n <= t:
        return np.arange(n)
    acc = np.asarray(acc[:n], dtype=np.float32)
    key = np.where(acc > 0, acc, np.float32(0))
    inner = np.arange(s, n - w)
    order = inner[np.lexsort((inner, -key[inner].astype(F64)))][:t - s - w]
    keep = np.zeros(n, dtype=bool)
    keep[:s] = True
    keep[order] = True
    low = np.arange(t - w)
    holes = low[~keep[:t - w]]
    high = np.arange(t - w, n)[keep[t - w:]]
    src = low.copy()
    src[holes] = high
    return np.concatenate([src, np.arange(n - w, n)])


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32).numpy()
