"""Prefill KV-cache token eviction (S1 * S2 scores) on NVIDIA B200: Python binding.

A thin layer over the C-ABI library ``libkvp.so`` (declared in ``include/kvp.h``): ctypes, and
for the paged cache's calls, which a decode makes for every token, ``_kvp_binding.so``. It only
marshals arguments: every step of the path - the split-L
log-sum-exp pass, the scoring pass, the selection and the compaction - runs in the
library's CUDA kernels. PyTorch provides device memory and streams.

The functions carry the C names:

* ``kvp_workspace_bytes(shape)``
* ``kvp_score(shape, q_win, k, v, score, s1=None, s2=None, workspace=None, stream=None)``
* ``kvp_select(shape, score, idx, workspace=None, stream=None)``
* ``kvp_select_policy(shape, policy, s1, s2, idx, stream=None)``
* ``kvp_leverage(shape, k, v, g, score, workspace=None, stream=None)``
* ``kvp_select_adaptive(shape, alpha, score, idx, counts, workspace=None, stream=None)``
* ``kvp_compact_ragged(shape, k, v, idx, counts, k_out, v_out, stream=None)``
* ``kvp_compact(shape, k, v, idx, k_out, v_out, stream=None)``
* ``kvp_workspace_status(workspace, stream=None)``
* ``kvp_cache_append(shape, k_new, v_new, k_pages, v_pages, table, lens, lens_out, acc=None, weight=None,
  counts=None, stream=None)``
* ``kvp_cache_attend(shape, q, k_pages, v_pages, table, lens, out, lse=None, acc=None, workspace=None,
  stream=None)``
* ``kvp_cache_evict(shape, evict, k_pages, v_pages, acc, acc_out, table, lens, lens_out, src=None,
  budgets=None, workspace=None, stream=None)``
* ``kvp_status_string(status)``

plus ``evict_layer``, which allocates the outputs and runs the first three calls, and
``LayerCache``, the paged cache that a decode reads: it takes what ``evict_layer`` kept, appends
and attends token by token, and keeps to a budget.

There is no fallback: if ``libkvp.so`` is missing or cannot be loaded, importing this package
raises; without ``_kvp_binding.so`` (or with a library that lacks them) the paged cache's calls do.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# KVP_LIBRARY may point at another build of the same library (e.g. one compiled with
# device-side bounds checks); the default is the in-tree build.
LIB_PATH = os.environ.get("KVP_LIBRARY", os.path.join(_HERE, "libkvp.so"))

KVP_OK = 0
STATUS_NAMES = {0: "KVP_OK", 1: "KVP_ERR_NULL", 2: "KVP_ERR_SHAPE", 3: "KVP_ERR_ALIGN",
                4: "KVP_ERR_WORKSPACE", 5: "KVP_ERR_CUDA", 6: "KVP_ERR_TIMEOUT"}


class KvpShape(ctypes.Structure):
    """Mirror of ``kvp_shape``: budget counts every kept position, window included."""
    _fields_ = [("batch", ctypes.c_int32), ("hq", ctypes.c_int32), ("hkv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("seq_len", ctypes.c_int32),
                ("window", ctypes.c_int32), ("budget", ctypes.c_int32)]

    def __repr__(self):
        return ("KvpShape(batch=%d, hq=%d, hkv=%d, head_dim=%d, seq_len=%d, window=%d, budget=%d)"
                % (self.batch, self.hq, self.hkv, self.head_dim, self.seq_len, self.window, self.budget))


RANK_PRODUCT, RANK_S1, RANK_S2 = 0, 1, 2


class KvpPolicy(ctypes.Structure):
    """Mirror of ``kvp_policy``: sinks always kept, S1 max-pooling kernel, ranking mode."""
    _fields_ = [("sinks", ctypes.c_int32), ("pool_kernel", ctypes.c_int32), ("mode", ctypes.c_int32)]


def make_policy(sinks=0, pool_kernel=1, mode=RANK_PRODUCT) -> KvpPolicy:
    return KvpPolicy(int(sinks), int(pool_kernel), int(mode))


class KvpCacheShape(ctypes.Structure):
    """Mirror of ``kvp_cache_shape``: a paged cache and the query heads that read it."""
    _fields_ = [("batch", ctypes.c_int32), ("hq", ctypes.c_int32), ("hkv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("dtype", ctypes.c_int32)]

    def __repr__(self):
        return "KvpCacheShape(%s)" % ", ".join("%s=%d" % (n, getattr(self, n)) for n, _ in self._fields_)


_DTYPES = (torch.bfloat16, torch.float16)     # by kvp_dtype


def make_cache_shape(batch, hq, hkv, head_dim, page_size, num_pages, max_pages,
                     dtype=torch.bfloat16) -> KvpCacheShape:
    if dtype not in _DTYPES:
        raise ValueError(f"a cache is torch.bfloat16 or torch.float16, got {dtype}")
    return KvpCacheShape(int(batch), int(hq), int(hkv), int(head_dim), int(page_size), int(num_pages),
                         int(max_pages), _DTYPES.index(dtype))


class KvpEvict(ctypes.Structure):
    """Mirror of ``kvp_evict``: rows a head keeps, the first and the last that always stay."""
    _fields_ = [("budget", ctypes.c_int32), ("sinks", ctypes.c_int32), ("window", ctypes.c_int32)]


def make_evict(budget, sinks=0, window=0) -> KvpEvict:
    return KvpEvict(int(budget), int(sinks), int(window))


class KvpError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = f"{what}: {kvp_status_string(status)}"
        if status == 5:
            msg += f" ({kvp_last_cuda_error()})"
        super().__init__(msg)


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python token_eviction_b200/build.py` "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(LIB_PATH)
    P, S = ctypes.c_void_p, ctypes.POINTER(KvpShape)
    lib.kvp_workspace_bytes.argtypes = [S]
    lib.kvp_workspace_bytes.restype = ctypes.c_size_t
    lib.kvp_score.argtypes = [S, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.kvp_score.restype = ctypes.c_int
    lib.kvp_select.argtypes = [S, P, P, P, ctypes.c_size_t, P]
    lib.kvp_select.restype = ctypes.c_int
    lib.kvp_select_policy.argtypes = [S, ctypes.POINTER(KvpPolicy), P, P, P, P]
    lib.kvp_select_policy.restype = ctypes.c_int
    lib.kvp_leverage.argtypes = [S, P, P, P, ctypes.c_int32, P, P, ctypes.c_size_t, P]
    lib.kvp_leverage.restype = ctypes.c_int
    lib.kvp_adaptive_workspace_bytes.argtypes = [S]
    lib.kvp_adaptive_workspace_bytes.restype = ctypes.c_size_t
    lib.kvp_select_adaptive.argtypes = [S, ctypes.c_float, P, P, P, P, ctypes.c_size_t, P]
    lib.kvp_select_adaptive.restype = ctypes.c_int
    lib.kvp_compact_ragged.argtypes = [S, P, P, P, P, P, P, P]
    lib.kvp_compact_ragged.restype = ctypes.c_int
    lib.kvp_compact.argtypes = [S, P, P, P, P, P, P]
    lib.kvp_compact.restype = ctypes.c_int
    lib.kvp_status_string.argtypes = [ctypes.c_int]
    lib.kvp_status_string.restype = ctypes.c_char_p
    lib.kvp_last_cuda_error.argtypes = []
    lib.kvp_last_cuda_error.restype = ctypes.c_char_p
    lib.kvp_workspace_status.argtypes = [P, P]
    lib.kvp_workspace_status.restype = ctypes.c_int
    lib.kvp_score_static.argtypes = [S, P, P, P, P, P, P, P]
    lib.kvp_score_static.restype = ctypes.c_int
    lib.kvp_score_static_status.argtypes = [P]
    lib.kvp_score_static_status.restype = ctypes.c_int
    return lib


class _Missing:
    """Stands for a part that cannot be loaded: whoever uses it is told why."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(f"the paged cache's calls: {self._why}: build it with "
                          "`python token_eviction_b200/build.py` (there is no fallback implementation)")


def _load_cache(lib):
    """The library as the paged cache's calls use it, and their entry. Where either is missing (a library
    from before them, a binding built for another torch), prefill eviction works without."""
    P = ctypes.c_void_p
    C, E = ctypes.POINTER(KvpCacheShape), ctypes.POINTER(KvpEvict)
    try:
        lib.kvp_cache_append.argtypes = [C, P, P, ctypes.c_int32, P, P, P, P, P, P, P, P, P]
        lib.kvp_cache_append.restype = ctypes.c_int
        lib.kvp_cache_attend_workspace_bytes.argtypes = [C, ctypes.c_int32]
        lib.kvp_cache_attend_workspace_bytes.restype = ctypes.c_size_t
        lib.kvp_cache_attend.argtypes = [C, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        lib.kvp_cache_attend.restype = ctypes.c_int
        lib.kvp_cache_evict_workspace_bytes.argtypes = [C, E]
        lib.kvp_cache_evict_workspace_bytes.restype = ctypes.c_size_t
        lib.kvp_cache_evict.argtypes = [C, E, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        lib.kvp_cache_evict.restype = ctypes.c_int
    except AttributeError as e:
        missing = _Missing(f"{LIB_PATH} does not have them ({e})")
        return missing, missing
    try:
        from . import _kvp_binding as binding
    except ImportError as e:
        return lib, _Missing(f"_kvp_binding.so cannot be loaded ({e})")
    binding.use(*(ctypes.cast(f, P).value for f in (lib.kvp_cache_append, lib.kvp_cache_attend, lib.kvp_cache_evict)))
    return lib, binding


_lib = _load()
_cache_lib, _kvp_binding = _load_cache(_lib)

# Kernel launches one layer's kvp_score + kvp_select + kvp_compact makes: the fused
# scoring kernel (both passes over K), the selection and the gather. kvp_score also
# enqueues one small memset of its workspace counters.
KERNELS_PER_LAYER = 3

EXPORTED = ("kvp_workspace_bytes", "kvp_score", "kvp_select", "kvp_select_policy", "kvp_leverage",
            "kvp_adaptive_workspace_bytes", "kvp_select_adaptive", "kvp_compact_ragged", "kvp_compact",
            "kvp_workspace_status", "kvp_cache_append", "kvp_cache_attend_workspace_bytes", "kvp_cache_attend",
            "kvp_cache_evict_workspace_bytes", "kvp_cache_evict",
            "kvp_score_static", "kvp_score_static_status", "kvp_status_string", "kvp_last_cuda_error")


def make_shape(batch, hq, hkv, head_dim, seq_len, window, budget) -> KvpShape:
    return KvpShape(int(batch), int(hq), int(hkv), int(head_dim), int(seq_len), int(window),
                    int(budget))


def _as_shape(shape) -> KvpShape:
    if isinstance(shape, KvpShape):
        return shape
    if isinstance(shape, dict):
        return make_shape(**shape)
    return make_shape(*shape)


def kvp_status_string(status: int) -> str:
    return _lib.kvp_status_string(int(status)).decode()


def kvp_last_cuda_error() -> str:
    return _lib.kvp_last_cuda_error().decode()


def kvp_workspace_bytes(shape) -> int:
    return int(_lib.kvp_workspace_bytes(ctypes.byref(_as_shape(shape))))


def _ptr(t, name, dtype, shape=None, optional=False):
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _current(stream, device):
    """`stream`, as the calls take it, made current for as long as the result is entered. What a call
    allocates for itself is allocated in it: the caching allocator then hands out no block that work
    on another stream still uses, and reuses the block behind the call's own work."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        # (0 and 1 are the default stream's handles, not those of a stream made elsewhere)
        stream = (torch.cuda.default_stream(device) if int(stream) in (0, 1)
                  else torch.cuda.ExternalStream(int(stream), device=device))
    return torch.cuda.stream(stream)


def workspace_for(shape, device=None) -> torch.Tensor:
    n = kvp_workspace_bytes(shape)
    if n == 0:
        raise KvpError(2, "kvp_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def kvp_score(shape, q_win, k, v, score, s1=None, s2=None, workspace=None, stream=None):
    sh = _as_shape(shape)
    b, hq, hkv, d, L, w = sh.batch, sh.hq, sh.hkv, sh.head_dim, sh.seq_len, sh.window
    args = (_ptr(q_win, "q_win", torch.bfloat16, (b, hq, w, d)),
            _ptr(k, "k", torch.bfloat16, (b, hkv, L, d)),
            _ptr(v, "v", torch.bfloat16, (b, hkv, L, d)),
            _ptr(score, "score", torch.float32, (b, hkv, L)),
            _ptr(s1, "s1", torch.float32, (b, hkv, L), optional=True),
            _ptr(s2, "s2", torch.float32, (b, hkv, L), optional=True))
    if workspace is None:
        with _current(stream, k.device):
            workspace = workspace_for(sh, k.device)
    st = _lib.kvp_score(ctypes.byref(sh), *args, workspace.data_ptr(), workspace.numel(),
                        _stream(stream))
    if st != KVP_OK:
        raise KvpError(st, "kvp_score")


def kvp_workspace_status(workspace, stream=None) -> int:
    """Device-side status of the last kvp_score on `workspace`: KVP_OK (0) or
    KVP_ERR_TIMEOUT (6) when one of its bounded waits gave up. Synchronises the stream."""
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda:
        raise ValueError("workspace must be a CUDA tensor")
    return int(_lib.kvp_workspace_status(workspace.data_ptr(), _stream(stream)))


def kvp_select(shape, score, idx, workspace=None, stream=None):
    sh = _as_shape(shape)
    b, hkv, L, B = sh.batch, sh.hkv, sh.seq_len, sh.budget
    ps = _ptr(score, "score", torch.float32, (b, hkv, L))
    pi = _ptr(idx, "idx", torch.int32, (b, hkv, B))
    if workspace is None:
        with _current(stream, score.device):
            workspace = workspace_for(sh, score.device)
    st = _lib.kvp_select(ctypes.byref(sh), ps, pi, workspace.data_ptr(), workspace.numel(),
                         _stream(stream))
    if st != KVP_OK:
        raise KvpError(st, "kvp_select")


def kvp_select_policy(shape, policy, s1, s2, idx, stream=None):
    """Kept positions under `policy` (a KvpPolicy, or a dict of make_policy's arguments):
    sinks, then the best candidates by the policy's key, then the window; ascending."""
    sh = _as_shape(shape)
    pol = policy if isinstance(policy, KvpPolicy) else make_policy(**policy)
    b, hkv, L, B = sh.batch, sh.hkv, sh.seq_len, sh.budget
    p1 = _ptr(s1, "s1", torch.float32, (b, hkv, L), optional=pol.mode == RANK_S2)
    p2 = _ptr(s2, "s2", torch.float32, (b, hkv, L), optional=pol.mode == RANK_S1)
    pi = _ptr(idx, "idx", torch.int32, (b, hkv, B))
    st = _lib.kvp_select_policy(ctypes.byref(sh), ctypes.byref(pol), p1, p2, pi, _stream(stream))
    if st != KVP_OK:
        raise KvpError(st, "kvp_select_policy")


def kvp_leverage(shape, k, v, g, score, workspace=None, stream=None):
    """CurDKV leverage scores of every position: squared row norms of K G and V G, their
    product, normalised per KV head. g: [d, r] bf16 CUDA tensor, 1 <= r <= 32."""
    sh = _as_shape(shape)
    b, hkv, d, L = sh.batch, sh.hkv, sh.head_dim, sh.seq_len
    if not isinstance(g, torch.Tensor) or g.dim() != 2 or g.shape[0] != d:
        raise ValueError(f"g must be a [{d}, r] tensor")
    args = (_ptr(k, "k", torch.bfloat16, (b, hkv, L, d)),
            _ptr(v, "v", torch.bfloat16, (b, hkv, L, d)),
            _ptr(g, "g", torch.bfloat16, tuple(g.shape)))
    ps = _ptr(score, "score", torch.float32, (b, hkv, L))
    if workspace is None:
        with _current(stream, k.device):
            workspace = workspace_for(sh, k.device)
    st = _lib.kvp_leverage(ctypes.byref(sh), *args, int(g.shape[1]), ps, workspace.data_ptr(),
                           workspace.numel(), _stream(stream))
    if st != KVP_OK:
        raise KvpError(st, "kvp_leverage")


def adaptive_workspace_for(shape, device=None) -> torch.Tensor:
    n = int(_lib.kvp_adaptive_workspace_bytes(ctypes.byref(_as_shape(shape))))
    if n == 0:
        raise KvpError(2, "kvp_adaptive_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def kvp_select_adaptive(shape, alpha, score, idx, counts, workspace=None, stream=None):
    """Adaptive per-head budgets (AdaKV with safeguard alpha): idx [b, hkv * B] packed
    head after head, counts [b, hkv]."""
    sh = _as_shape(shape)
    b, hkv, L, B = sh.batch, sh.hkv, sh.seq_len, sh.budget
    ps = _ptr(score, "score", torch.float32, (b, hkv, L))
    pi = _ptr(idx, "idx", torch.int32, (b, hkv * B))
    pc = _ptr(counts, "counts", torch.int32, (b, hkv))
    if workspace is None:
        with _current(stream, score.device):
            workspace = adaptive_workspace_for(sh, score.device)
    st = _lib.kvp_select_adaptive(ctypes.byref(sh), float(alpha), ps, pi, pc, workspace.data_ptr(),
                                  workspace.numel(), _stream(stream))
    if st != KVP_OK:
        raise KvpError(st, "kvp_select_adaptive")


def kvp_compact_ragged(shape, k, v, idx, counts, k_out, v_out, stream=None):
    sh = _as_shape(shape)
    b, hkv, d, L, B = sh.batch, sh.hkv, sh.head_dim, sh.seq_len, sh.budget
    args = (_ptr(k, "k", torch.bfloat16, (b, hkv, L, d)),
            _ptr(v, "v", torch.bfloat16, (b, hkv, L, d)),
            _ptr(idx, "idx", torch.int32, (b, hkv * B)),
            _ptr(counts, "counts", torch.int32, (b, hkv)),
            _ptr(k_out, "k_out", torch.bfloat16, (b, hkv * B, d)),
            _ptr(v_out, "v_out", torch.bfloat16, (b, hkv * B, d)))
    st = _lib.kvp_compact_ragged(ctypes.byref(sh), *args, _stream(stream))
    if st != KVP_OK:
        raise KvpError(st, "kvp_compact_ragged")


def kvp_compact(shape, k, v, idx, k_out, v_out, stream=None):
    sh = _as_shape(shape)
    b, hkv, d, L, B = sh.batch, sh.hkv, sh.head_dim, sh.seq_len, sh.budget
    args = (_ptr(k, "k", torch.bfloat16, (b, hkv, L, d)),
            _ptr(v, "v", torch.bfloat16, (b, hkv, L, d)),
            _ptr(idx, "idx", torch.int32, (b, hkv, B)),
            _ptr(k_out, "k_out", torch.bfloat16, (b, hkv, B, d)),
            _ptr(v_out, "v_out", torch.bfloat16, (b, hkv, B, d)))
    st = _lib.kvp_compact(ctypes.byref(sh), *args, _stream(stream))
    if st != KVP_OK:
        raise KvpError(st, "kvp_compact")


class LayerBuffers:
    """Device outputs and workspace of one layer's eviction, reusable across calls."""

    def __init__(self, shape, device="cuda", want_s1_s2=False):
        sh = _as_shape(shape)
        self.shape = sh
        b, hkv, d, L, B = sh.batch, sh.hkv, sh.head_dim, sh.seq_len, sh.budget
        self.score = torch.empty((b, hkv, L), dtype=torch.float32, device=device)
        self.s1 = torch.empty_like(self.score) if want_s1_s2 else None
        self.s2 = torch.empty_like(self.score) if want_s1_s2 else None
        self.idx = torch.empty((b, hkv, B), dtype=torch.int32, device=device)
        self.k_out = torch.empty((b, hkv, B, d), dtype=torch.bfloat16, device=device)
        self.v_out = torch.empty_like(self.k_out)
        self.workspace = workspace_for(sh, device)


def evict_layer(q_win, k, v, window: int, budget: int, buffers: LayerBuffers | None = None,
                stream=None):
    """Score, select and compact one layer; returns the LayerBuffers holding the results.

    q_win [b, hq, w, d], k and v [b, hkv, L, d]: bf16 CUDA tensors. Buffers that are not given are
    allocated on `stream`: they are that stream's memory, as if it had been the current one.
    """
    b, hq, w, d = q_win.shape
    _, hkv, L, _ = k.shape
    if w != window:
        raise ValueError("q_win must hold exactly `window` queries per head")
    sh = make_shape(b, hq, hkv, d, L, window, budget)
    if buffers is None:
        with _current(stream, k.device):
            buffers = LayerBuffers(sh, k.device)
    kvp_score(sh, q_win, k, v, buffers.score, buffers.s1, buffers.s2, buffers.workspace, stream)
    kvp_select(sh, buffers.score, buffers.idx, buffers.workspace, stream)
    kvp_compact(sh, k, v, buffers.idx, buffers.k_out, buffers.v_out, stream)
    return buffers


# ---- the paged cache


def _device_of(t):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("a paged cache's tensors must be CUDA tensors")
    return t.device


def _cache_workspace(nbytes, what, device):
    if nbytes == 0:
        raise KvpError(2, what)
    return torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")


def _structure(x, kind):
    if not isinstance(x, kind):
        raise ValueError(f"{type(x).__name__} where a {kind.__name__} is wanted")
    return x


def attend_workspace_for(shape, accumulate=False, device=None) -> torch.Tensor:
    _structure(shape, KvpCacheShape)
    n = int(_cache_lib.kvp_cache_attend_workspace_bytes(ctypes.byref(shape), int(bool(accumulate))))
    return _cache_workspace(n, "kvp_cache_attend_workspace_bytes", device)


def evict_workspace_for(shape, evict, device=None) -> torch.Tensor:
    _structure(shape, KvpCacheShape), _structure(evict, KvpEvict)
    n = int(_cache_lib.kvp_cache_evict_workspace_bytes(ctypes.byref(shape), ctypes.byref(evict)))
    return _cache_workspace(n, "kvp_cache_evict_workspace_bytes", device)


def kvp_cache_append(shape, k_new, v_new, k_pages, v_pages, table, lens, lens_out, acc=None, weight=None,
                     counts=None, stream=None):
    """Appends n rows per head: k_new and v_new [b, hkv, n, d], or packed head after head
    [b, hkv * n, d] with counts [b, hkv]. weight: the rows' first accumulated weights, shaped
    like k_new without its last dimension. lens_out may be lens."""
    st = _kvp_binding.append(shape, k_new, v_new, k_pages, v_pages, table, lens, lens_out, acc, weight, counts,
                             stream)
    if st != KVP_OK:
        raise KvpError(st, "kvp_cache_append")


def kvp_cache_attend(shape, q, k_pages, v_pages, table, lens, out, lse=None, acc=None, workspace=None,
                     stream=None):
    """Attention of one token q [b, hq, d] over the cache; acc gains each row's weights."""
    if workspace is None:
        with _current(stream, _device_of(q)):
            workspace = attend_workspace_for(shape, acc is not None, q.device)
    st = _kvp_binding.attend(shape, q, k_pages, v_pages, table, lens, out, lse, acc, workspace, stream)
    if st != KVP_OK:
        raise KvpError(st, "kvp_cache_attend")


def kvp_cache_evict(shape, evict, k_pages, v_pages, acc, acc_out, table, lens, lens_out, src=None,
                    budgets=None, workspace=None, stream=None):
    """Each head keeps its first `sinks` rows, its last `window` and the heaviest between them, up to
    its budget (a KvpEvict, or a dict of make_evict's arguments). In place; acc_out may be acc
    and lens_out lens."""
    ev = make_evict(**evict) if isinstance(evict, dict) else _structure(evict, KvpEvict)
    if workspace is None:
        with _current(stream, _device_of(k_pages)):
            workspace = evict_workspace_for(shape, ev, k_pages.device)
    st = _kvp_binding.evict(shape, ev, k_pages, v_pages, acc, acc_out, table, lens, lens_out, src, budgets,
                            workspace, stream)
    if st != KVP_OK:
        raise KvpError(st, "kvp_cache_evict")


class LayerCache:
    """One layer's paged cache through a decode: filled with the rows an eviction kept, then a token at
    a time appended, attended over and, where a budget is given, evicted by accumulated weight.

    Holds up to `capacity` rows per KV head, rounded up to whole pages, in pages of its own (table, pools
    and shape may be replaced by a program that shares a pool between layers or requests). Rows that no
    longer fit are dropped and attention goes on without them: a head whose `lens` stands at
    max_pages * page_size is full. `evict`: a KvpEvict; heads over its budget are cut back in every step, so capacity must exceed the budget.
    `budgets` [batch, hkv] int32: each head's own budget, up to evict's (the counts of
    kvp_select_adaptive, say, whose rows append(counts=) takes: without it every head that was
    given more rows than evict's budget is cut back to that, and the others grow up to it).
    """

    def __init__(self, batch, hq, hkv, head_dim, capacity, page_size=64, evict: KvpEvict | None = None,
                 dtype=torch.bfloat16, device="cuda", budgets=None):
        width = -(-capacity // page_size)
        if evict is None and budgets is not None:
            raise ValueError("budgets per head need an eviction policy: evict=make_evict(...)")
        if evict is not None and width * page_size <= evict.budget:
            raise ValueError("capacity must exceed the eviction's budget: a step appends before it evicts")
        self.shape = make_cache_shape(batch, hq, hkv, head_dim, page_size, batch * hkv * width, width, dtype)
        self.evict_policy, self.budgets = evict, budgets
        new = lambda shape, dt: torch.zeros(shape, dtype=dt, device=device)
        self.k_pages = new((self.shape.num_pages, page_size, head_dim), dtype)
        self.v_pages = torch.zeros_like(self.k_pages)
        self.table = torch.arange(self.shape.num_pages, dtype=torch.int32, device=device).view(batch, hkv, width)
        self.lens = new((batch, hkv), torch.int32)
        self.acc = new((self.shape.num_pages, page_size), torch.float32) if evict is not None else None
        self.out = new((batch, hq, head_dim), dtype)
        self.lse = new((batch, hq), torch.float32)
        self.workspace = attend_workspace_for(self.shape, evict is not None, device)
        self.evict_workspace = evict_workspace_for(self.shape, evict, device) if evict is not None else None

    def append(self, k_new, v_new, weight=None, counts=None, stream=None):
        """Rows behind those that each head holds: [b, hkv, n, d], or [b, hkv * n, d] with counts."""
        kvp_cache_append(self.shape, k_new, v_new, self.k_pages, self.v_pages, self.table, self.lens,
                         self.lens, self.acc, weight, counts, stream)

    def attend(self, q, stream=None) -> torch.Tensor:
        """Attention of q [b, hq, d] over the rows held; returns self.out (self.lse beside it)."""
        kvp_cache_attend(self.shape, q, self.k_pages, self.v_pages, self.table, self.lens, self.out,
                         self.lse, self.acc, self.workspace, stream)
        return self.out

    def evict(self, stream=None):
        """Cuts every head that is over the budget back to it."""
        if self.evict_policy is None:
            raise ValueError("this cache was made without an eviction policy: evict=make_evict(...)")
        kvp_cache_evict(self.shape, self.evict_policy, self.k_pages, self.v_pages, self.acc, self.acc,
                        self.table, self.lens, self.lens, None, self.budgets, self.evict_workspace, stream)

    def step(self, q, k_new, v_new, stream=None) -> torch.Tensor:
        """One decoded token: its key and value [b, hkv, 1, d] join the cache, q attends, and the cache is
        cut back to its budget."""
        self.append(k_new, v_new, stream=stream)
        out = self.attend(q, stream)
        if self.evict_policy is not None:
            self.evict(stream)
        return out
