"""A quantized key/value cache with the attention that reads it, and log
probabilities of tokens: the steps of a serving loop between the projections
and after the lm_head (C signatures and semantics in ``include/qmv.h``).

  KVCache                the pages of a cache, and what they hold
  cache_page_bytes       bytes of one page of keys or of values
  qmv_cache_write        quantizes new keys and values into slots
  qmv_cache_read         the values of slots
  qmv_cache_attention    attention of new tokens over the cache
  qmv_logprobs           log probabilities, entropy and most probable tokens

The names are attributes of the package as well.  Streams, outputs and
workspaces are as for the package's other entry points.
"""
import ctypes
import math
from collections import namedtuple

import bandwidth_bound_block_amd as _pkg

__all__ = ["KVCache", "cache_page_bytes", "qmv_cache_write", "qmv_cache_read", "qmv_cache_attention", "qmv_logprobs",
           "Logprobs"]

Logprobs = namedtuple("Logprobs", "logprobs entropy top_tokens top_logprobs")


class CacheStruct(ctypes.Structure):
    """qmv_cache of include/qmv.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("k_fmt", ctypes.c_int32),
                ("v_fmt", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def bind(L):
    """Argument types of the entry points."""
    P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    C = ctypes.POINTER(CacheStruct)
    L.qmv_cache_page_bytes.argtypes = [ctypes.c_int, i32, i32, i32]
    L.qmv_cache_attention_workspace_bytes.argtypes = [C, i64, i64, i32, i64]
    L.qmv_logprobs_workspace_bytes.argtypes = [i64, i64, i32]
    for name in ("qmv_cache_page_bytes", "qmv_cache_attention_workspace_bytes", "qmv_logprobs_workspace_bytes"):
        getattr(L, name).restype = sz
    L.qmv_cache_write.argtypes = [C, P, i64, i64, P, i64, i64, i32, P, i64, P]
    L.qmv_cache_read.argtypes = [C, P, i64, P, P, i32, P]
    L.qmv_cache_attention.argtypes = [C, P, i32, i64, i64, i64, i32, P, i64, P, P, i64, i64, ctypes.c_float, i32, P, P, P, sz, P]
    L.qmv_logprobs.argtypes = [P, i32, i64, i64, i64, P, i32, P, P, i32, P, P, P, sz, P]
    for name in ("qmv_cache_write", "qmv_cache_read", "qmv_cache_attention", "qmv_logprobs"):
        getattr(L, name).restype = i32


def cache_page_bytes(fmt, n_kv_heads, head_dim, page_size):
    """Bytes of one page of keys (or of values) in format fmt."""
    n = _pkg._lib.qmv_cache_page_bytes(_pkg._fmt(fmt), n_kv_heads, head_dim, page_size)
    if n == 0:
        raise ValueError("a cache has Q8_0, Q4_0 or Q4_1 pages of 16..4096 tokens (a power of two), heads of 64, 128 or 256")
    return n


class KVCache:
    """The pages of a cache: uint8 GPU tensors k and v of whole pages, their
    formats, and the sizes that make a page.  The memory is the caller's and
    may hold anything where no token was written.  The attributes are fixed."""
    __slots__ = ("k", "v", "k_fmt", "v_fmt", "n_kv_heads", "head_dim", "page_size", "n_pages", "_struct")

    def __init__(self, k, v, k_fmt, v_fmt, n_kv_heads, head_dim, page_size):
        kb, vb = (cache_page_bytes(f, n_kv_heads, head_dim, page_size) for f in (k_fmt, v_fmt))
        n = getattr(k, "numel", lambda: 0)() // kb
        kp, vp = _pkg._bytes_of(k, "k", n * kb), _pkg._bytes_of(v, "v", n * vb)
        if n < 1 or k.numel() != n * kb or v.numel() != n * vb:
            raise ValueError(f"k and v must hold the same number of whole pages, {kb} and {vb} bytes each")
        if k.get_device() != v.get_device():
            raise ValueError("k and v must be on one GPU")
        self.k, self.v, self.k_fmt, self.v_fmt = k, v, _pkg._fmt(k_fmt), _pkg._fmt(v_fmt)
        self.n_kv_heads, self.head_dim, self.page_size, self.n_pages = n_kv_heads, head_dim, page_size, n
        self._struct = CacheStruct(kp, vp, n, self.k_fmt, self.v_fmt, n_kv_heads, head_dim, page_size, 0)

    def __setattr__(self, name, value):
        if hasattr(self, "_struct"):      # set last: it has the pages' addresses
            raise AttributeError("a cache's pages and sizes are fixed")
        object.__setattr__(self, name, value)

    @classmethod
    def new(cls, n_pages, k_fmt, v_fmt, n_kv_heads, head_dim, page_size, device="cuda"):
        """A cache of n_pages pages in new memory."""
        torch = _pkg._torch()
        k, v = (torch.empty(n_pages * cache_page_bytes(f, n_kv_heads, head_dim, page_size), dtype=torch.uint8, device=device)
                for f in (k_fmt, v_fmt))
        return cls(k, v, k_fmt, v_fmt, n_kv_heads, head_dim, page_size)


def _one_gpu(like, **tensors):
    """All of a call's tensors are on like's GPU: a pointer of another one is not checked by the library."""
    at = like.get_device()
    for name, t in tensors.items():
        if t is not None and t.get_device() != at:
            raise ValueError(f"{name} must be on the same GPU as the others")


def _run(like, f, *args):
    """A library call on like's GPU, whichever is current: a launch goes to the current one."""
    torch = _pkg._torch()
    if like.get_device() == torch.cuda.current_device():
        _pkg._check(f(*args))
    else:
        with torch.cuda.device(like.get_device()):
            _pkg._check(f(*args))


def _heads(t, name, heads, dim):
    """Strides of a [tokens, heads, dim] tensor with unit inner stride."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim or t.stride(2) != 1:
        raise ValueError(f"{name} must be [tokens, {heads}, {dim}] with unit inner stride")
    return t.stride(0), t.stride(1)


def _ints(t, name):
    """Address of a contiguous one-dimensional int32 GPU tensor."""
    if getattr(t, "dim", lambda: 0)() != 1:
        raise ValueError(f"{name} must be a one-dimensional int32 GPU tensor")
    return _pkg._full(t, name, _pkg._torch().int32, t.shape)


def qmv_cache_write(cache, k, v, slots, stream=None):
    """Quantizes keys and values, float32, float16 or bfloat16 [tokens,
    kv_heads, head_dim], into the cache's slots (int32 [tokens]; a slot is
    page * page_size + place; one out of range is left out)."""
    xt = _pkg._type_of(k, "k")
    if _pkg._type_of(v, "v") != xt:
        raise ValueError("k and v must have one type")
    kt, kh = _heads(k, "k", cache.n_kv_heads, cache.head_dim)
    vt, vh = _heads(v, "v", cache.n_kv_heads, cache.head_dim)
    T = k.shape[0]
    s = _ints(slots, "slots")
    if v.shape[0] != T or slots.shape[0] != T:
        raise ValueError("k, v and slots must have as many tokens")
    _one_gpu(cache.k, k=k, v=v, slots=slots)
    _run(k, _pkg._lib.qmv_cache_write, cache._struct, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, xt, s, T, _pkg._on(stream, k))


def qmv_cache_read(cache, slots, dtype=None, k=None, v=None, stream=None):
    """The values of the cache's slots (int32 [tokens]): (k, v), each [tokens,
    kv_heads, head_dim] of dtype (float32 by default) or into given tensors."""
    torch = _pkg._torch()
    s = _ints(slots, "slots")
    shape = (slots.shape[0], cache.n_kv_heads, cache.head_dim)
    if dtype is None:
        dtype = k.dtype if k is not None else v.dtype if v is not None else torch.float32
    k, v = (_pkg._new(shape, dtype, slots, stream) if t is None else t for t in (k, v))
    ot = _pkg._type_of(k, "k")
    kp, vp = _pkg._full(k, "k", dtype, shape), _pkg._full(v, "v", dtype, shape)
    _one_gpu(cache.k, slots=slots, k=k, v=v)
    _run(k, _pkg._lib.qmv_cache_read, cache._struct, s, shape[0], kp, vp, ot, _pkg._on(stream, slots))
    return k, v


def qmv_cache_attention(cache, q, page_table, kv_lens, q_begin=None, max_q=None, scale=None, window=0, sinks=None, out=None,
                        workspace=None, stream=None):
    """Attention of new tokens over the cache (see qmv.h).

    q: float32, float16 or bfloat16 [tokens, heads, head_dim]; page_table
    int32 [requests, max_pages]; kv_lens int32 [requests], the new tokens
    counted in; q_begin int32 [requests + 1]: request r's queries are tokens
    q_begin[r] .. q_begin[r + 1] - 1, of which it may have max_q (an int, the
    most of any request; all tokens by default; those past it are left out).  Without q_begin every
    request has tokens / requests of them.  scale: 1 / sqrt(head_dim) by
    default; window 0: none; sinks float32 [heads] or None.  Returns out
    [tokens, heads, head_dim] of q's type; rows of no request are not
    written."""
    torch = _pkg._torch()
    xt = _pkg._type_of(q, "q")
    heads, D = (q.shape[1], cache.head_dim) if q.dim() == 3 else (0, 0)
    qt, qh = _heads(q, "q", heads, D)
    if getattr(page_table, "dim", lambda: 0)() != 2:
        raise ValueError("page_table must be an int32 [requests, max_pages] GPU tensor")
    R, pages = page_table.shape
    table = _pkg._full(page_table, "page_table", torch.int32, (R, pages))
    lens = _pkg._full(kv_lens, "kv_lens", torch.int32, (R,))
    T = q.shape[0]
    begin = None
    if q_begin is not None:
        begin = _pkg._full(q_begin, "q_begin", torch.int32, (R + 1,))
        max_q = T if max_q is None else max_q
    else:
        if R < 1 or T % R or (max_q is not None and max_q * R != T):
            raise ValueError("without q_begin, every request has tokens / requests (max_q) queries")
        max_q = T // R
    if not 0 <= window < 2 ** 31:
        raise ValueError("window must be 0 (none) .. 2^31 - 1")
    sk = _pkg._full(sinks, "sinks", torch.float32, (heads,)) if sinks is not None else None
    if out is None:
        out = _pkg._new((T, heads, D), q.dtype, q, stream)
    op = _pkg._full(out, "out", q.dtype, (T, heads, D))
    need = _pkg._lib.qmv_cache_attention_workspace_bytes(cache._struct, R, T, heads, max_q)
    ws = _pkg._scratch(workspace, "workspace", need, q, stream)
    _one_gpu(cache.k, q=q, page_table=page_table, kv_lens=kv_lens, q_begin=q_begin, sinks=sinks, out=out, workspace=ws)
    _run(q, _pkg._lib.qmv_cache_attention, cache._struct, q.data_ptr(), xt, qt, qh, T, heads, table, pages, lens, begin, R,
         max_q, 1.0 / math.sqrt(D) if scale is None else scale, window, sk, op, ws.data_ptr(), ws.numel(), _pkg._on(stream, q))
    return out


def qmv_logprobs(logits, targets=None, top_k=0, logprobs=None, entropy=None, top_tokens=None, top_logprobs=None,
                 workspace=None, stream=None):
    """Log probabilities under rows of logits, float32, float16 or bfloat16
    [rows, vocab]: of given tokens (targets int32 [rows] or [rows, n], or
    None), the rows' entropy, and the top_k most probable tokens (see qmv.h).
    Returns Logprobs(logprobs float32 as targets, entropy float32 [rows],
    top_tokens int32 [rows, top_k], top_logprobs float32 [rows, top_k]); what
    was not asked for is None."""
    lt = _pkg._type_of(logits, "logits")
    torch = _pkg._torch()
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be [rows, vocab] with unit inner stride")
    N, V = logits.shape
    if not 0 <= top_k <= 32:
        raise ValueError("top_k must be 0..32")
    i32, f32 = torch.int32, torch.float32
    tp = lp = bt = bl = None
    n = 0
    if targets is not None:
        if targets.dim() not in (1, 2) or targets.shape[0] != N:
            raise ValueError("targets must be [rows] or [rows, n]")
        n = 1 if targets.dim() == 1 else targets.shape[1]
        tp = _pkg._full(targets, "targets", i32, targets.shape)
        if logprobs is None:
            logprobs = _pkg._new(tuple(targets.shape), f32, logits, stream)
        lp = _pkg._full(logprobs, "logprobs", f32, targets.shape)
    elif logprobs is not None:
        raise ValueError("logprobs without targets")
    if entropy is None:
        entropy = _pkg._new((N,), f32, logits, stream)
    ep = _pkg._full(entropy, "entropy", f32, (N,))
    if top_k > 0:
        if top_tokens is None:
            top_tokens = _pkg._new((N, top_k), i32, logits, stream)
        if top_logprobs is None:
            top_logprobs = _pkg._new((N, top_k), f32, logits, stream)
        bt, bl = _pkg._full(top_tokens, "top_tokens", i32, (N, top_k)), _pkg._full(top_logprobs, "top_logprobs", f32, (N, top_k))
    elif top_tokens is not None or top_logprobs is not None:
        raise ValueError("top tokens without top_k")
    ws = _pkg._scratch(workspace, "workspace", _pkg._lib.qmv_logprobs_workspace_bytes(N, V, top_k), logits, stream)
    _one_gpu(logits, targets=targets, logprobs=logprobs, entropy=entropy, top_tokens=top_tokens, top_logprobs=top_logprobs,
             workspace=ws)
    _run(logits, _pkg._lib.qmv_logprobs, logits.data_ptr(), lt, logits.stride(0), N, V, tp, n, lp, ep, top_k, bt, bl,
         ws.data_ptr(), ws.numel(), _pkg._on(stream, logits))
    return Logprobs(logprobs, entropy, top_tokens, top_logprobs)
