"""Argument errors of the cache, its attention and the log probabilities: every call here is refused on the host before
anything is launched (no GPU)."""
import ctypes
import os
import re

import pytest

EINVAL, EALIGN, EUNSUPPORTED = 1, 2, 3
A = 0x10000          # a fake, aligned, never dereferenced device address


@pytest.fixture(scope="module")
def qmv():
    import bandwidth_bound_block_amd as q
    return q


GOOD = dict(k=A, v=A, n_pages=7, k_fmt=1, v_fmt=0, n_kv_heads=2, head_dim=128, page_size=32, reserved=0)
BAD = [(dict(k_fmt=3), EUNSUPPORTED, "format"), (dict(v_fmt=-1), EUNSUPPORTED, "format"), (dict(k=0), EINVAL, "null"),
       (dict(v=0), EINVAL, "null"), (dict(n_kv_heads=0), EINVAL, "n_kv_heads"), (dict(n_kv_heads=1025), EINVAL, "n_kv_heads"),
       (dict(head_dim=96), EINVAL, "head_dim"), (dict(head_dim=0), EINVAL, "head_dim"), (dict(page_size=8), EINVAL, "page_size"),
       (dict(page_size=48), EINVAL, "page_size"), (dict(page_size=8192), EINVAL, "page_size"), (dict(page_size=0), EINVAL, "page_size"),
       (dict(page_size=-16), EINVAL, "page_size"), (dict(n_pages=0), EINVAL, "n_pages"), (dict(n_pages=-1), EINVAL, "n_pages"),
       (dict(n_pages=1 << 26), EINVAL, "n_pages"), (dict(reserved=1), EINVAL, "reserved"), (dict(k=A + 8), EALIGN, "aligned"),
       (dict(v=A + 4), EALIGN, "aligned")]


def cache(qmv, **change):
    return ctypes.byref(qmv.serving.CacheStruct(**{**GOOD, **change}))


def check(qmv, name, good, changes):
    """good: argument names and values in order; changes: (changed arguments, code, word of the message)."""
    f = getattr(qmv.lib(), name)
    for change, code, word in changes:
        args = dict(good)
        assert set(change) <= set(args), change
        args.update(change)
        assert f(*args.values()) == code, (name, change, qmv.last_error())
        assert word in qmv.last_error(), (name, change, qmv.last_error())


def test_entry_points_are_declared_and_bound(qmv):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "qmv.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(qmv_\w+)\s*\(", src))
    for n in ("qmv_cache_write", "qmv_cache_read", "qmv_cache_attention", "qmv_logprobs"):
        assert n in names and n in qmv.serving.__all__ and getattr(qmv, n) is getattr(qmv.serving, n)
        assert getattr(qmv.lib(), n).argtypes
    for n in ("qmv_cache_page_bytes", "qmv_cache_attention_workspace_bytes", "qmv_logprobs_workspace_bytes"):
        assert n in names and getattr(qmv.lib(), n).restype is ctypes.c_size_t


def test_size_functions(qmv):
    L = qmv.lib()
    assert L.qmv_cache_page_bytes(0, 2, 64, 16) == 2 * 16 * 2 * 34 and L.qmv_cache_page_bytes(1, 1, 128, 16) == 16 * 4 * 18
    assert L.qmv_cache_page_bytes(2, 3, 256, 4096) == 3 * 4096 * 8 * 20
    for a in ((3, 2, 64, 16), (0, 0, 64, 16), (0, 2, 32, 16), (0, 2, 64, 15), (0, 2, 64, 24), (0, 1025, 64, 16), (-1, 2, 64, 16)):
        assert L.qmv_cache_page_bytes(*a) == 0
    with pytest.raises(ValueError):
        qmv.cache_page_bytes("q4_k", 2, 64, 16)
    w = L.qmv_cache_attention_workspace_bytes
    assert w(None, 1, 1, 2, 1) == 0 and w(cache(qmv, head_dim=80), 1, 1, 2, 1) == 0
    for a in ((0, 1, 2, 1), (65536, 1, 2, 1), (1, 0, 2, 1), (1, 1, 3, 1), (1, 1, 0, 1), (1, 1, 2, 0), (1, 1, 2, 2), (1, (1 << 24) + 1, 2, 1),
              (1, 1 << 24, 2 * 128, 1), (1, 1, 2 * 1025, 1)):
        assert w(cache(qmv), *a) == 0, a
    last = 0
    for n in (1, 2, 5, 100, 5000):      # more queries never need less
        b = w(cache(qmv), 3, 3 * n, 8, n)
        assert b >= last > -1 and b > 0
        last = b
    assert L.qmv_logprobs_workspace_bytes(0, 1, 0) == 0 and L.qmv_logprobs_workspace_bytes(1, 1, 33) == 0
    assert L.qmv_logprobs_workspace_bytes(1 << 20, 1 << 22, 0) == 0 and L.qmv_logprobs_workspace_bytes(1, (1 << 22) + 1, 0) == 0
    assert L.qmv_logprobs_workspace_bytes(1, -1, 0) == 0 and L.qmv_logprobs_workspace_bytes(1, 1, -1) == 0
    assert L.qmv_logprobs_workspace_bytes(1 << 17, 1 << 22, 32) > 1 << 32


def test_write_and_read_errors(qmv):
    w = dict(c=cache(qmv), k=A, kt=256, kh=128, v=A, vt=256, vh=128, xt=0, slots=A, n=5, stream=None)
    check(qmv, "qmv_cache_write", w, [
        (dict(c=None), EINVAL, "null"), *[(dict(c=cache(qmv, **b)), code, word) for b, code, word in BAD],
        *[({k: 0}, EINVAL, "null") for k in ("k", "v", "slots")], (dict(xt=3), EINVAL, "x_type"), (dict(xt=-1), EINVAL, "x_type"),
        (dict(n=0), EINVAL, "n_tokens"), (dict(n=(1 << 24) + 1), EINVAL, "n_tokens"), (dict(kh=127), EINVAL, "stride"),
        (dict(vh=0), EINVAL, "stride"), (dict(vh=-128), EINVAL, "stride"),
        (dict(k=A + 2), EALIGN, "aligned"), (dict(v=A + 1, xt=1), EALIGN, "aligned"), (dict(slots=A + 2), EALIGN, "aligned"),
    ])
    r = dict(c=cache(qmv), slots=A, n=5, k=A, v=A, xt=0, stream=None)
    check(qmv, "qmv_cache_read", r, [
        (dict(c=None), EINVAL, "null"), *[(dict(c=cache(qmv, **b)), code, word) for b, code, word in BAD],
        (dict(slots=0), EINVAL, "null"), (dict(k=0, v=0), EINVAL, "null"), (dict(xt=3), EINVAL, "out_type"),
        (dict(n=0), EINVAL, "n_tokens"), (dict(n=(1 << 24) + 1), EINVAL, "n_tokens"),
        (dict(k=A + 8), EALIGN, "aligned"), (dict(v=A + 4), EALIGN, "aligned"), (dict(slots=A + 1), EALIGN, "aligned"),
    ])


def test_attention_errors(qmv):
    need = qmv.lib().qmv_cache_attention_workspace_bytes(cache(qmv), 3, 12, 8, 4)
    good = dict(c=cache(qmv), q=A, xt=2, qt=1024, qh=128, tokens=12, heads=8, table=A, pages=9, lens=A, begin=A, requests=3,
                max_q=4, scale=0.1, window=0, sinks=None, out=A, ws=A, bytes=need, stream=None)
    check(qmv, "qmv_cache_attention", good, [
        (dict(c=None), EINVAL, "null"), *[(dict(c=cache(qmv, **b)), code, word) for b, code, word in BAD],
        *[({k: 0}, EINVAL, "null") for k in ("q", "table", "lens", "out", "ws")], (dict(xt=3), EINVAL, "x_type"),
        (dict(heads=7), EINVAL, "n_heads"), (dict(heads=0), EINVAL, "n_heads"), (dict(heads=2050), EINVAL, "n_heads"),
        (dict(tokens=0), EINVAL, "n_tokens"), (dict(tokens=(1 << 24) + 1), EINVAL, "n_tokens"), (dict(requests=0), EINVAL, "n_requests"),
        (dict(requests=65536), EINVAL, "n_requests"), (dict(max_q=0), EINVAL, "max_q"), (dict(max_q=13), EINVAL, "max_q"),
        (dict(begin=None, max_q=3), EINVAL, "q_begin"), (dict(pages=0), EINVAL, "max_pages"),
        (dict(pages=(1 << 25) + 1), EINVAL, "max_pages"), (dict(scale=0.0), EINVAL, "scale"), (dict(scale=-1.0), EINVAL, "scale"),
        (dict(scale=float("nan")), EINVAL, "scale"), (dict(scale=float("inf")), EINVAL, "scale"), (dict(window=-1), EINVAL, "window"),
        (dict(qh=127), EINVAL, "stride"), (dict(bytes=need - 1), EINVAL, "workspace"),
        (dict(q=A + 1), EALIGN, "aligned"), (dict(table=A + 2), EALIGN, "aligned"), (dict(lens=A + 2), EALIGN, "aligned"),
        (dict(begin=A + 2), EALIGN, "aligned"), (dict(sinks=A + 2), EALIGN, "aligned"), (dict(out=A + 8), EALIGN, "aligned"),
        (dict(ws=A + 8), EALIGN, "aligned"),
    ])


def test_logprobs_errors(qmv):
    need = qmv.lib().qmv_logprobs_workspace_bytes(3, 9000, 5)
    good = dict(l=A, lt=0, ld=9000, rows=3, vocab=9000, x=A, n=2, lp=A, e=A, top=5, tt=A, tl=A, ws=A, bytes=need, stream=None)
    check(qmv, "qmv_logprobs", good, [
        *[({k: 0}, EINVAL, "null") for k in ("l", "x", "lp", "tt", "tl", "ws")], (dict(lt=3), EINVAL, "logits_type"),
        (dict(n=-1), EINVAL, "n_targets"), (dict(n=1025), EINVAL, "n_targets"), (dict(rows=0), EINVAL, "n_rows"),
        (dict(rows=(1 << 20) + 1), EINVAL, "n_rows"), (dict(vocab=0), EINVAL, "vocab"), (dict(vocab=(1 << 22) + 1), EINVAL, "vocab"),
        (dict(top=33), EINVAL, "top_k"), (dict(top=-1), EINVAL, "top_k"), (dict(ld=8999), EINVAL, "ld"),
        (dict(bytes=need - 1), EINVAL, "workspace"), (dict(l=A + 2), EALIGN, "aligned"), (dict(x=A + 2), EALIGN, "aligned"),
        (dict(lp=A + 2), EALIGN, "aligned"), (dict(e=A + 1), EALIGN, "aligned"), (dict(tt=A + 2), EALIGN, "aligned"),
        (dict(tl=A + 2), EALIGN, "aligned"), (dict(ws=A + 8), EALIGN, "aligned"),
    ])
