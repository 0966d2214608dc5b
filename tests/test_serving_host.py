"""What the Python entry points of the cache, its attention and the log probabilities do on the host: no GPU."""
import contextlib

import pytest
import torch

from tests.test_operators_host import OnGpu, Stand, gpu, ids, raw


@pytest.fixture()
def stand(monkeypatch):
    import bandwidth_bound_block_amd as qmv
    st = Stand(monkeypatch, qmv)
    st.devices = []

    @contextlib.contextmanager
    def device(i):
        st.devices.append(i)
        yield
        st.devices.append(None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", device)
    return st, qmv


def cache(q, **k):
    return q.KVCache(raw(192), raw(192), "q8_0", "q4_0", 2, 64, 16)      # the stand-in's pages have 64 bytes


def f16(*shape):
    return gpu(*shape, dtype=torch.float16)


def tables(R=2, T=None):
    return ids(R, 3), ids(R), None if T is None else ids(R + 1)


CALLS = {
    "qmv_cache_read": lambda q, s: q.qmv_cache_read(cache(q), ids(5), stream=s),
    "qmv_cache_attention": lambda q, s: q.qmv_cache_attention(cache(q), gpu(6, 4, 64), *tables(2, 6), stream=s),
    "qmv_logprobs": lambda q, s: q.qmv_logprobs(gpu(3, 9), ids(3, 2), top_k=4, stream=s),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_new_tensors_come_from_the_pool_of_the_calls_stream(stand, name):
    st, qmv = stand
    out = CALLS[name](qmv, st.side)
    assert st.made and all(t.pool is st.side for t in st.made)
    assert st.current is st.main and [n for n, _ in st.calls] == [name]
    assert all(getattr(s, "value", s) == 22 for _, s in st.calls)
    for t in out if isinstance(out, tuple) else (out,):
        assert st.main in t.recorded


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("given", [False, True])
def test_nothing_is_recorded_on_the_current_stream(stand, name, given):
    st, qmv = stand
    CALLS[name](qmv, st.main if given else None)
    assert st.made and all(t.pool is st.main and not hasattr(t, "recorded") for t in st.made)
    assert all(getattr(s, "value", s) == 11 for _, s in st.calls)
    assert not st.devices


def test_writes_go_to_the_calls_stream_and_make_nothing(stand):
    st, qmv = stand
    c = cache(qmv)
    qmv.qmv_cache_write(c, f16(5, 2, 64), f16(5, 2, 64), ids(5))
    qmv.qmv_cache_write(c, f16(5, 2, 64), f16(5, 2, 64), ids(5), stream=st.side)
    assert not st.made and [(n, getattr(s, "value", s)) for n, s in st.calls] == [("qmv_cache_write", 11), ("qmv_cache_write", 22)]


class Elsewhere(OnGpu):
    def get_device(self):
        return 1


def elsewhere(t):
    return t.as_subclass(Elsewhere)


def test_calls_on_another_gpu_than_the_current_one(stand):
    """A launch goes to the current GPU: the call makes its tensors' GPU current, and the one before afterwards."""
    st, qmv = stand
    c = qmv.KVCache(elsewhere(raw(192)), elsewhere(raw(192)), "q4_1", "q4_0", 2, 64, 16)
    x = elsewhere(f16(5, 2, 64))
    qmv.qmv_cache_write(c, x, x, elsewhere(ids(5)))
    assert st.devices == [1, None]
    with pytest.raises(ValueError, match="same GPU"):
        qmv.qmv_cache_write(c, x, x, ids(5))
    with pytest.raises(ValueError, match="same GPU"):
        qmv.qmv_cache_write(cache(qmv), x, x, elsewhere(ids(5)))
    with pytest.raises(ValueError, match="one GPU"):
        qmv.KVCache(raw(192), elsewhere(raw(192)), "q4_1", "q4_0", 2, 64, 16)
    with pytest.raises(ValueError, match="same GPU"):
        qmv.qmv_cache_attention(cache(qmv), gpu(2, 4, 64), elsewhere(ids(2, 3)), ids(2))
    with pytest.raises(ValueError, match="same GPU"):
        qmv.qmv_logprobs(gpu(3, 9), elsewhere(ids(3)))


def test_a_cache_is_fixed(stand):
    """The library is given addresses: other pages are another cache."""
    _, qmv = stand
    c = cache(qmv)
    for name in ("k", "v", "n_pages", "k_fmt", "page_size"):
        with pytest.raises(AttributeError):
            setattr(c, name, getattr(c, name))
    assert c.n_pages == 3 and (c.k_fmt, c.v_fmt) == (qmv.Q8_0, qmv.Q4_0)


REFUSED = [
    lambda q: q.KVCache(raw(200), raw(192), "q8_0", "q4_0", 2, 64, 16),                     # no whole pages
    lambda q: q.KVCache(raw(128), raw(192), "q8_0", "q4_0", 2, 64, 16),
    lambda q: q.KVCache(raw(0), raw(0), "q8_0", "q4_0", 2, 64, 16),
    lambda q: q.KVCache(gpu(192), raw(192), "q8_0", "q4_0", 2, 64, 16),
    lambda q: q.KVCache(torch.zeros(192, dtype=torch.uint8), raw(192), "q8_0", "q4_0", 2, 64, 16),
    lambda q: q.KVCache(raw(192), raw(192), "q8", "q4_0", 2, 64, 16),
    lambda q: q.qmv_cache_write(cache(q), f16(5, 2, 64), gpu(5, 2, 64), ids(5)),            # two types
    lambda q: q.qmv_cache_write(cache(q), f16(5, 2, 64), f16(5, 2, 32), ids(5)),
    lambda q: q.qmv_cache_write(cache(q), f16(5, 3, 64), f16(5, 3, 64), ids(5)),
    lambda q: q.qmv_cache_write(cache(q), f16(5, 128), f16(5, 128), ids(5)),
    lambda q: q.qmv_cache_write(cache(q), f16(5, 2, 64), f16(4, 2, 64), ids(5)),
    lambda q: q.qmv_cache_write(cache(q), f16(5, 2, 64), f16(5, 2, 64), ids(4)),
    lambda q: q.qmv_cache_write(cache(q), f16(5, 2, 64), f16(5, 2, 64), ids(5, 1)),
    lambda q: q.qmv_cache_write(cache(q), f16(5, 2, 64), f16(5, 2, 64), gpu(5)),
    lambda q: q.qmv_cache_write(cache(q), f16(5, 2, 128)[..., ::2], f16(5, 2, 64), ids(5)),
    lambda q: q.qmv_cache_read(cache(q), gpu(5)),
    lambda q: q.qmv_cache_read(cache(q), ids(5), k=f16(5, 2, 32)),
    lambda q: q.qmv_cache_read(cache(q), ids(5), k=f16(5, 2, 64), v=gpu(5, 2, 64)),
    lambda q: q.qmv_cache_read(cache(q), ids(5), dtype=torch.int32),
    lambda q: q.qmv_cache_attention(cache(q), gpu(6, 256), ids(2, 3), ids(2)),
    lambda q: q.qmv_cache_attention(cache(q), gpu(6, 4, 32), ids(2, 3), ids(2)),
    lambda q: q.qmv_cache_attention(cache(q), gpu(6, 4, 64), ids(6), ids(2)),
    lambda q: q.qmv_cache_attention(cache(q), gpu(6, 4, 64), ids(2, 3), ids(3)),
    lambda q: q.qmv_cache_attention(cache(q), gpu(6, 4, 64), ids(2, 3), ids(2), ids(2)),
    lambda q: q.qmv_cache_attention(cache(q), gpu(5, 4, 64), ids(2, 3), ids(2)),            # 5 tokens of 2 requests
    lambda q: q.qmv_cache_attention(cache(q), gpu(6, 4, 64), ids(2, 3), ids(2), max_q=2),
    lambda q: q.qmv_cache_attention(cache(q), gpu(6, 4, 64), ids(0, 3), ids(0)),
    lambda q: q.qmv_cache_attention(cache(q), gpu(6, 4, 64), ids(2, 3), ids(2), sinks=gpu(3)),
    lambda q: q.qmv_cache_attention(cache(q), gpu(6, 4, 64), ids(2, 3), ids(2), out=f16(6, 4, 64)),
    lambda q: q.qmv_cache_attention(cache(q), gpu(6, 4, 64), ids(2, 3), ids(2), workspace=raw(63)),
    lambda q: q.qmv_cache_attention(cache(q), gpu(6, 4, 64), ids(2, 3), ids(2), window=-1),
    lambda q: q.qmv_cache_attention(cache(q), gpu(6, 4, 64), ids(2, 3), ids(2), window=1 << 32),
    lambda q: q.qmv_logprobs(gpu(9)),
    lambda q: q.qmv_logprobs(gpu(1, 9), top_k=-1),
    lambda q: q.qmv_logprobs(gpu(1, 9), top_k=1 << 32),
    lambda q: q.qmv_logprobs(gpu(3, 18)[:, ::2]),
    lambda q: q.qmv_logprobs(gpu(3, 9), ids(2)),
    lambda q: q.qmv_logprobs(gpu(3, 9), gpu(3)),
    lambda q: q.qmv_logprobs(gpu(3, 9), logprobs=gpu(3)),
    lambda q: q.qmv_logprobs(gpu(3, 9), top_tokens=ids(3, 1)),
    lambda q: q.qmv_logprobs(gpu(3, 9), top_k=2, top_tokens=ids(3, 1)),
    lambda q: q.qmv_logprobs(gpu(3, 9), entropy=gpu(4)),
    lambda q: q.qmv_logprobs(ids(3, 9)),
    lambda q: q.qmv_logprobs(gpu(3, 9), workspace=gpu(64)),
]


@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_refusals(stand, i):
    st, qmv = stand
    with pytest.raises((TypeError, ValueError, KeyError)):
        REFUSED[i](qmv)
    assert not st.calls
