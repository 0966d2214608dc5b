"""The example's answers: projections, cache, attention, experts, lm_head and log probabilities in a run together.

Each operator's outputs along the way are held against 64-bit values made of the inputs that it had there."""
import numpy as np
import pytest

from tests import cache_values as cv
from tests.test_gpu_logprobs import check

pytestmark = pytest.mark.gpu


def test_answers(monkeypatch):
    import torch
    from examples import serving_step as ex
    qmv, seen = ex.qmv, []

    def kept(name):
        f = getattr(qmv, name)

        def call(*a, **k):
            out = f(*a, **k)
            seen.append((name, a, k, out))
            return out
        monkeypatch.setattr(qmv, name, call)
    for name in ("qmv_cache_write", "qmv_cache_attention", "qmv_logprobs"):
        kept(name)
    rng = np.random.default_rng(6)
    lengths, n = [1, 15, 40, 16, 7, 90, 17], 6
    prompts = [rng.integers(0, ex.VOCAB, m).tolist() for m in lengths]
    R, H, D, P = len(lengths), ex.KV_HEADS, ex.DIM, ex.PAGE
    att = ex.Attention(sum(-(-(m + n) // P) for m in lengths), 1)
    att.cache.k.fill_(0xFF)          # NaN where nothing is written
    att.cache.v.fill_(0xFF)
    model = ex.Model(1)
    tokens, logprobs = ex.answer(model, att, prompts, n)
    assert tokens.shape == logprobs.shape == (R, n)
    assert [s[0] for s in seen] == (["qmv_cache_write", "qmv_cache_attention", "qmv_logprobs"] * n)

    G, lens, past = ex.HEADS // H, np.array(lengths), [[np.zeros((0, H, D))] * 2 for _ in range(R)]
    for step in range(n):
        (_, w, _, _), (_, a, kw, out), (_, l, _, best) = seen[3 * step:3 * step + 3]
        new = lens if step == 0 else np.ones(R, int)
        begin = np.concatenate([[0], np.cumsum(new)])
        coded = [cv.decode(*cv.encode(x.cpu().double().numpy(), f), f) for x, f in ((w[1], "q8_0"), (w[2], "q4_0"))]
        q, got = a[1].cpu().double().numpy(), out.cpu().double().numpy()
        assert a[3].tolist() == lens.tolist()
        for r in range(R):
            lo, hi = begin[r], begin[r + 1]
            past[r] = [np.concatenate([old, x[lo:hi]]) for old, x in zip(past[r], coded)]
            L = past[r][0].shape[0]
            assert L == lens[r]
            pos = np.repeat(np.arange(L - (hi - lo), L), G)
            for h in range(H):
                rows = q[lo:hi, h * G:(h + 1) * G].reshape(-1, D)
                want, bound = cv.attention(rows, past[r][0][:, h], past[r][1][:, h], D ** -0.5, pos, 0, None, "f32", rows.shape[0] <= 32)
                off = np.abs(got[lo:hi, h * G:(h + 1) * G].reshape(-1, D) - want)
                assert np.all(off <= bound), (step, r, h, (off / bound).max())
        check(torch, best, l[0].cpu().double().numpy(), None, 1)
        assert torch.equal(tokens[:, step], best.top_tokens[:, 0]) and torch.equal(logprobs[:, step], best.top_logprobs[:, 0])
        lens = lens + 1

    # the cache holds what was written, and nothing else
    slots = torch.cat([a[2][r, :-(-(m + n) // P)] for r, m in enumerate(lengths)])
    slots = slots[slots >= 0]
    back = qmv.qmv_cache_read(att.cache, (slots[:, None] * P + torch.arange(P, device="cuda", dtype=torch.int32)).view(-1))
    table = a[2].cpu().numpy()
    for got, which in zip(back, (0, 1)):
        got, at = got.cpu().numpy(), 0
        for r, m in enumerate(lengths):
            pages = int((table[r] >= 0).sum())
            g = got[at:at + pages * P]
            at += pages * P
            assert np.array_equal(g[:m + n - 1], past[r][which].astype(np.float32)) and np.all(np.isnan(g[m + n - 1:]))

    # the same again: the same bits
    again = ex.answer(model, att, prompts, n)
    assert torch.equal(again[0], tokens)
    with pytest.raises(ValueError):
        ex.answer(model, ex.Attention(2, 1), prompts, n)


def test_two_streams_at_once():
    """The operators in a row on two streams, each with memory of its own, while the other's run: what each gives alone."""
    import torch
    import bandwidth_bound_block_amd as qmv
    R, H, G, D, P, V = 9, 2, 4, 128, 16, 5000
    g = torch.Generator(device="cuda").manual_seed(4)
    lens = torch.tensor([1, 700, 33, 5, 2000, 64, 17, 300, 1200], dtype=torch.int32, device="cuda")
    pages = 126
    state = []
    for i in range(2):
        cache = qmv.KVCache.new(R * pages, "q8_0", "q4_1", H, D, P)
        table = torch.randperm(R * pages, generator=g, device="cuda").to(torch.int32).view(R, pages)
        at = [torch.arange(int(n), device="cuda") for n in lens]
        slots = torch.cat([(table[r, a // P] * P + a % P).to(torch.int32) for r, a in enumerate(at)])
        k, v = (torch.randn(slots.numel(), H, D, generator=g, device="cuda") for _ in range(2))
        q = torch.randn(R, H * G, D, generator=g, device="cuda")
        w = torch.randn(H * G * D, V, generator=g, device="cuda")
        state.append((cache, k, v, slots, q, table, w))

    def run(i, stream):
        cache, k, v, slots, q, table, w = state[i]
        qmv.qmv_cache_write(cache, k, v, slots, stream=stream)
        a = qmv.qmv_cache_attention(cache, q, table, lens, stream=stream)
        with torch.cuda.stream(stream):
            l = a.view(R, -1) @ w
        return (a,) + tuple(qmv.qmv_logprobs(l, None, top_k=7, stream=stream)[1:])
    want = []
    for i in range(2):
        want.append([t.clone() for t in run(i, torch.cuda.current_stream())])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for c, *_ in state:
        c.k.zero_()
        c.v.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        got = [run(i, streams[i]) for i in (0, 1)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
