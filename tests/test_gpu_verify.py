"""Verification of drafted tokens, on an MI355X, against 64-bit values.  The
outputs are whole numbers and have to be equal; the inputs are such that no
comparison is within 1e-12 of its border (checked here, on the CPU)."""
import numpy as np
import pytest

from tests import operator_values as ov

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)


@pytest.fixture(scope="module")
def env():
    import torch
    import bandwidth_bound_block_amd as qmv
    assert torch.cuda.is_available()
    return torch, qmv


def make(torch, Q, D, V, name, probs, seed, sharp=3.0):
    g = np.random.default_rng(seed)
    lt, l = ov.as_type(torch, sharp * g.standard_normal((Q, D + 1, V)), name)
    e = np.exp(l[:, :D] + 0.5 * g.standard_normal((Q, D, V)) - l[:, :D].max(-1, keepdims=True))
    q = (e / e.sum(-1, keepdims=True)).astype(np.float32) if probs else None
    x = np.empty((Q, D), dtype=np.int32)
    for r in range(Q):
        for i in range(D):
            x[r, i] = g.choice(V, p=q[r, i] / q[r, i].astype(np.float64).sum()) if probs else l[r, i].argmax()
    n = g.integers(0, D + 1, size=Q).astype(np.int32)
    u = (g.random((Q, D)) * (1.0 if probs else 0.2)).astype(np.float32)
    return lt, l, q, x, n, u, g.random(Q).astype(np.float32)


def expected(l, q, x, n, u, ul):
    Q, D1, V = l.shape
    tokens, kept, margin = np.full((Q, D1), -1), np.zeros(Q, int), np.inf
    for r in range(Q):
        k, t, m = ov.verify(l[r], None if q is None else q[r], x[r], min(max(int(n[r]), 0), D1 - 1),
                            u[r].astype(np.float64), float(ul[r]))
        margin = min(margin, m)
        kept[r] = k
        tokens[r, :k] = x[r, :k]
        tokens[r, k] = t
    return tokens, kept, margin


def call(torch, qmv, lt, q, x, n, u, ul, **kw):
    dev = [None if a is None else torch.from_numpy(a).cuda() for a in (q, x, n, u, ul)]
    tokens, kept = qmv.qmv_spec_verify(lt if lt.is_cuda else lt.cuda(), *dev, **kw)
    return tokens.cpu().numpy(), kept.cpu().numpy()


@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("Q,D,V", [(1, 1, 1), (3, 2, 5), (7, 7, 255), (20, 4, 4095), (9, 3, 4097), (5, 5, 9001), (2, 64, 300), (200, 2, 64)])
def test_against_64_bits(env, Q, D, V, name, probs):
    torch, qmv = env
    say("verify", Q, D, V, name, probs)
    lt, l, q, x, n, u, ul = make(torch, Q, D, V, name, probs, seed=Q * 100 + V)
    tokens, kept, margin = expected(l, q, x, n, u, ul)
    assert margin > 1e-12
    got = call(torch, qmv, lt, q, x, n, u, ul)
    assert np.array_equal(got[1], kept) and np.array_equal(got[0], tokens)


def test_both_ends_of_the_decisions_occur(env):
    """The inputs above keep all, some and none."""
    torch, _ = env
    _, l, q, x, n, u, ul = make(torch, 60, 5, 50, "f32", True, seed=1)
    kept = expected(l, q, x, n, u, ul)[1]
    assert (kept == n).any() and (kept < n).any() and (kept > 0).any() and (kept[n > 0] == 0).any()


def test_edges(env):
    """Masked logits, rows that are no distribution, ids out of range, counts out of range, u at its ends."""
    torch, qmv = env
    V, D = 37, 3
    inf = np.inf
    g = np.random.default_rng(0)
    base = g.standard_normal((D + 1, V))
    rows, q0 = [], np.full((D, V), 1.0 / V, dtype=np.float32)
    args = []

    def add(l, x, n, u, ul):
        rows.append(l)
        args.append((x, n, u, ul))
    add(base, [1, 2, 3], 3, [0, 0, 0], 0.0)                       # all kept; the first token with weight
    add(base, [1, 2, 3], 3, [0, 0, 0], np.float32(1 - 2 ** -24))  # the last ones
    l = base.copy(); l[0, 1:] = -inf
    add(l, [1, 2, 3], 3, [0, 0, 0], 0.7)                          # p(x) = 0: rejected, only token 0 left
    l = base.copy(); l[0] = -inf
    add(l, [1, 2, 3], 3, [0, 0, 0], 0.5)                          # masked throughout
    l = base.copy(); l[1, 5] = np.nan
    add(l, [1, 2, 3], 3, [0, 0, 0], 0.5)                          # NaN in row 1: one kept, none drawn
    l = base.copy(); l[3, 5] = inf
    add(l, [1, 2, 3], 3, [0, 0, 0], 0.5)                          # all kept, the last row no distribution
    l = base.copy(); l[0] = np.nan
    add(l, [1, 2, 3], 3, [0, 0, 0], 0.5)
    add(base, [1, V, 3], 3, [0, 0, 0], 0.4)                       # ids out of range
    add(base, [-1, 2, 3], 3, [0, 0, 0], 0.4)
    add(base, [1, 2, 3], 0, [0, 0, 0], 0.3)                       # no drafts
    add(base, [1, 2, 3], -5, [0, 0, 0], 0.3)
    add(base, [1, 2, 3], 99, [0, 0, 0], 0.3)
    l = base.copy(); l[2] = -inf; l[2, 7] = 500.0
    add(l, [1, 2, 7], 3, [0, 0, 0.99], 0.3)
    l = 1e4 * base
    add(l, [1, 2, 3], 2, [0.5, 0.5, 0.5], 0.3)                    # terms far below the largest
    lt, l64 = ov.as_type(torch, np.stack(rows), "f32")
    x = np.array([a[0] for a in args], dtype=np.int32)
    n = np.array([a[1] for a in args], dtype=np.int32)
    u = np.array([a[2] for a in args], dtype=np.float32)
    ul = np.array([a[3] for a in args], dtype=np.float32)
    for q in (None, np.broadcast_to(q0, (len(rows), D, V)).copy()):
        tokens, kept, margin = expected(l64, q, x, n, u, ul)
        got = call(torch, qmv, lt, q, x, n, u, ul)
        for r in range(len(rows)):
            assert got[1][r] == kept[r] and np.array_equal(got[0][r], tokens[r]), (r, got[1][r], kept[r], got[0][r], tokens[r])


def test_draft_equal_to_target_draws_from_p(env):
    """A rejection where p - q leaves nothing: the draw is from p."""
    torch, qmv = env
    V = 64
    l = torch.zeros(1, 2, V)
    q = np.full((1, 1, V), 1.0 / V, dtype=np.float32)
    x, n = np.array([[5]], dtype=np.int32), np.array([1], dtype=np.int32)
    u, ul = np.array([[1.0]], dtype=np.float32), np.array([0.505], dtype=np.float32)   # u = 1 rejects equality
    tokens, kept = call(torch, qmv, l, q, x, n, u, ul)
    assert kept[0] == 0 and tokens[0, 0] == int(0.505 * V)


def test_strides_alignment_repeats_stream_graph(env):
    torch, qmv = env
    Q, D, V = 6, 4, 5003
    lt, l, q, x, n, u, ul = make(torch, Q, D, V, "f32", True, seed=77)
    tokens, kept, margin = expected(l, q, x, n, u, ul)
    assert margin > 1e-12
    for pad, start in ((5, 0), (8, 4), (7, 3)):
        wide = torch.full((Q, D + 1, V + pad + start), float("nan"))
        wide[..., start:start + V] = lt
        wq = torch.full((Q, D, V + pad + start), float("nan"))
        wq[..., start:start + V] = torch.from_numpy(q)
        dev = [torch.from_numpy(a).cuda() for a in (x, n, u, ul)]
        t, k = qmv.qmv_spec_verify(wide.cuda()[..., start:start + V], wq.cuda()[..., start:start + V], *dev)
        assert np.array_equal(t.cpu().numpy(), tokens) and np.array_equal(k.cpu().numpy(), kept), (pad, start)
    lc, qc = lt.cuda(), torch.from_numpy(q).cuda()
    dev = [torch.from_numpy(a).cuda() for a in (x, n, u, ul)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        t, k = qmv.qmv_spec_verify(lc, qc, *dev, stream=side)
    side.synchronize()
    assert np.array_equal(t.cpu().numpy(), tokens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t, k = qmv.qmv_spec_verify(lc, qc, *dev)
    for i in range(4):
        perm = np.random.default_rng(i).permutation(Q)
        lc.copy_(lt[torch.from_numpy(perm)])
        qc.copy_(torch.from_numpy(q[perm]))
        for a, b in zip(dev, (x, n, u, ul)):
            a.copy_(torch.from_numpy(b[perm]))
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(t.cpu().numpy(), tokens[perm]) and np.array_equal(k.cpu().numpy(), kept[perm]), i


def test_large_vocabulary(env):
    torch, qmv = env
    lt, l, q, x, n, u, ul = make(torch, 2, 2, 151936, "f32", True, seed=5)
    tokens, kept, margin = expected(l, q, x, n, u, ul)
    assert margin > 1e-12
    got = call(torch, qmv, lt, q, x, n, u, ul)
    assert np.array_equal(got[1], kept) and np.array_equal(got[0], tokens)
