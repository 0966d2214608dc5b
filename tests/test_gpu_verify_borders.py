"""Verification close to its comparisons' borders, on an MI355X: exponentials hold to fp64, down to its smallest numbers.
Expected values are from 80-bit floats (2^-64)."""
import numpy as np
import pytest

from tests import operator_values as ov

pytestmark = pytest.mark.gpu
L = np.longdouble
NEAR, FAR = 1e-12, 3e-12          # relative distances from the border: past fp64's own error, 1e-15, by far


@pytest.fixture(scope="module")
def env():
    import torch
    import bandwidth_bound_block_amd as qmv
    assert torch.cuda.is_available()
    return torch, qmv


def call(torch, qmv, l, q, x, n, u, ul):
    dev = [None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (l, q, x, n, u, ul)]
    tokens, kept = qmv.qmv_spec_verify(*dev)
    return tokens.cpu().numpy(), kept.cpu().numpy()


def second(a):
    """p of the second token for logits (0, -a)."""
    e = np.exp(-a.astype(L))
    return e / (1 + e)


@pytest.mark.parametrize("at", [0.1, 0.3465, 0.34665, 1.0397, 5.8917, 30.15])     # near and at halves of ln 2, where e^x is worst
def test_acceptance_next_to_the_border(env, at):
    torch, qmv = env
    assert np.finfo(L).eps < 1e-18
    g = np.random.default_rng(int(at * 1e5))
    a = (at * (1 + 1e-4 * g.random(1_000_000))).astype(np.float32)
    p = second(a)
    q = (p * (1 + g.random(a.size))).astype(np.float32)
    u = (p / q.astype(L)).astype(np.float32)
    gap = u.astype(L) * q.astype(L) / p - 1
    pick = np.nonzero((np.abs(gap) > NEAR) & (np.abs(gap) < FAR))[0][:60]
    assert (gap[pick] > 0).sum() > 3 and (gap[pick] < 0).sum() > 3
    a, q, u, gap = a[pick], q[pick], u[pick], gap[pick]
    Q = a.size
    l = np.zeros((Q, 2, 2), dtype=np.float32)
    l[:, 0, 1] = -a
    qs = np.zeros((Q, 1, 2), dtype=np.float32)
    qs[:, 0, 1] = q
    x, n = np.ones((Q, 1), dtype=np.int32), np.ones(Q, dtype=np.int32)
    tokens, kept = call(torch, qmv, l, qs, x, n, u[:, None], np.full(Q, 0.25, dtype=np.float32))
    assert np.array_equal(kept, (gap < 0).astype(int))
    assert np.all(tokens[:, 0] == np.where(gap < 0, 1, 0))


@pytest.mark.parametrize("at", [0.1, 0.3465, 0.34665, 1.0397])
def test_draw_next_to_the_border(env, at):
    torch, qmv = env
    g = np.random.default_rng(int(at * 1e5) + 1)
    a = (at * (1 + 0.05 * g.random(3_000_000))).astype(np.float32)
    first = 1 / (1 + np.exp(-a.astype(L)))
    ul = first.astype(np.float32)
    gap = ul.astype(L) / first - 1
    pick = np.nonzero((np.abs(gap) > NEAR) & (np.abs(gap) < FAR))[0][:60]
    assert (gap[pick] > 0).sum() > 3 and (gap[pick] < 0).sum() > 3
    a, ul, gap = a[pick], ul[pick], gap[pick]
    Q = a.size
    l = np.zeros((Q, 2, 2), dtype=np.float32)
    l[:, 0, 1] = -a
    x, n = np.zeros((Q, 1), dtype=np.int32), np.zeros(Q, dtype=np.int32)
    tokens, kept = call(torch, qmv, l, None, x, n, np.zeros((Q, 1), dtype=np.float32), ul)
    assert (kept == 0).all() and np.array_equal(tokens[:, 0], (gap > 0).astype(int))


def test_terms_down_to_fp64s_smallest(env):
    """Probabilities down to e^-745 are numbers: u = 0 keeps their tokens, and u_last = 0 draws the first of them."""
    torch, qmv = env
    depths = np.array([600, 699, 701, 708, 720, 740, 744, 746, 800, 1e4, 3e38], dtype=np.float32)
    Q = depths.size
    l = np.zeros((Q, 2, 3), dtype=np.float32)
    l[:, 0, 0] = l[:, 1, 0] = -depths
    l[:, 0, 2] = l[:, 1, 2] = -np.inf
    there = np.exp(-depths.astype(np.float64)) > 0
    assert there.sum() == 7
    zero = np.zeros((Q, 1), dtype=np.float32)
    for name in ("f32", "bf16"):
        lt, l64 = ov.as_type(torch, l, name)
        # bf16 rounds the depths, and the borders with them
        on = np.exp(l64[:, 0, 0]) > 0
        for token, want in ((0, on), (1, np.ones(Q, bool)), (2, np.zeros(Q, bool))):
            x, n = np.full((Q, 1), token, dtype=np.int32), np.ones(Q, dtype=np.int32)
            dev = [torch.from_numpy(v).cuda() for v in (x, n, zero, zero[:, 0].copy())]
            tokens, kept = qmv.qmv_spec_verify(lt.cuda(), None, *dev)
            tokens, kept = tokens.cpu().numpy(), kept.cpu().numpy()
            assert np.array_equal(kept, want.astype(int)), (name, token)
            # where it is kept, the next row's first token with any weight
            assert np.array_equal(tokens[want, 1], np.where(on[want], 0, 1)), (name, token)
