"""qmv_logprobs on an MI355X against 64-bit values."""
import numpy as np
import pytest

from tests import cache_values as cv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import bandwidth_bound_block_amd as qmv
    assert torch.cuda.is_available()
    return torch, qmv


def typed(torch, a, x):
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to({"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[x])
    return t, t.to(torch.float64).numpy()


def check(torch, got, l, targets, top):
    lp, H, tt, tl = (None if t is None else t.cpu().numpy() for t in got)
    for r in range(l.shape[0]):
        row = l[r]
        if not np.any(row > -np.inf) or np.any(np.isnan(row)) or np.any(row == np.inf):
            assert np.isnan(H[r])
            assert lp is None or np.all(np.isnan(lp[r]))
            assert top == 0 or (np.all(tt[r] == -1) and np.all(np.isnan(tl[r])))
            continue
        p, h, bp, bh = cv.logprobs(row)
        assert abs(H[r] - h) <= bh, (r, H[r], h, bh)
        if lp is not None:
            for i, x in enumerate(np.atleast_1d(targets[r])):
                g = np.atleast_1d(lp[r])[i]
                if not 0 <= x < row.size:
                    assert np.isnan(g)
                elif p[x] == -np.inf:
                    assert g == -np.inf
                else:
                    assert abs(g - p[x]) <= bp[x], (r, x, g, p[x], bp[x])
        if top:
            order = np.argsort(-row, kind="stable")[:top]
            order = order[row[order] > -np.inf]
            n = order.size
            assert np.array_equal(tt[r, :n], order), (r, tt[r], order)
            assert np.all(tt[r, n:] == -1) and np.all(tl[r, n:] == -np.inf)
            assert np.all(np.abs(tl[r, :n] - p[order]) <= bp[order])


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,V,top,given", [(1, 1, 1, 1), (1, 5, 32, 3), (3, 64, 0, 1), (2, 4095, 5, 2), (5, 4096, 32, 0),
                                              (2, 4097, 20, 1), (7, 13003, 20, 4), (3, 128256, 5, 1), (2, 151936, 32, 1024)])
def test_rows(env, x, rows, V, top, given):
    torch, qmv = env
    print(x, rows, V, top, given, flush=True)
    rng = np.random.default_rng(V + top)
    t, l = typed(torch, 3 * rng.standard_normal((rows, V)), x)
    ids = rng.integers(-1, V + 1, (rows, given)).astype(np.int32)
    got = qmv.qmv_logprobs(t.cuda(), torch.from_numpy(ids).cuda() if given else None, top_k=top)
    check(torch, got, l, ids, top)


@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_rows_that_are_special(env, x):
    """Masked tokens, masks of the type's lowest value, rows with nothing left, NaN, infinities, certain rows, ties."""
    torch, qmv = env
    print(x, flush=True)
    rng = np.random.default_rng(3)
    V = 9001
    a = 3 * rng.standard_normal((14, V))
    a[0, rng.random(V) < 0.9] = -np.inf
    a[1] = -np.inf
    a[2] = -np.inf
    a[2, [5, 8000]] = 1.0, 2.0                         # two tokens have a probability
    a[3, 77] = np.nan
    a[4, 8999] = np.inf
    a[5] = 0.25                                        # all alike
    a[6, 4500] = 60.0                                  # certain: what is left is 1e-22
    a[7, 100] = 18.0                                   # nearly
    a[8, 50:4200] = 9.0                                # many largest ones, over a chunk's border
    a[9] = np.round(a[9])                              # ties throughout
    a[10, rng.random(V) < 0.5] = -3.3e38               # a finite mask
    a[11] *= 1e3
    a[12] -= 30000.0
    a[13, 3] = 3.3e38
    t, l = typed(torch, a, x)
    ids = rng.integers(0, V, (14, 3)).astype(np.int32)
    ids[2] = [5, 8000, 6]
    ids[6, 0], ids[7, 0] = 4500, 100
    for top in (0, 1, 20, 32):
        got = qmv.qmv_logprobs(t.cuda(), torch.from_numpy(ids).cuda(), top_k=top)
        check(torch, got, l, ids, top)


def test_many_chunks_with_ties(env):
    """More candidates than are counted in LDS: every chunk's list has the same values."""
    torch, qmv = env
    V = 300001
    l = torch.zeros(2, V, device="cuda")
    l[1] = torch.arange(V, device="cuda") % 7
    got = qmv.qmv_logprobs(l, None, top_k=32)
    check(torch, got, l.cpu().double().numpy(), None, 32)


@pytest.mark.parametrize("x", ["f32", "f16"])
def test_strides_and_alignment(env, x):
    torch, qmv = env
    print(x, flush=True)
    rng = np.random.default_rng(8)
    V = 5003
    t, l = typed(torch, 2 * rng.standard_normal((4, V)), x)
    ids = torch.tensor([1, V - 1, 0, 2500], dtype=torch.int32)
    want = qmv.qmv_logprobs(t.cuda(), ids.cuda(), top_k=9)
    for lead, pad in ((1, 0), (3, 2), (0, 1), (4, 9)):
        buf = torch.full((4, lead + V + pad), 50.0, dtype=t.dtype, device="cuda")
        buf[:, lead:lead + V] = t.cuda()
        got = qmv.qmv_logprobs(buf[:, lead:lead + V], ids.cuda(), top_k=9)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (lead, pad)
    check(torch, want, l, ids.numpy(), 9)


def test_captured_and_replayed(env):
    torch, qmv = env
    rng = np.random.default_rng(4)
    l = torch.from_numpy(rng.standard_normal((3, 20000)).astype(np.float32)).cuda()
    ids = torch.tensor([1, 2, 3], dtype=torch.int32).cuda()
    qmv.qmv_logprobs(l, ids, top_k=6)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = qmv.qmv_logprobs(l, ids, top_k=6)
    for i in range(4):
        l.copy_(torch.from_numpy((1 + i) * rng.standard_normal((3, 20000)).astype(np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        want = qmv.qmv_logprobs(l, ids, top_k=6)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
