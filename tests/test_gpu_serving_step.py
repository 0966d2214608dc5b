"""The example serving step: its parts together give what the parts' plain forms give."""
import numpy as np
import pytest

import workloads as wl
from tests import operator_values as ov

pytestmark = pytest.mark.gpu


def test_serving_step():
    import torch
    from examples import serving_step as ex
    model = ex.Model(1)
    requests, drafts = 9, 3
    drafted, tokens, kept = ex.step(model, requests, drafts, seed=2)
    again = ex.step(model, requests, drafts, seed=2)
    assert torch.equal(tokens, again[1]) and torch.equal(kept, again[2])
    drafted, tokens, kept = drafted.cpu().numpy(), tokens.cpu().numpy(), kept.cpu().numpy()
    for r in range(requests):
        assert np.array_equal(tokens[r, :kept[r]], drafted[r, :kept[r]])
        assert 0 <= tokens[r, kept[r]] < ex.VOCAB and np.all(tokens[r, kept[r] + 1:] == -1)
    assert 0 < kept.sum() < requests * drafts


def test_logits_against_64_bits():
    """Projection, adapters, experts and head in 64 bits; the bfloat16 steps between them are roundings of at most half a
    step each, which the router's choice (a gap between scores) has to survive."""
    import torch
    from examples import serving_step as ex
    model = ex.Model(3)
    T, H, F = 40, ex.HIDDEN, ex.FFN
    g = torch.Generator().manual_seed(5)
    x = torch.randn(T, H, generator=g).bfloat16()
    ids = torch.randint(-1, ex.ADAPTERS, (T,), generator=g).to(torch.int32)
    got = model.logits(x.cuda(), ids.cuda()).cpu().double().numpy()

    def weights(fmt, tag, n, k, std=0.02):
        raw = wl.quant_weights(fmt, f"example/3/{tag}", n, k, std=std)
        return ov.oracle.dequant(fmt, raw, n, k).astype(np.float64).reshape(n, k)
    xv = x.double().numpy()
    A, B = model.A.cpu().double().numpy(), model.B.cpu().double().numpy()
    d, _ = ov.adapters(xv, A, B, np.ones(ex.ADAPTERS), ids.numpy())
    h = torch.from_numpy(xv @ weights("q4_0", "proj", H, H).T + d).bfloat16().double().numpy()
    scores = h @ model.router.cpu().double().numpy()
    order = np.argsort(-scores, axis=1)[:, :ex.TOP_K]
    top = np.take_along_axis(scores, order, 1)
    w = np.exp(top - top.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    gu = weights("q4_k", "gu", ex.EXPERTS * 2 * F, H).reshape(ex.EXPERTS, 2 * F, H)
    dn = weights("q4_k", "down", ex.EXPERTS * H, F).reshape(ex.EXPERTS, H, F)
    y = np.zeros((T, H))
    for t in range(T):
        for s in range(ex.TOP_K):
            a = gu[order[t, s]] @ h[t]
            y[t] += w[t, s] * (dn[order[t, s]] @ (ov.silu(a[:F]) * a[F:]))
    head = weights("q8_0", "head", ex.VOCAB, H, std=0.2)
    out = (h + y) @ head.T
    # bfloat16 roundings of h, e, the sum y and h + y, 2^-8 each of values no larger than |h| + |y|'s row norms
    norm = np.linalg.norm(h, axis=1, keepdims=True) + 3 * np.linalg.norm(y, axis=1, keepdims=True)
    bound = 4 * ov.HALF["bf16"] * norm * np.linalg.norm(head, axis=1)[None]
    gap = np.sort(scores, axis=1)[:, ::-1]
    clear = (gap[:, ex.TOP_K - 1] - gap[:, ex.TOP_K]) > 0.05 * np.abs(gap[:, 0])
    assert clear.sum() > T // 2
    assert np.all(np.abs(got - out)[clear] <= bound[clear])
