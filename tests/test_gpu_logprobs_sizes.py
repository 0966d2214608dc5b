"""qmv_logprobs at the ends of its chunks of 8192 logits, over many of them, and with more rows than a launch is high."""
import numpy as np
import pytest

from tests.test_gpu_logprobs import check, typed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import bandwidth_bound_block_amd as qmv
    assert torch.cuda.is_available()
    return torch, qmv


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [8191, 8192, 8193, 16383, 16384, 16385, 24576, 63, 65])
def test_ends_of_chunks(env, x, V):
    torch, qmv = env
    print(x, V, flush=True)
    rng = np.random.default_rng(V)
    a = 3 * rng.standard_normal((4, V))
    a[1, -1] = 30.0                            # the last of the row, the first, and those beside the chunks' ends
    a[2, 0] = 30.0
    a[3, [min(8191, V - 1), min(8192, V - 1), V - 1, V - 2]] = [20.0, 20.5, 21.0, 21.5]
    t, l = typed(torch, a, x)
    ids = rng.integers(0, V, (4, 3)).astype(np.int32)
    ids[:, 0], ids[:, 1] = V - 1, min(8191, V - 1)
    for top in (0, 1, 32):
        check(torch, qmv.qmv_logprobs(t.cuda(), torch.from_numpy(ids).cuda(), top_k=top), l, ids, top)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("V", [300001, 524288, 600011, 1 << 22])
def test_many_chunks(env, x, V):
    """Distinct logits, the largest ones late: groups past those that a thread keeps, chunks past those that a lane has one of."""
    torch, qmv = env
    print(x, V, flush=True)
    rng = np.random.default_rng(V)
    a = 2 * rng.standard_normal((2, V))
    late = V - 1 - rng.choice(min(V // 8, 200000), 40, replace=False)
    a[0, late] = 12.0 + 0.125 * np.arange(40)             # of bf16's numbers: distinct
    a[1, late[::5]] = 11.0
    t, l = typed(torch, a, x)
    ids = np.stack([late[:4], rng.integers(0, V, 4)]).astype(np.int32)
    got = qmv.qmv_logprobs(t.cuda(), torch.from_numpy(ids).cuda(), top_k=32)
    check(torch, got, l, ids, 32)


@pytest.mark.parametrize("V", [5, 70])
def test_more_rows_than_a_launch_is_high(env, V):
    torch, qmv = env
    R = 65535 + 700
    print(V, R, flush=True)
    rng = np.random.default_rng(V)
    t, l = typed(torch, 3 * rng.standard_normal((R, V)), "f32")
    ids = rng.integers(0, V, (R, 1)).astype(np.int32)
    got = qmv.qmv_logprobs(t.cuda(), torch.from_numpy(ids).cuda(), top_k=3)
    rows = np.concatenate([np.arange(40), np.arange(65500, 65600), np.arange(R - 40, R)])
    at = torch.from_numpy(rows).cuda()
    check(torch, [g[at] for g in got], l[rows], ids[rows], 3)
    # the others by what holds of every row: the probabilities of all tokens
    z = torch.log_softmax(t.cuda().double(), 1)
    assert float((got.logprobs[:, 0].double() - z.gather(1, torch.from_numpy(ids).cuda().long())[:, 0]).abs().max()) < 1e-5
    assert torch.equal(got.top_tokens[:, 0].long(), z.argmax(1))
    assert float((got.entropy.double() + (z.exp() * z).sum(1)).abs().max()) < 1e-5
