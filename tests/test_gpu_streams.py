"""Calls on a stream that is not the current one, on an MI355X: what they make is theirs from the call on until they are done,
whatever the current stream has queued before or allocates after."""
import numpy as np
import pytest

import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import bandwidth_bound_block_amd as qmv
    assert torch.cuda.is_available()
    return torch, qmv


class Calls:
    """Inputs on the GPU, and calls that return their outputs as a tuple."""

    def __init__(self, torch, qmv):
        g = torch.Generator().manual_seed(3)
        N, K, T, S, E, F, V = 96, 256, 40, 2, 4, 64, 700

        def put(fmt, tag, n, k):
            return torch.from_numpy(wl.quant_weights(fmt, f"t/streams/{tag}", n, k).reshape(-1)).cuda()

        def randn(*shape):
            return torch.randn(*shape, generator=g).cuda()
        W, x = put("q4_0", "w", N, K), randn(T, K)
        ids = torch.randint(0, E, (T, S), generator=g, dtype=torch.int32).cuda()
        owner = torch.randint(-1, 3, (T,), generator=g, dtype=torch.int32).cuda()
        A, B, scales, weights = randn(3, 8, K), randn(3, N, 8), randn(3), randn(T, S)
        W1, W2 = put("q4_0", "gu", E * 2 * F, K), put("q4_0", "down", E * K, F)
        s1, s2 = 2 * F * qmv.row_bytes("q4_0", K), K * qmv.row_bytes("q4_0", F)
        logits, x8 = randn(6, 4, V), randn(8, F)
        q = torch.softmax(randn(6, 3, V), -1)
        drafted = torch.randint(0, V, (6, 3), generator=g, dtype=torch.int32).cuda()
        n, u, ul = torch.full((6,), 3, dtype=torch.int32).cuda(), torch.rand(6, 3, generator=g).cuda(), torch.rand(6, generator=g).cuda()

        def experts(s):
            plan = qmv.qmv_group_plan(ids, E, stream=s)
            h = qmv.qmv_moe_grouped_swiglu("q4_0", W1, s1, E, F, K, plan, S, x, stream=s)
            y = qmv.qmv_moe_grouped("q4_0", W2, s2, E, K, F, plan, S, h, stream=s)
            return (qmv.qmv_moe_weighted_sum(y, weights, stream=s),)
        self.calls = {
            "experts": experts,
            "lora": lambda s: (qmv.qmv_lora("q4_0", W, N, K, x, A, B, scales, owner, stream=s),),
            "lora few": lambda s: (qmv.qmv_lora("q4_0", W, N, K, x[:4], A, B, scales, owner[:4], stream=s),),
            "verify": lambda s: qmv.qmv_spec_verify(logits, q, drafted, n, u, ul, stream=s),
            "matvec": lambda s: (qmv.qmv_matvec_xt("q4_0", W, N, K, x[:8], stream=s),),
            "moe": lambda s: (qmv.qmv_moe("q4_0", W2, s2, E, K, F, ids[:8], x8, stream=s),),
        }
        # sizes in bytes that the calls above ask for, about
        self.sizes = sorted({4 * T * K, 4 * T * S * K, 4 * T * S * F, 4 * T * N, 16 * N, 32 * N, 32 * S * K, 4 * T * 8 * 16, 4096, 512,
                             1024, 2048, 8192, 16384})
        self.busy = randn(4096, 4096)


NAMES = ["experts", "lora", "lora few", "verify", "matvec", "moe"]


@pytest.fixture(scope="module")
def made(env):
    return Calls(*env)


def work(c):
    """A few milliseconds of the current stream."""
    m = c.busy
    for _ in range(20):
        m = m @ c.busy * 0.01
    return m


@pytest.mark.parametrize("name", NAMES)
def test_memory_that_queued_work_still_writes(env, made, name):
    """The current stream has writes queued to tensors that are freed already: a call on another stream gets none of them."""
    torch, _ = env
    print(name, flush=True)
    want = [t.cpu() for t in made.calls[name](None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    work(made)
    mine = set()
    for size in made.sizes:
        t = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
        for v in t:
            v.fill_(255)
            mine.add(v.data_ptr())
        del t, v
    got = made.calls[name](side)
    assert all(t.data_ptr() not in mine for t in got)
    side.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_call_still_uses(env, made, name):
    """The call waits on its stream; meanwhile the current stream allocates and writes: what the call holds is not among it."""
    torch, _ = env
    print(name, flush=True)
    want = [t.cpu() for t in made.calls[name](None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        work(made)
    got = made.calls[name](side)
    for _ in range(3):
        for size in made.sizes:
            torch.empty(size, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.cpu(), b)


def test_an_output_dropped_while_the_current_stream_reads_it(env, made):
    torch, _ = env
    side = torch.cuda.Stream()
    want = made.calls["lora"](None)[0].cpu()
    torch.cuda.synchronize()
    y = made.calls["lora"](side)[0]
    torch.cuda.current_stream().wait_stream(side)
    work(made)
    copy = y.clone()
    at = y.data_ptr()
    del y
    more = [made.calls["lora"](side)[0] for _ in range(4)]      # of the same size, while the copy has not begun
    assert all(t.data_ptr() != at for t in more)
    torch.cuda.synchronize()
    assert torch.equal(copy.cpu(), want)


def test_a_plan_used_on_another_stream(env):
    torch, qmv = env
    E, N, K, T = 4, 64, 256, 50
    g = torch.Generator().manual_seed(1)
    W = torch.from_numpy(wl.quant_weights("q4_0", "t/streams/plan", E * N, K).reshape(-1)).cuda()
    stride = N * qmv.row_bytes("q4_0", K)
    ids = torch.randint(0, E, (T, 1), generator=g, dtype=torch.int32).cuda()
    x = torch.randn(T, K, generator=g).cuda()
    want = qmv.qmv_moe_grouped("q4_0", W, stride, E, N, K, qmv.qmv_group_plan(ids, E), 1, x).cpu()
    busy = torch.randn(4096, 4096, generator=g).cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    plan = qmv.qmv_group_plan(ids, E)
    size = plan.buffer.numel()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m = busy
        for _ in range(20):
            m = m @ busy * 0.01
    got = qmv.qmv_moe_grouped("q4_0", W, stride, E, N, K, plan, 1, x, stream=side)
    at = plan.buffer.data_ptr()
    del plan
    others = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(4)]     # while the product has not begun
    assert all(t.data_ptr() != at for t in others)
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy(), want.numpy())
