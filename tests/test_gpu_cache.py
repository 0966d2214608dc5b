"""qmv_cache_write and qmv_cache_read on an MI355X: the stored bytes are those of the encoders in 64 bits, whole pages compared."""
import numpy as np
import pytest

from tests import cache_values as cv

pytestmark = pytest.mark.gpu

FMTS = ["q8_0", "q4_0", "q4_1"]


@pytest.fixture(scope="module")
def env():
    import torch
    import bandwidth_bound_block_amd as qmv
    assert torch.cuda.is_available()
    return torch, qmv


def typed(torch, a, x):
    """float64 numpy -> a CPU tensor of the type, and its exact values."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to({"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[x])
    return t, t.to(torch.float64).numpy()


def cache_of(torch, qmv, kp, vp, kf, vf, heads, D, P):
    put = lambda a: torch.from_numpy(a.reshape(-1).copy()).cuda()      # noqa: E731
    return qmv.KVCache(put(kp), put(vp), kf, vf, heads, D, P)


def stored(cache, side, shape):
    return getattr(cache, side).cpu().numpy().reshape(shape)


def values(rng, T, heads, D, hard):
    """Keys or values, with blocks that are hard to encode among them."""
    x = rng.standard_normal((T, heads, D)) * np.exp(rng.standard_normal((1, heads, D)))
    if not hard:
        return x
    b = x.reshape(T, heads, -1, 32)
    kinds = rng.integers(0, 14, b.shape[:-1])
    for at in np.ndindex(*kinds.shape):
        k, w = kinds[at], b[at]
        if k == 1:
            w[:] = 0.0
        elif k == 2:
            w[:] = -0.0
        elif k == 3:                              # exactly between codes: the scale is a power of two
            w[:] = np.sign(w) * (np.floor(np.abs(w) * 4) + 0.5) * 2.0 ** -6
            w[0] = 127 * 2.0 ** -6
        elif k == 4:                              # the same for 4 bits
            w[:] = (rng.integers(-8, 8, 32) + 0.5) * 0.25
            w[5] = -2.0
        elif k == 5:                              # largest values of both signs
            w[rng.integers(0, 32)] = 3.5
            w[rng.integers(0, 32)] = -3.5
            w[:] = np.clip(w, -3.5, 3.5)
        elif k == 6:
            w *= 1e-7                             # scales below fp16's normal numbers, and 0
        elif k == 7:
            w *= 1e-9
        elif k == 8:
            w *= 1e-30
        elif k == 9:
            w *= 30000.0                          # past the limit
        elif k == 10:
            w[:] = 1000.0 + 0.01 * w              # a small spread far from 0
        elif k == 11:
            w[:] = w[0]
    return x


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kf,vf", [("q8_0", "q4_1"), ("q4_0", "q8_0"), ("q4_1", "q4_0")])
@pytest.mark.parametrize("heads,D,P,T", [(1, 64, 16, 1), (3, 64, 32, 37), (2, 128, 16, 70), (5, 256, 64, 19)])
def test_written_bytes(env, x, kf, vf, heads, D, P, T):
    torch, qmv = env
    print(x, kf, vf, heads, D, P, T, flush=True)
    rng = np.random.default_rng(7 * T + D + heads)
    n = T // P + 3
    with np.errstate(over="ignore"):
        k, ke = typed(torch, np.clip(values(rng, T, heads, D, True), -60000, 60000) if x == "f16" else values(rng, T, heads, D, True), x)
        v, ve = typed(torch, np.clip(values(rng, T, heads, D, True), -60000, 60000) if x == "f16" else values(rng, T, heads, D, True), x)
    slots = rng.permutation(n * P)[:T].astype(np.int32)
    left = slots.copy()
    for i in range(0, T, 5):                      # padding
        left[i] = [-1, n * P, -2 ** 31, 2 ** 31 - 1][i // 5 % 4] if T > 1 else left[i]
    kp, vp = cv.empty_pages(kf, n, heads, D, P), cv.empty_pages(vf, n, heads, D, P)
    cache = cache_of(torch, qmv, kp, vp, kf, vf, heads, D, P)
    qmv.qmv_cache_write(cache, k.cuda(), v.cuda(), torch.from_numpy(left).cuda())
    for pages, e, f in ((kp, ke, kf), (vp, ve, vf)):
        c, d, m = cv.encode(e, f)
        for t in range(T):
            if 0 <= left[t] < n * P:
                for h in range(heads):
                    cv.put(pages, f, D, P, left[t] // P, left[t] % P, h, c[t, h], d[t, h], None if m is None else m[t, h])
    assert np.array_equal(stored(cache, "k", kp.shape), kp)
    assert np.array_equal(stored(cache, "v", vp.shape), vp)
    # and back, in every type, one slot twice
    ids = np.concatenate([left, left[:1]])
    for y in ("f32", "f16", "bf16"):
        dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[y]
        got = qmv.qmv_cache_read(cache, torch.from_numpy(ids).cuda(), dtype=dt)
        for g, e, f in zip(got, (ke, ve), (kf, vf)):
            want = cv.decode(*cv.encode(e, f), f)
            want = np.concatenate([want, want[:1]])
            want[(ids < 0) | (ids >= n * P)] = np.nan
            with np.errstate(over="ignore"):
                want = torch.from_numpy(want).to(torch.float32).to(dt)
            assert torch.equal(torch.nan_to_num(g.cpu(), nan=77.0), torch.nan_to_num(want, nan=77.0)), (y, f)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_values_that_are_not_finite(env, fmt, x):
    """A block with one reads back as NaN throughout, the blocks beside it as they are."""
    torch, qmv = env
    print(fmt, x, flush=True)
    rng = np.random.default_rng(5)
    T, heads, D, P = 6, 2, 128, 16
    a = values(rng, T, heads, D, False)
    for i, bad in enumerate((np.nan, np.inf, -np.inf, np.nan)):
        a[i, i % 2, 40 * i % D] = bad
    k, e = typed(torch, a, x)
    cache = qmv.KVCache.new(1, fmt, fmt, heads, D, P)
    slots = torch.arange(T, dtype=torch.int32).cuda()
    qmv.qmv_cache_write(cache, k.cuda(), k.cuda(), slots)
    got = qmv.qmv_cache_read(cache, slots)[0].cpu().numpy()
    want = cv.decode(*cv.encode(e, fmt), fmt)
    assert np.isnan(want).sum() == 4 * 32
    assert np.array_equal(np.nan_to_num(got, nan=77.0), np.nan_to_num(want, nan=77.0).astype(np.float32))


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
def test_strides_and_alignment(env, x):
    """Rows of a fused q, k, v projection, one element off 16 bytes, tokens in reverse: the same bytes."""
    torch, qmv = env
    print(x, flush=True)
    rng = np.random.default_rng(11)
    T, heads, D, P = 21, 2, 64, 16
    k, _ = typed(torch, values(rng, T, heads, D, True).clip(-60000, 60000), x)
    v, _ = typed(torch, values(rng, T, heads, D, True).clip(-60000, 60000), x)
    slots = torch.from_numpy(rng.permutation(3 * P)[:T].astype(np.int32)).cuda()
    k, v = k.cuda(), v.cuda()

    def pages(kk, vv):
        c = qmv.KVCache(*(torch.zeros(3 * qmv.cache_page_bytes(f, heads, D, P), dtype=torch.uint8, device="cuda") for f in ("q4_0", "q8_0")),
                        "q4_0", "q8_0", heads, D, P)
        qmv.qmv_cache_write(c, kk, vv, slots)
        return torch.cat([c.k, c.v]).cpu()
    want = pages(k, v)
    for lead, pad in ((1, 0), (8, 8), (3, 5), (4, 4)):
        rows = torch.full((T, lead + 2 * heads * (D + pad) + pad), 9.0, dtype=k.dtype, device="cuda")
        kk = rows[:, lead:lead + heads * (D + pad)].unflatten(1, (heads, D + pad))[..., :D]
        vv = rows[:, lead + heads * (D + pad):lead + 2 * heads * (D + pad)].unflatten(1, (heads, D + pad))[..., :D]
        kk.copy_(k)
        vv.copy_(v)
        assert torch.equal(pages(kk, vv), want), (lead, pad)
    # the same token for all slots (stride 0)
    one = pages(k[:1].expand(T, heads, D), v[:1].expand(T, heads, D))
    assert torch.equal(one, pages(k[:1].repeat(T, 1, 1), v[:1].repeat(T, 1, 1)))


def test_many_tokens_and_only_one_output(env):
    """More tokens than the grid has threads at a time is a loop; keys alone."""
    torch, qmv = env
    T, heads, D, P = 30000, 64, 64, 4096
    print(T, heads, flush=True)
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.randn(T, heads, D, generator=g, device="cuda", dtype=torch.float16)
    cache = qmv.KVCache.new(8, "q8_0", "q8_0", heads, D, P)
    slots = torch.randperm(8 * P, generator=g, device="cuda")[:T].to(torch.int32)
    qmv.qmv_cache_write(cache, k, k, slots)
    got = torch.full((T, heads, D), 5.0, device="cuda")
    lib = qmv.lib()
    assert lib.qmv_cache_read(cache._struct, slots.data_ptr(), T, got.data_ptr(), 0, 0, torch.cuda.current_stream().cuda_stream) == 0
    d = (k.float().unflatten(-1, (2, 32)).abs().amax(-1) / 127).half().float()
    # half a step, and the rounding of the scale: the largest value is 127 steps
    off = (got - k.float()).unflatten(-1, (2, 32)).abs()
    assert bool((off <= (0.5 + 127 * 2.0 ** -11 + 0.01) * d.unsqueeze(-1)).all())


def test_captured_and_replayed(env):
    torch, qmv = env
    rng = np.random.default_rng(2)
    T, heads, D, P = 9, 2, 128, 16
    k, v = (torch.from_numpy(rng.standard_normal((T, heads, D)).astype(np.float32)).cuda() for _ in range(2))
    slots = torch.arange(3, 3 + T, dtype=torch.int32).cuda()
    cache = qmv.KVCache.new(2, "q4_0", "q4_1", heads, D, P)
    ko, vo = torch.empty(T, heads, D, device="cuda"), torch.empty(T, heads, D, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        qmv.qmv_cache_write(cache, k, v, slots)
        qmv.qmv_cache_read(cache, slots, k=ko, v=vo)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmv.qmv_cache_write(cache, k, v, slots)
        qmv.qmv_cache_read(cache, slots, k=ko, v=vo)
    for i in range(4):
        k.copy_(torch.from_numpy(rng.standard_normal((T, heads, D)).astype(np.float32)))
        v.mul_(1.5)
        slots.add_(2)
        graph.replay()
        torch.cuda.synchronize()
        for g, e, f in ((ko, k, "q4_0"), (vo, v, "q4_1")):
            want = cv.decode(*cv.encode(e.cpu().double().numpy(), f), f).astype(np.float32)
            assert np.array_equal(g.cpu().numpy(), want), (i, f)
        torch.randn(1000, device="cuda").sum()
