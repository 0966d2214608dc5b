"""qmv_cache_attention where one key has nearly all of the weight and no value: the output is what the others' weights make."""
import pytest

from tests import attention_bounds as ab

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import bandwidth_bound_block_amd as qmv
    assert torch.cuda.is_available()
    return torch, qmv


TYPES = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}


def sink_cache(torch, qmv, g, kf, vf, H, D, P, L, gap, at):
    """One sequence whose key `at` scores `gap` above all others, for queries near u [H, D], and has the value 0; the other
    values are about 1000."""
    u = torch.sign(torch.randn(H, D, generator=g, device="cuda"))
    k = 0.3 * torch.randn(L, H, D, generator=g, device="cuda")
    v = 1000.0 + 400.0 * torch.randn(L, H, D, generator=g, device="cuda")
    k[at] = u * (gap * D ** -0.5)
    v[at] = 0.0
    pages = -(-L // P)
    cache = qmv.KVCache.new(pages + 2, kf, vf, H, D, P)
    cache.k.fill_(0xFF)
    cache.v.fill_(0xFF)
    table = torch.randperm(pages + 2, generator=g, device="cuda")[:pages].to(torch.int32)
    j = torch.arange(L, device="cuda")
    qmv.qmv_cache_write(cache, k, v, (table[j // P] * P + j % P).to(torch.int32))
    return cache, table, u


# requests, heads: 64 of 4 fill the GPU, a wave of the kernel for few rows has many blocks of keys; one of one is split
@pytest.mark.parametrize("gap", [12, 16, 18, 20, 24])
@pytest.mark.parametrize("new,G", [(1, 4), (3, 7), (40, 2)])
@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("R,H,L,at", [(64, 4, 1500, 0), (1, 1, 2500, 1100)])
def test_small_weights(env, R, H, L, at, x, new, G, gap):
    torch, qmv = env
    print(R, H, L, at, x, new, G, gap, flush=True)
    D, P = 128, 32
    g = torch.Generator(device="cuda").manual_seed(gap + new)
    cache, row, u = sink_cache(torch, qmv, g, "q8_0", "q8_0", H, D, P, L, gap, at)
    q = u.repeat_interleave(G, 0) + 0.02 * torch.randn(R * new, H * G, D, generator=g, device="cuda")
    q = q.to(getattr(torch, TYPES[x]))
    table = row.expand(R, -1).contiguous()
    lens = torch.full((R,), L, dtype=torch.int32, device="cuda")
    got = qmv.qmv_cache_attention(cache, q, table, lens)
    for r in sorted({0, R // 2, R - 1}):
        rows = slice(r * new, (r + 1) * new)
        want, bound = ab.of_cache(qmv, cache, q[rows], table[:1], [L], [0, new], D ** -0.5, x)
        ab.close(got[rows], want, bound)


@pytest.mark.parametrize("kf,vf", [("q4_0", "q4_0"), ("q4_1", "q4_1"), ("q8_0", "q4_1")])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [2, 50])
@pytest.mark.parametrize("x", ["f16", "bf16"])
def test_formats_with_a_sink(env, x, new, D, kf, vf):
    """The same in other formats and sizes, beside a logit of a sink that is as large as the key's score."""
    torch, qmv = env
    print(x, new, D, kf, vf, flush=True)
    H, G, P, L, R, gap = 4, 2, 16, 900, 48, 17
    g = torch.Generator(device="cuda").manual_seed(D + new)
    cache, row, u = sink_cache(torch, qmv, g, kf, vf, H, D, P, L, gap, 5)
    q = (u.repeat_interleave(G, 0) + 0.02 * torch.randn(R * new, H * G, D, generator=g, device="cuda")).to(getattr(torch, TYPES[x]))
    table = row.expand(R, -1).contiguous()
    lens = torch.full((R,), L, dtype=torch.int32, device="cuda")
    sinks = torch.tensor([17.0, 15.0, 18.0, -5.0, 16.5, 0.0, 17.5, 16.0], device="cuda")
    got = qmv.qmv_cache_attention(cache, q, table, lens, sinks=sinks)
    for r in (0, R - 1):
        rows = slice(r * new, (r + 1) * new)
        want, bound = ab.of_cache(qmv, cache, q[rows], table[:1], [L], [0, new], D ** -0.5, x, sinks=sinks,
                                  k_spread=3.0 if kf == "q4_1" else 1.0)
        ab.close(got[rows], want, bound)
