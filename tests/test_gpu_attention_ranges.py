"""qmv_cache_attention with queries, scales, sinks and stored blocks at the ends of their ranges."""
import pytest

from tests import attention_bounds as ab

pytestmark = pytest.mark.gpu

TYPES = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}


@pytest.fixture(scope="module")
def env():
    import torch
    import bandwidth_bound_block_amd as qmv
    assert torch.cuda.is_available()
    return torch, qmv


def filled(torch, qmv, k, v, kf, vf, P=16):
    """One sequence in a cache, its pages in reverse."""
    L, H, D = k.shape
    pages = -(-L // P)
    cache = qmv.KVCache.new(pages, kf, vf, H, D, P)
    cache.k.fill_(0xFF)
    cache.v.fill_(0xFF)
    table = torch.arange(pages - 1, -1, -1, device="cuda", dtype=torch.int32)
    j = torch.arange(L, device="cuda")
    qmv.qmv_cache_write(cache, k, v, (table[j // P] * P + j % P).to(torch.int32))
    return cache, table.view(1, -1)


@pytest.mark.parametrize("size", [1e4, 1e6, 1e7, 3e7, 1e8, 1e9])
@pytest.mark.parametrize("new", [2, 45])
@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_scores_past_24_bits(env, x, new, size):
    """Scores whose last bit is more than 1: outputs are still between the values, and equal scores share the weight."""
    torch, qmv = env
    print(x, new, size, flush=True)
    H, G, D, L = 2, 2, 64, 300
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.randn(L, H, D, generator=g, device="cuda") * 0.2
    same = [3, 40, 41, 200]
    k[same] = torch.sign(k[3:4])                            # by far the largest scores, bit for bit alike
    v = torch.randn(L, H, D, generator=g, device="cuda")
    cache, table = filled(torch, qmv, k, v, "q8_0", "q8_0")
    q = (size * torch.sign(k[3]).repeat_interleave(G, 0) * (1 + 0.3 * torch.rand(new, H * G, 1, generator=g, device="cuda"))).to(
        getattr(torch, TYPES[x]))
    got = qmv.qmv_cache_attention(cache, q, table, torch.tensor([L], dtype=torch.int32, device="cuda"))
    at = torch.tensor([int(table[0, i // 16]) * 16 + i % 16 for i in same], dtype=torch.int32, device="cuda")
    vals = qmv.qmv_cache_read(cache, at)[1].double()
    want = vals.mean(0).repeat_interleave(G, 0).expand(new, -1, -1)
    mean = vals.abs().mean(0).repeat_interleave(G, 0).expand(new, -1, -1)
    # four weights of a quarter, their quotient and sums: a few roundings; each value's own, as above; the output's
    bound = mean * ((ab.H16 * 3 if x == "bf16" else 0) + 32 * ab.U) * 1.01 + 2.0 ** -25
    ab.close(got, want, bound + ab.HALF[x] * (want.abs() + bound))


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", [1e12, 1e25, 1e30, 1e34, 1e37, 3e38])
@pytest.mark.parametrize("kf", ["q8_0", "q4_0", "q4_1"])
@pytest.mark.parametrize("new", [2, 45])
@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_large_queries(env, x, new, kf, size, sign):
    """All of the weight is on the key with the largest score, also where all scores are far below zero or past fp32."""
    torch, qmv = env
    print(x, new, kf, size, sign, flush=True)
    H, G, D, L, best = 2, 2, 128, 333, 77
    g = torch.Generator(device="cuda").manual_seed(1)
    u = torch.sign(torch.randn(H, D, generator=g, device="cuda"))
    # scores sign * c: the largest is c = 2 of 0.5..1.5, or 0.5 of 1..2
    c = 0.5 + torch.rand(L, generator=g, device="cuda")
    c[best] = 2.0
    c = sign * (c if sign > 0 else c + 0.5)
    if sign < 0:
        c[best] = -0.5
    v = torch.randn(L, H, D, generator=g, device="cuda")
    cache, table = filled(torch, qmv, c[:, None, None] * u, v, kf, "q8_0")
    q = (size * u.repeat_interleave(G, 0)).expand(new, -1, -1).to(getattr(torch, TYPES[x])).contiguous()
    assert bool(torch.isfinite(q.float()).all())
    # read back the order holds, by more than a score's rounding
    s = torch.einsum("lhd,hd->lh", qmv.qmv_cache_read(cache, torch.arange(cache.n_pages * 16, dtype=torch.int32, device="cuda"))[0][
        (table[0].long()[:, None] * 16 + torch.arange(16, device="cuda")).flatten()[:L]].double(), u.double())
    two = s.topk(2, dim=0)
    assert bool((two.indices[0] == best).all()) and bool((two.values[0] - two.values[1] > 0.05 * s.abs().amax(0)).all())
    got = qmv.qmv_cache_attention(cache, q, table.contiguous(), torch.tensor([L], dtype=torch.int32, device="cuda"))
    at = (table[0, best // 16] * 16 + best % 16).to(torch.int32).view(1)
    want = qmv.qmv_cache_read(cache, at)[1].double().repeat_interleave(G, 1).expand(new, -1, -1)
    seen = torch.arange(L - new, L, device="cuda") >= best
    assert bool(seen.all())
    # weight 1 and the value as fp16 (beside an offset's rounding, half a scale at most) or two pieces, the output rounded
    half = ab.HALF[x] + (2 * ab.H16 if x == "bf16" else 8 * ab.U)
    ab.close(got, want, want.abs() * half * 1.01 + 2.0 ** -25)


@pytest.mark.parametrize("power", [20, 60, 100, 120])
@pytest.mark.parametrize("new", [2, 45])
@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_small_queries_with_a_large_scale(env, x, new, power):
    """Powers of two moved from the queries to the scale change nothing."""
    torch, qmv = env
    print(x, new, power, flush=True)
    H, G, D, L = 2, 2, 128, 200
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(L, H, D, generator=g, device="cuda") for _ in range(2))
    cache, table = filled(torch, qmv, k, v, "q8_0", "q4_0")
    q = torch.randn(new, H * G, D, generator=g, device="cuda").to(getattr(torch, TYPES[x]))
    q = torch.where(q.abs() < 2.0 ** -5, torch.zeros_like(q), q)      # no element is below the type's normal numbers
    n = torch.tensor([L], dtype=torch.int32, device="cuda")
    got = qmv.qmv_cache_attention(cache, q * 2.0 ** -power, table, n, scale=2.0 ** power * D ** -0.5)
    ab.close(got, *ab.of_cache(qmv, cache, q, table, [L], [0, new], D ** -0.5, x))


@pytest.mark.parametrize("L,new", [(40, 1), (700, 2), (700, 45), (0, 1), (0, 45)])
@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
def test_sinks_without_bound(env, x, L, new):
    """A sink of +infinity (or past fp32 in units of log 2) leaves nothing for the keys, one of -infinity is none."""
    torch, qmv = env
    print(x, L, new, flush=True)
    H, G, D = 2, 4, 64
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn(max(L, 1), H, D, generator=g, device="cuda") for _ in range(2))
    cache, table = filled(torch, qmv, k, v, "q4_0", "q8_0")
    q = torch.randn(new, H * G, D, generator=g, device="cuda").to(getattr(torch, TYPES[x]))
    n = torch.tensor([L], dtype=torch.int32, device="cuda")
    inf = float("inf")
    sinks = torch.tensor([inf, 3.4e38, 3e38, 2e38, -inf, -3.4e38, -3e38, -1e30], device="cuda")
    got = qmv.qmv_cache_attention(cache, q, table, n, sinks=sinks)
    plain = qmv.qmv_cache_attention(cache, q, table, n)
    assert bool((got[:, :4] == 0).all())
    assert torch.equal(got[:, 4:], plain[:, 4:])


@pytest.mark.parametrize("new", [2, 45])
@pytest.mark.parametrize("kf,vf", [("q4_1", "q4_1"), ("q8_0", "q4_1"), ("q4_1", "q4_0")])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
def test_blocks_of_both_ends_of_the_range(env, x, D, kf, vf, new):
    """Q4_1 blocks with values near 65024 of both signs: code times scale is past fp16 though no value is."""
    torch, qmv = env
    print(x, D, kf, vf, new, flush=True)
    H, G, L = 2, 2, 150
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn(L, H, D, generator=g, device="cuda") for _ in range(2))
    for t, f in ((k, kf), (v, vf)):
        if f == "q4_1":
            for j in (0, 17, 60, 149 - new):
                t[j, j % H, 5:D:32] = 64000.0
                t[j, j % H, 9:D:32] = -65024.0
    cache, table = filled(torch, qmv, k, v, kf, vf)
    assert float(qmv.qmv_cache_read(cache, torch.arange(L, dtype=torch.int32, device="cuda"))[1 if vf == "q4_1" else 0].abs().nan_to_num().max()) > 6e4
    # queries so small that the large keys have ordinary scores
    q = ((2e-5 if kf == "q4_1" else 1.0) * torch.randn(new, H * G, D, generator=g, device="cuda")).to(getattr(torch, TYPES[x]))
    got = qmv.qmv_cache_attention(cache, q, table, torch.tensor([L], dtype=torch.int32, device="cuda"))
    ab.close(got, *ab.of_cache(qmv, cache, q, table, [L], [0, new], D ** -0.5, x, k_spread=3.0 if kf == "q4_1" else 1.0))
