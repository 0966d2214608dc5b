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
