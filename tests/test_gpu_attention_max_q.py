"""qmv_cache_attention where requests have more query tokens than max_q: query i of n stands at kv_lens - n + i whether the last
ones are left out or not, and sees no token behind it."""
import numpy as np
import pytest

from tests import attention_bounds as ab
from tests.test_gpu_attention import random_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import bandwidth_bound_block_amd as qmv
    assert torch.cuda.is_available()
    return torch, qmv


@pytest.mark.parametrize("window", [0, 9])
@pytest.mark.parametrize("x,D,G,lens,new,most", [
    ("bf16", 64, 2, [50, 40, 44, 0, 60], [3, 0, 2, 0, 7], 2),
    ("f16", 128, 1, [50, 9, 44, 3], [4, 9, 1, 3], 3),
    ("bf16", 64, 2, [90, 40, 44, 0, 70], [60, 0, 3, 0, 45], 40),
    ("f32", 64, 4, [700, 5, 130], [100, 5, 120], 64),
    ("bf16", 128, 3, [400], [130], 77),
    ("bf16", 128, 1, [40, 3, 2], [10, 8, 50], 4),        # more query tokens than there are keys: positions before the sequence
    ("f16", 64, 2, [40, 60], [90, 61], 30),
    ("f32", 256, 1, [35], [36], 35),
])
def test_more_queries_than_max_q(env, x, D, G, lens, new, most, window):
    torch, qmv = env
    print(x, D, G, lens, new, most, window, flush=True)
    g = torch.Generator(device="cuda").manual_seed(3)
    H = 2
    cache, table = random_cache(torch, qmv, g, "q8_0", "q4_0", H, D, 16, lens)
    begin = np.concatenate([[0], np.cumsum(new)])
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[x]
    q = torch.randn(int(begin[-1]) + 2, H * G, D, generator=g, device="cuda").to(dt)
    out = torch.full(q.shape, 7.0, dtype=dt, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qmv.qmv_cache_attention(cache, q, table, n, torch.from_numpy(begin.astype(np.int32)).cuda(), most, window=window, out=out)
    want, bound = ab.of_cache(qmv, cache, q, table, lens, begin, D ** -0.5, x, window)
    kept = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    for r in range(len(new)):
        kept[begin[r]:begin[r] + min(new[r], most)] = True
    assert bool((out[~kept] == 7).all())
    ab.close(out[kept], want[kept], bound[kept])


def test_bounds_of_requests_that_are_out_of_order_or_out_of_range(env):
    """Nothing outside the tensors is touched, whatever q_begin holds."""
    torch, qmv = env
    g = torch.Generator(device="cuda").manual_seed(5)
    cache, table = random_cache(torch, qmv, g, "q4_0", "q4_1", 2, 64, 16, [50, 40, 44, 1, 60])
    n = torch.tensor([50, 40, 44, 0, 60], dtype=torch.int32, device="cuda")
    q = torch.randn(75, 4, 64, generator=g, device="cuda").bfloat16()
    around = torch.full((80, 4, 64), 7.0, dtype=q.dtype, device="cuda")
    for most in (1, 2, 39, 75):
        for b in ([0, 3, 1, 2, 2, 4], [-5, 0, 1, 2, 3, 2 ** 31 - 1], [9, 9, 9, 0, 0, 0], [75, 0, 0, 0, 0, 75], [-2 ** 31, 60, 2, 70, 71, 90]):
            print(most, b, flush=True)
            qmv.qmv_cache_attention(cache, q, table, n, torch.tensor(b, dtype=torch.int32, device="cuda"), most, out=around[2:77])
            torch.cuda.synchronize()
            assert bool((around[:2] == 7).all()) and bool((around[77:] == 7).all())
