"""qmv_cache_attention in the forms between single tokens and prompts: 17 to 32 rows of queries a request, 33 to 128, heads of
256, every pair of formats, and more tiles of rows than a launch has workgroups for."""
import numpy as np
import pytest

from tests import attention_bounds as ab
from tests.test_gpu_attention import random_cache

pytestmark = pytest.mark.gpu

PAIRS = [(a, b) for a in ("q8_0", "q4_0", "q4_1") for b in ("q8_0", "q4_0", "q4_1")]
TYPES = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}


@pytest.fixture(scope="module")
def env():
    import torch
    import bandwidth_bound_block_amd as qmv
    assert torch.cuda.is_available()
    return torch, qmv


# heads of queries per key/value head, new tokens of each request: rows are their products
@pytest.mark.parametrize("pair", PAIRS, ids="-".join)
@pytest.mark.parametrize("x,D,G,new,window", [
    ("bf16", 128, 4, [5, 1, 8], 0),          # 20, 4, 32
    ("bf16", 128, 7, [3, 4], 100),           # 21, 28
    ("bf16", 64, 4, [5, 8, 6], 0),
    ("bf16", 256, 4, [5, 1, 3], 0),
    ("bf16", 256, 16, [1, 2], 0),
    ("f32", 128, 4, [7, 5], 0),
    ("bf16", 128, 8, [5, 16, 9, 1], 0),      # 40, 128, 72, 8
    ("bf16", 64, 8, [9, 5], 70),
    ("f16", 128, 8, [5, 12], 0),
    ("bf16", 256, 8, [5, 8], 0),
])
def test_rows_between(env, x, D, G, new, window, pair):
    torch, qmv = env
    print(x, D, G, new, window, pair, flush=True)
    kf, vf = pair
    H, P = 2, 32
    g = torch.Generator(device="cuda").manual_seed(D + G)
    lens = [[701, 90, 333, 40][i] for i in range(len(new))]
    cache, table = random_cache(torch, qmv, g, kf, vf, H, D, P, lens)
    q = torch.randn(sum(new), H * G, D, generator=g, device="cuda").to(getattr(torch, TYPES[x]))
    begin = np.concatenate([[0], np.cumsum(new)])
    got = qmv.qmv_cache_attention(cache, q, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                  torch.from_numpy(begin.astype(np.int32)).cuda(), max(new), window=window)
    ab.close(got, *ab.of_cache(qmv, cache, q, table, lens, begin, D ** -0.5, x, window, k_spread=3.0 if kf == "q4_1" else 1.0))


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
def test_as_many_parts_as_workgroups(env, x):
    """Many requests of 20 rows, each many blocks of keys: a workgroup's share is parts of several units."""
    torch, qmv = env
    print(x, flush=True)
    R, H, G, D, P, new = 90, 4, 4, 128, 64, 5
    g = torch.Generator(device="cuda").manual_seed(7)
    lens = [1900]
    cache, table = random_cache(torch, qmv, g, "q4_0", "q4_0", H, D, P, lens)
    n = torch.randint(new, 1900, (R,), generator=g, device="cuda").to(torch.int32)
    table = table.expand(R, -1).contiguous()
    q = torch.randn(R * new, H * G, D, generator=g, device="cuda").to(getattr(torch, TYPES[x]))
    got = qmv.qmv_cache_attention(cache, q, table, n)
    for r in (0, 1, 44, 88, 89):
        rows = slice(r * new, (r + 1) * new)
        ab.close(got[rows], *ab.of_cache(qmv, cache, q[rows], table[:1], [int(n[r])], [0, new], D ** -0.5, x))


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 256])
def test_more_tiles_than_workgroups(env, x, D):
    """A launch has 2^22 workgroups: past that one of them goes over several tiles of rows, here all of a request's."""
    torch, qmv = env
    H, P, R, most = 1024, 16, 4100, 600
    assert H * R > 1 << 22
    g = torch.Generator(device="cuda").manual_seed(9)
    new = [1] * R
    at = (1, R - 2)
    new[at[0]], new[at[1]] = most, 300
    lens = [1 + r % 40 for r in range(R)]
    lens[at[0]], lens[at[1]] = 640, 500
    print(x, D, sum(new), flush=True)
    cache = qmv.KVCache.new(40, "q4_0", "q8_0", H, D, P)
    for p in range(40):
        k, v = (torch.randn(P, H, D, generator=g, device="cuda") for _ in range(2))
        qmv.qmv_cache_write(cache, k, v, torch.arange(p * P, (p + 1) * P, dtype=torch.int32, device="cuda"))
    table = torch.stack([torch.randperm(40, generator=g, device="cuda") for _ in range(R)]).to(torch.int32)
    q = torch.randn(sum(new), H, D, generator=g, device="cuda").to(getattr(torch, TYPES[x]))
    begin = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = qmv.qmv_cache_attention(cache, q, table, n, begin, most)
    for r in at:        # alone, a workgroup has one tile
        rows = slice(int(begin[r]), int(begin[r + 1]))
        want = qmv.qmv_cache_attention(cache, q[rows], table[r:r + 1], n[r:r + 1])
        assert torch.equal(got[rows], want)
        few = slice(rows.start + 260, rows.start + 300)
        part, bound = ab.of_cache(qmv, cache, q[few], table[r:r + 1], [int(n[r]) - (new[r] - 300)], [0, 40], D ** -0.5, x)
        ab.close(got[few], part, bound)
    for r in (0, 2, R // 2, R - 1):
        rows = slice(int(begin[r]), int(begin[r + 1]))
        want, bound = ab.of_cache(qmv, cache, q[rows], table[r:r + 1], n[r:r + 1].tolist(), [0, 1], D ** -0.5, x)
        ab.close(got[rows], want, bound)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("G,most", [(2, 90), (4, 8), (64, 3)])
def test_replayed_with_other_requests(env, G, most, x):
    """q_begin, lengths and tables change between replays of one graph, and with them which kernel has a request."""
    torch, qmv = env
    print(G, most, x, flush=True)
    g = torch.Generator(device="cuda").manual_seed(11)
    rng = np.random.default_rng(most)
    H, D, P, R, T = 2, 64, 16, 6, 3 * most
    cache, full = random_cache(torch, qmv, g, "q8_0", "q4_0", H, D, P, [900] * R)
    q = torch.randn(T, H * G, D, generator=g, device="cuda").to(getattr(torch, TYPES[x]))
    table, n = full.clone(), torch.full((R,), 40, dtype=torch.int32, device="cuda")
    begin = torch.zeros(R + 1, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    ws = torch.empty(qmv.lib().qmv_cache_attention_workspace_bytes(cache._struct, R, T, H * G, most), dtype=torch.uint8, device="cuda")

    def call(to, workspace):
        return qmv.qmv_cache_attention(cache, q, table, n, begin, most, window=500, out=to, workspace=workspace)
    call(out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, ws)
    for i in range(8):
        new = rng.integers(0, most + 1, R) * rng.integers(0, 2, R) if i else np.zeros(R, int)
        while new.sum() > T:
            new[rng.integers(R)] = rng.integers(0, 2)
        at = np.concatenate([[0], np.cumsum(new)])
        lens = np.maximum(rng.integers(1, 900, R), new)
        begin.copy_(torch.from_numpy(at.astype(np.int32)))
        n.copy_(torch.from_numpy(lens.astype(np.int32)))
        table.copy_(full[torch.randperm(R, generator=g, device="cuda")])
        q.normal_(generator=g)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert bool((out[at[-1]:] == 7).all())
        assert torch.equal(out, call(torch.full_like(out, 7.0), None)), i
        if at[-1]:
            want, bound = ab.of_cache(qmv, cache, q, table, lens, at, D ** -0.5, x, 500)
            ab.close(out[:at[-1]], want[:at[-1]], bound[:at[-1]])
        torch.randn(5000, device="cuda").sum()


@pytest.mark.parametrize("x,new", [("bf16", 1), ("f32", 2), ("bf16", 40)])
def test_millions_of_keys(env, x, new):
    """One request whose weights are all alike in size: sums of 3 million of them."""
    torch, qmv = env
    L, D, P = 3_000_001, 64, 4096
    print(x, new, L, flush=True)
    g = torch.Generator(device="cuda").manual_seed(13)
    pages = -(-L // P)
    cache = qmv.KVCache.new(pages, "q4_0", "q8_0", 1, D, P)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    for c in range(0, L, 1 << 18):
        j = torch.arange(c, min(c + (1 << 18), L), device="cuda")
        k = torch.randn(j.numel(), 1, D, generator=g, device="cuda")
        v = 1.0 + torch.randn(j.numel(), 1, D, generator=g, device="cuda")
        qmv.qmv_cache_write(cache, k, v, (table[j // P] * P + j % P).to(torch.int32))
    q = torch.randn(new, 1, D, generator=g, device="cuda").to(getattr(torch, TYPES[x]))
    n = torch.tensor([L], dtype=torch.int32, device="cuda")
    got = qmv.qmv_cache_attention(cache, q, table.view(1, -1), n)
    total, out = torch.zeros(new, 1, dtype=torch.float64, device="cuda"), torch.zeros(new, D, dtype=torch.float64, device="cuda")
    pos = torch.arange(L - new, L, device="cuda")[:, None]
    for c in range(0, L, 1 << 18):
        j = torch.arange(c, min(c + (1 << 18), L), device="cuda")
        k, v = (t[:, 0].double() for t in qmv.qmv_cache_read(cache, (table[j // P] * P + j % P).to(torch.int32)))
        w = torch.exp(torch.matmul(q[:, 0].double(), k.t().contiguous()) * D ** -0.5).masked_fill(j > pos, 0.0)
        total += w.sum(1, keepdim=True)
        out += torch.matmul(w, v)
    want = (out / total)[:, None]
    # outputs are means of values about 1, of roundings of random signs but for those of the sums: a wave adds some 1500 (two
    # rounds of 32 keys) or, in the kernel for many rows, 3000 times at most, each 2^-24 of a part of the sum
    off = float((got.double() - want).abs().max())
    print("off", off, flush=True)
    assert off <= ab.HALF[x] * 1.5 + (2 * ab.H16 if x == "bf16" else 0) + 6000 * ab.U
