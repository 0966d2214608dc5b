"""qmv_cache_attention on an MI355X against 64-bit values.  Memory that no query sees is full of NaN scales, and table entries
of pages that none sees are out of range."""
import numpy as np
import pytest

from tests import cache_values as cv

pytestmark = pytest.mark.gpu

FEW = 32          # rows of queries of a request up to which DEQ(K) is used as codes


@pytest.fixture(scope="module")
def env():
    import torch
    import bandwidth_bound_block_amd as qmv
    assert torch.cuda.is_available()
    return torch, qmv


def typed(torch, a, x):
    t = torch.from_numpy(np.ascontiguousarray(a)).to({"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[x])
    return t, t.to(torch.float64).numpy()


class Setup:
    """A cache with the tokens of some requests in pages anywhere."""

    def __init__(self, torch, qmv, seed, kf, vf, H, D, P, lens, spare=2, kstd=1.0, first=None):
        """first: the first position that is stored, per request (what a window leaves of the sequence)."""
        rng = np.random.default_rng(seed)
        self.torch, self.qmv, self.rng = torch, qmv, rng
        self.H, self.D, self.P, self.kf, self.vf = H, D, P, kf, vf
        first = [0] * len(lens) if first is None else first
        need = [range(f // P, -(-n // P)) for n, f in zip(lens, first)]
        pages = sum(len(p) for p in need) + 1
        order = rng.permutation(pages)
        self.max_pages = max(1, max(-(-n // P) for n in lens)) + spare
        self.table = rng.choice([-1, -2 ** 31, pages, 2 ** 31 - 1], (len(lens), self.max_pages)).astype(np.int32)
        kp, vp = (cv.empty_pages(f, pages, H, D, P, 0xFF) for f in (kf, vf))
        self.k, self.v = [], []
        at = 0
        for r, n in enumerate(lens):
            for p in need[r]:
                self.table[r, p] = order[at]
                at += 1
            both = []
            for f, dest, std in ((kf, kp, kstd), (vf, vp, 1.0)):
                x = (rng.standard_normal((n, H, D)) * std + (0.5 if f == "q4_1" else 0.0)).astype(np.float32).astype(np.float64)
                c, d, m = cv.encode(x, f)
                for j in range(first[r], n):
                    for h in range(H):
                        cv.put(dest, f, D, P, self.table[r, j // P], j % P, h, c[j, h], d[j, h], None if m is None else m[j, h])
                both.append(cv.decode(c, d, m, f))
            self.k.append(both[0])
            self.v.append(both[1])
        self.lens = np.array(lens, np.int32)
        self.kp, self.vp = kp, vp
        self.upload()

    def upload(self):
        put = lambda a: self.torch.from_numpy(np.ascontiguousarray(a).reshape(-1).copy()).cuda()      # noqa: E731
        self.cache = self.qmv.KVCache(put(self.kp), put(self.vp), self.kf, self.vf, self.H, self.D, self.P)

    def gpu(self, a):
        return self.torch.from_numpy(np.ascontiguousarray(a)).cuda()

    def queries(self, new, G, x, std=1.0):
        n = int(sum(new))
        begin = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        q, qe = typed(self.torch, std * self.rng.standard_normal((n, self.H * G, self.D)), x)
        return q, qe, begin

    def want(self, qe, begin, G, x, scale, window=0, sinks=None):
        out, bound = np.zeros(qe.shape), np.zeros(qe.shape)
        for r in range(len(self.lens)):
            a, b = begin[r], begin[r + 1]
            n, L = b - a, int(self.lens[r])
            if n == 0:
                continue
            pos = np.repeat(np.arange(L - n, L), G)
            for h in range(self.H):
                q = qe[a:b, h * G:(h + 1) * G].reshape(n * G, self.D)
                sk = None if sinks is None else np.tile(sinks[h * G:(h + 1) * G], n)
                o, e = cv.attention(q, self.k[r][:, h], self.v[r][:, h], scale, pos, window, sk, x, n * G <= FEW, self.kf)
                out[a:b, h * G:(h + 1) * G] = o.reshape(n, G, self.D)
                bound[a:b, h * G:(h + 1) * G] = e.reshape(n, G, self.D)
        return out, bound


def close(got, want, bound):
    g = got.cpu().double().numpy()
    off = np.abs(g - want)
    assert np.all(np.isfinite(g)), np.argwhere(~np.isfinite(g))[:5]
    worst = np.unravel_index(np.argmax(off / bound), off.shape)
    print("worst", off[worst] / bound[worst], "rms", np.sqrt((off ** 2).mean() / (want ** 2).mean()), flush=True)
    assert np.all(off <= bound), (worst, g[worst], want[worst], bound[worst])


PAIRS = [(a, b) for a in ("q8_0", "q4_0", "q4_1") for b in ("q8_0", "q4_0", "q4_1")]
# x, D, H, G, page, lens, new tokens, window, sinks
SHAPES = [
    ("bf16", 128, 2, 4, 16, [1, 17, 300], [1, 1, 1], 0, False),
    ("f16", 64, 3, 1, 32, [33, 32, 31, 64], [1, 2, 1, 3], 0, True),
    ("f32", 128, 1, 5, 16, [5, 129, 260], [5, 3, 1], 0, False),
    ("f32", 256, 2, 2, 64, [100, 1], [4, 1], 40, True),
    ("bf16", 256, 1, 8, 16, [77, 200], [3, 1], 0, False),
    ("f16", 128, 1, 16, 32, [150], [1], 20, True),
    ("bf16", 64, 2, 7, 16, [90, 16, 333], [2, 4, 1], 7, False),
    ("f32", 64, 1, 20, 16, [70, 40], [1, 1], 0, True),
    ("bf16", 128, 1, 71, 16, [50, 100], [1, 2], 0, False),
    ("f16", 128, 2, 4, 16, [180, 70, 40], [100, 33, 1], 0, True),
    ("bf16", 64, 1, 2, 32, [270], [131], 50, False),
    ("f32", 256, 1, 3, 16, [120, 65], [60, 20], 0, False),
    ("f32", 128, 2, 2, 16, [140, 9, 80], [70, 9, 2], 33, True),
    ("bf16", 256, 1, 4, 16, [150], [90], 0, True),
]


@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("pair", PAIRS, ids="-".join)
def test_against_64_bits(env, pair, i):
    torch, qmv = env
    x, D, H, G, P, lens, new, window, sink = SHAPES[i]
    print(pair, SHAPES[i], flush=True)
    first = [max(0, n - m - window + 1) // 16 * 16 if window else 0 for n, m in zip(lens, new)]
    s = Setup(torch, qmv, 100 + i, *pair, H, D, P, lens, first=first)
    q, qe, begin = s.queries(new, G, x, 1.5)
    scale = D ** -0.5
    sinks = np.float32(s.rng.standard_normal(H * G) + 1.0) if sink else None
    out = torch.full(q.shape, 3.0, dtype=q.dtype, device="cuda")
    got = qmv.qmv_cache_attention(s.cache, q.cuda(), s.gpu(s.table), s.gpu(s.lens), s.gpu(begin), max(new), window=window,
                                  sinks=None if sinks is None else s.gpu(sinks), out=out)
    close(got, *s.want(qe, begin, G, x, scale, window, sinks))
    again = qmv.qmv_cache_attention(s.cache, q.cuda(), s.gpu(s.table), s.gpu(s.lens), s.gpu(begin), max(new), window=window,
                                    sinks=None if sinks is None else s.gpu(sinks))
    assert torch.equal(got, again)


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("new", [1, 40])
def test_rows_that_see_nothing_and_lengths_out_of_range(env, x, new):
    torch, qmv = env
    print(x, new, flush=True)
    G, D = 2, 64
    s = Setup(torch, qmv, 5, "q4_0", "q8_0", 2, D, 16, [0, 3, 60, 60, 60], spare=1)
    q, qe, begin = s.queries([new, new, new, new, new], G, x)
    for sinks in (None, np.float32([0.5, -1.0, 2.0, 30.0])):
        lens = s.lens.copy()
        lens[3], lens[4] = -1, s.max_pages * 16 + 1
        want, bound = s.want(qe, begin, G, x, 0.2, 0, sinks)
        got = qmv.qmv_cache_attention(s.cache, q.cuda(), s.gpu(s.table), s.gpu(lens), scale=0.2,
                                      sinks=None if sinks is None else s.gpu(sinks))
        assert bool(torch.isnan(got[3 * new:].float()).all())
        assert bool((got[:new] == 0).all())
        if new > 3:
            assert bool((got[new:2 * new - 3] == 0).all())      # positions before the sequence
        close(got[:3 * new], want[:3 * new], bound[:3 * new])


@pytest.mark.parametrize("new,G", [(1, 4), (5, 4), (9, 4), (70, 2)])
def test_pages_out_of_range(env, new, G):
    """The queries that see a position of such a page are NaN, the others as they were."""
    torch, qmv = env
    print(new, G, flush=True)
    D, P, L = 128, 16, 205
    s = Setup(torch, qmv, 6, "q4_0", "q4_0", 1, D, P, [L, L, L], spare=0)
    q, qe, begin = s.queries([new] * 3, G, "bf16")
    want, bound = s.want(qe, begin, G, "bf16", D ** -0.5, 0)
    table = s.table.copy()
    table[0, (L - 1) // P] = -1                                 # the last page
    table[1, (L - 1) // P - 1] = s.cache.n_pages                # the one before
    got = qmv.qmv_cache_attention(s.cache, q.cuda(), s.gpu(table), s.gpu(s.lens))
    pos = np.arange(L - new, L)
    for r, first in ((0, (L - 1) // P * P), (1, ((L - 1) // P - 1) * P), (2, L)):
        bad = pos >= first
        rows = got[r * new:(r + 1) * new]
        assert bool(torch.isnan(rows[torch.from_numpy(bad).cuda()].float()).all())
        ok = np.concatenate([np.zeros(r * new, bool), ~bad, np.zeros((2 - r) * new, bool)])
        if ok.any():
            close(got[torch.from_numpy(ok).cuda()], want[ok], bound[ok])


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["q8_0", "q4_1"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,G", [(6, 2), (60, 2)])
def test_values_that_are_not_finite(env, x, fmt, D, new, G):
    """A block of V that reads back as NaN makes that block NaN for the queries that see it; one of K, their whole rows."""
    torch, qmv = env
    print(x, fmt, D, new, G, flush=True)
    L, P = 150, 16
    s = Setup(torch, qmv, 8, fmt, fmt, 2, D, P, [L, L], spare=0)
    at = {(0, 0): (L - 3, 1), (0, 1): (L - 5, 0)}                # (request, head): position and block of V
    nb, row = D // 32, D if fmt == "q8_0" else D // 2

    def spoil(pages, r, h, j, b, value):
        head = pages[s.table[r, j // P], h]
        head[P * row + 2 * b * P + 2 * (j % P):][:2] = np.float16(value).reshape(1).view(np.uint8)
    for (r, h), (j, b) in at.items():
        spoil(s.vp, r, h, j, b, np.nan if h else np.inf)
    spoil(s.kp, 1, 1, L - 2, nb - 1, np.nan)
    s.upload()
    q, qe, begin = s.queries([new, new], G, x)
    want, bound = s.want(qe, begin, G, x, D ** -0.5)
    nan = np.zeros(want.shape, bool)
    pos = np.arange(L - new, L)
    for (r, h), (j, b) in at.items():
        nan[r * new:(r + 1) * new][pos >= j, h * G:(h + 1) * G, 32 * b:32 * b + 32] = True
    nan[new:][pos >= L - 2, G:2 * G] = True
    got = qmv.qmv_cache_attention(s.cache, q.cuda(), s.gpu(s.table), s.gpu(s.lens)).cpu()
    assert np.array_equal(torch.isnan(got.float()).numpy(), nan)
    close(torch.where(torch.from_numpy(nan), torch.zeros((), dtype=got.dtype), got), np.where(nan, 0, want), bound)


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("new", [3, 50])
def test_queries_that_are_not_finite_or_of_odd_size(env, x, new):
    torch, qmv = env
    print(x, new, flush=True)
    G, D, L = 4, 64, 90
    s = Setup(torch, qmv, 9, "q8_0", "q8_0", 1, D, 16, [L], spare=0)
    q, qe, begin = s.queries([new], G, x)
    sizes = [1e-30, 1e-7, 0.0, 30.0] if x != "f16" else [1e-7, 1e-3, 0.0, 30.0]
    for h in range(G):
        qe[0, h] *= sizes[h]
    q, qe = typed(torch, qe, x)
    q[1, 2, 5] = float("nan")
    q[2, 0, 63] = float("inf")
    got = qmv.qmv_cache_attention(s.cache, q.cuda(), s.gpu(s.table), s.gpu(s.lens)).cpu()
    qe[1, 2], qe[2, 0] = 0, 0
    want, bound = s.want(qe, begin, G, x, D ** -0.5)
    assert bool(torch.isnan(got[1, 2].float()).all()) and bool(torch.isnan(got[2, 0].float()).all())
    got[1, 2], got[2, 0] = 0, 0
    want[1, 2], want[2, 0] = 0, 0
    close(got, want, bound)


@pytest.mark.parametrize("new", [[1, 0, 2, 0, 1], [40, 0, 3, 0, 25]])
def test_rows_of_no_request_and_more_than_max_q(env, new):
    torch, qmv = env
    print(new, flush=True)
    G, D = 2, 64
    s = Setup(torch, qmv, 10, "q4_0", "q4_1", 2, D, 16, [50, 40, 44, 0, 60])
    q, qe, begin = s.queries(new, G, "bf16")
    want, bound = s.want(qe, begin, G, "bf16", D ** -0.5)
    T = q.shape[0]
    more = torch.cat([q, q[:1].expand(5, -1, -1)]).cuda()
    out = torch.full(more.shape, 7.0, dtype=more.dtype, device="cuda")
    qmv.qmv_cache_attention(s.cache, more, s.gpu(s.table), s.gpu(s.lens), s.gpu(begin), max(new), out=out)
    assert bool((out[T:] == 7).all())
    close(out[:T], want, bound)
    # a request has more queries than max_q: the rest is left, the first are as without the limit
    most = max(new) - 1
    out.fill_(7.0)
    lens = s.lens - np.maximum(np.diff(begin) - most, 0).astype(np.int32)     # so that they stand where they stood
    qmv.qmv_cache_attention(s.cache, more, s.gpu(s.table), s.gpu(lens), s.gpu(begin), most, out=out)
    left = np.ones(T, bool)
    for r in range(len(new)):
        left[begin[r]:begin[r] + min(new[r], most)] = False
    assert bool((out[:T][torch.from_numpy(left).cuda()] == 7).all())
    keep = torch.from_numpy(~left).cuda()
    close(out[:T][keep], want[~left], bound[~left])
    # q_begin that is out of order or out of range stays within the tensors
    for b in ([0, 3, 1, 2, 2, 4], [-5, 0, 1, 2, 3, 2 ** 31 - 1], [9, 9, 9, 0, 0, 0]):
        qmv.qmv_cache_attention(s.cache, more, s.gpu(s.table), s.gpu(s.lens), s.gpu(np.array(b, np.int32)), most, out=out)
    torch.cuda.synchronize()


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("new", [2, 30])
def test_strides_and_alignment(env, x, new):
    torch, qmv = env
    print(x, new, flush=True)
    G, D, H = 3, 64, 2
    s = Setup(torch, qmv, 12, "q4_0", "q4_0", H, D, 32, [100, 65])
    q, qe, begin = s.queries([new, new], G, x)
    want = qmv.qmv_cache_attention(s.cache, q.cuda(), s.gpu(s.table), s.gpu(s.lens))
    close(want, *s.want(qe, begin, G, x, D ** -0.5))
    for lead, pad in ((1, 0), (8, 8), (3, 5), (4, 4)):
        rows = torch.full((2 * new, lead + H * G * (D + pad)), 9.0, dtype=q.dtype, device="cuda")
        v = rows[:, lead:].unflatten(1, (H * G, D + pad))[..., :D]
        v.copy_(q)
        assert torch.equal(qmv.qmv_cache_attention(s.cache, v, s.gpu(s.table), s.gpu(s.lens)), want), (lead, pad)


def of_reads(torch, qmv, cache, q, table, lens, begin, scale, window, x):
    """float64 on the GPU from qmv_cache_read's values, request by request."""
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    G = q.shape[1] // cache.n_kv_heads
    for r in range(table.shape[0]):
        a, b, L = int(begin[r]), int(begin[r + 1]), int(lens[r])
        if a == b:
            continue
        j = torch.arange(L, device="cuda")
        slots = (table[r][j // cache.page_size].long() * cache.page_size + j % cache.page_size).to(torch.int32)
        k, v = (t.double().transpose(0, 1) for t in qmv.qmv_cache_read(cache, slots))
        qq = q[a:b].double().view(b - a, -1, G, q.shape[2]).permute(1, 0, 2, 3).flatten(1, 2)
        s = torch.matmul(qq, k.transpose(1, 2)) * scale
        pos = torch.arange(L - (b - a), L, device="cuda").repeat_interleave(G)[:, None]
        hide = j > pos
        if window:
            hide |= j <= pos - window
        w = torch.softmax(s.masked_fill(hide, float("-inf")), -1)
        out[a:b] = torch.matmul(w, v).unflatten(1, (b - a, G)).permute(1, 0, 2, 3).flatten(1, 2)
    return out


def random_cache(torch, qmv, g, kf, vf, H, D, P, lens, spare=0):
    each = [-(-n // P) for n in lens]
    pages = sum(each) + spare
    cache = qmv.KVCache.new(pages, kf, vf, H, D, P)
    order = torch.randperm(pages, generator=g, device="cuda")
    table = torch.full((len(lens), max(each)), -1, device="cuda", dtype=torch.int32)
    at = 0
    for r, (n, e) in enumerate(zip(lens, each)):
        table[r, :e] = order[at:at + e].to(torch.int32)
        at += e
        for c in range(0, n, 8192):
            j = torch.arange(c, min(c + 8192, n), device="cuda")
            slots = (table[r][j // P].long() * P + j % P).to(torch.int32)
            kv = [torch.randn(j.numel(), H, D, generator=g, device="cuda") for _ in range(2)]
            qmv.qmv_cache_write(cache, *kv, slots)
    return cache, table


# relative to the rms of the outputs: sums of random signs; one rounding of the output, of V, of the weights and of the scores each,
# every one at most half a step and on average a third of it or less
FAR = {"bf16": 2.0 ** -8, "f16": 2.5 * 2.0 ** -11, "f32": 2e-6}


def near(torch, got, want, x):
    off = float((got.double() - want).norm() / want.norm())
    print("off", off, flush=True)
    assert off <= FAR[x]


@pytest.mark.parametrize("x,kf,vf,H,G,D,P,lens,new,window", [
    ("bf16", "q4_0", "q4_0", 8, 4, 128, 64, [70001], [1], 0),
    ("f32", "q8_0", "q4_1", 2, 8, 64, 256, [40000, 3], [2, 1], 0),
    ("f16", "q4_0", "q8_0", 1, 1, 256, 16, [20000], [1], 5000),
    ("bf16", "q4_0", "q4_0", 2, 4, 128, 64, [5000, 700], [1500, 700], 0),
    ("f16", "q8_0", "q4_0", 2, 5, 64, 16, [3000, 20], [1100, 1], 400),
    ("f32", "q4_0", "q4_0", 1, 4, 128, 32, [2500], [600], 0),
    ("f16", "q4_1", "q4_1", 1, 2, 256, 128, [2100, 2100], [777, 5], 0),
    ("bf16", "q4_0", "q4_0", 1, 8, 128, 64, [30000], [200], 0),
])
def test_long(env, x, kf, vf, H, G, D, P, lens, new, window):
    torch, qmv = env
    print(x, kf, vf, H, G, D, P, lens, new, window, flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    cache, table = random_cache(torch, qmv, g, kf, vf, H, D, P, lens)
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[x]
    q = torch.randn(sum(new), H * G, D, generator=g, device="cuda").to(dt)
    begin = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = qmv.qmv_cache_attention(cache, q, table, n, begin, max(new), window=window)
    near(torch, got, of_reads(torch, qmv, cache, q, table, n, begin, D ** -0.5, window, x), x)


@pytest.mark.parametrize("R,most", [(300, 1), (700, 3), (270, 40)])
def test_many_requests(env, R, most):
    """More requests than a workgroup has threads, some without queries."""
    torch, qmv = env
    print(R, most, flush=True)
    g = torch.Generator(device="cuda").manual_seed(2)
    rng = np.random.default_rng(R)
    lens = list(rng.integers(1, 120, R))
    new = [int(min(rng.integers(0, most + 1), n)) for n in lens]
    cache, table = random_cache(torch, qmv, g, "q4_0", "q4_0", 1, 64, 16, lens)
    q = torch.randn(sum(new), 2, 64, generator=g, device="cuda").half()
    begin = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = qmv.qmv_cache_attention(cache, q, table, n, begin, most)
    near(torch, got, of_reads(torch, qmv, cache, q, table, n, begin, 0.125, 0, "f16"), "f16")


def test_a_cache_past_32_bits(env):
    """The last pages of a cache of more than 4 GiB a side."""
    torch, qmv = env
    H, D, P = 8, 128, 256
    pages = (9 << 30) // 2 // qmv.cache_page_bytes("q4_0", H, D, P)
    cache = qmv.KVCache.new(pages, "q4_0", "q8_0", H, D, P)
    print(pages, cache.k.numel(), cache.v.numel(), flush=True)
    assert cache.k.numel() > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(4)
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device="cuda")
    L = 700
    j = torch.arange(L, device="cuda")
    slots = (table[0][j // P].long() * P + j % P).to(torch.int32)
    k, v = (torch.randn(L, H, D, generator=g, device="cuda") for _ in range(2))
    qmv.qmv_cache_write(cache, k, v, slots)
    kk, vv = qmv.qmv_cache_read(cache, slots)
    assert float((kk - k).abs().max()) < 0.5 and float((vv - v).abs().max()) < 0.05
    n = torch.tensor([L], dtype=torch.int32, device="cuda")
    for new in (1, 100):
        q = torch.randn(new, 2 * H, D, generator=g, device="cuda").half()
        begin = torch.tensor([0, new], dtype=torch.int32, device="cuda")
        got = qmv.qmv_cache_attention(cache, q, table, n)
        near(torch, got, of_reads(torch, qmv, cache, q, table, n, begin, D ** -0.5, 0, "f16"), "f16")


@pytest.mark.parametrize("new", [1, 33])
def test_captured_and_replayed(env, new):
    """Lengths, tables and queries change between replays of one graph."""
    torch, qmv = env
    print(new, flush=True)
    g = torch.Generator(device="cuda").manual_seed(6)
    rng = np.random.default_rng(1)
    H, G, D, P, R = 2, 2, 128, 16, 5
    cache, full = random_cache(torch, qmv, g, "q4_0", "q4_0", H, D, P, [2000] * R)
    q = torch.randn(R * new, H * G, D, generator=g, device="cuda").half()
    table, n = full.clone(), torch.full((R,), 40, dtype=torch.int32, device="cuda")
    begin = torch.arange(R + 1, device="cuda", dtype=torch.int32) * new
    qmv.qmv_cache_attention(cache, q, table, n, begin, new)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = qmv.qmv_cache_attention(cache, q, table, n, begin, new)
    for i in range(5):
        q.normal_(generator=g)
        n.copy_(torch.from_numpy(rng.integers(new, 2000, R).astype(np.int32)))
        table.copy_(full[torch.randperm(R, generator=g, device="cuda")])
        graph.replay()
        torch.cuda.synchronize()
        want = qmv.qmv_cache_attention(cache, q, table, n, begin, new)
        assert torch.equal(got, want), i
        near(torch, got, of_reads(torch, qmv, cache, q, table, n, begin, D ** -0.5, 0, "f16"), "f16")
