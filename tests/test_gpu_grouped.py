"""Products grouped by expert, on an MI355X, against 64-bit values."""
import numpy as np
import pytest

import workloads as wl
from tests import operator_values as ov

pytestmark = pytest.mark.gpu

FORMATS = ["q8_0", "q4_0", "q4_1", "q4_k", "q6_k"]


def say(*a):
    print(*a, flush=True)


@pytest.fixture(scope="module")
def env():
    import torch
    import bandwidth_bound_block_amd as qmv
    assert torch.cuda.is_available()
    return torch, qmv


def experts(fmt, tag, E, rows, K, gap=0):
    """E expert matrices, `gap` bytes apart: the buffer, the stride and each expert's bytes."""
    per = wl.block_bytes(fmt, rows, K)
    W = wl.quant_weights(fmt, tag, E * rows, K).reshape(E, per)
    buf = np.full(((E - 1) * (per + gap) + per,), 0xAB, dtype=np.uint8)
    for e in range(E):
        buf[e * (per + gap):e * (per + gap) + per] = W[e]
    return buf, per + gap, W


def expect(fmt, W, rows, K, ids, x):
    """Values and bounds [T][S][rows]; x [T][K] or [T][S][K] float64."""
    T, S = ids.shape
    y, e = np.full((T, S, rows), np.nan), np.zeros((T, S, rows))
    for g in np.unique(ids):
        if 0 <= g < len(W):
            t, s = np.nonzero(ids == g)
            xs = x[t] if x.ndim == 2 else x[t, s]
            y[t, s], e[t, s] = ov.product(fmt, W[g].reshape(rows, -1), rows, K, xs)
    return y, e


def assert_close(got, y, e, what=""):
    got = got.detach().to("cpu").double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(y)), what
    ok = ~np.isnan(y)
    over = np.abs(got[ok] - y[ok]) - e[ok]
    assert not over.size or over.max() <= 0, (what, float(np.max(np.abs(got[ok] - y[ok]) / e[ok])))


def run(torch, qmv, fmt, buf, stride, E, rows, K, ids, x, top_k, **kw):
    d = torch.from_numpy(np.ascontiguousarray(ids, dtype=np.int32)).cuda()
    plan = qmv.qmv_group_plan(d, E)
    W = torch.from_numpy(buf).cuda()
    return qmv.qmv_moe_grouped(fmt, W, stride, E, rows, K, plan, top_k, x, **kw)


# ------------------------------------------------------------------ the plan
@pytest.mark.parametrize("n,E", [(1, 1), (7, 3), (64, 1024), (1023, 5), (1024, 128), (1025, 128), (5000, 37), (40000, 1024),
                                 (16384, 128), (16385, 128), (20000, 8), (200001, 300)])
@pytest.mark.parametrize("kind", ["even", "one", "bad"])
def test_plan_is_a_stable_sort(env, n, E, kind):
    torch, qmv = env
    say("plan", n, E, kind)
    g = np.random.default_rng(n * 31 + E)
    ids = g.integers(0, E, size=n) if kind == "even" else np.full(n, E // 2)
    if kind == "bad":
        ids = g.integers(-3, E + 3, size=n)
        ids[g.integers(0, n)] = 2 ** 31 - 1
        ids[g.integers(0, n)] = -2 ** 31
    plan = qmv.qmv_group_plan(torch.from_numpy(ids.astype(np.int32)).cuda(), E)
    p = plan.buffer.cpu().numpy().view(np.int32)
    assert p[1] == n and p[2] == E
    tile, tiles = int(p[3]), int(p[4])
    key = np.where((ids >= 0) & (ids < E), ids, E)
    order = np.argsort(key, kind="stable")
    counts = np.bincount(key, minlength=E + 1)
    offs = np.concatenate([[0], np.cumsum(counts)])
    assert np.array_equal(p[8:8 + E + 2], offs)
    assert np.array_equal(p[len(p) - n:][:n], order)
    at = (8 + E + 2 + 3) // 4 * 4
    got = p[at:at + 4 * tiles].reshape(-1, 4)
    want = [(k, offs[k] + i, min(tile, counts[k] - i)) for k in range(E + 1) for i in range(0, counts[k], tile)]
    assert [tuple(r[:3]) for r in got] == want
    assert at + 4 * tiles <= len(p) - n


# ------------------------------------------------------------------ products
@pytest.mark.parametrize("x_name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,S,E,rows,blocks", [(1, 1, 1, 1, 1), (3, 2, 5, 37, 3), (33, 3, 4, 130, 2), (150, 2, 2, 129, 9),
                                               (260, 1, 1, 256, 4)])
def test_product(env, fmt, x_name, T, S, E, rows, blocks):
    torch, qmv = env
    K = blocks * (256 if fmt in ("q4_k", "q6_k") else 32)
    say("grouped", fmt, x_name, T, S, E, rows, K)
    buf, stride, W = experts(fmt, f"t/grp/{fmt}/{rows}/{K}", E, rows, K, gap=0 if E == 1 else 48)
    g = np.random.default_rng(T + rows)
    ids = g.integers(0, E, size=(T, S))
    xt, x = ov.as_type(torch, g.standard_normal((T, K)), x_name)
    y, e = expect(fmt, W, rows, K, ids, x)
    for y_name, dtype in (("f32", torch.float32), ("bf16", torch.bfloat16), ("f16", torch.float16)):
        got = run(torch, qmv, fmt, buf, stride, E, rows, K, ids, xt.cuda(), S, y_dtype=dtype)
        assert got.dtype == dtype
        assert_close(got, y, e + (ov.rounded(np.abs(y) + e, y_name) if y_name != "f32" else 0), (fmt, y_name))


@pytest.mark.parametrize("x_name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E,rows,blocks", [(300, 1, 16500, 3), (170, 2, 16500, 1), (60, 4, 17000, 2), (40, 2, 16500, 2),
                                             (20, 1, 200, 43), (70, 1, 90, 11), (40, 1, 9000, 9), (33, 1, 4500, 37)])
def test_every_tile_shape(env, fmt, x_name, T, E, rows, blocks):
    """Shapes that take each tile: wide ones, narrow ones whose waves share rows or not, odd numbers of eight-block pieces."""
    torch, qmv = env
    K = blocks * (256 if fmt in ("q4_k", "q6_k") and blocks < 40 else 32 if fmt not in ("q4_k", "q6_k") else 256)
    say("tiles", fmt, x_name, T, E, rows, K)
    buf, stride, W = experts(fmt, f"t/grp/shape/{fmt}/{rows}/{K}", E, rows, K)
    g = np.random.default_rng(T + E)
    ids = g.integers(0, E, size=(T, 1))
    xt, x = ov.as_type(torch, g.standard_normal((T, K)), x_name)
    y, e = expect(fmt, W, rows, K, ids, x)
    assert_close(run(torch, qmv, fmt, buf, stride, E, rows, K, ids, xt.cuda(), 1), y, e, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("x_name", ["f32", "f16"])
@pytest.mark.parametrize("T,E,F", [(300, 1, 8300), (140, 2, 8300), (60, 4, 8500), (20, 1, 72),
                                   (20, 1, 8500), (60, 2, 8500)])
def test_swiglu_in_every_tile_shape(env, fmt, x_name, T, E, F):
    torch, qmv = env
    H = 256
    say("swiglu tiles", fmt, x_name, T, E, F)
    buf, stride, W = experts(fmt, f"t/grp/gush/{fmt}/{F}", E, 2 * F, H)
    g = np.random.default_rng(T)
    ids = g.integers(0, E, size=(T, 1))
    xt, x = ov.as_type(torch, 3 * g.standard_normal((T, H)), x_name)
    a, ea = expect(fmt, W, 2 * F, H, ids, x)
    h, eh = ov.swiglu(a[..., :F], ea[..., :F], a[..., F:], ea[..., F:])
    plan = qmv.qmv_group_plan(torch.from_numpy(ids.astype(np.int32)).cuda(), E)
    got = qmv.qmv_moe_grouped_swiglu(fmt, torch.from_numpy(buf).cuda(), stride, E, F, H, plan, 1, xt.cuda())
    assert_close(got, h, eh, fmt)


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0", "q6_k"])
def test_experts_two_bytes_past_a_word(env, fmt):
    """Odd rows of an odd number of 2-byte-aligned units: every other expert starts 2 bytes past a word, the last ends there."""
    torch, qmv = env
    rows, E, T = 33, 4, 50
    K = 256 if fmt == "q6_k" else 32 * 11
    buf, stride, W = experts(fmt, f"t/grp/two/{fmt}", E, rows, K)
    assert stride % 4 == 2 and buf.size % 4 == 0
    for n in (E, E - 1):              # the buffer's end on a word, and 2 bytes past one
        g = np.random.default_rng(n)
        ids = g.integers(0, n, size=(T, 1))
        xt, x = ov.as_type(torch, g.standard_normal((T, K)), "bf16")
        y, e = expect(fmt, W[:n], rows, K, ids, x)
        got = run(torch, qmv, fmt, buf[:(n - 1) * stride + W.shape[1]], stride, n, rows, K, ids, xt.cuda(), 1)
        assert_close(got, y, e, (fmt, n))


@pytest.mark.parametrize("fmt", FORMATS)
def test_invalid_ids_give_nan_and_touch_nothing_else(env, fmt):
    torch, qmv = env
    T, S, E, rows, K = 50, 3, 6, 70, 512
    buf, stride, W = experts(fmt, f"t/grp/bad/{fmt}", E, rows, K)
    g = np.random.default_rng(5)
    ids = g.integers(-2, E + 2, size=(T, S))
    ids[0] = E                     # a token with no valid slot
    xt, x = ov.as_type(torch, g.standard_normal((T, K)), "bf16")
    y, e = expect(fmt, W, rows, K, ids, x)
    assert_close(run(torch, qmv, fmt, buf, stride, E, rows, K, ids, xt.cuda(), S), y, e)
    # every id invalid
    ids[:] = -1
    assert np.isnan(run(torch, qmv, fmt, buf, stride, E, rows, K, ids, xt.cuda(), S).cpu().numpy()).all()


@pytest.mark.parametrize("x_name", ["f32", "f16", "bf16"])
def test_per_slot_inputs_strides_and_alignment(env, x_name):
    """x [T, S, K] views: a padded row stride, and a start that no 16-byte load can take."""
    torch, qmv = env
    fmt, T, S, E, rows, K = "q8_0", 45, 2, 3, 100, 96
    buf, stride, W = experts(fmt, "t/grp/strides", E, rows, K)
    g = np.random.default_rng(8)
    ids = g.integers(0, E, size=(T, S))
    xt, x = ov.as_type(torch, g.standard_normal((T, S, K)), x_name)
    y, e = expect(fmt, W, rows, K, ids, x)
    for pad, start in ((0, 0), (16, 16), (5, 3), (1, 1)):
        wide = torch.zeros(T, S, K + pad + start, dtype=xt.dtype)
        wide[..., start:start + K] = xt
        v = wide.cuda()[..., start:start + K]
        assert_close(run(torch, qmv, fmt, buf, stride, E, rows, K, ids, v, S), y, e, (pad, start))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("x_name", ["f32", "bf16"])
def test_swiglu_and_weighted_sum(env, fmt, x_name):
    torch, qmv = env
    for T, S, E, F, H in ((5, 2, 4, 256, 256), (140, 3, 3, 512, 256), (30, 1, 1, 256, 512)):
        say("swiglu", fmt, x_name, T, S, E, F, H)
        b1, s1, W1 = experts(fmt, f"t/grp/gu/{fmt}/{F}", E, 2 * F, H, gap=16)
        g = np.random.default_rng(T)
        ids = g.integers(0, E, size=(T, S))
        ids[T // 2, 0] = -1
        xt, x = ov.as_type(torch, 3 * g.standard_normal((T, H)), x_name)
        a, ea = expect(fmt, W1, 2 * F, H, ids, x)
        h, eh = ov.swiglu(a[..., :F], ea[..., :F], a[..., F:], ea[..., F:])
        d = torch.from_numpy(ids.astype(np.int32)).cuda()
        plan = qmv.qmv_group_plan(d, E)
        dtype = xt.dtype
        got = qmv.qmv_moe_grouped_swiglu(fmt, torch.from_numpy(b1).cuda(), s1, E, F, H, plan, S, xt.cuda(), h_dtype=dtype)
        assert_close(got, h, eh + (ov.rounded(np.abs(h) + eh, x_name) if x_name != "f32" else 0), "h")
        # the down product takes h as it is, [T, S, F]
        b2, s2, W2 = experts(fmt, f"t/grp/down/{fmt}/{F}", E, H, F)
        hv = got.cpu().double().numpy()
        y, ey = expect(fmt, W2, H, F, ids, hv)
        down = qmv.qmv_moe_grouped(fmt, torch.from_numpy(b2).cuda(), s2, E, H, F, plan, S, got)
        assert_close(down, y, ey, "down")
        w = g.random((T, S)).astype(np.float32)
        yv = down.cpu().double().numpy()
        out = (yv * w[..., None]).sum(1)
        eo = (S + 1) * ov.U * (np.abs(yv) * w[..., None]).sum(1)
        for name, ot in (("f32", torch.float32), ("bf16", torch.bfloat16), ("f16", torch.float16)):
            o = qmv.qmv_moe_weighted_sum(down, torch.from_numpy(w).cuda(), out_dtype=ot)
            assert_close(o, out, eo + ov.rounded(np.abs(out) + eo, name) + 2.0 ** -120, name)


@pytest.mark.parametrize("n", [1, 3, 4, 5, 130])
@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
def test_weighted_sum_odd_rows(env, n, name):
    torch, qmv = env
    T, S = 9, 5
    g = np.random.default_rng(n)
    yt, y = ov.as_type(torch, g.standard_normal((T, S, n)), name)
    w = g.standard_normal((T, S)).astype(np.float32)
    out = (y * w[..., None]).sum(1)
    bound = (S + 1) * ov.U * (np.abs(y) * np.abs(w[..., None])).sum(1) + 2.0 ** -120
    assert_close(qmv.qmv_moe_weighted_sum(yt.cuda(), torch.from_numpy(w).cuda()), out, bound)


@pytest.mark.parametrize("T", [20, 200])
@pytest.mark.parametrize("fmt", FORMATS)
def test_zero_heavy_rows(env, fmt, T):
    """Rows of mostly zero weights with large activations on them: errors stay relative to sum |w x|."""
    torch, qmv = env
    rows, K = 40, 512
    raw, x = wl.zero_heavy(fmt, f"t/grp/zh/{fmt}", rows, K, B=T)
    ids = np.zeros((T, 1), dtype=np.int64)
    y, e = expect(fmt, [raw], rows, K, ids, x.astype(np.float64))
    got = run(torch, qmv, fmt, raw.reshape(-1), raw.size, 1, rows, K, ids, torch.from_numpy(x).cuda(), 1)
    assert_close(got, y, e + 0.0, fmt)


@pytest.mark.parametrize("x_name", ["f32", "f16", "bf16"])
def test_values_at_the_edges_of_the_types(env, x_name):
    """Subnormal and largest activations; a token of NaN or inf leaves the others alone."""
    torch, qmv = env
    fmt, T, rows, K = "q8_0", 40, 64, 128
    buf, stride, W = experts(fmt, "t/grp/edge", 1, rows, K)
    g = np.random.default_rng(3)
    a = g.standard_normal((T, K))
    a[1] *= {"f32": 1e-36, "f16": 1e-6, "bf16": 1e-36}[x_name]
    a[2] *= {"f32": 1e30, "f16": 1e4, "bf16": 1e30}[x_name]
    xt, x = ov.as_type(torch, a, x_name)
    ids = np.zeros((T, 1), dtype=np.int64)
    y, e = expect(fmt, W, rows, K, ids, x)
    got = run(torch, qmv, fmt, buf, stride, 1, rows, K, ids, xt.cuda(), 1)
    # pieces of tiny fp32 activations end at bf16's smallest step, 2^-133, its half each
    tiny = 2.0 ** -134 * np.abs(ov.oracle.dequant(fmt, W[0].reshape(rows, -1), rows, K)).sum(1) if x_name == "f32" else 0
    assert_close(got, y, e + tiny, x_name)
    xt[5], xt[6, 3], xt[7, 9] = float("nan"), float("inf"), float("-inf")
    bad = run(torch, qmv, fmt, buf, stride, 1, rows, K, ids, xt.cuda(), 1).cpu().numpy()
    keep = np.ones(T, bool)
    keep[[5, 6, 7]] = False
    assert np.array_equal(bad[keep], got.cpu().numpy()[keep]) and not np.isfinite(bad[~keep]).any()


@pytest.mark.parametrize("T", [30, 300])
def test_items_do_not_depend_on_each_other(env, T):
    """The same item among other items, in another order, twice: the same bits where the tile is the same."""
    torch, qmv = env
    fmt, E, rows, K = "q4_k", 3, 64, 512
    buf, stride, _ = experts(fmt, "t/grp/order", E, rows, K)
    g = np.random.default_rng(1)
    ids = g.integers(0, E, size=(T, 1))
    xt, _ = ov.as_type(torch, g.standard_normal((T, K)), "bf16")
    a = run(torch, qmv, fmt, buf, stride, E, rows, K, ids, xt.cuda(), 1).cpu().numpy()
    b = run(torch, qmv, fmt, buf, stride, E, rows, K, ids, xt.cuda(), 1).cpu().numpy()
    assert np.array_equal(a, b)
    p = g.permutation(T)
    c = run(torch, qmv, fmt, buf, stride, E, rows, K, ids[p], xt[torch.from_numpy(p)].cuda(), 1).cpu().numpy()
    assert np.array_equal(a[p], c)


def test_plan_of_other_sizes_writes_nothing(env):
    torch, qmv = env
    fmt, E, rows, K, T = "q4_0", 4, 32, 64, 10
    buf, stride, _ = experts(fmt, "t/grp/other", E, rows, K)
    plan = qmv.qmv_group_plan(torch.zeros(T + 5, dtype=torch.int32).cuda(), E)
    x = torch.ones(T, K).cuda()
    with pytest.raises(ValueError):
        qmv.qmv_moe_grouped(fmt, torch.from_numpy(buf).cuda(), stride, E, rows, K, plan, 1, x)
    lie = qmv.GroupPlan(plan.buffer, T, E)      # what a C caller could pass
    y = torch.full((T, 1, rows), 7.0).cuda()
    qmv.qmv_moe_grouped(fmt, torch.from_numpy(buf).cuda(), stride, E, rows, K, lie, 1, x, y=y)
    torch.cuda.synchronize()
    assert (y == 7.0).all()


def test_other_stream_and_graph(env):
    torch, qmv = env
    fmt, E, F, H, T, S = "q4_0", 5, 64, 96, 21, 2
    b1, s1, _ = experts(fmt, "t/grp/g1", E, 2 * F, H)
    b2, s2, _ = experts(fmt, "t/grp/g2", E, H, F)
    W1, W2 = torch.from_numpy(b1).cuda(), torch.from_numpy(b2).cuda()
    g = torch.Generator().manual_seed(4)
    ids = torch.randint(0, E, (T, S), generator=g, dtype=torch.int32).cuda()
    w = torch.rand(T, S, generator=g).cuda()
    x = torch.randn(T, H, generator=g).cuda()

    def block(stream=None):
        plan = qmv.qmv_group_plan(ids, E, stream=stream)
        h = qmv.qmv_moe_grouped_swiglu(fmt, W1, s1, E, F, H, plan, S, x, stream=stream)
        y = qmv.qmv_moe_grouped(fmt, W2, s2, E, H, F, plan, S, h, stream=stream)
        return qmv.qmv_moe_weighted_sum(y, w, stream=stream)
    eager = block().cpu()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = block(side)
    side.synchronize()
    assert torch.equal(other.cpu(), eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block()
    for k in range(4):
        x.copy_(torch.randn(T, H, generator=g))
        ids.copy_(torch.randint(0, E, (T, S), generator=g, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = out.cpu()
        assert torch.equal(got, block().cpu()), k


def test_offsets_past_32_bits(env):
    """The last expert begins past 4 GiB; token and output offsets pass 2^31 elements only by stride."""
    torch, qmv = env
    fmt, rows, K, E = "q8_0", 64, 64, 3
    per = wl.block_bytes(fmt, rows, K)
    stride = (1 << 32) // 2 + 4096
    raw = wl.quant_weights(fmt, "t/grp/far", E * rows, K).reshape(E, per)
    W = torch.zeros((E - 1) * stride + per, dtype=torch.uint8, device="cuda")
    for e in range(E):
        W[e * stride:e * stride + per] = torch.from_numpy(raw[e]).cuda()
    T = 6
    g = np.random.default_rng(2)
    ids = np.array([[2], [0], [1], [2], [2], [0]])
    xt, x = ov.as_type(torch, g.standard_normal((T, K)), "f32")
    far = torch.zeros(5 * (1 << 29) + K, device="cuda")     # rows 2^29 elements apart
    v = far.as_strided((T, K), (1 << 29, 1))
    v.copy_(xt)
    y, e = expect(fmt, list(raw), rows, K, ids, x)
    plan = qmv.qmv_group_plan(torch.from_numpy(ids.astype(np.int32)).cuda(), E)
    assert_close(qmv.qmv_moe_grouped(fmt, W, stride, E, rows, K, plan, 1, v), y, e)
