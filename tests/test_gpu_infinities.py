"""Activations outside the accuracy contract, on an MI355X: infinities, and finite ones too large for the products' pieces and
block sums.  Sums are those of the weights' own products in 64 bits, NaN and infinities among them."""
import numpy as np
import pytest

import workloads as wl
from tests import operator_values as ov

pytestmark = pytest.mark.gpu

FORMATS = ["q8_0", "q4_0", "q4_1", "q4_k", "q6_k"]
CHECKED = 14                 # tokens held to 64 bits: those with such values, and a few others
HUGE = {"f32": 3.4028234e38, "bf16": 3.3895314e38, "f16": 65504.0}


@pytest.fixture(scope="module")
def env():
    import torch
    import bandwidth_bound_block_amd as qmv
    assert torch.cuda.is_available()
    return torch, qmv


def activations(torch, T, K, name, seed):
    """Tokens 0..6 hold, in a few columns: inf; -inf; inf twice; both; the largest float; NaN beside inf; inf throughout.
    The others are ordinary, and so are tokens 7 and 8 but for a value that only bf16's rounding takes past the largest."""
    g = np.random.default_rng(seed)
    a = g.standard_normal((T, K))
    c = g.permutation(K)
    a[0, c[0]] = np.inf
    a[1, c[1]] = -np.inf
    a[2, c[:2]] = np.inf
    a[3, c[2]], a[3, c[3]] = np.inf, -np.inf
    a[4] = 0.0
    a[4, c[4]] = HUGE[name]
    a[5, c[5]], a[5, c[6]] = np.inf, np.nan
    a[6] = np.inf
    a[7, c[7]] = HUGE[name]
    a[8, c[8]] = -HUGE[name]
    return ov.as_type(torch, a, name)


def values(fmt, raw, N, K, x):
    """y and its bound by formula; a number where every product is one, else what the products' sum is."""
    w = ov.oracle.dequant(fmt, raw, N, K).astype(np.float64).reshape(N, K)
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.empty((x.shape[0], N))
        e = np.empty((x.shape[0], N))
        for t in range(x.shape[0]):
            p = w * x[t]
            y[t], e[t] = p.sum(1), np.abs(p).sum(1)
    return y, 3 * (K // 32 + 40) * ov.U * e + 2.0 ** -120


def assert_same(got, y, e, what):
    got = got.detach().cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(y)), (what, np.argwhere(np.isnan(got) != np.isnan(y))[:5])
    inf = np.isinf(y)
    assert np.array_equal(got[inf], y[inf]), what
    ok = np.isfinite(y)
    # a sum past fp32's largest rounds to an infinity
    big = ok & (np.abs(y) + e > 3.4e38)
    ok &= ~big
    assert np.all(np.abs(got[ok] - y[ok]) <= e[ok]), (what, float(np.max(np.abs(got[ok] - y[ok]) / e[ok])))


def size(fmt, blocks):
    return blocks * (256 if fmt in ("q4_k", "q6_k") else 32)


@pytest.mark.parametrize("x_name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E,rows,blocks", [(20, 1, 90, 9), (40, 1, 4500, 37), (60, 4, 8200, 2), (60, 4, 17000, 1), (300, 1, 16500, 1)])
def test_products(env, fmt, x_name, T, E, rows, blocks):
    torch, qmv = env
    K = size(fmt, blocks if blocks < 37 or fmt not in ("q4_k", "q6_k") else 5)
    print("inf", fmt, x_name, T, E, rows, K, flush=True)
    per = wl.block_bytes(fmt, rows, K)
    W = wl.quant_weights(fmt, f"t/inf/{fmt}/{rows}/{K}", E * rows, K).reshape(E, per)
    ids = np.random.default_rng(T).integers(0, E, size=(T, 1))
    xt, x = activations(torch, T, K, x_name, T + rows)
    y, e = np.empty((CHECKED, 1, rows)), np.empty((CHECKED, 1, rows))
    for g in range(E):
        t = np.nonzero(ids[:CHECKED, 0] == g)[0]
        y[t, 0], e[t, 0] = values(fmt, W[g].reshape(rows, -1), rows, K, x[t])
    plan = qmv.qmv_group_plan(torch.from_numpy(ids.astype(np.int32)).cuda(), E)
    got = qmv.qmv_moe_grouped(fmt, torch.from_numpy(W.reshape(-1)).cuda(), per, E, rows, K, plan, 1, xt.cuda())
    assert_same(got[:CHECKED], y, e, fmt)
    # the ordinary tokens have the bits that they have among ordinary ones
    xt[:9] = 0.5
    clean = qmv.qmv_moe_grouped(fmt, torch.from_numpy(W.reshape(-1)).cuda(), per, E, rows, K, plan, 1, xt.cuda())
    assert torch.equal(got[9:], clean[9:])


@pytest.mark.parametrize("x_name", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,F", [(20, 72), (300, 8300)])
def test_swiglu(env, fmt, x_name, T, F):
    torch, qmv = env
    K = 256
    raw = wl.quant_weights(fmt, f"t/inf/gu/{fmt}/{F}", 2 * F, K)
    xt, x = activations(torch, T, K, x_name, T)
    a, ea = values(fmt, raw, 2 * F, K, x[:CHECKED])
    with np.errstate(invalid="ignore", over="ignore"):
        h, eh = ov.swiglu(a[:, :F], ea[:, :F], a[:, F:], ea[:, F:])
    plan = qmv.qmv_group_plan(torch.zeros((T, 1), dtype=torch.int32).cuda(), 1)
    got = qmv.qmv_moe_grouped_swiglu(fmt, torch.from_numpy(raw.reshape(-1)).cuda(), raw.size, 1, F, K, plan, 1, xt.cuda())
    got, large = got[:CHECKED, 0], np.abs(a).max(1) > 1e30       # SiLU times up of two large sums: past fp32, or cancelled exponentials
    assert_same(got[~torch.from_numpy(large)], h[~large], eh[~large], fmt)
    g = got.cpu().double().numpy()
    for t in (0, 1, 2, 3, 5, 6):
        assert np.array_equal(np.isnan(g[t]), np.isnan(h[t])) and np.array_equal(g[t][np.isinf(h[t])], h[t][np.isinf(h[t])]), t


@pytest.mark.parametrize("x_name,a_name", [("f32", "f32"), ("f32", "bf16"), ("f16", "f16"), ("f16", "bf16"), ("f16", "f32"), ("bf16", "bf16"),
                                           ("bf16", "f16")])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,N,blocks,R", [(20, 90, 9, 16), (40, 300, 40, 5), (300, 8300, 1, 72)])
def test_adapters(env, fmt, x_name, a_name, T, N, blocks, R):
    torch, qmv = env
    K, G = size(fmt, blocks if fmt not in ("q4_k", "q6_k") else (blocks + 7) // 8), 4
    print("inf lora", fmt, x_name, a_name, T, N, K, R, flush=True)
    raw = wl.quant_weights(fmt, f"t/inf/lora/{fmt}/{N}/{K}", N, K)
    xt, x = activations(torch, T, K, x_name, T + N)
    g = np.random.default_rng(R)
    At, A = ov.as_type(torch, g.standard_normal((G, R, K)) / np.sqrt(K), a_name)
    Bt, B = ov.as_type(torch, g.standard_normal((G, N, R)), a_name)
    scales = g.uniform(0.5, 2, size=G).astype(np.float32)
    ids = np.arange(T) % (G + 2) - 1                       # -1, 0..3, and 4: no adapter of these
    y, e = values(fmt, raw, N, K, x[:CHECKED])
    with np.errstate(invalid="ignore", over="ignore"):
        d, ed = ov.adapters(x[:CHECKED], A, B, scales, ids)
        out, bound = y + d, e + ed + 2 * ov.U * (np.abs(y) + np.abs(d))
    out[ids[:CHECKED] >= G] = np.nan
    got = qmv.qmv_lora(fmt, torch.from_numpy(raw.reshape(-1)).cuda(), N, K, xt.cuda(), At.cuda(), Bt.cuda(),
                       torch.from_numpy(scales).cuda(), torch.from_numpy(ids.astype(np.int32)).cuda())
    got, large = got[:CHECKED], np.zeros(CHECKED, bool)
    large[[4, 7, 8]] = x_name != "f16"          # the adapters' sums of the largest floats pass fp32
    assert_same(got[~torch.from_numpy(large)], out[~large], bound[~large], fmt)


@pytest.mark.parametrize("x_name,a_name", [("f32", "bf16"), ("f16", "f16"), ("f16", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("first,T", [(0, 8), (1, 8), (0, 1), (1, 2), (3, 4)])
def test_adapters_on_few_tokens(env, fmt, x_name, a_name, first, T):
    """The base is the matvec's, on its matrix cores at some of these sizes: 256-column rows of 16-byte aligned blocks."""
    torch, qmv = env
    N, K, R, G = 1100, 512, 8, 3
    raw = wl.quant_weights(fmt, f"t/inf/few/{fmt}", N, K)
    xt, x = activations(torch, 9, K, x_name, 5)
    xt, x = xt[first:first + T], x[first:first + T]
    g = np.random.default_rng(R)
    At, A = ov.as_type(torch, g.standard_normal((G, R, K)) / np.sqrt(K), a_name)
    Bt, B = ov.as_type(torch, g.standard_normal((G, N, R)), a_name)
    scales = g.uniform(0.5, 2, size=G).astype(np.float32)
    for ids in (np.full(T, -1), np.arange(T) % (G + 2) - 1):
        y, _ = values(fmt, raw, N, K, x)
        w = ov.oracle.dequant(fmt, raw, N, K).astype(np.float64).reshape(N, K)
        with np.errstate(invalid="ignore", over="ignore"):
            e = np.stack([1e-4 * np.abs(w * v).sum(1) + 1e-6 for v in x])       # the matvec's contract
            d, ed = ov.adapters(x, A, B, scales, ids)
            out, bound = y + d, e + ed + 2 * ov.U * (np.abs(y) + np.abs(d))
        out[ids >= G] = np.nan
        got = qmv.qmv_lora(fmt, torch.from_numpy(raw.reshape(-1)).cuda(), N, K, xt.cuda(), At.cuda(), Bt.cuda(),
                           torch.from_numpy(scales).cuda(), torch.from_numpy(ids.astype(np.int32)).cuda())
        keep = np.array([first + t not in (4, 7, 8) or x_name == "f16" or ids[t] == -1 for t in range(T)])
        assert_same(got[torch.from_numpy(keep)], out[keep], bound[keep], (fmt, list(ids)))
