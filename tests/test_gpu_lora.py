"""Shared projections with a low-rank adapter per token, on an MI355X,
against 64-bit values.  Up to 8 tokens the base is the matvec, held to its
contract (1e-4 of sum |w x|); past that it is the tile product."""
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


class Case:
    def __init__(self, torch, fmt, T, N, K, R, G, x_name, a_name, seed=0, ids=None):
        g = np.random.default_rng(1000 * T + N + seed)
        self.fmt, self.T, self.N, self.K = fmt, T, N, K
        self.raw = wl.quant_weights(fmt, f"t/lora/{fmt}/{N}/{K}", N, K)
        self.xt, self.x = ov.as_type(torch, g.standard_normal((T, K)), x_name)
        self.At, self.A = ov.as_type(torch, g.standard_normal((G, R, K)) / np.sqrt(K), a_name)
        self.Bt, self.B = ov.as_type(torch, g.standard_normal((G, N, R)), a_name)
        self.scales = g.uniform(-2, 2, size=G).astype(np.float32)
        self.ids = g.integers(-1, G, size=T) if ids is None else np.asarray(ids)

    def expect(self):
        y, e = ov.product(self.fmt, self.raw, self.N, self.K, self.x)
        if self.T <= 8:
            w = ov.oracle.dequant(self.fmt, self.raw, self.N, self.K).astype(np.float64).reshape(self.N, self.K)
            e = 1e-4 * np.abs(self.x) @ np.abs(w).T + 1e-6
        d, ed = ov.adapters(self.x, self.A, self.B, self.scales, self.ids)
        out = y + d
        G = self.A.shape[0]
        out[(self.ids < -1) | (self.ids >= G)] = np.nan
        return out, e + ed + 2 * ov.U * (np.abs(y) + np.abs(d)), d

    def run(self, torch, qmv, **kw):
        return qmv.qmv_lora(self.fmt, torch.from_numpy(self.raw.reshape(-1)).cuda(), self.N, self.K,
                            kw.pop("x", None) if "x" in kw else self.xt.cuda(), self.At.cuda(), self.Bt.cuda(),
                            torch.from_numpy(self.scales).cuda(), torch.from_numpy(self.ids.astype(np.int32)).cuda(), **kw)


def assert_close(got, y, e, what=""):
    got = got.detach().cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(y)), what
    ok = ~np.isnan(y)
    assert np.all(np.abs(got[ok] - y[ok]) <= e[ok]), (what, float(np.max(np.abs(got[ok] - y[ok]) / e[ok])))


@pytest.mark.parametrize("x_name,a_name", [("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,N,blocks,R,G", [(1, 33, 1, 1, 1), (2, 130, 3, 5, 3), (8, 300, 4, 16, 8), (9, 65, 2, 8, 4), (40, 257, 5, 3, 70),
                                            (150, 128, 2, 64, 2), (33, 70, 8, 128, 3), (300, 200, 3, 17, 5)])
def test_against_64_bits(env, fmt, x_name, a_name, T, N, blocks, R, G):
    torch, qmv = env
    K = blocks * (256 if fmt in ("q4_k", "q6_k") else 32)
    say("lora", fmt, x_name, a_name, T, N, K, R, G)
    c = Case(torch, fmt, T, N, K, R, G, x_name, a_name)
    y, e, _ = c.expect()
    assert_close(c.run(torch, qmv), y, e)


@pytest.mark.parametrize("x_name,a_name", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,N,blocks,R,G", [(300, 16500, 1, 8, 3), (40, 2000, 9, 24, 40), (100, 600, 5, 72, 9)])
def test_every_tile_shape(env, fmt, x_name, a_name, T, N, blocks, R, G):
    torch, qmv = env
    K = blocks * (256 if fmt in ("q4_k", "q6_k") else 32)
    say("lora tiles", fmt, x_name, T, N, K, R, G)
    c = Case(torch, fmt, T, N, K, R, G, x_name, a_name, seed=3)
    y, e, _ = c.expect()
    assert_close(c.run(torch, qmv), y, e)


@pytest.mark.parametrize("T", [1, 7, 60, 260])
def test_no_adapter_is_the_base_and_bad_ids_are_nan(env, T):
    torch, qmv = env
    c = Case(torch, "q4_0", T, 96, 256, 8, 3, "bf16", "bf16", ids=np.full(T, -1))
    base = c.run(torch, qmv)
    if T <= 8:
        same = qmv.qmv_matvec_xt("q4_0", torch.from_numpy(c.raw.reshape(-1)).cuda(), 96, 256, c.xt.cuda())
        assert torch.equal(base, same.view_as(base))
    y, e, _ = c.expect()
    assert_close(base, y, e)
    c.ids = np.where(np.arange(T) % 3 == 0, 3, np.where(np.arange(T) % 3 == 1, -2, 1))
    y, e, _ = c.expect()
    got = c.run(torch, qmv)
    assert_close(got, y, e)
    # a token's outputs do not depend on the other tokens' adapters
    c.ids[0] = -1
    again = c.run(torch, qmv)
    assert torch.equal(again[0], base[0])
    if T > 1:
        assert np.array_equal(got[1:].cpu().numpy(), again[1:].cpu().numpy(), equal_nan=True)


def test_strides_and_an_output_given(env):
    torch, qmv = env
    for T in (3, 50):
        for pad, start in ((8, 0), (3, 1)):
            c = Case(torch, "q8_0", T, 70, 128, 6, 4, "f32", "bf16")
            y, e, _ = c.expect()
            wide = torch.zeros(T, 128 + pad + start)
            wide[:, start:start + 128] = c.xt
            out = torch.full((T, 90), 5.0).cuda()
            got = c.run(torch, qmv, x=wide.cuda()[:, start:start + 128], y=out[:, 7:77])
            assert_close(got, y, e, (T, pad))
            assert (out[:, :7] == 5).all() and (out[:, 77:] == 5).all()


def test_adapters_off_16_bytes(env):
    """Adapter rows whose length or start allows no wide loads."""
    torch, qmv = env
    for T in (2, 40):
        for R in (3, 16):
            c = Case(torch, "q4_1", T, 75, 96, R, 3, "bf16", "bf16")
            y, e, _ = c.expect()
            A = torch.empty(c.At.numel() + 1, dtype=c.At.dtype, device="cuda")[1:].view_as(c.At)
            B = torch.empty(c.Bt.numel() + 3, dtype=c.Bt.dtype, device="cuda")[3:].view_as(c.Bt)
            A.copy_(c.At)
            B.copy_(c.Bt)
            got = qmv.qmv_lora("q4_1", torch.from_numpy(c.raw.reshape(-1)).cuda(), 75, 96, c.xt.cuda(), A, B,
                               torch.from_numpy(c.scales).cuda(), torch.from_numpy(c.ids.astype(np.int32)).cuda())
            assert_close(got, y, e, (T, R))


@pytest.mark.parametrize("T", [20, 200])
def test_token_of_nan_stays_alone(env, T):
    torch, qmv = env
    c = Case(torch, "q6_k", T, 64, 256, 8, 2, "f16", "f16", ids=np.arange(T) % 2)
    clean = c.run(torch, qmv).cpu().numpy()
    c.xt[4] = float("nan")
    c.xt[9, 2] = float("inf")
    got = c.run(torch, qmv).cpu().numpy()
    keep = np.ones(T, bool)
    keep[[4, 9]] = False
    assert np.array_equal(got[keep], clean[keep]) and not np.isfinite(got[~keep]).any()


@pytest.mark.parametrize("T", [4, 33, 200])
def test_other_stream_graph_and_repeats(env, T):
    torch, qmv = env
    c = Case(torch, "q4_0", T, 160, 256, 16, 5, "bf16", "bf16")
    W, A, B = torch.from_numpy(c.raw.reshape(-1)).cuda(), c.At.cuda(), c.Bt.cuda()
    s, ids, x = torch.from_numpy(c.scales).cuda(), torch.from_numpy(c.ids.astype(np.int32)).cuda(), c.xt.cuda()

    def call(stream=None):
        return qmv.qmv_lora("q4_0", W, 160, 256, x, A, B, s, ids, stream=stream)
    eager = call().cpu()
    assert torch.equal(call().cpu(), eager)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call(side)
    side.synchronize()
    assert torch.equal(other.cpu(), eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    gen = torch.Generator().manual_seed(T)
    for k in range(4):
        x.copy_(torch.randn(T, 256, generator=gen))
        ids.copy_(torch.randint(-1, 5, (T,), generator=gen, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), call().cpu()), k
