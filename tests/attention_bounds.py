"""Attention of one request in 64 bits, with a bound that has no allowance for weights that are lost: a weight may be off by its
roundings, relative to itself, and by 2^-39 of the row's largest, the last bit of fp16 under weights of up to 2^14.

A rounding to a type is off by at most half a step, eps / 2 relative to the value: 2^-24 in fp32, 2^-11 in fp16, 2^-8 in bf16.
"""
import torch

U, H16 = 2.0 ** -24, 2.0 ** -11
HALF = {"f32": U, "f16": H16, "bf16": 2.0 ** -8}


def attention(q, k, v, scale, pos, x, many, window=0, sink=None, k_size=None):
    """q [heads, rows, D], k and v [heads, L, D] float64, pos [rows] (positions), sink [heads, rows] or None; x the type of the
    queries, many whether a request has more than 32 rows (K is made fp16); k_size: sizes of the terms that k is the sum of
    (|k| by default).  Returns (out, bound)."""
    D, L = q.shape[-1], k.shape[1]
    two = x != "bf16"
    j = torch.arange(L, device=q.device)
    seen = j <= pos[:, None]
    if window:
        seen &= j > pos[:, None] - window
    s = scale * torch.matmul(q, k.transpose(1, 2).contiguous())
    size = scale * torch.matmul(q.abs(), (k.abs() if k_size is None else k_size).transpose(1, 2).contiguous())
    top = s.masked_fill(~seen, -float("inf")).amax(-1)
    if sink is not None:
        top = torch.maximum(top, sink)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p = torch.exp((s - top[..., None]).masked_fill(~seen, -float("inf")))
    total = p.sum(-1)
    if sink is not None:
        total = total + torch.exp(sink - top)
    w = p / torch.where(total > 0, total, torch.ones_like(total))[..., None]
    out = torch.matmul(w, v)
    # a score: up to 2 D + 64 roundings of partial sums and scales in fp32; pieces of queries 2^-22 twice, and of keys where they
    # are made fp16; single pieces of keys 2^-11, codes below fp16's normal numbers 2^-20; its multiple of log 2 and the
    # difference to the maximum 4 more, of which the exponential adds 2^-22
    es = (2 * D + 64 + (24 if two else 0)) * U * size + (0 if two else H16 if many else 2.0 ** -20) * size
    es = (es + 4 * U * s.abs() + 4 * U * top.abs()[..., None] + 8 * U).masked_fill(~seen, 0.0)
    # weights and values: one rounding each (22 bits each in two pieces), their sums' up to L + 128
    rel = 2 * es + 2 * (8 * U if two else H16) + (L + 128) * U
    a = v.abs()
    wa = torch.matmul(w, a)
    bound = torch.matmul(w * rel, a) + wa * ((w * es).sum(-1, keepdim=True) * 2 + (8 * U if two else H16) + (L + 128) * U)
    # a weight's last bit, and that of a value (2^-25; 2^-36 with a second piece that has its own)
    bound = bound + 2.0 ** -39 * torch.matmul(seen.double().expand_as(w), a) / total.clamp(min=1e-300)[..., None]
    bound = bound + 2.0 ** -25
    return out, bound * 1.01 + HALF[x] * (out.abs() + bound) + 2.0 ** -120


def of_cache(qmv, cache, q, table, lens, begin, scale, x, window=0, sinks=None, k_spread=1.0):
    """All requests' outputs and bounds [tokens, heads, D] from the values that qmv_cache_read gives; rows of no request are 0.
    k_spread: how many times the block's largest value the terms of a stored key may be (3 for Q4_1)."""
    out, bound = torch.zeros(q.shape, dtype=torch.float64, device=q.device), torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    D, P, H = q.shape[2], cache.page_size, cache.n_kv_heads
    G = q.shape[1] // H
    for r in range(table.shape[0]):
        a, b, L = int(begin[r]), int(begin[r + 1]), int(lens[r])
        if a == b or L == 0:
            continue
        j = torch.arange(L, device=q.device)
        slots = (table[r][j // P].long() * P + j % P).to(torch.int32)
        k, v = (t.double().transpose(0, 1).contiguous() for t in qmv.qmv_cache_read(cache, slots))
        qq = q[a:b].double().view(b - a, H, G, D).permute(1, 0, 2, 3).flatten(1, 2)
        pos = torch.arange(L - (b - a), L, device=q.device).repeat_interleave(G)
        sk = None if sinks is None else sinks.double().view(H, 1, G).expand(H, b - a, G).flatten(1)
        size = k.abs()
        if k_spread != 1.0:
            c = size.unflatten(-1, (D // 32, 32))
            size = (k_spread * c.amax(-1, keepdim=True)).expand_as(c).flatten(-2)
        o, e = attention(qq, k, v, scale, pos, x, (b - a) * G > 32, window, sk, size)
        for dest, t in ((out, o), (bound, e)):
            dest[a:b] = t.unflatten(1, (b - a, G)).permute(1, 0, 2, 3).flatten(1, 2)
    return out, bound


def close(got, want, bound):
    g = got.double()
    assert bool(torch.isfinite(g).all()), torch.nonzero(~torch.isfinite(g))[:5].tolist()
    off = (g - want).abs()
    at = int((off / bound).argmax())
    f = [t.flatten()[at].item() for t in (off, bound, g, want)]
    print("worst", f[0] / f[1], "off", float((g - want).norm() / want.norm()), flush=True)
    assert bool((off <= bound).all()), (at, f)
