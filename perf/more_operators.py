"""The operators of a quantized key/value cache and of token log probabilities, as they are measured.

Four operators, each in plain torch operations (``own`` false) and through the library's entry points (``own`` true):

write      new keys and values quantized into the pages of a cache (blocks of 32 values, Q8_0, Q4_0 or Q4_1), then read back: the
           values that the stored blocks stand for.
read       tokens of a cache, from any pages, as values.
attention  softmax(q k^T scale) v over such a cache, one request's tokens behind each other in its pages: causal, grouped heads,
           one or a few new tokens per request, or a piece of a prompt; optionally a sliding window and sink logits.
logprobs   log probabilities of given tokens under rows of logits, with the rows' entropy and most probable tokens.

A page of a cache holds `page` tokens of every key/value head: for each head the tokens' codes (4 or 8 bits, rows of `dim` values),
then fp16 scales [dim / 32][page], and for Q4_1 fp16 minimums [dim / 32][page].  In a row the 8 values 32 b + 8 g .. + 7 lie at
place g * (dim / 32) + b, as 8 bytes, or as 4 bytes with value 2 j in nibble j and value 2 j + 1 in nibble j + 4.  Q8_0 stands for
d * (signed byte), Q4_0 for d * (c - 8), Q4_1 for d * c + m.

Head shapes and vocabularies are those of the layer sets in ``workloads``, and generic odd ones.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
BITS = {"q8_0": 8, "q4_0": 4, "q4_1": 4}
ROW = {"q8_0": 34, "q4_0": 18, "q4_1": 20}      # bytes of 32 values
LIMIT = 65024.0                                 # larger values are stored as this


def listed():
    return [
        # a decode step's new tokens, one of each of 48 requests, into their pages: latency
        dict(name="write 48 q4_0 bf16", op="write", tokens=48, run=1, kv_heads=8, dim=128, page=16, k_fmt="q4_0", v_fmt="q4_0", x="bf16"),
        # a prompt's keys in 8 bits and values in 4, from fp32 projections
        dict(name="write 6000 q8_0 q4_1 f32", op="write", tokens=6000, run=1500, kv_heads=8, dim=128, page=64, k_fmt="q8_0",
             v_fmt="q4_1", x="f32"),
        # a short prefix of small heads, odd count
        dict(name="read 333 q4_1 f32", op="read", tokens=333, run=333, kv_heads=4, dim=64, page=32, k_fmt="q4_1", v_fmt="q4_1", x="f32"),
        # a shared prefix brought back to 16 bits for a kernel that needs it so
        dict(name="read 65536 q4_0 bf16", op="read", tokens=65536, run=16384, kv_heads=8, dim=128, page=64, k_fmt="q4_0",
             v_fmt="q4_0", x="bf16"),
        # one request, one new token, the 8B set's heads, a short chat: latency
        dict(name="attention decode 1x700 q4_0", op="attention", requests=1, heads=32, kv_heads=8, dim=128, page=16, k_fmt="q4_0",
             v_fmt="q4_0", x="bf16", new=1, ragged=False, short=700, long=700, window=0, sinks=False),
        # a busy server's decode step: 64 requests of very different lengths
        dict(name="attention decode 64 q4_0", op="attention", requests=64, heads=32, kv_heads=8, dim=128, page=64, k_fmt="q4_0",
             v_fmt="q4_0", x="bf16", new=1, ragged=False, short=200, long=8000, window=0, sinks=False),
        # one long document, keys in 8 bits: the whole GPU on one request
        dict(name="attention decode 1x131000 f16", op="attention", requests=1, heads=32, kv_heads=4, dim=128, page=256, k_fmt="q8_0",
             v_fmt="q4_0", x="f16", new=1, ragged=False, short=131000, long=131000, window=0, sinks=False),
        # drafted tokens of 16 requests under verification, the 0.6B set's heads, queries as the matvec gives them
        dict(name="attention verify 16x5 q8_0 f32", op="attention", requests=16, heads=16, kv_heads=8, dim=128, page=32, k_fmt="q8_0",
             v_fmt="q8_0", x="f32", new=5, ragged=False, short=900, long=4000, window=0, sinks=False),
        # a chunk of a long prompt behind what is in the cache already: bound by arithmetic
        dict(name="attention prefill 2048 q4_0", op="attention", requests=1, heads=32, kv_heads=8, dim=128, page=64, k_fmt="q4_0",
             v_fmt="q4_0", x="bf16", new=2048, ragged=False, short=8192, long=8192, window=0, sinks=False),
        # a mixed step: pieces of prompts and single tokens, a sliding window with sinks, odd head group, small heads
        dict(name="attention mixed 13 q4_1", op="attention", requests=13, heads=14, kv_heads=2, dim=64, page=16, k_fmt="q4_1",
             v_fmt="q4_1", x="f16", new=301, ragged=True, short=1, long=5000, window=1024, sinks=True),
        # one request's next token with its alternatives: latency
        dict(name="logprobs 1x128256 f32", op="logprobs", rows=1, vocab=128256, x="f32", given=1, top=5),
        # scoring a batch of prompts' tokens
        dict(name="logprobs 500x151936 bf16", op="logprobs", rows=500, vocab=151936, x="bf16", given=1, top=20),
    ]


def _between(rng, lo, hi):
    """A whole number in lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attention", "attention", "attention", "logprobs"])
    x = rng.choice(["f32", "f16", "bf16"])
    if op == "logprobs":
        vocab = _between(rng, 1000, 151936)
        return dict(op=op, rows=_between(rng, 1, min(2000, 75_000_000 // vocab)), vocab=vocab, x=x, given=rng.choice([0, 1, 1, 4]),
                    top=rng.choice([0, 1, 5, 20, 32]))
    dim, kv_heads, page = rng.choice([64, 128, 256]), rng.randint(1, 8), 1 << rng.randint(4, 8)
    k_fmt, v_fmt = rng.choice(list(BITS)), rng.choice(list(BITS))
    common = dict(op=op, kv_heads=kv_heads, dim=dim, page=page, k_fmt=k_fmt, v_fmt=v_fmt, x=x)
    if op != "attention":
        tokens = _between(rng, 1, 6_000_000 // (kv_heads * dim) if op == "write" else 40_000_000 // (kv_heads * dim))
        return dict(common, tokens=tokens, run=_between(rng, 1, tokens))
    group = rng.choice([1, 2, 4, 4, 5, 7, 8, 16])
    new = rng.choice([1, 1, 1, rng.randint(2, 8), _between(rng, 9, 1500)])
    requests = _between(rng, 1, 64) if new <= 8 else _between(rng, 1, 8)
    if new > 8:
        new = min(new, int(math.sqrt(5e10 / (requests * kv_heads * group * dim))))
    # as much work as the largest listed case at most: 500e6 values read, and the products of the queries
    long = _between(rng, 1, max(64, min(100_000, 200_000_000 // (requests * kv_heads * dim), int(2e10 / (requests * new * kv_heads * group * dim)))))
    return dict(common, requests=requests, heads=kv_heads * group, new=new, ragged=new > 1 and rng.random() < 0.6, short=_between(rng, 1, long),
                long=max(long, new), window=rng.choice([0, 0, _between(rng, 1, 4096)]), sinks=rng.random() < 0.3)


# ---------------------------------------------------------------- inputs
def _pages(fmt, n, heads, page, dim, gen):
    """uint8 [n, heads, bytes of a head] of values about N(0, 1): scales that vary by block, codes as such values give."""
    dev, nb = gen.device, dim // 32
    sd, mid, lo, hi = (50.0, 0.0, -127, 127) if fmt == "q8_0" else (3.3, 8.0 if fmt == "q4_0" else 7.5, 0, 15)
    c = torch.randn(n, heads, page, dim, generator=gen, device=dev, dtype=torch.float16).mul_(sd).add_(mid).round_().clamp_(lo, hi)
    c = c.to(torch.int8).view(torch.uint8)
    if fmt != "q8_0":
        c = c[..., :dim // 2] | (c[..., dim // 2:] << 4)      # which value is in which nibble does not matter: they are alike
    d = (0.7 + 0.6 * torch.rand(n, heads, nb, page, generator=gen, device=dev)) / sd
    parts = [c.reshape(n, heads, -1), d.half().view(n, heads, -1).view(torch.uint8)]
    if fmt == "q4_1":
        parts.append((-7.5 * d).half().view(n, heads, -1).view(torch.uint8))
    return torch.cat(parts, dim=-1)


def _cache(st, n, gen):
    st["k_pages"] = _pages(st["k_fmt"], n, st["kv_heads"], st["page"], st["dim"], gen)
    st["v_pages"] = _pages(st["v_fmt"], n, st["kv_heads"], st["page"], st["dim"], gen)


def _randn(gen, dtype, *shape):
    return torch.randn(*shape, generator=gen, device=gen.device).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * int(seed) + 29)
    st, dev, x = dict(case), "cuda", DTYPES[case["x"]]
    if case["op"] == "logprobs":
        R, V = case["rows"], case["vocab"]
        st["logits"] = torch.randn(R, V, generator=gen, device=dev).mul_(3.0).to(x)
        # tokens that were drawn from about these probabilities
        noise = torch.rand(R, V, generator=gen, device=dev).clamp_(1e-6, 1 - 1e-6).log_().neg_().log_().neg_()
        first = noise.add_(st["logits"]).argmax(dim=1, keepdim=True)
        others = torch.randint(0, V, (R, 3), generator=gen, device=dev)
        st["tokens"] = torch.cat([first, others], dim=1)[:, :case["given"]].to(torch.int32).contiguous()
        return st
    H, D, P = case["kv_heads"], case["dim"], case["page"]
    if case["op"] in ("write", "read"):
        # runs of `run` tokens behind each other, each from the middle of a page on, their pages anywhere
        T, run = case["tokens"], case["run"]
        runs = -(-T // run)
        each = -(-(run + P) // P)
        order = torch.randperm(runs * each + 3, generator=gen, device=dev)[:runs * each].view(runs, each)
        at = torch.arange(T, device=dev)
        begin = torch.randint(0, P, (runs,), generator=gen, device=dev)
        place = begin[at // run] + at % run
        st["slots"] = (order[at // run, place // P] * P + place % P).to(torch.int32)
        _cache(st, runs * each + 3, gen)
        if case["op"] == "write":
            # channels of different size, as keys have them
            size = torch.exp(0.5 * torch.randn(1, H, D, generator=gen, device=dev))
            st["k"], st["v"] = (_randn(gen, torch.float32, T, H, D) * size).to(x), _randn(gen, x, T, H, D)
        return st
    R, new = case["requests"], case["new"]
    if case["ragged"]:
        # most requests have a token or a few, some a piece of a prompt
        n = torch.exp(torch.linspace(0.0, 1.0, R, device=dev) ** 2 * math.log(new + 0.5)).long().clamp_(1, new)
        n = n[torch.randperm(R, generator=gen, device=dev)]
    else:
        n = torch.full((R,), new, device=dev)
    st["q_begin"] = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), n.cumsum(0)]).to(torch.int32)
    st["most"] = new
    lo, hi = math.log(case["short"]), math.log(case["long"])
    lens = torch.exp(lo + (hi - lo) * torch.rand(R, generator=gen, device=dev)).round_().long()
    lens[0] = case["long"]
    lens = torch.maximum(lens.clamp_(1, case["long"]), n)      # the new tokens are in the cache
    st["lens"] = lens.to(torch.int32)
    each = -(-case["long"] // P)
    pages = R * each + 3
    st["table"] = torch.randperm(pages, generator=gen, device=dev)[:R * each].view(R, each).to(torch.int32)
    _cache(st, pages, gen)
    total = int(st["q_begin"][-1])
    st["q"] = (1.5 * _randn(gen, torch.float32, total, case["heads"], D)).to(x)
    st["scale"] = 1.0 / math.sqrt(D)
    st["sink"] = _randn(gen, torch.float32, case["heads"]) + 2.0 if case["sinks"] else None
    return st


# ---------------------------------------------------------------- plain forms
def _planes(pages, fmt, P, D):
    """Views of a cache's pages: codes [n, heads, P, bytes of a row], scales and minimums [n, heads, D / 32, P]."""
    nb, codes = D // 32, P * D * BITS[fmt] // 8
    half = pages[..., codes:].view(torch.float16).unflatten(-1, (-1, nb, P))
    return pages[..., :codes].unflatten(-1, (P, -1)), half[:, :, 0], half[:, :, 1] if fmt == "q4_1" else None


def _octets(rows, fmt, D):
    """Codes [..., D] as float32 of rows of stored bytes, in the values' order."""
    if fmt == "q8_0":
        c = rows.view(torch.int8).float().unflatten(-1, (4, D // 32, 8))
    else:
        b = rows.unflatten(-1, (4, D // 32, 4))
        # bytes 0, 1 hold values 0, 2, 4, 6, bytes 2, 3 values 1, 3, 5, 7
        nib = torch.stack([b & 15, b >> 4], dim=-1).flatten(-2)
        c = nib.unflatten(-1, (2, 4)).transpose(-1, -2).flatten(-2).float()
    return c.transpose(-2, -3).flatten(-3)


def _stored(rows, d, m, fmt, D):
    """float32 [..., D] of stored rows, d and m [..., D / 32]."""
    c = _octets(rows, fmt, D).unflatten(-1, (D // 32, 32))
    if fmt == "q4_0":
        c = c - 8.0
    v = c * d.float().unsqueeze(-1)
    if fmt == "q4_1":
        v = v + m.float().unsqueeze(-1)
    return v.flatten(-2)


def _read_plain(pages, fmt, slots, P, D):
    codes, d, m = _planes(pages, fmt, P, D)
    page, off = slots.long() // P, slots.long() % P
    return _stored(codes[page, :, off], d[page, :, :, off], m[page, :, :, off] if m is not None else None, fmt, D)


def _away(v):
    return torch.sign(v) * torch.floor(v.abs() + 0.5)


def _encoded(x, fmt):
    """Codes [..., D], scales and minimums [..., D / 32]: in 64 bits, next to the borders between codes."""
    w = x.double().clamp(-LIMIT, LIMIT).unflatten(-1, (-1, 32))
    if fmt == "q8_0":
        d, m = (w.abs().amax(-1) / 127.0).half(), None
        q = torch.where(d.unsqueeze(-1) != 0, _away(w / d.double().unsqueeze(-1)).clamp(-127, 127), 0.0)
    elif fmt == "q4_0":
        place = torch.arange(32, device=w.device)
        at = torch.where(w.abs() == w.abs().amax(-1, keepdim=True), place, 31).amin(-1, keepdim=True)      # the first of the largest
        d, m = (torch.gather(w, -1, at).squeeze(-1) / -8.0).half(), None
        q = torch.where(d.unsqueeze(-1) != 0, (_away(w / d.double().unsqueeze(-1)) + 8.0).clamp(0, 15), 8.0)
    else:
        m = w.amin(-1).half()
        d = ((w.amax(-1) - w.amin(-1)) / 15.0).half()
        q = torch.where(d.unsqueeze(-1) != 0, _away((w - m.double().unsqueeze(-1)) / d.double().unsqueeze(-1)).clamp(0, 15), 0.0)
    return q.flatten(-2), d, m


def _write_plain(pages, fmt, x, slots, P, D):
    q, d, m = _encoded(x, fmt)
    q = q.unflatten(-1, (D // 32, 4, 8)).transpose(-2, -3)
    if fmt == "q8_0":
        rows = q.to(torch.int8).view(torch.uint8).flatten(-3)
    else:
        u = q.to(torch.uint8)
        rows = (u[..., [0, 4, 1, 5]] | (u[..., [2, 6, 3, 7]] << 4)).flatten(-3)
    codes, dp, mp = _planes(pages, fmt, P, D)
    page, off = slots.long() // P, slots.long() % P
    codes[page, :, off] = rows
    dp[page, :, :, off] = d
    if m is not None:
        mp[page, :, :, off] = m


def _attention_plain(st):
    R, Hq, H, D, P, n = st["requests"], st["heads"], st["kv_heads"], st["dim"], st["page"], st["most"]
    G = Hq // H
    L = st["table"].shape[1] * P

    def values(pages, fmt):
        codes, d, m = _planes(pages[st["table"].long()].flatten(0, 1), fmt, P, D)
        v = _stored(codes, d.transpose(-1, -2), m.transpose(-1, -2) if m is not None else None, fmt, D)
        return v.view(R, -1, H, P, D).transpose(1, 2).reshape(R, H, L, D)
    lens, begin = st["lens"].long(), st["q_begin"].long()
    i, j = torch.arange(n, device=lens.device), torch.arange(L, device=lens.device)
    mine = begin[1:] - begin[:-1]
    at = (begin[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"].float()[at].view(R, n, H, G, D).transpose(1, 2).reshape(R, H, n * G, D)
    s = torch.matmul(q, values(st["k_pages"], st["k_fmt"]).transpose(-1, -2).contiguous()).view(R, H, n, G, L)
    pos = (lens - mine)[:, None] + i
    seen = j <= pos[..., None]
    if st["window"]:
        seen &= j > pos[..., None] - st["window"]
    s = (s * st["scale"]).masked_fill_(~seen[:, None, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    if st["sink"] is not None:
        sink = st["sink"].view(1, H, 1, G, 1)
        top = torch.maximum(top, sink)
    top = top.clamp(min=-1e30)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    if st["sink"] is not None:
        total = total + torch.exp(sink - top)
    o = torch.matmul(p.view(R, H, n * G, L), values(st["v_pages"], st["v_fmt"])).view(R, H, n, G, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(R, n, Hq, D)
    return o[i < mine[:, None]].to(st["q"].dtype)


def _logprobs_plain(st):
    l = st["logits"].float()
    V, k = l.shape[1], st["top"]
    top = l.amax(1, keepdim=True)
    z = l - top
    e = torch.exp(z)
    # sums without the largest term, so that what is left of a certain row is not lost beside 1
    e.scatter_(1, z.argmax(1, keepdim=True), 0.0)
    rest = e.double().sum(1)
    log_total = torch.log1p(rest)
    entropy = (log_total - (e.double() * z).sum(1) / (1.0 + rest)).float()
    out = {"entropy": entropy}
    if st["given"]:
        out["logprobs"] = (z.gather(1, st["tokens"].long()) - log_total[:, None]).float()
    if k:
        best = torch.sort(z, dim=1, descending=True, stable=True)
        out["top_tokens"] = best.indices[:, :k].to(torch.int32)
        out["top_logprobs"] = (best.values[:, :k] - log_total[:, None]).float()
    return out


# ---------------------------------------------------------------- the library's calls
def _own(st):
    import bandwidth_bound_block_amd as qmv
    if st["op"] == "logprobs":
        r = qmv.qmv_logprobs(st["logits"], st["tokens"] if st["given"] else None, top_k=st["top"])
        out = {"entropy": r.entropy}
        if st["given"]:
            out["logprobs"] = r.logprobs
        if st["top"]:
            out["top_tokens"], out["top_logprobs"] = r.top_tokens, r.top_logprobs
        return out
    cache = qmv.KVCache(st["k_pages"], st["v_pages"], st["k_fmt"], st["v_fmt"], st["kv_heads"], st["dim"], st["page"])
    if st["op"] == "write":
        qmv.qmv_cache_write(cache, st["k"], st["v"], st["slots"])
        return qmv.qmv_cache_read(cache, st["slots"])
    if st["op"] == "read":
        return qmv.qmv_cache_read(cache, st["slots"], dtype=DTYPES[st["x"]])
    return qmv.qmv_cache_attention(cache, st["q"], st["table"], st["lens"], q_begin=st["q_begin"], max_q=st["most"],
                                   scale=st["scale"], window=st["window"], sinks=st["sink"])


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "logprobs":
        return _logprobs_plain(state)
    if op == "attention":
        return _attention_plain(state)
    P, D, slots = state["page"], state["dim"], state["slots"]
    if op == "write":
        _write_plain(state["k_pages"], state["k_fmt"], state["k"], slots, P, D)
        _write_plain(state["v_pages"], state["v_fmt"], state["v"], slots, P, D)
    dtype = torch.float32 if op == "write" else DTYPES[state["x"]]
    return (_read_plain(state["k_pages"], state["k_fmt"], slots, P, D).to(dtype),
            _read_plain(state["v_pages"], state["v_fmt"], slots, P, D).to(dtype))


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    size = SIZE[case["x"]]
    if case["op"] == "logprobs":
        R, V = case["rows"], case["vocab"]
        return {"bytes": R * V * float(size) + R * (4.0 + 8.0 * case["given"] + 8.0 * case["top"]), "flops": 4.0 * R * V}
    H, D = case["kv_heads"], case["dim"]
    stored = H * (D // 32) * (ROW[case["k_fmt"]] + ROW[case["v_fmt"]])      # bytes of a token
    if case["op"] == "write":
        T = case["tokens"]
        return {"bytes": T * (2.0 * H * D * (size + 4) + 2.0 * stored + 4.0), "flops": 8.0 * T * H * D}
    if case["op"] == "read":
        T = case["tokens"]
        return {"bytes": T * (2.0 * H * D * size + stored + 4.0), "flops": 4.0 * T * H * D}
    R, Hq, new, W = case["requests"], case["heads"], case["new"], case["window"]
    lo, hi = case["short"], case["long"]
    mean = (hi - lo) / math.log(hi / lo) if hi > lo else float(lo)          # of lengths even over their logarithm
    n = new * 0.4 if case["ragged"] and new > 8 else (new + 1) / 2.0 if case["ragged"] else float(new)
    mean = max(mean, n)
    per_query = max(mean - (n - 1) / 2.0, 1.0)
    read = mean
    if W:
        per_query, read = min(per_query, W), min(read, W + n)
    return {"bytes": R * (read * stored + 2.0 * n * Hq * D * size), "flops": 4.0 * R * n * Hq * D * per_query}


# ---------------------------------------------------------------- the same in 64 bits
def _rows64(pages, fmt, P, D, page, off):
    """float64 [tokens, heads, D]: value by value from the bytes at their offsets."""
    n, H, size = pages.shape
    e = torch.arange(D, device=pages.device)
    place = ((e // 8) % 4) * (D // 32) + e // 32
    i = e % 8
    head = (page[:, None, None] * H + torch.arange(H, device=pages.device)[None, :, None]) * size
    flat = pages.reshape(-1)
    codes = P * D * BITS[fmt] // 8

    def half(at):
        return torch.stack([flat[at], flat[at + 1]], dim=-1).view(torch.float16).squeeze(-1).double()
    at = head + codes + 2 * ((e // 32) * P + off[:, None, None])
    d = half(at)
    if fmt == "q8_0":
        b = flat[head + off[:, None, None] * D + place * 8 + i].to(torch.int32)
        return d * ((b + 128) % 256 - 128)
    b = flat[head + off[:, None, None] * (D // 2) + place * 4 + (i % 2) * 2 + (i // 2) // 2].to(torch.int32)
    c = torch.where((i // 2) % 2 == 1, b // 16, b % 16)
    return d * (c - 8) if fmt == "q4_0" else d * c + half(at + 2 * (D // 32) * P)


def _nearest64(x, fmt):
    """The values that x is stored as, block by block, in 64 bits."""
    T, H, D = x.shape
    w = x.to(torch.float64).clamp(-LIMIT, LIMIT).reshape(-1, 32)
    if fmt == "q4_1":
        base = w.min(1, keepdim=True).values
        step = ((w.max(1, keepdim=True).values - base) / 15).to(torch.float16).double()
        base = base.to(torch.float16).double()
        code = torch.nan_to_num(torch.floor((w - base) / step + 0.5), nan=0.0, posinf=0.0, neginf=0.0).clamp(0, 15)
        return (code * step + base).view(T, H, D)
    # the first of the largest: a stable order by size
    big = w.gather(1, torch.sort(w.abs(), dim=1, descending=True, stable=True).indices[:, :1])
    step = (big.abs() / 127 if fmt == "q8_0" else -big / 8).to(torch.float16).double()
    t = torch.nan_to_num(w / step, nan=0.0, posinf=0.0, neginf=0.0)
    code = torch.where(t < 0, -torch.floor(0.5 - t), torch.floor(t + 0.5))
    code = code.clamp(-127, 127) if fmt == "q8_0" else code.clamp(-8, 7)
    return (code * step).view(T, H, D)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "logprobs":
        l = st["logits"]
        out = {"entropy": torch.empty(case["rows"], dtype=torch.float64, device=l.device)}
        if case["given"]:
            out["logprobs"] = torch.empty(case["rows"], case["given"], dtype=torch.float64, device=l.device)
        if case["top"]:
            out["top_tokens"], out["top_logprobs"] = None, torch.empty(case["rows"], case["top"], dtype=torch.float64, device=l.device)
        for a in range(0, case["rows"], 64):
            z = torch.log_softmax(l[a:a + 64].double(), dim=1)
            out["entropy"][a:a + 64] = -(z.exp() * z).sum(1)
            if case["given"]:
                out["logprobs"][a:a + 64] = z.gather(1, st["tokens"][a:a + 64].long())
            if case["top"]:
                out["top_logprobs"][a:a + 64] = z.topk(case["top"], dim=1).values
        return out
    P, D, H = case["page"], case["dim"], case["kv_heads"]
    if op == "write":
        return _nearest64(st["k"], case["k_fmt"]), _nearest64(st["v"], case["v_fmt"])
    if op == "read":
        page, off = st["slots"].long() // P, st["slots"].long() % P
        return (_rows64(st["k_pages"], case["k_fmt"], P, D, page, off), _rows64(st["v_pages"], case["v_fmt"], P, D, page, off))
    G = case["heads"] // H
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    begins, lens = st["q_begin"].tolist(), st["lens"].tolist()
    for r in range(case["requests"]):
        a, b, n = begins[r], begins[r + 1], lens[r]
        j = torch.arange(n, device="cuda")
        page, off = st["table"][r].long()[j // P], j % P
        k, v = _rows64(st["k_pages"], case["k_fmt"], P, D, page, off), _rows64(st["v_pages"], case["v_fmt"], P, D, page, off)
        pos = torch.arange(n - (b - a), n, device="cuda")[:, None]
        hidden = (j > pos) | ((j <= pos - case["window"]) if case["window"] else False)
        for h in range(H):
            for c in range(0, b - a, 256):
                q = st["q"][a:b][c:c + 256, h * G:(h + 1) * G].double().transpose(0, 1)
                z = (q @ k[:, h].t()) * st["scale"]
                z = z.masked_fill(hidden[c:c + 256], -math.inf)
                if case["sinks"]:
                    z = torch.cat([z, st["sink"][h * G:(h + 1) * G].double().view(G, 1, 1).expand(G, z.shape[1], 1)], dim=-1)
                out[a:b][c:c + 256, h * G:(h + 1) * G] = (torch.softmax(z, dim=-1)[..., :n] @ v[:, h]).transpose(0, 1)
    return out
