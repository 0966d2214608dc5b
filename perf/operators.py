"""The operators of many-request serving, as they are measured.

Three operators, each in plain torch operations (``own`` false) and through the library's entry points (``own`` true):

experts  MoE expert products grouped by expert, for more tokens than a matvec takes.  form "product": one projection,
         y[t, s] = DEQ(W_e) x_t; form "block": gate||up with SwiGLU, down, and the router-weighted sum over the slots.
lora     a projection of quantized weights shared by all tokens plus each token's own low-rank adapter,
         y_t = DEQ(W) x_t + s_a B_a (A_a x_t).
verify   drafted tokens accepted or replaced by the target's probabilities, from given random numbers.

Weights are block-quantized (Q8_0, Q4_0, Q4_1, Q4_K, Q6_K) with codes and scales distributed as encoded Gaussian weights have
them; shapes are those of the 8B layer set and of the 128-expert set in ``workloads``, and generic odd ones.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ROW_BYTES = {"q8_0": (32, 34), "q4_0": (32, 18), "q4_1": (32, 20), "q4_k": (256, 144), "q6_k": (256, 210)}


def listed():
    return [
        # a few requests decoding together, one token more than the matvec's widest call: every routed expert streams from memory
        dict(name="experts decode 9 q4_0", op="experts", form="block", fmt="q4_0", tokens=9, top_k=8, experts=128, ff=768,
             hidden=2048, x="bf16", skew=0.0),
        # a busy server's decode step
        dict(name="experts decode 64 q6_k", op="experts", form="block", fmt="q6_k", tokens=64, top_k=8, experts=128, ff=768,
             hidden=2048, x="f16", skew=0.5),
        # one projection of large experts, odd token count, fp32 activations
        dict(name="experts product 77 q4_1", op="experts", form="product", fmt="q4_1", tokens=77, top_k=2, experts=8, ff=3584,
             hidden=4096, x="f32", skew=0.5),
        # a long prompt's prefill chunk, experts unevenly loaded
        dict(name="experts prefill 2048 q4_k", op="experts", form="block", fmt="q4_k", tokens=2048, top_k=8, experts=128,
             ff=768, hidden=2048, x="bf16", skew=0.5),
        # the same through one 8-bit projection of larger experts: bound by arithmetic
        dict(name="experts product 4096 q8_0", op="experts", form="product", fmt="q8_0", tokens=4096, top_k=2, experts=8,
             ff=2048, hidden=4096, x="bf16", skew=0.3),
        # one request's decode step with its adapter on the o projection: latency
        dict(name="lora decode 1 q4_0", op="lora", fmt="q4_0", tokens=1, rows=4096, cols=4096, rank=16, adapters=64,
             runs=1, x="bf16", a="bf16"),
        # eight requests, each with its own adapter, on the fused q+k+v rows
        dict(name="lora decode 8 q8_0", op="lora", fmt="q8_0", tokens=8, rows=6144, cols=4096, rank=16, adapters=64,
             runs=8, x="f32", a="f16"),
        # a mixed step: some requests decode, some run a piece of their prompt; down projection
        dict(name="lora mixed 101 q4_k", op="lora", fmt="q4_k", tokens=101, rows=4096, cols=14336, rank=8, adapters=32,
             runs=40, x="f16", a="f16"),
        # prompts of several tenants in one chunk, gate projection, a large rank
        dict(name="lora prefill 2048 q4_0", op="lora", fmt="q4_0", tokens=2048, rows=14336, cols=4096, rank=64, adapters=16,
             runs=11, x="bf16", a="bf16"),
        # one request, four drafted tokens, the 8B set's vocabulary: latency
        dict(name="verify 1x4 128256", op="verify", requests=1, drafts=4, vocab=128256, logits="f32", probs=True, ragged=False),
        # a batch of requests with ragged draft counts, drafts looked up in the prompt (no draft probabilities), odd vocabulary
        dict(name="verify 16x5 50257", op="verify", requests=16, drafts=5, vocab=50257, logits="bf16", probs=False, ragged=True),
        # the largest batch at the widest matvec, the largest vocabulary of the shape sets
        dict(name="verify 64x7 151936", op="verify", requests=64, drafts=7, vocab=151936, logits="f32", probs=True, ragged=True),
    ]


def _between(rng, lo, hi):
    """A whole number in lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["experts", "experts", "lora", "lora", "verify"])
    fmt = rng.choice(["q8_0", "q4_0", "q4_1", "q4_k", "q6_k"])
    unit = ROW_BYTES[fmt][0]
    x = rng.choice(["f32", "f16", "bf16"])
    if op == "experts":
        # the hidden size and the expert width are both some product's row length: whole blocks of the format
        form, top_k = rng.choice(["block", "product"]), rng.randint(1, 8)
        hidden, ff = unit * _between(rng, 256 // unit, 4096 // unit), unit * _between(rng, 256 // unit, 2048 // unit)
        if form == "product":
            ff = _between(rng, 100, 2048)
        weights = (3 if form == "block" else 1) * ff * hidden
        experts = min(_between(rng, 8, 128), max(8, 600_000_000 // weights))
        tokens = min(_between(rng, 1, 4096), int(1.5e11 / (2 * top_k * weights)))
        return dict(op=op, form=form, fmt=fmt, tokens=tokens, top_k=top_k, experts=experts, ff=ff,
                    hidden=hidden, x=x, skew=round(rng.uniform(0, 1), 2))
    if op == "lora":
        tokens, rows = _between(rng, 1, 2048), _between(rng, 500, 6000)
        return dict(op=op, fmt=fmt, tokens=tokens, rows=rows, cols=unit * _between(rng, 512 // unit, 8192 // unit),
                    rank=_between(rng, 4, 64), adapters=_between(rng, 1, 64), runs=_between(rng, 1, min(tokens, 64)), x=x,
                    a=rng.choice(["f32", "f16", "bf16"]))
    return dict(op=op, requests=_between(rng, 1, 64), drafts=rng.randint(1, 7), vocab=_between(rng, 1000, 150000), logits=x,
                probs=rng.random() < 0.6, ragged=rng.random() < 0.7)


# ---------------------------------------------------------------- inputs
def _half_bytes(v):
    return v.to(torch.float16).unsqueeze(-1).view(torch.uint8)


def _blocks(fmt, rows, cols, gen):
    """Stored bytes [rows, row bytes] of weights about N(0, 0.02^2): scales that vary by block, codes as such weights give."""
    dev = gen.device

    def scale(*shape, at):
        return at * (0.7 + 0.6 * torch.rand(*shape, generator=gen, device=dev))

    def codes(*shape, sd, mid, lo, hi):
        # float16 normals: the codes are small integers
        return (torch.randn(*shape, generator=gen, device=dev, dtype=torch.float16) * sd + mid).round_().clamp_(lo, hi)

    if fmt == "q8_0":
        nb = cols // 32
        d = _half_bytes(scale(rows, nb, at=0.02 / 50))
        q = codes(rows, nb, 32, sd=50.0, mid=0.0, lo=-127, hi=127).to(torch.int8).view(torch.uint8)
        return torch.cat([d, q], dim=-1).reshape(rows, -1)
    if fmt in ("q4_0", "q4_1"):
        nb = cols // 32
        c = codes(rows, nb, 32, sd=3.3, mid=8.0 if fmt == "q4_0" else 7.5, lo=0, hi=15).to(torch.uint8)
        d = scale(rows, nb, at=0.02 / 3.3)
        head = _half_bytes(d) if fmt == "q4_0" else torch.cat([_half_bytes(d), _half_bytes(-7.5 * d)], dim=-1)
        return torch.cat([head, c[..., :16] | (c[..., 16:] << 4)], dim=-1).reshape(rows, -1)
    ns = cols // 256
    if fmt == "q4_k":
        c = codes(rows, ns, 4, 2, 32, sd=3.3, mid=7.5, lo=0, hi=15).to(torch.uint8)
        sc = torch.randint(30, 64, (rows, ns, 8), generator=gen, device=dev, dtype=torch.uint8)
        d = scale(rows, ns, at=0.02 / 3.3 / 47)
        mn = (sc.to(torch.int32) * 15 // 16).to(torch.uint8)   # dmin mn about 7.5 d sc
        b = torch.cat([sc[..., :4] | ((sc[..., 4:] >> 4) << 6), mn[..., :4] | ((mn[..., 4:] >> 4) << 6),
                       (sc[..., 4:] & 15) | ((mn[..., 4:] & 15) << 4)], dim=-1)
        q = (c[..., 0, :] | (c[..., 1, :] << 4)).reshape(rows, ns, 128)
        return torch.cat([_half_bytes(d), _half_bytes(8.0 * d), b, q], dim=-1).reshape(rows, -1)
    c = codes(rows, ns, 2, 4, 32, sd=13.0, mid=32.0, lo=0, hi=63).to(torch.uint8)
    low, high = c & 15, c >> 4
    ql = torch.cat([low[..., 0, :] | (low[..., 2, :] << 4), low[..., 1, :] | (low[..., 3, :] << 4)], dim=-1)
    qh = high[..., 0, :] | (high[..., 1, :] << 2) | (high[..., 2, :] << 4) | (high[..., 3, :] << 6)
    sc = torch.randint(60, 128, (rows, ns, 16), generator=gen, device=dev, dtype=torch.uint8)
    return torch.cat([ql.reshape(rows, ns, 128), qh.reshape(rows, ns, 64), sc,
                      _half_bytes(scale(rows, ns, at=0.02 / 13.0 / 94))], dim=-1).reshape(rows, -1)


def _rand(gen, *shape):
    return torch.rand(*shape, generator=gen, device=gen.device)


def _randn(gen, dtype, *shape):
    return torch.randn(*shape, generator=gen, device=gen.device).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * int(seed) + 17)
    st = dict(case)
    if case["op"] == "experts":
        E, F, H, T, S = case["experts"], case["ff"], case["hidden"], case["tokens"], case["top_k"]
        first = (2 * F if case["form"] == "block" else F, H)
        st["W1"] = _blocks(case["fmt"], E * first[0], first[1], gen).reshape(-1)
        if case["form"] == "block":
            st["W2"] = _blocks(case["fmt"], E * H, F, gen).reshape(-1)
        # a router's choice: per token the top_k of noisy scores, some experts liked more than others
        liked = case["skew"] * torch.randn(E, generator=gen, device="cuda")
        noise = -torch.log(-torch.log(_rand(gen, T, E).clamp_(1e-6, 1 - 1e-6)))
        top = torch.topk(liked + noise, S, dim=1)
        st["ids"] = top.indices.to(torch.int32)
        st["weights"] = torch.softmax(top.values, dim=1)
        st["x_in"] = _randn(gen, DTYPES[case["x"]], T, H)
        st["most"] = int(torch.bincount(st["ids"].reshape(-1).long(), minlength=E).max())   # sizes a padded batch
    elif case["op"] == "lora":
        T, N, K, R, G = case["tokens"], case["rows"], case["cols"], case["rank"], case["adapters"]
        st["W"] = _blocks(case["fmt"], N, K, gen).reshape(-1)
        a = DTYPES[case["a"]]
        st["A"] = (_randn(gen, torch.float32, G, R, K) / math.sqrt(K)).to(a)
        st["B"] = (_randn(gen, torch.float32, G, N, R) * 0.1).to(a)
        st["scales"] = 0.5 + _rand(gen, G)
        # `runs` requests' tokens lie next to each other; about one request in eight has no adapter
        cuts = torch.sort(torch.randperm(max(T - 1, 1), generator=gen, device="cuda")[: case["runs"] - 1]).values + 1
        run_of = torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)
        owner = torch.randint(0, G, (case["runs"],), generator=gen, device="cuda")
        if case["runs"] > 1:
            owner = torch.where(_rand(gen, case["runs"]) < 0.125, torch.full_like(owner, -1), owner)
        st["ids"] = owner[run_of].to(torch.int32)
        st["x_in"] = _randn(gen, DTYPES[case["x"]], T, K)
        st["most"] = int(torch.bincount(st["ids"].long() + 1, minlength=G + 1).max())
    else:
        Q, D, V = case["requests"], case["drafts"], case["vocab"]
        logits = 3.0 * torch.randn(Q, D + 1, V, generator=gen, device="cuda")
        st["logits"] = logits.to(DTYPES[case["logits"]])
        near = torch.softmax(logits[:, :D] + 0.5 * torch.randn(Q, D, V, generator=gen, device="cuda"), dim=-1)
        if case["probs"]:
            st["q"] = near
            pick = torch.searchsorted(near.double().cumsum(-1), 0.999999 * _rand(gen, Q, D, 1).double()).squeeze(-1)
        else:
            st["q"] = None
            pick = logits[:, :D].argmax(dim=-1)
        st["drafted"] = pick.clamp_(0, V - 1).to(torch.int32)
        n = torch.randint(0, D + 1, (Q,), generator=gen, device="cuda") if case["ragged"] else torch.full((Q,), D, device="cuda")
        st["n_draft"] = n.to(torch.int32)
        # lookups are accepted often enough to matter when their random numbers are those of a confident target
        st["u"] = _rand(gen, Q, D) * (1.0 if case["probs"] else 0.1)
        st["u_last"] = _rand(gen, Q)
    return st


# ---------------------------------------------------------------- plain forms
def _values(fmt, raw, rows, cols):
    """float32 [rows, cols] of stored bytes."""
    if fmt == "q8_0":
        b = raw.view(rows, cols // 32, 34)
        return (b[..., :2].contiguous().view(torch.float16).float() * b[..., 2:].contiguous().view(torch.int8)).view(rows, cols)
    if fmt in ("q4_0", "q4_1"):
        b = raw.view(rows, cols // 32, ROW_BYTES[fmt][1])
        d = b[..., :2].contiguous().view(torch.float16).float()
        qs = b[..., -16:]
        c = torch.cat([qs & 15, qs >> 4], dim=-1).float()
        v = d * (c - 8.0) if fmt == "q4_0" else d * c + b[..., 2:4].contiguous().view(torch.float16).float()
        return v.view(rows, cols)
    b = raw.view(rows, cols // 256, ROW_BYTES[fmt][1])
    if fmt == "q4_k":
        d, dmin = b[..., 0:2].contiguous().view(torch.float16).float(), b[..., 2:4].contiguous().view(torch.float16).float()
        x, y, z = b[..., 4:8], b[..., 8:12], b[..., 12:16]
        sc = torch.cat([x & 63, (z & 15) | ((x >> 6) << 4)], dim=-1).float()
        mn = torch.cat([y & 63, (z >> 4) | ((y >> 6) << 4)], dim=-1).float()
        q = b[..., 16:].reshape(rows, cols // 256, 4, 1, 32)
        c = torch.cat([q & 15, q >> 4], dim=3).reshape(rows, cols // 256, 8, 32).float()
        return ((d * sc).unsqueeze(-1) * c - (dmin * mn).unsqueeze(-1)).view(rows, cols)
    ql, qh = b[..., :128].reshape(rows, -1, 2, 1, 64), b[..., 128:192].reshape(rows, -1, 2, 1, 32)
    low = torch.cat([ql & 15, ql >> 4], dim=3).view(rows, -1, 2, 4, 32)
    high = torch.cat([qh & 3, (qh >> 2) & 3, (qh >> 4) & 3, qh >> 6], dim=3)
    c = ((low | (high << 4)).float() - 32.0).view(rows, -1, 16, 16)
    sc = b[..., 192:208].contiguous().view(torch.int8).float() * b[..., 208:].contiguous().view(torch.float16).float()
    return (c * sc.unsqueeze(-1)).view(rows, cols)


def _places(ids, groups, most):
    """Each item's place in a padded [groups, most] batch, by group, in order."""
    flat = ids.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    of = flat[order]
    begin = torch.searchsorted(of, torch.arange(groups, device=of.device))
    return order, of, torch.arange(of.numel(), device=of.device) - begin[of]


def _padded(rows, of, at, groups, most):
    out = torch.zeros(groups, most, rows.shape[1], device=rows.device)
    out[of, at] = rows
    return out


def _experts_plain(st):
    E, F, H, T, S = st["experts"], st["ff"], st["hidden"], st["tokens"], st["top_k"]
    order, of, at = _places(st["ids"], E, st["most"])
    block = st["form"] == "block"
    w1 = _values(st["fmt"], st["W1"], E * (2 * F if block else F), H).view(E, -1, H)
    a = torch.bmm(_padded(st["x_in"].float()[order // S], of, at, E, st["most"]), w1.transpose(1, 2))
    y = torch.empty(T * S, F if not block else H, device=a.device)
    if not block:
        y[order] = a[of, at]
        return y.view(T, S, F)
    g, u = a[..., :F], a[..., F:]
    h = (g / (1.0 + torch.exp(-g)) * u).to(st["x_in"].dtype).float()   # the activations' type between the two products
    w2 = _values(st["fmt"], st["W2"], E * H, F).view(E, H, F)
    y[order] = torch.bmm(h, w2.transpose(1, 2))[of, at]
    return (y.view(T, S, H) * st["weights"].unsqueeze(-1)).sum(1).to(st["x_in"].dtype)


def _lora_plain(st):
    x = st["x_in"].float()
    y = x @ _values(st["fmt"], st["W"], st["rows"], st["cols"]).t()
    order, of, at = _places(st["ids"] + 1, st["adapters"] + 1, st["most"])
    zero = torch.zeros(1, 1, 1, device=x.device)
    A = torch.cat([zero.expand(1, *st["A"].shape[1:]), st["A"].float()])   # adapter 0: none
    B = torch.cat([zero.expand(1, *st["B"].shape[1:]), st["B"].float()])
    s = torch.cat([zero.view(1), st["scales"]]).view(-1, 1, 1)
    v = torch.bmm(_padded(x[order], of, at, st["adapters"] + 1, st["most"]), A.transpose(1, 2)) * s
    return y.index_add_(0, order, torch.bmm(v, B.transpose(1, 2))[of, at])


def _verify_plain(st):
    Q, D, V = st["requests"], st["drafts"], st["vocab"]
    l = st["logits"].double()   # the choices are comparisons: 64 bits
    e = torch.exp(l - l.amax(-1, keepdim=True))
    p = e / e.sum(-1, keepdim=True)
    x = st["drafted"].long().unsqueeze(-1)
    px = p[:, :D].gather(-1, x).squeeze(-1)
    qx = st["q"].gather(-1, x).squeeze(-1).double() if st["q"] is not None else torch.ones_like(px)
    place = torch.arange(D, device=l.device)
    n = st["n_draft"].long().unsqueeze(1)
    ok = (st["u"].double() * qx < px) & (place < n)
    kept = ok.long().cumprod(1).sum(1)
    at = kept.view(Q, 1, 1).expand(Q, 1, V)
    r = p.gather(1, at).squeeze(1)
    stopped = (kept < n.squeeze(1)).unsqueeze(1)
    last = kept.clamp(max=D - 1)
    if st["q"] is not None:
        taken = st["q"].gather(1, last.view(Q, 1, 1).expand(Q, 1, V)).squeeze(1).double()
    else:
        taken = torch.zeros_like(r).scatter_(1, x.squeeze(-1).gather(1, last.unsqueeze(1)), 1.0)
    left = torch.where(stopped, (r - taken).clamp_min(0.0), r)
    r = torch.where(left.sum(1, keepdim=True) > 0, left, r)
    c = r.cumsum(1)
    token = (c <= st["u_last"].double().unsqueeze(1) * c[:, -1:]).sum(1).clamp(max=V - 1)
    place = torch.arange(D + 1, device=l.device)
    padded = torch.cat([st["drafted"].long(), torch.zeros(Q, 1, dtype=torch.long, device=l.device)], dim=1)
    k = kept.unsqueeze(1)
    out = torch.where(place < k, padded, torch.where(place == k, token.unsqueeze(1), torch.full_like(padded, -1)))
    return out.to(torch.int32), kept.to(torch.int32)


# ---------------------------------------------------------------- the library's calls
def _experts_own(st):
    import bandwidth_bound_block_amd as qmv
    E, F, H, T, S, fmt = st["experts"], st["ff"], st["hidden"], st["tokens"], st["top_k"], st["fmt"]
    plan = qmv.qmv_group_plan(st["ids"], E)
    if st["form"] == "product":
        return qmv.qmv_moe_grouped(fmt, st["W1"], F * qmv.row_bytes(fmt, H), E, F, H, plan, S, st["x_in"])
    h = qmv.qmv_moe_grouped_swiglu(fmt, st["W1"], 2 * F * qmv.row_bytes(fmt, H), E, F, H, plan, S, st["x_in"],
                                   h_dtype=st["x_in"].dtype)
    y = qmv.qmv_moe_grouped(fmt, st["W2"], H * qmv.row_bytes(fmt, F), E, H, F, plan, S, h)
    return qmv.qmv_moe_weighted_sum(y, st["weights"], out_dtype=st["x_in"].dtype)


def _lora_own(st):
    import bandwidth_bound_block_amd as qmv
    return qmv.qmv_lora(st["fmt"], st["W"], st["rows"], st["cols"], st["x_in"], st["A"], st["B"], st["scales"], st["ids"])


def _verify_own(st):
    import bandwidth_bound_block_amd as qmv
    return qmv.qmv_spec_verify(st["logits"], st["q"], st["drafted"], st["n_draft"], st["u"], st["u_last"])


def run(state):
    op = state["op"]
    if own:
        return _experts_own(state) if op == "experts" else _lora_own(state) if op == "lora" else _verify_own(state)
    return _experts_plain(state) if op == "experts" else _lora_plain(state) if op == "lora" else _verify_plain(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2}
    if case["op"] == "experts":
        E, F, H, T, S = case["experts"], case["ff"], case["hidden"], case["tokens"], case["top_k"]
        unit, nbytes = ROW_BYTES[case["fmt"]]
        touched = E * (1.0 - (1.0 - S / E) ** T) if S < E else E    # experts that some token takes, choices even
        weights = (3 if case["form"] == "block" else 1) * F * H
        written = T * H * size[case["x"]] if case["form"] == "block" else T * S * F * 4
        return {"bytes": touched * weights * nbytes / unit + T * H * size[case["x"]] + written + 8.0 * T * S,
                "flops": 2.0 * T * S * weights}
    if case["op"] == "lora":
        T, N, K, R = case["tokens"], case["rows"], case["cols"], case["rank"]
        unit, nbytes = ROW_BYTES[case["fmt"]]
        G = case["adapters"] * (1.0 - (1.0 - 1.0 / case["adapters"]) ** case["runs"])
        return {"bytes": N * K * nbytes / unit + G * R * (N + K) * size[case["a"]] + T * K * size[case["x"]] + T * N * 4.0,
                "flops": 2.0 * T * (N * K + R * (N + K))}
    Q, D, V = case["requests"], case["drafts"], case["vocab"]
    rows = Q * ((D / 2.0 if case["ragged"] else D) + 1)
    return {"bytes": rows * V * size[case["logits"]] + (Q * V * 4.0 if case["probs"] else 0.0), "flops": 4.0 * rows * V}


# ---------------------------------------------------------------- the same in 64 bits
def _weights64(fmt, raw, n, k):
    """float64 [n, k], bit fields taken from whole numbers."""
    def num(v):
        return v.contiguous().view(torch.float16).to(torch.float64).squeeze(-1)
    unit, nbytes = ROW_BYTES[fmt]
    b = raw.reshape(n * (k // unit), nbytes)
    w = torch.empty(b.shape[0], unit, dtype=torch.float64, device=raw.device)
    d = num(b[:, 208:210] if fmt == "q6_k" else b[:, 0:2])[:, None]
    i = b.to(torch.int32)
    if fmt == "q8_0":
        w[:] = d * ((i[:, 2:] + 128) % 256 - 128)
    elif fmt == "q4_0":
        w[:, :16], w[:, 16:] = d * (i[:, 2:] % 16 - 8), d * (i[:, 2:] // 16 - 8)
    elif fmt == "q4_1":
        m = num(b[:, 2:4])[:, None]
        w[:, :16], w[:, 16:] = d * (i[:, 4:] % 16) + m, d * (i[:, 4:] // 16) + m
    elif fmt == "q4_k":
        m = num(b[:, 2:4])[:, None]
        for s in range(8):
            if s < 4:
                sc, mn = i[:, 4 + s] % 64, i[:, 8 + s] % 64
            else:
                sc, mn = i[:, 8 + s] % 16 + 16 * (i[:, s] // 64), i[:, 8 + s] // 16 + 16 * (i[:, 4 + s] // 64)
            q = i[:, 16 + 32 * (s // 2):48 + 32 * (s // 2)]
            c = q // 16 if s % 2 else q % 16
            w[:, 32 * s:32 * s + 32] = d * sc[:, None] * c - m * mn[:, None]
    else:
        for j in range(8):
            h, q = j // 4, j % 4
            lo = i[:, 64 * h + 32 * (q % 2):64 * h + 32 * (q % 2) + 32]
            lo = lo // 16 if q >= 2 else lo % 16
            hi = (i[:, 128 + 32 * h:160 + 32 * h] // 4 ** q) % 4
            sc = ((i[:, 192 + 2 * j:194 + 2 * j] + 128) % 256 - 128).repeat_interleave(16, dim=1)
            w[:, 32 * j:32 * j + 32] = d * sc * (lo + 16 * hi - 32)
    return w.view(n, k)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "experts":
        E, F, H, T, S = case["experts"], case["ff"], case["hidden"], case["tokens"], case["top_k"]
        block = case["form"] == "block"
        x, ids = st["x_in"].double(), st["ids"].long()
        out = torch.zeros((T, H) if block else (T, S, F), dtype=torch.float64, device=x.device)
        raw1 = st["W1"].view(E, -1)
        for e in range(E):
            t, s = torch.nonzero(ids == e, as_tuple=True)
            if t.numel() == 0:
                continue
            a = x[t] @ _weights64(case["fmt"], raw1[e], 2 * F if block else F, H).t()
            if not block:
                out[t, s] = a
                continue
            h = a[:, :F] * torch.sigmoid(a[:, :F]) * a[:, F:]
            y = h @ _weights64(case["fmt"], st["W2"].view(E, -1)[e], H, F).t()
            out.index_add_(0, t, y * st["weights"].double()[t, s][:, None])
        return out
    if case["op"] == "lora":
        x = st["x_in"].double()
        y = x @ _weights64(case["fmt"], st["W"], case["rows"], case["cols"]).t()
        for g in range(case["adapters"]):
            t = torch.nonzero(st["ids"] == g).squeeze(1)
            if t.numel():
                y[t] += float(st["scales"][g]) * ((x[t] @ st["A"][g].double().t()) @ st["B"][g].double().t())
        return y
    return None   # whole numbers: they have to be equal
