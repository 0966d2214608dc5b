"""Plain 64-bit values of the quantized cache, its attention and the log
probabilities, with the error bounds their tests hold outputs to.

A rounding to a type is off by at most half a step, eps / 2 relative to the
value: 2^-24 in fp32, 2^-11 in fp16, 2^-8 in bf16.
"""
import numpy as np

U, H16 = 2.0 ** -24, 2.0 ** -11
HALF = {"f32": U, "f16": H16, "bf16": 2.0 ** -8}
LIMIT = 65024.0
ROW = {"q8_0": 34, "q4_0": 18, "q4_1": 20}


def away(v):
    return np.sign(v) * np.floor(np.abs(v) + 0.5)


def half(v):
    """fp64 -> fp32 -> fp16, as the scales are rounded; zeros are +0."""
    with np.errstate(over="ignore"):
        return np.asarray(v, np.float64).astype(np.float32).astype(np.float16) + np.float16(0)


def encode(x, fmt):
    """x float64 [..., D] -> codes [..., D] (signed for q8_0, else 0..15), d and m fp16 [..., D / 32] (m None but for q4_1).
    Blocks with values that are not finite get d = NaN."""
    fin = np.isfinite(x).reshape(*x.shape[:-1], x.shape[-1] // 32, 32).all(-1)
    w = np.clip(np.nan_to_num(x, nan=0.0, posinf=LIMIT, neginf=-LIMIT), -LIMIT, LIMIT).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    m = None
    if fmt == "q8_0":
        d = half(np.abs(w).max(-1) / 127.0)
    elif fmt == "q4_0":
        at = np.abs(w).argmax(-1)[..., None]
        d = half(np.take_along_axis(w, at, -1)[..., 0] / -8.0)
    else:
        m = half(w.min(-1))
        d = half((w.max(-1) - w.min(-1)) / 15.0)
    dd = d.astype(np.float64)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        if fmt == "q8_0":
            c = np.where(dd != 0, np.clip(away(w / dd), -127, 127), 0)
        elif fmt == "q4_0":
            c = np.where(dd != 0, np.clip(away(w / dd) + 8, 0, 15), 8)
        else:
            c = np.where(dd != 0, np.clip(away((w - m.astype(np.float64)[..., None]) / dd), 0, 15), 0)
    d = np.where(fin, d, np.float16(np.nan))
    return c.reshape(x.shape).astype(np.int64), d, m


def decode(c, d, m, fmt):
    """float64 [..., D]."""
    v = c.reshape(*c.shape[:-1], c.shape[-1] // 32, 32) - (8 if fmt == "q4_0" else 0)
    v = v * d.astype(np.float64)[..., None]
    if m is not None:
        v = v + m.astype(np.float64)[..., None]
    return v.reshape(c.shape)


def place(D):
    """Octet's place in a stored row, by octet."""
    o = np.arange(D // 8)
    return (o % 4) * (D // 32) + o // 4


def empty_pages(fmt, n, heads, D, P, fill=0xA5):
    return np.full((n, heads, P * (D // 32) * ROW[fmt]), fill, dtype=np.uint8)


def put(pages, fmt, D, P, page, off, h, c, d, m):
    """Stores one token's head: codes [D], d, m [D / 32]."""
    nb, row = D // 32, D if fmt == "q8_0" else D // 2
    oct_ = np.zeros((D // 8, 8), np.int64)
    oct_[place(D)] = c.reshape(-1, 8)
    if fmt == "q8_0":
        b = oct_.astype(np.int8).view(np.uint8).reshape(-1)
    else:
        word = np.zeros(D // 8, np.uint32)
        for i in range(8):
            word |= oct_[:, i].astype(np.uint32) << np.uint32(4 * (i // 2) + 16 * (i % 2))
        b = word.view(np.uint8)
    head = pages[page, h]
    head[off * row:(off + 1) * row] = b
    for j, s in enumerate([d] if m is None else [d, m]):
        plane = head[P * row + 2 * j * nb * P:][:2 * nb * P].view(np.float16).reshape(nb, P)
        plane[:, off] = s


def filled(rng, fmt, n, heads, D, P, std=1.0):
    """Pages full of N(0, std^2) values -> (uint8 pages, float64 values [n, heads, P, D])."""
    x = rng.standard_normal((n, heads, P, D)).astype(np.float32).astype(np.float64) * std
    c, d, m = encode(x, fmt)
    pages = empty_pages(fmt, n, heads, D, P)
    for i in range(n):
        for h in range(heads):
            for o in range(P):
                put(pages, fmt, D, P, i, o, h, c[i, h, o], d[i, h, o], None if m is None else m[i, h, o])
    return pages, decode(c, d, m, fmt)


def spread(v, fmt):
    """Sizes of the terms that a stored value is the sum of, at most: |d c| + |m| for q4_1."""
    if fmt != "q4_1":
        return np.abs(v)
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    return np.broadcast_to(3 * np.abs(b).max(-1, keepdims=True), b.shape).reshape(v.shape)


def attention(q, k, v, scale, pos, window, sink, x, few, k_fmt="q8_0"):
    """One request, one key/value head.  q [rows, D] float64, k, v [L, D], pos [rows], sink [rows] or None.
    Returns (out, bound): x the query type, few whether DEQ(K) is used as codes (else rounded to fp16)."""
    L, D = k.shape
    j = np.arange(L)
    seen = j <= pos[:, None]
    if window:
        seen &= j > pos[:, None] - window
    s = scale * (q @ k.T)
    size = scale * (np.abs(q) @ spread(k, k_fmt).T)
    with np.errstate(invalid="ignore"):
        top = np.where(seen, s, -np.inf).max(1, initial=-np.inf)
    if sink is not None:
        top = np.maximum(top, sink)
    top = np.where(np.isfinite(top), top, 0.0)
    p = np.where(seen, np.exp(np.where(seen, s, 0.0) - top[:, None]), 0.0)
    total = p.sum(1)
    if sink is not None:
        total = total + np.exp(sink - top)
    w = p / np.where(total > 0, total, 1.0)[:, None]
    out = w @ v
    # a score: products exact, up to 2 D + 64 roundings of partial sums and scales in fp32 (the queries' pieces: two of 2^-22
    # more); keys as fp16 values one of 2^-11 each; its multiple of log 2 and the difference to the maximum two more, and e^x 2^-22
    two = x != "bf16"
    es = (2 * D + 64 + (16 if two else 0)) * U * size + (0 if few or two else H16 * size) + (0 if few or not two else 8 * U * size)
    es = np.where(seen, es, 0.0)
    es = es + 4 * U * np.where(seen, np.abs(s), 0.0) + 4 * U * np.abs(top)[:, None] + 8 * U
    # weights and values: one fp16 rounding each (22 bits in two pieces), fp16's smallest step beside a weight of 1; sums of L
    ew = 8 * U if two else H16
    smallest = 2.0 ** -24 if not two else 2.0 ** -25 * 2 ** -10
    rel = 2 * es + 2 * ew + (L + 128) * U
    bound = (w * rel) @ np.abs(v) + (w @ np.abs(v)) * (w * es).sum(1, keepdims=True) * 2
    bound = bound + (seen * smallest) @ np.abs(v) / np.maximum(total, 1e-30)[:, None] + L * 2.0 ** -25 * (0 if two else 1) * w.max(1, initial=0)[:, None]
    bound = bound * 1.01 + HALF[x] * (np.abs(out) + bound) + (2.0 ** -25 if x == "f16" else 0) + 2.0 ** -120
    return out, bound


def logprobs(l):
    """One row, float64: (log p, entropy, bound of log p, bound of the entropy)."""
    m = l.max()
    z = l - m
    e = np.exp(z)
    first = int(np.argmax(z))
    rest = np.delete(e, first).sum()
    lt = np.log1p(rest)
    with np.errstate(invalid="ignore"):
        ez = np.where(e > 0, e * -z, 0.0)
        zs = np.where(np.isfinite(z), np.abs(z), 0.0)
    a = ez.sum()
    p, H = z - lt, lt + a / (1 + rest)
    # a term: z's rounding is an error of the exponent, e^z 2^-22 more (twice where chunks meet); sums round some 64 times
    et = ((np.delete(e, first) * (np.delete(zs, first) * 2 + 8 + 64)).sum()) * U
    ea = (ez * (zs * 2 + 8 + 64 + 2)).sum() * U + (e * zs).sum() * 2 * U
    bl = et / (1 + rest) + 8 * U * lt
    bp = bl + 2 * U * (zs + lt) + 2.0 ** -126
    bh = bl + (ea + a * et / (1 + rest)) / (1 + rest) + 4 * U * H + 2.0 ** -126
    return p, H, bp * 1.01, bh * 1.01
