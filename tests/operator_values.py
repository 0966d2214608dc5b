"""Plain 64-bit values of the grouped products, the adapters and the
verification, with the error bounds their tests hold outputs to.

A rounding to a type is off by at most half a step, eps / 2 relative to the
value; U = 2^-24 is fp32's.
"""
import numpy as np

import oracle

U = 2.0 ** -24
HALF = {"f32": U, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def as_type(torch, a, name):
    """float64 numpy -> a CPU tensor of the type, and its exact float64 values."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(
        {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name])
    return t, t.to(torch.float64).numpy()


def rounded(y, name):
    """Bound of rounding y to a type once (fp16's smallest step included)."""
    return HALF[name] * np.abs(y) + (2.0 ** -25 if name == "f16" else 2.0 ** -134)


def product(fmt, raw, N, K, x):
    """y = DEQ(W) x for rows of x, and the bound of its fp32 evaluation: a
    block's 32 products and their sum, its scale, and the sum over blocks
    round at most 40 + K / 32 times; where a format carries codes about a
    pivot, its two terms are at most 3 |w x| together."""
    w = oracle.dequant(fmt, raw, N, K).astype(np.float64).reshape(N, K)
    y = x @ w.T
    S = np.abs(x) @ np.abs(w).T
    return y, 3 * (K // 32 + 40) * U * S + 2.0 ** -120


def silu(g):
    return g / (1.0 + np.exp(-g))


def swiglu(g, eg, u, eu):
    """SiLU(g) u and its bound: |SiLU'| < 1.1; e^-g is off by about |g| + 2
    roundings, the sum, quotient and product by three more."""
    h = silu(g) * u
    return h, 1.1 * eg * np.abs(u) + np.abs(silu(g)) * eu + 1.1 * eg * eu + (np.abs(g) + 8) * U * np.abs(h) + 2.0 ** -120


def adapters(x, A, B, scales, ids):
    """s B (A x) per token and the bound of its fp32 evaluation."""
    T, K = x.shape
    N, R = B.shape[1:]
    y, e = np.zeros((T, N)), np.zeros((T, N))
    for t in range(T):
        a = ids[t]
        if 0 <= a < A.shape[0]:
            s = abs(float(scales[a]))
            v, V = A[a] @ x[t], np.abs(A[a]) @ np.abs(x[t])
            y[t] = float(scales[a]) * (B[a] @ v)
            e[t] = s * (np.abs(B[a]) @ ((K + R + 4) * U * V))
    return y, e


def verify(l, q, x, n, u, u_last):
    """Kept tokens and the token drawn for one request from float64 logits
    [D + 1][V], and the smallest distance of a comparison from its border
    (relative to the row's mass)."""
    margin = np.inf
    V = l.shape[1]

    def softmax(row):
        if not np.any(row > -np.inf) or np.any(np.isnan(row)) or np.any(row == np.inf):
            return None
        e = np.exp(row - row.max())
        return e / e.sum()
    i, p = 0, None
    for i in range(n + 1):
        p = softmax(l[i])
        if i == n or p is None:
            break
        if not 0 <= x[i] < V:
            break
        qx = q[i, x[i]] if q is not None else 1.0
        margin = min(margin, abs(u[i] * qx - p[x[i]]))
        if not u[i] * qx < p[x[i]]:
            break
    if p is None:
        return i, -1, margin
    r = p
    if i < n:
        t = np.zeros(V)
        if q is not None:
            t = q[i].astype(np.float64)
        elif 0 <= x[i] < V:
            t[x[i]] = 1.0
        r = np.maximum(p - t, 0.0)
        if not r.sum() > 0:
            r = p
    c = np.cumsum(r)
    goal = u_last * c[-1]
    at = int(np.argmax(c > goal)) if np.any(c > goal) else int(np.nonzero(r)[0][-1])
    margin = min(margin, np.abs(c - goal)[r > 0].min() if goal > 0 else np.inf)
    return i, at, margin
