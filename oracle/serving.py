"""The operators around the cache in 64 bits (oracle): rotary positions, causal
attention over one prompt, attention of a drafted tree, and the walk that verifies
one.  Plain definitions, one sequence at a time, sharing nothing with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np


def rope_freqs(rot: int, base: float, scaling: str = "none", factor: float = 1.0,
               length: float = 0.0, low: float = 1.0, high: float = 4.0, fast: float = 32.0,
               slow: float = 1.0):
    """(radians per position of each pair [rot/2], magnitude of cos and sin)."""
    out, mag = [], 1.0
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "banded":
            turns = length * f / (2 * math.pi)
            w = min(1.0, max(0.0, (turns - low) / (high - low)))
            f = w * f + (1 - w) * f / factor
        elif scaling == "yarn":
            e = lambda n: rot * math.log(length / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
            lo, hi = max(math.floor(e(fast)), 0), min(math.ceil(e(slow)), rot - 1)
            w = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
            f = (1 - w) * f + w * f / factor
        out.append(f)
    if scaling == "yarn" and factor > 1:
        mag = 0.1 * math.log(factor) + 1.0
    return np.array(out), mag


def rope(x, pos, freqs, mag: float, layout: str) -> np.ndarray:
    """x [n, H, d] turned to positions pos [n] -> fp64."""
    y = np.asarray(x).astype(np.float64).copy()
    r = 2 * len(freqs)
    ang = np.asarray(pos, dtype=np.float64)[:, None] * freqs
    c, s = mag * np.cos(ang)[:, None], mag * np.sin(ang)[:, None]
    ia = np.arange(r // 2) if layout == "half" else np.arange(0, r, 2)
    ib = ia + (r // 2 if layout == "half" else 1)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def attention(q, k, v, see, scale: float | None = None, rounded=None):
    """q [n, Hq, d], k and v [T, Hkv, d], see [n, T] truth -> (o [n, Hq, d], bound).

    `bound` is how far a kernel may be that rounds each probability (times its value
    row's scale) and the output to fp16 once (2^-11 each) and works in fp32 otherwise:
    with A = sum p max(|v|, w), w [T, Hkv, 1] = `rounded` the size of what multiplies
    the rounded probability where that is not v itself (a zero point is added apart:
    v = code * scale + z), and delta the error of a logit, d + 8 roundings of 2^-24 of
    sigma sum |q_c k_c|, plus 2^-22 of the logit for its scaling and the exponential,
      2^-11 (A + |o|) + (2 delta + 2^-20 + T 2^-23) (A + |o|) + 2^-24.
    A row that sees nothing gives 0."""
    q, k, v = (np.asarray(x).astype(np.float64) for x in (q, k, v))
    n, Hq, d = q.shape
    G = Hq // k.shape[1]
    sigma = 1.0 / math.sqrt(d) if not scale else float(scale)
    o, bound = np.zeros((n, Hq, d)), np.full((n, Hq, d), 2.0 ** -24)
    for h in range(Hq):
        kh, vh = k[:, h // G], v[:, h // G]
        x = sigma * (q[:, h] @ kh.T)
        big = sigma * (np.abs(q[:, h]) @ np.abs(kh).T)
        for i in range(n):
            j = np.nonzero(see[i])[0]
            if len(j) == 0:
                continue
            p = np.exp(x[i, j] - x[i, j].max())
            p /= p.sum()
            o[i, h] = p @ vh[j]
            size = np.abs(vh[j]) if rounded is None else np.maximum(np.abs(vh[j]),
                                                                    rounded[j, h // G])
            a = p @ size + np.abs(o[i, h])
            delta = (d + 8) * 2.0 ** -24 * big[i, j].max() + 2.0 ** -22 * np.abs(x[i, j]).max()
            bound[i, h] += (2.0 ** -11 + 2 * delta + 2.0 ** -20 + len(j) * 2.0 ** -23) * a
    return o, bound


def causal(n: int) -> np.ndarray:
    return np.tril(np.ones((n, n), dtype=bool))


def tree_sees(parents, n: int, cached: int) -> np.ndarray:
    """[n, cached + n] truth: node i sees every cached token, itself and its ancestors."""
    see = np.zeros((n, cached + n), dtype=bool)
    see[:, :cached] = True
    for i in range(n):
        a = i
        while a >= 0:
            see[i, cached + a] = True
            p = int(parents[a])
            a = p if 0 <= p < a else -1
    return see


def verify(p, q, tokens, parents, u, us, n: int):
    """One tree: p [m, V], q [m, V] or None -> (path list, next token)."""
    V = p.shape[1]
    if n <= 0:
        return [], -1
    node, path = 0, []
    while True:
        r, z, hit = p[node].astype(np.float64), 1.0, False
        for c in range(1, n):
            if parents[c] != node or not 0 <= tokens[c] < V:
                continue
            x = int(tokens[c])
            qx = 1.0 if q is None else float(q[node, x])
            if float(u[c]) * qx * z < r[x]:
                path.append(c)
                node, hit = c, True
                break
            if q is None:
                z -= r[x]
                r[x] = 0.0
            else:
                r = np.maximum(r - z * q[node].astype(np.float64), 0.0)
                z = r.sum()
        if not hit:
            break
    if r.sum() <= 0:
        r = p[node].astype(np.float64)
    cum = np.cumsum(r)
    return path, min(V - 1, int(np.searchsorted(cum, float(us) * cum[-1], side="right")))
