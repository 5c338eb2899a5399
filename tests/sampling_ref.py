"""Sampling and verification by their definition, in 64 bits on the CPU (numpy), one row at a time.

Each function also says how near its decisions are to a border, as shares of the mass: `near` is the smallest distance
of a sum from what it was held against. Weights of the kernels are good to 4e-14 and are rounded to 2^-45 at n = 2^17
(2^-38 at 2^24), so sums differ by less than n 2^-45 + 1e-13 of a mass that is at least 1: decisions further than BORDER
from their border are the same.
"""
import numpy as np

BORDER = 1e-8     # n 2^-(62 - ceil log2 n) is 4e-9 at n = 2^17


def tame(x):
    x = np.asarray(x, np.float64).copy()
    x[np.isnan(x)] = -np.inf
    x[x == np.inf] = float(np.finfo(np.float32).max)
    return x


def weights(x, T=1.0, k=0, p=1.0, m=0.0):
    """(weights over the columns, 0 of what the settings leave out; near). x: one row, float64 of the logits' own values."""
    x = tame(x)
    n = len(x)
    T, p, m = (float(np.float32(v)) for v in (T, p, m))
    live = x > -np.inf
    w = np.zeros(n)
    if not live.any():
        return w, 1.0
    if not T > 0:
        T, k = 1.0, 1
    if k <= 0 or k > n:
        k = n
    hi = x.max()
    with np.errstate(over="ignore", invalid="ignore"):
        d = np.where(live, (x - hi) / T if np.isfinite(T) else 0.0, -np.inf)
    order = np.argsort(-x, kind="stable")[:int(live.sum())][:k]
    e = np.exp(np.maximum(d[order], -1e4))
    near = 1.0
    keep = len(order)
    if p < 1:
        mass = e.sum()
        before = np.concatenate([[0.0], np.cumsum(e)[:-1]])
        ok = before < max(p, 0.0) * mass
        ok[0] = True
        keep = int(ok.sum())
        if keep > 1 or p > 0:
            near = min(near, float(np.abs(before[1:] - p * mass).min(initial=1.0) / mass))
    if m > 0:
        m = min(m, 1.0)
        keep = min(keep, int((d[order] >= np.log(m)).sum()))
        gap = np.abs(d[order] - np.log(m))
        near = min(near, float(gap[gap != 0].min(initial=1.0)))
    w[order[:keep]] = e[:keep]
    return w, near


def draw(w, u):
    """(column, near) of u in the weights; column -1 without any."""
    c = np.cumsum(w)
    total = c[-1]
    if not total > 0:
        return -1, 1.0
    u = float(u)
    u = 0.0 if np.isnan(u) else min(max(u, 0.0), 1.0)
    at = int(np.searchsorted(c, u * total, side="right"))
    last = int(np.flatnonzero(w > 0)[-1])
    edges = c[w > 0][:-1]    # borders between columns that can be drawn
    near = float(np.abs(edges / total - u).min(initial=1.0))
    return min(at, last), near


def verify(x, token, ids, probs, u, settings):
    """(tokens, near) of one sequence: x [s+1, n], token [s], ids / probs [s, k] or None, u [s+1]."""
    s, n = len(token), x.shape[1]
    near, out = 1.0, []
    for j in range(s + 1):
        w, c = weights(x[j], **settings)
        near = min(near, c)
        total = w.sum()
        p = w / total if total > 0 else w
        if j < s:
            q = np.zeros(n)
            if ids is None:
                if 0 <= token[j] < n:
                    q[token[j]] = 1.0
                qt = 1.0
            else:
                for i, v in zip(ids[j], probs[j]):
                    v = 0.0 if not v > 0 else float(v)
                    if 0 <= i < n:
                        q[i] += v
                qt = sum(float(v) for i, v in zip(ids[j], probs[j]) if i == token[j] and v > 0)
            pt = p[token[j]] if 0 <= token[j] < n else 0.0
            if not (pt == 0.0 or qt == 0.0):
                near = min(near, abs(float(u[j]) * qt - pt))
            if float(u[j]) * qt < pt:
                out.append(int(token[j]))
                continue
            rest = np.maximum(p - q, 0.0)
            if rest.sum() > 0:
                near = min(near, float(rest.sum()))     # a rest of roundings alone says nothing
                p = rest
        at, c = draw(p, u[s])
        near = min(near, c)
        if at >= 0:
            out.append(at)
        break
    return out, near
