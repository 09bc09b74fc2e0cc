"""The definition of the truncated distribution, the draw and sampled
verification in float64 numpy, for the tests of the sampling operators."""

import numpy as np


def order_of(z):
    """Token ids above -inf, by logit descending, equal logits by smaller id."""
    z = np.where(np.isnan(z), -np.inf, z)
    o = np.lexsort((np.arange(len(z)), -z))
    return o[z[o] > -np.inf]


def masses(z, t=1.0, k=0, p=1.0, m=0.0):
    """[V] float64 masses of the kept tokens (0 elsewhere)."""
    z = np.asarray(z, np.float64)
    out = np.zeros(len(z))
    o = order_of(z)
    if len(o) == 0:
        return out
    if not t > 0:
        out[o[0]] = 1.0
        return out
    if k > 0:
        o = o[:k]
    top = z[o[0]]
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.where(z[o] == top, 1.0, np.exp((z[o] - top) / t))
    if p < 1:
        c = np.cumsum(e)
        n = max(1, int(np.searchsorted(c, p * c[-1], side="left")) + 1)
        o, e = o[:n], e[:n]
    if m > 0:
        stay = e >= min(m, 1.0)
        o, e = o[stay], e[stay]
    out[o] = e
    return out


def draw(mass, u):
    c = np.cumsum(mass)
    if c[-1] == 0:
        return -1
    u = min(max(float(u), 0.0), float(np.float32(0.99999994)))
    return int(np.searchsorted(c, u * c[-1], side="right"))


def verify(z, path, n, settings, u_accept, u):
    """One sequence: (accepted, emitted token)."""
    for i in range(n + 1):
        w = masses(z[i], *settings)
        if i == n:
            return n, draw(w, u)
        x = int(path[i])
        px = w[x] if 0 <= x < len(w) else 0.0
        if not float(u_accept[i]) * w.sum() < px:
            if 0 <= x < len(w):
                w[x] = 0.0
            return i, draw(w, u)
