"""Plain 64-bit forms of the paged-cache operators, the attention over a paged cache and the changes to logits, for
their tests.  Row by row, from the definitions in include/dflash2.h."""

import numpy as np


def bf16(x):
    """float64 values rounded to bfloat16 (nearest, ties to even), as float64; NaN and infinities stay."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126))), -126) - 7)
        return np.where(np.isfinite(x), np.rint(x / step) * step, x)


def e4m3_values():
    """The 256 codes' values (float64; NaN for 0x7f and 0xff)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    mag = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    mag = np.where((c & 127) == 127, np.nan, mag)
    return np.where(c >= 128, -mag, mag)


def quantise_row(x):
    """(codes, exponent byte) of one head's row, by looking at every byte and every code."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x)
    top = np.abs(x[fine]).max() if fine.any() else 0.0
    b = next(b for b in range(1, 256) if top <= 448 * 2.0 ** (b - 127))
    grid = e4m3_values()[:127]  # non-negative, ascending
    codes = np.empty(x.size, np.uint8)
    for i, v in enumerate(x):
        if not fine[i]:
            codes[i] = 0x7f
            continue
        y = abs(v) * 2.0 ** (127 - b)
        hi = int(np.searchsorted(grid, y))
        lo = max(0, hi - 1)
        hi = min(hi, 126)
        up, down = grid[hi] - y, y - grid[lo]
        pick = hi if up < down or (up == down and hi % 2 == 0) else lo
        codes[i] = pick | (0x80 if np.signbit(v) else 0)
    return codes, b


def attend(q, k, v, scale, causal, window):
    """One sequence: q [n, nq, d], k and v [keys, nkv, d] -> (outputs, sums of weight times |value|), [n, nq, d]."""
    n, nq, d = q.shape
    keys, nkv = k.shape[:2]
    out, mag = np.zeros((n, nq, d)), np.zeros((n, nq, d))
    for t in range(n):
        hi = keys - (n - 1 - t) if causal else keys
        lo = max(0, hi - window) if window else 0
        if hi <= lo:
            continue
        for h in range(nq):
            kk, vv = k[lo:hi, h // (nq // nkv)], v[lo:hi, h // (nq // nkv)]
            z = kk @ q[t, h] * scale
            p = np.exp(z - z.max())
            p /= p.sum()
            out[t, h] = p @ vv
            mag[t, h] = p @ np.abs(vv)
    return out, mag


def adjust(z, tokens, prompt, drafts, rho, presence, frequency, bias, mask):
    """One row of float64 logits; tokens and drafts: lists of ids; bias: list of (id, value); mask: bits or None."""
    z = np.array(z, np.float64)
    count, seen = {}, set()
    for i, t in enumerate(list(tokens) + [d for d in drafts if d >= 0]):
        if not 0 <= t < z.size:
            continue
        seen.add(t)
        if i >= prompt or i >= len(tokens):
            count[t] = count.get(t, 0) + 1
    for t in seen:
        z[t] = z[t] / rho if z[t] > 0 else z[t] * rho
    for t, c in count.items():
        z[t] = (z[t] - frequency * c) - presence
    for t, b in {t: b for t, b in bias if 0 <= t < z.size}.items():
        z[t] += b
    if mask is not None:
        z[~np.asarray(mask[:z.size], bool)] = -np.inf
    return z
