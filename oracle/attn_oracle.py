"""CPU oracle of the attention-side operators (numpy, float64 or wider):
rotary positions, head norms with the rotation, and scored attention with its
gradients.  Test infrastructure only; written from the formulas, head by head
and pair by pair, with nothing of the library in it."""

from __future__ import annotations

import math

import numpy as np


# ------------------------------------------------------------------- rotary
def rope_frequencies(r, base, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=4.0):
    """Angle per position of each of the r/2 pairs (long double)."""
    ld = np.longdouble
    base, factor = ld(base), ld(factor)
    if scaling == "base" and r > 2:
        base = base * factor ** (ld(r) / ld(r - 2))
    out = []
    for i in range(r // 2):
        w = base ** (ld(-2 * i) / ld(r))
        if scaling == "linear":
            w = w / factor
        elif scaling == "bands":
            turns = ld(original_len) * w / (2 * ld(np.pi))
            if turns <= low:
                w = w / factor
            elif turns < high:
                s = (turns - ld(low)) / (ld(high) - ld(low))
                w = w * s + w / factor * (1 - s)
        elif scaling == "ramp":
            def index(n):
                return r * math.log(original_len / (2 * math.pi * n)) / (2 * math.log(float(base)))
            first, last = max(math.floor(index(high)), 0), min(math.ceil(index(low)), r - 1)
            span = last - first if last > first else 0.001
            g = min(1.0, max(0.0, (i - first) / span))
            w = w * ld(1 - g) + w / factor * ld(g)
        out.append(w)
    return np.array(out, dtype=np.longdouble)


def rope_rotate(x, positions, freqs, layout="half", amplitude=1.0, inverse=False):
    """x [T, heads, D] -> each head's pairs turned by position * freq."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    two_pi = 2 * np.longdouble("3.14159265358979323846264338327950288")
    n = len(freqs)
    for i in range(n):
        a, b = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
        f = np.mod(np.asarray(positions).astype(np.longdouble) * freqs[i], two_pi)
        c, s = np.cos(f).astype(np.float64), np.sin(f).astype(np.float64)
        if inverse:
            s = -s
        c, s = amplitude * c[:, None], amplitude * s[:, None]
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y


def head_norm(x, w, eps):
    """x [T, heads, D]: x / rms(x) * w over the last dimension."""
    x = np.asarray(x, np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if w is None else w)


def head_norm_backward(x, w, g, eps):
    """(dx, dw) of head_norm for the upstream gradient g."""
    x, g = np.asarray(x, np.float64), np.asarray(g, np.float64)
    rms = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xhat = x / rms
    dw = (g * xhat).sum((0, 1))
    gw = g * (1.0 if w is None else w)
    return (gw - xhat * (gw * xhat).mean(-1, keepdims=True)) / rms, dw


# ------------------------------------------------------- scored attention
def visible(T, causal, doc_offsets=None, prefix=None):
    """([T, T] bool: row i sees key j, [T] bool: row i lies in a document)."""
    seen, inside = np.zeros((T, T), bool), np.zeros(T, bool)
    offs = [0, T] if doc_offsets is None else list(doc_offsets)
    for d, (a, b) in enumerate(zip(offs, offs[1:])):
        a, b = max(a, 0), min(b, T)
        for i in range(a, b):
            inside[i] = True
            seen[i, a:(i + 1 if causal else b)] = True
            if causal and prefix is not None:
                seen[i, a:min(b, a + max(prefix[d], 0))] = True
    return seen, inside


def scores(q, k, scale, cap=0.0, slope=0.0):
    """(z [Tq, Tk], tanh or None) of one head; distances |i - j|."""
    z = scale * (np.asarray(q, np.float64) @ np.asarray(k, np.float64).T)
    t = None
    if cap:
        t = np.tanh(z / cap)
        z = cap * t
    i, j = np.arange(z.shape[0]), np.arange(z.shape[1])
    return z - slope * np.abs(i[:, None] - j[None, :]), t


def scored_head(q, k, v, seen, scale, cap=0.0, slope=0.0):
    """(O, LSE) of one head over the keys that each row sees; rows that see
    nothing give 0 and -inf."""
    z, _ = scores(q, k, scale, cap, slope)
    z = np.where(seen, z, -np.inf)
    m = z.max(1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    e = np.exp(z - m)
    l = e.sum(1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        o = np.where(l > 0, (e @ np.asarray(v, np.float64)) / l, 0.0)
        return o, (m + np.log(l))[:, 0]


def scored_head_backward(q, k, v, do, seen, scale, cap=0.0, slope=0.0):
    """(dq, dk, dv) of one head for the upstream gradient do."""
    q, k, v, do = (np.asarray(x, np.float64) for x in (q, k, v, do))
    z, t = scores(q, k, scale, cap, slope)
    _, lse = scored_head(q, k, v, seen, scale, cap, slope)
    P = np.where(seen, np.exp(np.where(seen, z, 0.0) - np.where(np.isfinite(lse), lse, 0.0)[:, None]), 0.0)
    dP = do @ v.T
    dz = P * (dP - (P * dP).sum(1, keepdims=True))
    if t is not None:
        dz = dz * (1 - t * t)
    dz = dz * scale
    return dz @ k, dz.T @ q, P.T @ do


def scored_row(q, k, v, scale, cap=0.0, slope=0.0):
    """(o, lse) of one query behind the keys k (the last one its own)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n = len(k)
    if n == 0:
        return np.zeros(q.shape), -np.inf
    z = scale * (k @ q)
    if cap:
        z = cap * np.tanh(z / cap)
    z = z - slope * np.arange(n - 1, -1, -1)
    e = np.exp(z - z.max())
    return (e @ v) / e.sum(), z.max() + math.log(e.sum())
